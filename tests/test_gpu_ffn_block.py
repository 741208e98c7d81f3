"""The feed-forward side's operators together, as a block uses them: layer norm,
gated feed-forward, down projection, and back; streams and captured graphs."""
import numpy as np
import pytest
import torch

import _ffn_ref as R
from _gpu_ffn import dev, empty, host
from sparse_linear_layers_group_amd import bitlinear as bl
from sparse_linear_layers_group_amd.layer import BitLinearWeight, BlockFeedForward

pytestmark = pytest.mark.gpu
K, N = 640, 1152


def block(seed=0, keep=torch.int8, act=bl.BL_ACT_RELU2, center=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lws, codes = [], []
    for n_out, k in ((N, K), (N, K), (K, N)):
        lw, wq = BitLinearWeight(n_out, k), empty(n_out, k, dtype=torch.int8)
        lw.quantize((torch.randn(n_out, k, generator=gen, device="cuda") * 0.02).bfloat16(), wq=wq)
        lws.append(lw)
        codes.append(wq.cpu().numpy())
    w = 1 + 0.2 * torch.randn(K, generator=gen, device="cuda")
    b = 0.1 * torch.randn(K, generator=gen, device="cuda")
    return BlockFeedForward(*lws, act=act, norm_weight=w, norm_bias=b, center=center, keep=keep), codes


@pytest.mark.parametrize("t", [1, 16, 70, 300])
@pytest.mark.parametrize("keep,act,center,x", [
    (torch.int8, bl.BL_ACT_RELU2, False, torch.float32), (torch.bfloat16, bl.BL_ACT_SILU, True, torch.bfloat16),
    (torch.float32, bl.BL_ACT_RELU2, True, torch.float32)])
def test_step_against_its_parts(t, keep, act, center, x):
    """Each step of the block on the values that the step before it gave: the
    operators' own bounds are tested beside them, so this checks that the block
    hands the right things on."""
    ffn, codes = block(keep=keep, act=act, center=center)
    X = torch.randn(t, K, device="cuda").to(x)
    Y, kept = ffn.fwd(X)
    kind = "relu2" if act == bl.BL_ACT_RELU2 else "silu"
    gm = [float(lw.gamma.item()) for lw in (ffn.gate, ffn.up, ffn.down)]
    xq, xs, hs = (host(kept[n]) for n in ("xq", "x_scale", "h_scale"))
    hq = host(kept["hq"]).reshape(t, N)
    y64, mean, rstd = R.norm(host(X), host(ffn.norm_weight), host(ffn.norm_bias), ffn.eps, center)
    # int8 activations of the norm's rows: half a step of 1/127, and bf16's rounding before it
    assert np.all(np.abs(xq * xs[:, None] - y64) <= xs[:, None] * 0.502 + 2 * R.UBF * np.abs(y64))
    g, u = (R.project(xq, xs, codes[i], gm[i]) for i in range(2))
    h = R.act(g, kind)[0] * u
    # (half a step of h's own 1/127, and bf16's rounding, of which a_t = max|h| feels one too)
    assert np.all(np.abs(hq * hs[:, None] - h) <= hs[:, None] * 0.502 + 2.1 * R.UBF * np.abs(h) + 1e-30)
    assert np.array_equal(host(Y), R.project(hq, hs, codes[2], gm[2]))
    values = lambda p: host(p[0]) if p[1] is None else R.ckpt_values(host(p[0]), host(p[1]))  # noqa: E731
    for p, want in ((kept["G"], g), (kept["U"], u)):
        assert np.array_equal(values(p), R.ckpt_values(*R.ckpt(want)) if keep == torch.int8 else
                              R.bf16(want) if keep == torch.bfloat16 else want)
    dY = torch.randn(t, K, device="cuda").bfloat16()
    dR = torch.randn(t, K, device="cuda")
    grads = ffn.bwd(dY, kept, dR=dR)
    # the whole chain in binary64 from what was kept.  Each product rounds operands to bf16 (2^-8 at most, half that and
    # less on average): 2-norms of the results agree to 1e-2 as for the BitLinears' own backward
    c = [v.astype(np.float64) for v in codes]
    dh = host(dY).astype(np.float64) @ c[2] * gm[2]
    (dn, _), (dwg, _), (dwu, _) = R.glu_bwd(dh, values(kept["G"]), values(kept["U"]), kind, xq, xs, codes[:2], gm[:2])
    dwd = (host(dY).astype(np.float64) * hs[:, None]).T @ hq.astype(np.float64)
    dx, dw, db = R.norm_bwd(values(kept["X"]), host(ffn.norm_weight), mean, rstd, dn, host(dR), center)
    for name, want in (("X", dx), ("gate", dwg), ("up", dwu), ("down", dwd), ("norm_weight", dw), ("norm_bias", db)):
        got = host(grads[name])
        assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want) + 1e-30, name


def test_inference_keeps_nothing_and_gives_the_same():
    ffn, _ = block()
    X = torch.randn(50, K, device="cuda")
    Y, kept = ffn.fwd(X, train=False)
    assert kept is None and torch.equal(Y, ffn.fwd(X)[0])


def test_rows_may_be_overwritten_after_a_forward_that_keeps_8_bits():
    ffn, _ = block()
    X, dY = torch.randn(50, K, device="cuda"), torch.randn(50, K, device="cuda").bfloat16()
    want = ffn.bwd(dY, ffn.fwd(X)[1])
    _, kept = ffn.fwd(X)
    X.fill_(float("nan"))
    got = ffn.bwd(dY, kept)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("keep", [torch.int8, torch.float32])
def test_no_tokens(keep):
    ffn, _ = block(keep=keep)
    y, kept = ffn.fwd(torch.empty(0, K, device="cuda"))
    assert y.shape == (0, K)
    grads = ffn.bwd(torch.empty(0, K, device="cuda", dtype=torch.bfloat16), kept)
    assert grads["X"].shape == (0, K)
    for name in ("gate", "up", "down", "norm_weight", "norm_bias"):
        assert not grads[name].any(), name


def test_refused_blocks():
    a, b, c = BitLinearWeight(N, K), BitLinearWeight(N, K, 4, 8), BitLinearWeight(K, N)
    with pytest.raises(ValueError):
        BlockFeedForward(a, b, c)
    with pytest.raises(ValueError):
        BlockFeedForward(a, a, a)
    with pytest.raises(ValueError):
        BlockFeedForward(a, a, c, keep=torch.float16)


def test_calls_run_on_the_stream_they_name():
    """Inputs are made on one stream, the calls run on another that waits for it."""
    ffn, _ = block()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    X, dY = torch.randn(200, K, device="cuda"), torch.randn(200, K, device="cuda").bfloat16()
    want_y, kept = ffn.fwd(X)
    want = ffn.bwd(dY, kept)
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        torch.cuda._sleep(20_000_000)
        x2 = X * 1
    s2.wait_stream(s1)
    with torch.cuda.stream(s2):
        y, kept = ffn.fwd(x2)
        got = ffn.bwd(dY, kept)
    s2.synchronize()
    assert torch.equal(y, want_y) and all(torch.equal(got[n], want[n]) for n in want)


def test_two_streams_at_once():
    ffn, _ = block()
    xs = [torch.randn(300, K, device="cuda") for _ in range(2)]
    dY = torch.randn(300, K, device="cuda").bfloat16()
    want = []
    for x in xs:
        y, kept = ffn.fwd(x)
        want.append((y, ffn.bwd(dY, kept)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                y, kept = ffn.fwd(xs[i])
                got[i] = (y, ffn.bwd(dY, kept))
    torch.cuda.synchronize()
    for (y, g), (wy, wg) in zip(got, want):
        assert torch.equal(y, wy) and all(torch.equal(g[n], wg[n]) for n in wg)


@pytest.mark.parametrize("t", [1, 40, 300, 4700])
def test_captured_step_replays(t):
    """Forward and backward in one graph, replayed with other inputs, with eager
    work between the replays; every replay equals the eager step's bits."""
    ffn, _ = block()
    X, dY = torch.randn(t, K, device="cuda"), torch.randn(t, K, device="cuda").bfloat16()

    def step():
        y, kept = ffn.fwd(X)
        return y, ffn.bwd(dY, kept)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, grads = step()
    for i in range(4):
        X.copy_(torch.randn(t, K, device="cuda") * (i + 1))
        dY.copy_(torch.randn(t, K, device="cuda"))
        want_y, want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and all(torch.equal(grads[n], want[n]) for n in want)


def test_training_step_changes_the_weights():
    """quantise, forward, backward, update: the latent weights move against the
    gradient, by what the update's definition says."""
    from sparse_linear_layers_group_amd.layer import LatentWeights
    ffn, _ = block()
    lat = LatentWeights((torch.randn(N, K, device="cuda") * 0.02).bfloat16())
    ffn.gate.quantize(lat.W)
    X, dY = torch.randn(64, K, device="cuda"), torch.randn(64, K, device="cuda").bfloat16()
    _, kept = ffn.fwd(X)
    grads = ffn.bwd(dY, kept)
    before = lat.master.clone()
    lat.update(grads["gate"], 0.5)
    want = (before.double() - 0.5 * grads["gate"].double()).float()
    assert torch.equal(lat.master, want)
    ffn.gate.quantize(lat.W)
    ffn.fwd(X)
