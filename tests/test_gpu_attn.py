"""Packed causal attention (bitlinear_attn_fwd, bitlinear_attn_bwd) on the GPU
against the 64-bit form, within the bounds its roundings allow."""
import math

import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def cu(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def inputs(q_lens, k_lens, hq, hkv, d, seed, extra=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    tq, tk = sum(q_lens) + extra, sum(k_lens) + extra
    return (n(tq, hq, d) * std).to(BF), n(tk, hkv, d).to(BF), (n(tk, hkv, d) + 0.25).to(BF), n(tq, hq, d)


def ws_for(fn, *a):
    n = fn(*a)
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def forward(q, k, v, q_lens, k_lens, scale, lse=True, stream=None):
    tq, hq, d = q.shape
    tk, hkv = k.shape[:2]
    b = len(q_lens)
    o = torch.full((tq, hq, d), 7.0, dtype=BF, device="cuda")
    l = torch.full((hq, tq), 7.0, device="cuda") if lse else None
    ws = ws_for(bl.bitlinear_attn_fwd_workspace_bytes, b, tq, tk, hq, hkv, d)
    bl.bitlinear_attn_fwd(q, k, v, cu(q_lens), cu(k_lens), b, hq, hkv, d, scale, o, l, ws=ws, stream=stream)
    return o, l


def backward(q, k, v, o, lse, do, q_lens, k_lens, scale):
    tq, hq, d = q.shape
    tk, hkv = k.shape[:2]
    b = len(q_lens)
    dq = torch.full((tq, hq, d), 7.0, dtype=BF, device="cuda")
    dk, dv = (torch.full((tk, hkv, d), 7.0, dtype=BF, device="cuda") for _ in range(2))
    ws = ws_for(bl.bitlinear_attn_bwd_workspace_bytes, b, tq, tk, hq, hkv, d)
    if ws is not None:
        ws.fill_(0xff)  # NaN patterns: nothing is read that was not written
    bl.bitlinear_attn_bwd(q, k, v, o, lse, do, cu(q_lens), cu(k_lens), b, hq, hkv, d, scale, dq, dk, dv, ws=ws)
    return dq, dk, dv


def check(q, k, v, do, q_lens, k_lens, scale=None, do_f32=False):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    do = do if do_f32 else do.to(BF)
    o, lse = forward(q, k, v, q_lens, k_lens, scale)
    ref = R.attention(q, k, v, q_lens, k_lens, scale, do, do_f32)
    R.assert_within(o, ref["o"], ref["o_err"], "O")
    R.assert_within(lse, ref["lse"], ref["lse_err"], "lse")
    tq, tk = sum(q_lens), sum(k_lens)
    assert (o[tq:] == 7).all() and (lse[:, tq:] == 7).all(), "rows behind the last sequence"
    dq, dk, dv = backward(q, k, v, o, lse, do, q_lens, k_lens, scale)
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        R.assert_within(x, ref[n], ref[n + "_err"], n)
    assert (dq[tq:] == 7).all() and (dk[tk:] == 7).all() and (dv[tk:] == 7).all(), "gradients behind the last sequence"
    return o, lse, dq, dk, dv


LAYOUTS = [(1, 1, 64), (4, 2, 64), (14, 2, 64), (5, 5, 128), (8, 2, 128), (12, 2, 128), (7, 1, 128)]


@pytest.mark.parametrize("hq,hkv,d", LAYOUTS)
@pytest.mark.parametrize("lens", [[1], [31, 33], [64], [65, 1, 127], [128, 129, 2], [200, 0, 257], [500]])
def test_self_attention(hq, hkv, d, lens):
    q, k, v, do = inputs(lens, lens, hq, hkv, d, seed=hq * 100 + len(lens))
    check(q, k, v, do, lens, lens)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (6, 2, 128)])
@pytest.mark.parametrize("q_lens,k_lens", [
    ([1, 1, 1], [1, 64, 333]),           # single tokens
    ([17, 130], [400, 131]),             # a prompt's next piece
    ([100, 3, 140], [40, 0, 9]),         # more queries than keys: rows that see none
    ([0, 5, 0], [7, 0, 130]),            # no queries, no keys
    ([70, 0, 64], [300, 64, 64]),
])
def test_unequal_lengths(hq, hkv, d, q_lens, k_lens):
    q, k, v, do = inputs(q_lens, k_lens, hq, hkv, d, seed=3)
    check(q, k, v, do, q_lens, k_lens)


def test_binary32_output_gradient():
    lens = [130, 77]
    q, k, v, do = inputs(lens, lens, 4, 2, 128, seed=4)
    check(q, k, v, do, lens, lens, do_f32=True)


@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_behind_a_sequence_does_not_matter(d):
    lens, extra = [70, 33], 40
    q, k, v, do = inputs(lens, lens, 4, 2, d, seed=5, extra=extra)
    n = sum(lens)
    for x in (q, k, v, do):
        x[n:] = float("nan")
    k[n] = float("inf")
    check(q, k, v, do, lens, lens)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores_and_flat_rows(d):
    lens = [150]
    q, k, v, do = inputs(lens, lens, 2, 1, d, seed=6, std=20.0)  # scores of hundreds: one key takes all
    check(q, k, v, do, lens, lens)
    check(torch.zeros_like(q), k, v, do, lens, lens)             # equal scores: plain means
    up = (torch.arange(150, device="cuda") * 0.5).to(BF)[:, None, None].expand(150, 1, d).contiguous()
    check(torch.full_like(q, 0.5), up, v, do, lens, lens)        # the maximum grows with every key


def test_strided_rows_of_one_projection():
    lens, hq, hkv, d = [65, 40], 6, 2, 64
    q, k, v, do = inputs(lens, lens, hq, hkv, d, seed=7)
    t = sum(lens)
    wide = torch.cat([x.reshape(t, -1) for x in (q, k, v)], 1)
    qs, ks, vs = wide[:, :hq * d], wide[:, hq * d:(hq + hkv) * d], wide[:, (hq + hkv) * d:]
    o, lse, dq, dk, dv = check(q, k, v, do, lens, lens)
    b, s = len(lens), d ** -0.5
    o2, l2 = torch.empty_like(o), torch.empty_like(lse)
    bl.bitlinear_attn_fwd(qs, ks, vs, cu(lens), cu(lens), b, hq, hkv, d, s, o2, l2)
    g = [torch.empty_like(x) for x in (dq, dk, dv)]
    ws = ws_for(bl.bitlinear_attn_bwd_workspace_bytes, b, t, t, hq, hkv, d)
    bl.bitlinear_attn_bwd(qs, ks, vs, o2, l2, do.to(BF), cu(lens), cu(lens), b, hq, hkv, d, s, *g, ws=ws)
    for x, y in zip((o, lse, dq, dk, dv), (o2, l2, *g)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("batch", [64, 257, 300])
def test_many_short_sequences(batch):
    lens = [(i * 7) % 5 + (130 if i % 50 == 3 else 0) for i in range(batch)]
    q, k, v, do = inputs(lens, lens, 2, 1, 64, seed=8)
    check(q, k, v, do, lens, lens)


def test_long_sequence_and_reruns_are_bit_identical():
    lens = [2300, 700]
    q, k, v, do = inputs(lens, lens, 4, 1, 128, seed=9)
    first = check(q, k, v, do, lens, lens)
    o, lse = forward(q, k, v, lens, lens, 128 ** -0.5)
    again = (o, lse, *backward(q, k, v, o, lse, do.to(BF), lens, lens, 128 ** -0.5))
    for x, y in zip(first, again):
        assert torch.equal(x, y)


def test_offsets_outside_the_buffers_are_cut_off():
    hq, hkv, d, t = 2, 1, 64, 100
    q, k, v, do = inputs([t], [t], hq, hkv, d, seed=10)
    o, lse = torch.empty_like(q), torch.empty(hq, t, device="cuda")
    c = torch.tensor([-5, 40, 30, 1 << 30], dtype=torch.int32, device="cuda")  # [0, 40), [40, 40), [30, 100)
    bl.bitlinear_attn_fwd(q, k, v, c, c, 3, hq, hkv, d, 0.125, o, lse)
    ref = R.attention(q[:30], k[:30], v[:30], [30], [30], 0.125)
    R.assert_within(o[:30], ref["o"], ref["o_err"], "O")
    ref = R.attention(q[40:], k[30:], v[30:], [60], [70], 0.125)
    assert torch.isfinite(o.float()).all()


def test_gradient_against_differences():
    """<dX, u> of the kernel against the central difference of the 64-bit loss
    sum(O dO) along u; the bound is the rounding bound along |u|."""
    lens, hq, hkv, d, s = [90, 41], 4, 2, 64, 0.125
    q, k, v, do = inputs(lens, lens, hq, hkv, d, seed=11)
    do = do.to(BF)
    o, lse = forward(q, k, v, lens, lens, s)
    grads = dict(zip("qkv", backward(q, k, v, o, lse, do, lens, lens, s)))
    ref = R.attention(q, k, v, lens, lens, s, do)
    x = {"q": q.double(), "k": k.double(), "v": v.double()}
    gen = torch.Generator(device="cuda").manual_seed(12)
    for n in "qkv":
        u = torch.randn(x[n].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        loss = [float((R.attention(**{**x, n: x[n] + e * u}, q_lens=lens, k_lens=lens, scale=s)["o"] * do.double()).sum())
                for e in (h, -h)]
        diff = (loss[0] - loss[1]) / (2 * h)
        bound = float((ref[f"d{n}_err"] * u.abs()).sum()) + 1e-6 * abs(diff) + 1e-6
        assert abs(float((grads[n].double() * u).sum()) - diff) <= bound


def test_captured_graph_replays_with_other_lengths():
    hq, hkv, d, t, s = 4, 2, 64, 200, 0.125
    q, k, v, do = inputs([t], [t], hq, hkv, d, seed=13)
    do = do.to(BF)
    c = cu([120, 80])
    o, lse = torch.empty_like(q), torch.empty(hq, t, device="cuda")
    g = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
    wf = ws_for(bl.bitlinear_attn_fwd_workspace_bytes, 2, t, t, hq, hkv, d)
    wb = ws_for(bl.bitlinear_attn_bwd_workspace_bytes, 2, t, t, hq, hkv, d)

    def step():
        bl.bitlinear_attn_fwd(q, k, v, c, c, 2, hq, hkv, d, s, o, lse, ws=wf)
        bl.bitlinear_attn_bwd(q, k, v, o, lse, do, c, c, 2, hq, hkv, d, s, *g, ws=wb)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([120, 80], [1, 199], [64, 136], [200, 0]):
        c.copy_(cu(lens))
        q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (o, lse, *g)]
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (o, lse, *g)):
            assert torch.equal(x, y)
        ref = R.attention(q, k, v, lens, lens, s, do)
        R.assert_within(got[0], ref["o"], ref["o_err"], "O")
        R.assert_within(got[3], ref["dk"], ref["dk_err"], "dk")


def test_another_stream_and_no_lse():
    lens = [100, 28]
    q, k, v, _ = inputs(lens, lens, 4, 2, 128, seed=14)
    want, _ = forward(q, k, v, lens, lens, 0.1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o, lse = forward(q, k, v, lens, lens, 0.1, lse=False, stream=st)
    st.synchronize()
    # the outputs were filled on the default stream before
    torch.cuda.synchronize()
    assert lse is None
    with torch.cuda.stream(st):
        o2, _ = forward(q, k, v, lens, lens, 0.1, lse=False)
    st.synchronize()
    assert torch.equal(o2, want)


def test_no_rows():
    e = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    k = torch.randn(9, 1, 64, device="cuda").to(BF)
    o, lse = forward(e, k, k, [0], [9], 0.125)
    dq, dk, dv = backward(e, k, k, o, lse, e, [0], [9], 0.125)
    assert (dk == 0).all() and (dv == 0).all()
    q = torch.randn(5, 2, 64, device="cuda").to(BF)
    none = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    o, lse = forward(q, none, none, [5], [0], 0.125)
    assert (o == 0).all() and (lse == -math.inf).all()
    dq, _, _ = backward(q, none, none, o, lse, q, [5], [0], 0.125)
    assert (dq == 0).all()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (6, 2, 128), (8, 1, 128)])
@pytest.mark.parametrize("q_lens,k_lens", [
    ([5], [4100]),                       # few rows, many keys: the keys are shared out
    ([130, 1], [3000, 2500]),
    ([64, 200, 3], [1700, 200, 4000]),   # one short sequence among them: parts without tiles
    ([40, 100], [4000, 20]),             # and rows that see no key
])
def test_few_rows_with_many_keys(hq, hkv, d, q_lens, k_lens):
    assert bl.bitlinear_attn_fwd_workspace_bytes(len(q_lens), sum(q_lens), sum(k_lens), hq, hkv, d) > 0
    q, k, v, do = inputs(q_lens, k_lens, hq, hkv, d, seed=20, extra=3)
    check(q, k, v, do, q_lens, k_lens)


@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_may_hold_anything(d):
    """Not-a-number rows of one sequence stay in it, forward and backward."""
    lens = [70, 33, 190]
    q, k, v, do = inputs(lens, lens, 4, 2, d, seed=21)
    do = do.to(BF)
    clean = forward(q, k, v, lens, lens, 0.1)
    grads = backward(q, k, v, *clean, do, lens, lens, 0.1)
    q2, k2, v2, do2 = (t.clone() for t in (q, k, v, do))
    for t in (q2, k2, v2, do2):
        t[70:103] = float("nan")
    o, lse = forward(q2, k2, v2, lens, lens, 0.1)
    keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep[70:103] = False
    assert torch.equal(o[keep], clean[0][keep]) and torch.equal(lse[:, keep], clean[1][:, keep])
    for x, y in zip(backward(q2, k2, v2, o, lse, do2, lens, lens, 0.1), grads):
        assert torch.equal(x[keep], y[keep])


def test_two_streams_at_once():
    """Two calls of different sizes, each with its own buffers."""
    a, b = [300, 40], [129, 513, 7]
    qa, qb = inputs(a, a, 4, 2, 128, seed=22), inputs(b, b, 4, 2, 128, seed=23)
    want = [forward(*q[:3], n, n, 0.1) for q, n in ((qa, a), (qb, b))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st, q, n in zip(streams, (qa, qb), (a, b)):
        with torch.cuda.stream(st):
            got.append(forward(*q[:3], n, n, 0.1))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("q_lens,k_lens", [([1] * 40, [300] * 40), ([1] * 300, [40] * 300), ([3] * 16, [800] * 16)])
def test_a_few_rows_of_many_sequences(q_lens, k_lens):
    q, k, v, do = inputs(q_lens, k_lens, 4, 2, 64, seed=24)
    check(q, k, v, do, q_lens, k_lens)


@pytest.mark.parametrize("hq,hkv", [(300, 1), (96, 96), (520, 4)])
def test_many_heads(hq, hkv):
    lens = [5, 70]
    q, k, v, do = inputs(lens, lens, hq, hkv, 64, seed=25)
    check(q, k, v, do, lens, lens)


def test_captured_graph_of_shared_out_keys():
    """Few rows, many keys: parts, their join and the backward's splits, with
    lengths that change what is split; eager work between the replays."""
    hq, hkv, d, tq, tk, s = 4, 2, 128, 70, 4000, 0.1
    q, k, v, do = inputs([tq], [tk], hq, hkv, d, seed=26)
    do = do.to(BF)
    cq, ck = cu([30, 40]), cu([1000, 3000])
    nf = bl.bitlinear_attn_fwd_workspace_bytes(2, tq, tk, hq, hkv, d)
    assert nf > 0
    wf = torch.full((nf,), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((bl.bitlinear_attn_bwd_workspace_bytes(2, tq, tk, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(hq, tq, device="cuda")
    g = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]

    def step():
        bl.bitlinear_attn_fwd(q, k, v, cq, ck, 2, hq, hkv, d, s, o, lse, ws=wf)
        bl.bitlinear_attn_bwd(q, k, v, o, lse, do, cq, ck, 2, hq, hkv, d, s, *g, ws=wb)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for ql, kl in (([30, 40], [1000, 3000]), ([1, 69], [4000, 0]), ([70, 0], [20, 3980]), ([35, 35], [2000, 2000])):
        cq.copy_(cu(ql))
        ck.copy_(cu(kl))
        for x in (o, lse, *g):
            x.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (o, lse, *g)]
        ref = R.attention(q, k, v, ql, kl, s, do)
        R.assert_within(got[0], ref["o"], ref["o_err"], "O")
        for x, n in zip(got[2:], ("dq", "dk", "dv")):
            R.assert_within(x, ref[n], ref[n + "_err"], n)
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (o, lse, *g)):
            assert torch.equal(x, y)


def test_two_graphs_with_workspaces_of_their_own():
    """Replayed in turn, each keeps its results."""
    runs = []
    for seed, lens in ((27, [200, 56]), (28, [100, 300])):
        q, k, v, do = inputs(lens, lens, 4, 2, 64, seed=seed)
        do = do.to(BF)
        b, t = len(lens), sum(lens)
        c = cu(lens)
        o, lse = torch.empty_like(q), torch.empty(4, t, device="cuda")
        g = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
        ws = ws_for(bl.bitlinear_attn_bwd_workspace_bytes, b, t, t, 4, 2, 64)

        def step(q=q, k=k, v=v, do=do, c=c, o=o, lse=lse, g=g, ws=ws, b=b):
            bl.bitlinear_attn_fwd(q, k, v, c, c, b, 4, 2, 64, 0.125, o, lse)
            bl.bitlinear_attn_bwd(q, k, v, o, lse, do, c, c, b, 4, 2, 64, 0.125, *g, ws=ws)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (o, lse, *g)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((graph, want, (o, lse, *g), step))  # (step holds the inputs and the workspace)
    for _ in range(3):
        for graph, _, outs, _ in runs:
            for x in outs:
                x.fill_(3.0)
            graph.replay()
        torch.cuda.synchronize()
        for _, want, outs, _ in runs:
            for x, y in zip(want, outs):
                assert torch.equal(x, y)


@pytest.mark.parametrize("scale", [1e-30, 1e-12])
def test_scales_that_flatten_every_row(scale):
    """Scores that vanish: the mean of the visible V, and its gradients."""
    lens = [70, 200]
    q, k, v, do = inputs(lens, lens, 2, 1, 64, seed=29)
    do = do.to(BF)
    o, lse = forward(q, k, v, lens, lens, scale)
    ref = R.attention(q, k, v, lens, lens, scale, do)
    R.assert_within(o, ref["o"], ref["o_err"], "O")
    _, _, dv = backward(q, k, v, o, lse, do, lens, lens, scale)
    R.assert_within(dv, ref["dv"], ref["dv_err"], "dv")
