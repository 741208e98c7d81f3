"""The attention side of a block together with its BitLinears, as a training
step and a serving loop run them: every stage against the 64-bit form of its
own inputs, gradients through to the q, k, v projections, and decoding over a
paged cache against the prompt's attention."""
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from sparse_linear_layers_group_amd import bitlinear as bl
from sparse_linear_layers_group_amd import synth
from sparse_linear_layers_group_amd.layer import BitLinearWeight, BlockAttention, bf16_tensor

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HQ, HKV, D, HID = 6, 2, 64, 384
N, M = 6, 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def projections(seed):
    out = []
    for i, n_out in enumerate((HQ * D, HKV * D, HKV * D, HID)):
        lw = BitLinearWeight(n_out, HID, N, M)
        lw.quantize(bf16_tensor(synth.weights(n_out, HID, seed=seed, layer=i)))
        out.append(lw)
    return out


def project(lws, x, tokens):
    """float32 q, k, v rows of one quantised input, and that input's codes."""
    xq = torch.empty(tokens * HID, dtype=torch.int8, device="cuda")
    sc = torch.empty(tokens, dtype=torch.float32, device="cuda")
    bl.bitlinear_act_quant(x, tokens, HID, xq, sc)
    ys = [torch.empty(tokens, lw.n_out, device="cuda") for lw in lws]
    items = bl.make_contract_items([dict(packed=lw.packed, gamma=lw.gamma, Y=y, n_out=lw.n_out) for lw, y in zip(lws, ys)],
                                   tokens)
    n = bl.bitlinear_contract_group_workspace_bytes(items, 3, tokens, HID)
    bl.bitlinear_contract_group(items, 3, xq, sc, tokens, HID, N, M,
                                ws=torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None)
    return ys, xq, sc


def angles(att, pos):
    t = att.table.double()[pos.long()]
    return t[..., 0], t[..., 1]


def block(norm, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)] if norm else [None, None]
    return projections(seed), BlockAttention(HQ, HKV, D, 2048, q_weight=w[0], k_weight=w[1])


@pytest.mark.parametrize("norm", [False, True])
def test_training_step(norm):
    lens = [70, 1, 130]
    tokens = sum(lens)
    (wq, wk, wv, wo), att = block(norm)
    x = bf16_tensor(synth.activations(tokens, HID, seed=2))
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    cu = torch.tensor([0, 70, 71, 201], dtype=torch.int32, device="cuda")

    (yq, yk, yv), xq, sc = project((wq, wk, wv), x, tokens)
    qr, kr, vr = att.rotate(yq, yk, yv, pos)
    o, lse = att.attend(qr, kr, vr, cu, cu)
    fo = wo.fwd(o, tokens)
    dy = bf16_tensor(synth.grad_output(tokens, HID, seed=3))
    do, _ = wo.bwd(dy, fo["xq"], fo["x_scale"], tokens)  # binary32
    dqr, dkr, dv = att.attend_bwd(qr, kr, vr, o, lse, do, cu, cu)
    dq, dk, gq, gk = att.rotate_bwd(yq, yk, pos, dqr, dkr)
    dx = [torch.empty(tokens * HID, device="cuda") for _ in range(3)]
    dw = [torch.empty(lw.n_out * HID, device="cuda") for lw in (wq, wk, wv)]
    items = bl.make_bwd_items([dict(dY=d, xq=xq, x_scale=sc, packed=lw.packed, gamma=lw.gamma, dX=a, dW=b, k=HID,
                                    n_out=lw.n_out) for d, lw, a, b in zip((dq, dk, dv), (wq, wk, wv), dx, dw)], tokens)
    ws = torch.empty(bl.bitlinear_bwd_group_workspace_bytes(items, 3, tokens), dtype=torch.uint8, device="cuda")
    bl.bitlinear_bwd_group(items, 3, tokens, N, M, ws=ws)
    torch.cuda.synchronize()

    c, s = angles(att, pos)
    for got, y, w, h in ((qr, yq, att.q_weight, HQ), (kr, yk, att.k_weight, HKV)):
        want, err = R.rope(y.view(tokens, h, D), c, s, w, att.eps)
        R.assert_within(got.view(tokens, h, D), want, err, "rotated")
    q3, k3, v3 = (t.view(tokens, -1, D) for t in (qr, kr, vr))
    ref = R.attention(q3, k3, v3, lens, lens, att.scale, do.view(tokens, HQ, D), do_f32=True)
    R.assert_within(o.view(tokens, HQ, D), ref["o"], ref["o_err"], "O")
    for got, n in ((dqr, "dq"), (dkr, "dk"), (dv, "dv")):
        R.assert_within(got.view(tokens, -1, D), ref[n], ref[n + "_err"], n)
    for got, gw, y, dy_, w, h in ((dq, gq, yq, dqr, att.q_weight, HQ), (dk, gk, yk, dkr, att.k_weight, HKV)):
        want, err, dwt, dwe = R.rope_bwd(y.view(tokens, h, D), dy_.view(tokens, h, D), c, s, w, att.eps)
        R.assert_within(got.view(tokens, h, D), want, err, "gradient before the rotation")
        if norm:
            R.assert_within(gw, dwt, dwe, "norm weight")
    assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in dx + dw)


def test_serving_over_a_paged_cache():
    """A prompt, then tokens one at a time, then a drafted chain, over pages:
    the rows of one packed causal attention over all of it."""
    lens, page, new = [45, 9], 16, 4
    (wq, wk, wv, wo), att = block(True, seed=5)
    total = [n + new for n in lens]
    x = [bf16_tensor(synth.activations(n, HID, seed=10 + b)) for b, n in enumerate(total)]
    pages = torch.tensor([[5, 0, 7, 2], [3, -1, -1, -1]], dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((8 * page, HKV * D), float("nan"), dtype=BF, device="cuda") for _ in range(2))

    def slots(b, p):
        return pages[b].long()[p // page] * page + p % page

    # everything at once, as packed prompts
    ys, _, _ = project((wq, wk, wv), torch.cat(x), sum(total))
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in total]).cuda()
    cu = torch.tensor([0, total[0], sum(total)], dtype=torch.int32, device="cuda")
    qr, kr, vr = att.rotate(*ys, pos)
    want, _ = att.attend(qr, kr, vr, cu, cu)
    ref = R.attention(*(t.view(sum(total), -1, D) for t in (qr, kr, vr)), total, total, att.scale)

    def rows(b, a, e):
        return slice(int(cu[b]) + a, int(cu[b]) + e)

    # the prompts' rows into the cache
    for b, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        r = rows(b, 0, n)
        att.rotate(*(y[r] for y in ys), p.int(), cache=(kc, vc), slots=slots(b, p))
    # one token of each sequence at a time
    for i in range(new):
        p = torch.tensor([n + i for n in lens], device="cuda")
        at = [rows(b, n + i, n + i + 1) for b, n in enumerate(lens)]
        q, _, _ = att.rotate(*(torch.cat([y[r] for r in at]) for y in ys), p.int(), cache=(kc, vc),
                             slots=torch.stack([slots(b, p[b]) for b in range(2)]))
        o = att.attend_cache(q, (kc, vc), pages, page, (p + 1).int())
        for b, r in enumerate(at):
            R.assert_within(o[b].view(1, HQ, D), ref["o"][r], ref["o_err"][r], f"token {i} of sequence {b}")
    # the same tokens as a drafted chain
    q = torch.cat([qr[rows(b, n, n + new)] for b, n in enumerate(lens)])
    o = att.attend_cache(q, (kc, vc), pages, page, torch.tensor(total, dtype=torch.int32, device="cuda"))
    for b, n in enumerate(lens):
        r = rows(b, n, n + new)
        R.assert_within(o[b * new:(b + 1) * new].view(new, HQ, D), ref["o"][r], ref["o_err"][r], f"chain {b}")
    # and the o projection takes the result
    assert torch.isfinite(wo.fwd(o, 2 * new)["Y"]).all() and torch.isfinite(want.float()).all()
