"""Head norms with the rotation (bitlinear_qk_rope and its backward) and the
rotation table on the GPU against the 64-bit form."""
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def table_of(max_pos, d, base=10000.0):
    t = torch.empty(max_pos, d // 2, 2, device="cuda")
    bl.bitlinear_rope_table(max_pos, d, base, t)
    return t


def case(tokens, hq, hkv, d, dtype, norm, seed, max_pos=4096, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, (hq + 2 * hkv) * d, generator=g, device="cuda").to(dtype)
    q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, max_pos, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)] if norm else [None, None]
    return q, k, v, pos, w


def angles(table, pos):
    t = table.double()[pos.long()]
    return t[..., 0], t[..., 1]


@pytest.mark.parametrize("max_pos,d,base", [(1, 64, 10000.0), (1000, 128, 10000.0), (131072, 128, 1e6), (70000, 64, 500000.0)])
def test_table(max_pos, d, base):
    t = table_of(max_pos, d, base).double()
    p = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None]
    a = p * base ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))
    # half a step of binary32, and the binary64 angle's own error (p * 2^-50)
    err = R.F32 + max_pos * 2.0 ** -50
    assert (t[..., 0] - a.cos()).abs().max() <= err and (t[..., 1] - a.sin()).abs().max() <= err


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (14, 2, 64), (8, 8, 64), (12, 2, 128), (20, 5, 128), (3, 1, 128)])
@pytest.mark.parametrize("tokens", [1, 3, 130])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("norm", [False, True])
def test_forward_and_backward(hq, hkv, d, tokens, dtype, norm):
    table = table_of(4096, d)
    for fused in (False, True):
        q, k, v, pos, (qw, kw) = case(tokens, hq, hkv, d, dtype, norm, seed=tokens + hq, fused=fused)
        qo = torch.full((tokens, hq * d), 7.0, dtype=BF, device="cuda")
        ko, vo = (torch.full((tokens + 2, hkv * d), 7.0, dtype=BF, device="cuda") for _ in range(2))
        bl.bitlinear_qk_rope(q, k, v, tokens, hq, hkv, d, qw, kw, EPS, table, pos, qo, ko, vo)
        c, s = angles(table, pos)
        for got, x, w, h, n in ((qo, q, qw, hq, "q"), (ko[:tokens], k, kw, hkv, "k")):
            y, err = R.rope(x.reshape(tokens, h, d), c, s, w, EPS)
            R.assert_within(got.view(tokens, h, d), y, err, n)
        assert torch.equal(vo[:tokens], v.to(BF))
        assert (ko[tokens:] == 7).all() and (vo[tokens:] == 7).all()

        g = torch.Generator(device="cuda").manual_seed(99)
        dq, dk = (torch.randn(tokens, h * d, generator=g, device="cuda").to(BF) for h in (hq, hkv))
        gq, gk = torch.empty_like(dq), torch.empty_like(dk)
        gqw, gkw = (torch.empty(d, device="cuda"), torch.empty(d, device="cuda")) if norm else (None, None)
        ws = torch.full((bl.bitlinear_qk_rope_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
        bl.bitlinear_qk_rope_bwd(q if norm else None, k if norm else None, tokens, hq, hkv, d, qw, kw, EPS, table, pos,
                                 dq, dk, gq, gk, gqw, gkw, ws=ws if norm else None)
        for got, gw, x, dy, w, h, n in ((gq, gqw, q, dq, qw, hq, "dq"), (gk, gkw, k, dk, kw, hkv, "dk")):
            dx, err, dw, dwe = R.rope_bwd(x.reshape(tokens, h, d), dy.view(tokens, h, d), c, s, w, EPS)
            R.assert_within(got.view(tokens, h, d), dx, err, n)
            if norm:
                R.assert_within(gw, dw, dwe, n + " weight")


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_rows_go_to_their_slots(dtype):
    tokens, hq, hkv, d, rows = 37, 4, 2, 128, 500
    table = table_of(4096, d)
    q, k, v, pos, (qw, kw) = case(tokens, hq, hkv, d, dtype, True, seed=5)
    slots = torch.randperm(rows, device="cuda")[:tokens].contiguous()
    slots[3], slots[9], slots[20] = -1, rows, 1 << 40  # padding
    outs = [torch.empty(tokens, hq * d, dtype=BF, device="cuda")] + [torch.full((rows, hkv * d), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    bl.bitlinear_qk_rope(q, k, v, tokens, hq, hkv, d, qw, kw, EPS, table, pos, *outs, slots=slots)
    plain = [torch.empty(tokens, h * d, dtype=BF, device="cuda") for h in (hq, hkv, hkv)]
    bl.bitlinear_qk_rope(q, k, v, tokens, hq, hkv, d, qw, kw, EPS, table, pos, *plain)
    assert torch.equal(outs[0], plain[0])
    kept = (slots >= 0) & (slots < rows)
    for got, rowwise in zip(outs[1:], plain[1:]):
        want = torch.full((rows, hkv * d), 7.0, dtype=BF, device="cuda")
        want[slots[kept]] = rowwise[kept]
        assert torch.equal(got, want)


def test_position_outside_the_table_gives_nan():
    tokens, hq, hkv, d = 5, 2, 1, 64
    table = table_of(16, d)
    q, k, v, pos, _ = case(tokens, hq, hkv, d, torch.float32, False, seed=6, max_pos=16)
    pos[1], pos[3] = -1, 16
    qo, ko, vo = (torch.empty(tokens, h * d, dtype=BF, device="cuda") for h in (hq, hkv, hkv))
    bl.bitlinear_qk_rope(q, k, v, tokens, hq, hkv, d, None, None, 0.0, table, pos, qo, ko, vo)
    bad = torch.tensor([False, True, False, True, False], device="cuda")
    assert torch.equal(torch.isnan(qo).all(1), bad) and torch.equal(torch.isnan(qo).any(1), bad)
    assert torch.equal(torch.isnan(ko).all(1), bad) and torch.equal(vo, v.to(BF))


def test_large_and_zero_rows():
    """Rows of zeros (eps keeps them finite) and of large values."""
    tokens, hq, hkv, d = 4, 2, 1, 128
    table = table_of(64, d)
    q, k, v, pos, (qw, kw) = case(tokens, hq, hkv, d, torch.float32, True, seed=7, max_pos=64)
    q[1], q[2] = 0, q[2] * 1e15
    qo, ko = (torch.empty(tokens, h * d, dtype=BF, device="cuda") for h in (hq, hkv))
    bl.bitlinear_qk_rope(q, k, None, tokens, hq, hkv, d, qw, kw, EPS, table, pos, qo, ko, None)
    c, s = angles(table, pos)
    y, err = R.rope(q.view(tokens, hq, d), c, s, qw, EPS)
    R.assert_within(qo.view(tokens, hq, d), y, err, "q")


def test_weight_gradients_over_many_rows_and_reruns():
    tokens, hq, hkv, d = 5000, 8, 2, 128
    table = table_of(8192, d)
    q, k, v, pos, (qw, kw) = case(tokens, hq, hkv, d, torch.float32, True, seed=8, max_pos=8192)
    g = torch.Generator(device="cuda").manual_seed(9)
    dq, dk = (torch.randn(tokens, h * d, generator=g, device="cuda").to(BF) for h in (hq, hkv))
    ws = torch.empty(bl.bitlinear_qk_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    runs = []
    for _ in range(2):
        out = [torch.empty_like(dq), torch.empty_like(dk), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
        bl.bitlinear_qk_rope_bwd(q, k, tokens, hq, hkv, d, qw, kw, EPS, table, pos, dq, dk, *out, ws=ws)
        runs.append(out)
    assert all(torch.equal(x, y) for x, y in zip(*runs))
    c, s = angles(table, pos)
    for i, (x, dy, w, h) in enumerate(((q, dq, qw, hq), (k, dk, kw, hkv))):
        _, _, dw, dwe = R.rope_bwd(x.view(tokens, h, d), dy.view(tokens, h, d), c, s, w, EPS)
        R.assert_within(runs[0][2 + i], dw, dwe, "weight gradient")


def test_gradient_against_differences():
    tokens, hq, hkv, d = 7, 2, 2, 64
    table = table_of(512, d)
    q, k, v, pos, (qw, kw) = case(tokens, hq, hkv, d, torch.float32, True, seed=10, max_pos=512)
    g = torch.Generator(device="cuda").manual_seed(11)
    dq, dk = (torch.randn(tokens, h * d, generator=g, device="cuda").to(BF) for h in (hq, hkv))
    out = [torch.empty_like(dq), torch.empty_like(dk), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    ws = torch.empty(bl.bitlinear_qk_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    bl.bitlinear_qk_rope_bwd(q, k, tokens, hq, hkv, d, qw, kw, EPS, table, pos, dq, dk, *out, ws=ws)
    c, s = angles(table, pos)
    x, dy = q.double().view(tokens, hq, d), dq.double().view(tokens, hq, d)
    dx, dxe, dw, dwe = R.rope_bwd(x, dy, c, s, qw, EPS)
    h = 1e-5
    loss = lambda x, w: float((R.rope(x, c, s, w, EPS)[0] * dy).sum())  # noqa: E731
    u = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    diff = (loss(x + h * u, qw.double()) - loss(x - h * u, qw.double())) / (2 * h)
    assert abs(float((out[0].double().view_as(u) * u).sum()) - diff) <= float((dxe * u.abs()).sum()) + 1e-6 * abs(diff) + 1e-6
    u = torch.randn(d, generator=g, device="cuda", dtype=torch.float64)
    diff = (loss(x, qw.double() + h * u) - loss(x, qw.double() - h * u)) / (2 * h)
    assert abs(float((out[2].double() * u).sum()) - diff) <= float((dwe * u.abs()).sum()) + 1e-6 * abs(diff) + 1e-6


def test_no_tokens():
    d = 64
    table = table_of(4, d)
    e = torch.empty(0, d, dtype=torch.float32, device="cuda")
    eb = e.to(BF)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    w = torch.ones(d, device="cuda")
    bl.bitlinear_qk_rope(e, e, e, 0, 1, 1, d, w, w, EPS, table, pos, eb, eb, eb)
    gq, gk = torch.full((d,), 5.0, device="cuda"), torch.full((d,), 5.0, device="cuda")
    ws = torch.empty(bl.bitlinear_qk_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    bl.bitlinear_qk_rope_bwd(e, e, 0, 1, 1, d, w, w, EPS, table, pos, eb, eb, eb, eb, gq, gk, ws=ws)
    assert (gq == 0).all() and (gk == 0).all()


def test_captured_graph_and_another_stream():
    tokens, hq, hkv, d = 70, 4, 2, 64
    table = table_of(4096, d)
    q, k, v, pos, (qw, kw) = case(tokens, hq, hkv, d, torch.float32, True, seed=20)
    outs = [torch.empty(tokens, h * d, dtype=BF, device="cuda") for h in (hq, hkv, hkv)]
    grads = [torch.empty(tokens, h * d, dtype=BF, device="cuda") for h in (hq, hkv)]
    gw = [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.full((bl.bitlinear_qk_rope_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")

    def step():
        bl.bitlinear_qk_rope(q, k, v, tokens, hq, hkv, d, qw, kw, EPS, table, pos, *outs)
        bl.bitlinear_qk_rope_bwd(q, k, tokens, hq, hkv, d, qw, kw, EPS, table, pos, outs[0], outs[1], *grads, *gw, ws=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        pos.copy_(torch.randint(0, 4096, (tokens,), generator=g, device="cuda", dtype=torch.int32))
        q.normal_(generator=g)
        for x in (*outs, *grads, *gw):
            x.fill_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*outs, *grads, *gw)]
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (*outs, *grads, *gw)):
            assert torch.equal(x, y)
        c, s = angles(table, pos)
        y, err = R.rope(q.view(tokens, hq, d), c, s, qw, EPS)
        R.assert_within(got[0].view(tokens, hq, d), y, err, "q")
