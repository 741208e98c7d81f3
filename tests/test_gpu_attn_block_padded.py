"""BlockAttention on a batch padded behind its last sequence: the padding's rows
of every result are zeros, so sums over tokens further back (the norms' and the
projections' weight gradients) are those of the sequences alone."""
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from sparse_linear_layers_group_amd.layer import BlockAttention

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def poison(*sizes):
    """Leaves NaN in the memory that the allocator hands out next."""
    held = [torch.full((n,), float("nan"), dtype=BF, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_padded_batch(d, norm):
    hq, hkv, used, pad = 4, 2, 150, 50
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = [1 + 0.2 * n(d), 1 + 0.2 * n(d)] if norm else [None, None]
    att = BlockAttention(hq, hkv, d, 256, q_weight=w[0], k_weight=w[1])
    total = used + pad
    x, do = [n(total, h * d) for h in (hq, hkv, hkv)], n(total, hq * d)
    pos = torch.cat([torch.arange(100), torch.arange(50), torch.zeros(pad)]).int().cuda()
    cu = torch.tensor([0, 100, used], dtype=torch.int32, device="cuda")

    poison(total * hq * d, total * hkv * d)
    r = att.rotate(*x, pos)
    poison(total * hq * d, total * hkv * d)
    o, lse = att.attend(*r, cu, cu)
    poison(total * hq * d, total * hkv * d)
    dr = att.attend_bwd(*r, o, lse, do, cu, cu)
    dx = att.rotate_bwd(x[0], x[1], pos, dr[0], dr[1])

    ref = R.attention(*(t.view(total, -1, d) for t in r), [100, 50], [100, 50], att.scale, do.view(total, hq, d), do_f32=True)
    for t, n in ((o, "o"), (dr[0], "dq"), (dr[1], "dk"), (dr[2], "dv")):
        R.assert_within(t.view(total, -1, d), ref[n], ref[n + "_err"], n)
        assert (t[used:] == 0).all(), f"padding of {n}"
    t = att.table.double()[pos.long()][:used]
    for i, h in enumerate((hq, hkv)):
        want, err, dw, dwe = R.rope_bwd(x[i][:used].view(used, h, d), dr[i][:used].view(used, h, d), t[..., 0], t[..., 1],
                                        w[i], att.eps)
        R.assert_within(dx[i][:used].view(used, h, d), want, err, "gradient before the rotation")
        assert (dx[i][used:] == 0).all()
        if norm:
            R.assert_within(dx[2 + i], dw, dwe, "norm weight")


@pytest.mark.parametrize("q_total,k_total", [(200, 200), (60, 3000)])
def test_padded_batch_in_a_graph(q_total, k_total):
    """Captured with one set of lengths, replayed with others: rows that were a
    sequence's before are padding now, and zeros."""
    hq, hkv, d = 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    att = BlockAttention(hq, hkv, d, 256)
    q, k, v, do = n(q_total, hq * d), n(k_total, hkv * d), n(k_total, hkv * d), n(q_total, hq * d)
    cq, ck = (torch.tensor([0, t // 2, t], dtype=torch.int32, device="cuda") for t in (q_total, k_total))

    def step():
        o, lse = att.attend(q, k, v, cq, ck)
        return o, *att.attend_bwd(q, k, v, o, lse, do, cq, ck)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for used in ((1.0, 1.0), (0.3, 0.5), (0.1, 0.9), (1.0, 0.4)):
        ql = [int(q_total * used[0] * 0.5), int(q_total * used[0] * 0.4)]
        kl = [int(k_total * used[1] * 0.4), int(k_total * used[1] * 0.5)]
        for c, l in ((cq, ql), (ck, kl)):
            c.copy_(torch.tensor([0, l[0], sum(l)], dtype=torch.int32))
        poison(q_total * hq * d, k_total * hkv * d)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        ref = R.attention(*(t.view(t.shape[0], -1, d) for t in (q, k, v)), ql, kl, att.scale, do.view(q_total, hq, d))
        for x, name, rows in zip(got, ("o", "dq", "dk", "dv"), (sum(ql), sum(ql), sum(kl), sum(kl))):
            R.assert_within(x.view(x.shape[0], -1, d), ref[name], ref[name + "_err"], name)
            assert (x[rows:] == 0).all()
        for x, y in zip(got, step()):
            assert torch.equal(x, y)
