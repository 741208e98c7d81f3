"""Sequence offsets outside the buffers are cut off there: every row of every
output, forward and backward."""
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cq,q_lens,ck,k_lens", [
    # (offsets given, lengths that remain; total_q 230 and total_k 300)
    ([-5, 40, 1 << 30], [40, 190], [-7, 40, 1 << 30], [40, 260]),
    ([-(1 << 31), 0, 200, (1 << 31) - 1], [0, 200, 30], [0, 130, 299, 5000], [130, 169, 1]),
    ([-3, -1, 230, 231], [0, 230, 0], [-3, 150, 300, 301], [150, 150, 0]),
    ([0, 230, 1 << 20], [230, 0], [0, 1 << 20, 1 << 21], [300, 0]),
])
def test_every_row(d, cq, q_lens, ck, k_lens):
    hq, hkv, tq, tk, b, scale = 4, 2, 230, 300, len(q_lens), 0.1
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda t, h: torch.randn(t, h, d, generator=g, device="cuda").to(BF)  # noqa: E731
    # what lies around the buffers is theirs too: rows before and behind in one allocation, left alone
    pad = 64
    whole = [torch.full((t + 2 * pad, h, d), float("nan"), dtype=BF, device="cuda") for t, h in
             ((tq, hq), (tk, hkv), (tk, hkv), (tq, hq))]
    q, k, v, do = (t[pad:-pad] for t in whole)
    for t, x in zip((q, k, v, do), (n(tq, hq), n(tk, hkv), n(tk, hkv), n(tq, hq))):
        t.copy_(x)
    outs = [torch.full((t + 2 * pad, h, d), 7.0, dtype=BF, device="cuda") for t, h in ((tq, hq), (tq, hq), (tk, hkv), (tk, hkv))]
    o, dq, dk, dv = (t[pad:-pad] for t in outs)
    lse = torch.full((hq + 2, tq), 7.0, device="cuda")
    cqt, ckt = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cq, ck))
    nf = bl.bitlinear_attn_fwd_workspace_bytes(b, tq, tk, hq, hkv, d)
    ws = torch.full((nf,), 255, dtype=torch.uint8, device="cuda") if nf else None
    bl.bitlinear_attn_fwd(q, k, v, cqt, ckt, b, hq, hkv, d, scale, o, lse[1:-1], ws=ws)
    ws = torch.full((bl.bitlinear_attn_bwd_workspace_bytes(b, tq, tk, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    bl.bitlinear_attn_bwd(q, k, v, o, lse[1:-1], do, cqt, ckt, b, hq, hkv, d, scale, dq, dk, dv, ws=ws)
    ref = R.attention(q, k, v, q_lens, k_lens, scale, do)
    assert sum(q_lens) == tq and sum(k_lens) == tk
    for x, name in ((o, "o"), (lse[1:-1], "lse"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        assert not torch.isnan(ref[name]).any()
        R.assert_within(x, ref[name], ref[name + "_err"], name)
    for t in outs:
        assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()
    assert (lse[0] == 7).all() and (lse[-1] == 7).all()
