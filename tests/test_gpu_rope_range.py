"""Head norms of rows whose squares leave binary32."""
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


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-6, 1e30])
def test_large_and_small_rows(dtype, d, eps):
    """Rows from 2^-100 to the largest numbers beside ordinary ones: the norm of
    each, forward and backward, within the bounds of ordinary rows (powers of
    two scale them exactly)."""
    powers = [0, 60, 64, 100, 120, 125, 1, -40, -60, -63, -70, -100, 0]
    tokens, hq, hkv = len(powers), 3, 1
    table = torch.empty(32, d // 2, 2, device="cuda")
    bl.bitlinear_rope_table(32, d, 10000.0, table)
    g = torch.Generator(device="cuda").manual_seed(1)
    by = (2.0 ** torch.tensor(powers, device="cuda", dtype=torch.float64))[:, None]

    def rows(h):
        return ((torch.rand(tokens, h * d, generator=g, device="cuda", dtype=torch.float64) * 6 - 3) * by).to(dtype)
    q, k = rows(hq), rows(hkv)
    assert torch.isfinite(q.float()).all()
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    pos = torch.arange(tokens, device="cuda", dtype=torch.int32)
    qo, ko = (torch.empty(tokens, h * d, dtype=BF, device="cuda") for h in (hq, hkv))
    bl.bitlinear_qk_rope(q, k, None, tokens, hq, hkv, d, *w, eps, table, pos, qo, ko, None)
    t = table.double()[pos.long()]
    c, s = t[..., 0], t[..., 1]
    eps32 = float(torch.tensor(eps, dtype=torch.float32))
    tiny = 2.0 ** -133  # half the smallest step of bf16, and results below its normal numbers
    for got, x, wt, h, n in ((qo, q, w[0], hq, "q"), (ko, k, w[1], hkv, "k")):
        y, err = R.rope(x.view(tokens, h, d), c, s, wt, eps32)
        R.assert_within(got.view(tokens, h, d), y, err + tiny, n)

    # gradients as large as the rows, so that dx (about dy / x) stays in range
    dq, dk = ((torch.randn(tokens, h * d, generator=g, device="cuda", dtype=torch.float64) * by.clamp(2.0 ** -90, 2.0 ** 90)
               ).to(BF) for h in (hq, hkv))
    for i in range(tokens):  # each alone: the weights' gradients differ by too much to be summed
        out = [torch.empty(1, hq * d, dtype=BF, device="cuda"), torch.empty(1, hkv * d, dtype=BF, device="cuda"),
               torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
        ws = torch.empty(bl.bitlinear_qk_rope_bwd_workspace_bytes(d), dtype=torch.uint8, device="cuda")
        one = [x[i:i + 1].contiguous() for x in (q, k, dq, dk)]
        bl.bitlinear_qk_rope_bwd(one[0], one[1], 1, hq, hkv, d, *w, eps, table, pos[i:i + 1].contiguous(), one[2], one[3],
                                 *out, ws=ws)
        for j, (h, n) in enumerate(((hq, "dq"), (hkv, "dk"))):
            dx, err, dw, dwe = R.rope_bwd(one[j].view(1, h, d), one[2 + j].view(1, h, d), c[i:i + 1], s[i:i + 1], w[j], eps32)
            R.assert_within(out[j].view(1, h, d), dx, err + tiny, f"{n} of 2^{powers[i]}")
            R.assert_within(out[2 + j], dw, dwe + tiny, f"{n} weight of 2^{powers[i]}")
