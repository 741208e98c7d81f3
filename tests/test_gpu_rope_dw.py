"""The norm weights' gradients within what their summation allows."""
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
import _rope_dw_ref as W
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("tokens,hq,hkv,d", [(5000, 8, 2, 128), (3071, 14, 2, 64), (700, 40, 4, 128), (1, 3, 1, 64),
                                             (20000, 2, 1, 64), (257, 1, 1, 128)])
def test_weight_gradients(tokens, hq, hkv, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    n = lambda h: torch.randn(tokens, h * d, generator=g, device="cuda")  # noqa: E731
    q, k, dq, dk = n(hq).to(dtype), n(hkv).to(dtype), n(hq).to(BF), n(hkv).to(BF)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    pos = torch.randint(0, 4096, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.empty(4096, d // 2, 2, device="cuda")
    bl.bitlinear_rope_table(4096, d, 10000.0, table)
    out = [torch.empty_like(dq), torch.empty_like(dk), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    ws = torch.full((bl.bitlinear_qk_rope_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    bl.bitlinear_qk_rope_bwd(q, k, tokens, hq, hkv, d, *w, EPS, table, pos, dq, dk, *out, ws=ws)
    t = table.double()[pos.long()]
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    for x, dy, h, got in ((q, dq, hq, out[2]), (k, dk, hkv, out[3])):
        dw, err = W.weight_gradient(x.view(tokens, h, d), dy.view(tokens, h, d), t[..., 0], t[..., 1], eps, hq + hkv)
        R.assert_within(got, dw, err, "weight gradient")
