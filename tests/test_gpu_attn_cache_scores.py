"""Attention over a paged cache whose scores are large (exact products of
whole numbers, so that the softmax alone is compared)."""
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from test_gpu_attn_scores import SCALES, softmax_rows, whole
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("hq,hkv,d,draft,lens", [
    (4, 2, 64, 1, [1, 33, 700]), (16, 2, 128, 1, [5000]), (8, 1, 128, 7, [7, 40, 900]), (4, 4, 64, 40, [41, 3000]),
])
def test_large_scores(scale, hq, hkv, d, draft, lens):
    page, batch = 16, len(lens)
    g = torch.Generator(device="cuda").manual_seed(4)
    per = -(-max(lens) // page)
    q, v = whole(g, -4, 4, batch * draft, hq, d), torch.randn(batch * per * page, hkv, d, generator=g, device="cuda").to(BF)
    k = whole(g, -4, 4, batch * per * page, hkv, d)
    pages = torch.randperm(batch * per, generator=g, device="cuda").int().view(batch, per).contiguous()
    o = torch.full_like(q, 7.0)
    ws = torch.full((bl.bitlinear_attn_cache_workspace_bytes(batch, draft, hq, hkv, d),), 255, dtype=torch.uint8,
                    device="cuda")
    bl.bitlinear_attn_cache(q, k, v, pages, page, torch.tensor(lens, dtype=torch.int32, device="cuda"), None, batch, draft,
                            hq, hkv, d, scale, o, ws=ws)
    for b, n in enumerate(lens):
        rows = (pages[b].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        see = torch.ones(draft, n, dtype=torch.bool, device="cuda").tril(n - draft)
        for h in range(hq):
            i = h // (hq // hkv)
            want, err, _ = softmax_rows(q[b * draft:(b + 1) * draft, h], k[rows, i], v[rows, i], see, scale)
            R.assert_within(o[b * draft:(b + 1) * draft, h], want, err, "O")
