"""Scores that are not a number show in everything attention returns for the
row: a -infinity in lse means that a row sees no key, and nothing else."""
import math

import pytest
import torch

import _gpu_helpers as H
from test_gpu_attn_scores import cu
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,k_lens", [([40], [200]), ([140, 30], [140, 10]), ([9], [4000])])
def test_not_a_number_in_a_row_of_q(d, q_lens, k_lens):
    hq, hkv, b = 4, 2, len(q_lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    tq, tk = sum(q_lens), sum(k_lens)
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(BF) for n, h in ((tq, hq), (tk, hkv), (tk, hkv)))
    q[5, 2, 3] = float("nan")
    o, lse = torch.full_like(q, 7.0), torch.full((hq, tq), 7.0, device="cuda")
    n = bl.bitlinear_attn_fwd_workspace_bytes(b, tq, tk, hq, hkv, d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    bl.bitlinear_attn_fwd(q, k, v, cu(q_lens), cu(k_lens), b, hq, hkv, d, 0.1, o, lse, ws=ws)
    bad = torch.zeros(hq, tq, dtype=torch.bool, device="cuda")
    bad[2, 5] = True
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(o).all(2).t(), bad) and torch.equal(torch.isnan(o).any(2).t(), bad)
    none = torch.zeros(hq, tq, dtype=torch.bool, device="cuda")
    if k_lens[-1] < q_lens[-1]:
        none[:, tq - q_lens[-1]:tq - k_lens[-1]] = True  # rows before the last sequence's first key
    assert torch.equal(lse == -math.inf, none)
