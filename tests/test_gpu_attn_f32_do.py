"""A binary32 output gradient (what bitlinear_bwd of the o BitLinear writes)
where keys and dK / dV tiles are shared out between workgroups."""
import pytest

import _gpu_helpers as H
from test_gpu_attn import check, inputs
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (6, 2, 128), (8, 1, 128)])
@pytest.mark.parametrize("q_lens,k_lens", [
    ([300, 129, 83], [300, 129, 83]),       # dK / dV tiles shared out
    ([130, 1, 33], [3000, 2500, 700]),      # keys shared out, some of them to parts of one sequence only
    ([1900], [1900]),
    ([40, 100], [4000, 20]),                # rows that see no key
])
def test_shared_out(hq, hkv, d, q_lens, k_lens):
    q, k, v, do = inputs(q_lens, k_lens, hq, hkv, d, seed=30, extra=5)
    do[sum(q_lens):] = float("nan")
    shared = bl.bitlinear_attn_fwd_workspace_bytes(len(q_lens), sum(q_lens) + 5, sum(k_lens) + 5, hq, hkv, d) > 0
    assert shared or q_lens[0] == 300
    check(q, k, v, do, q_lens, k_lens, do_f32=True)
