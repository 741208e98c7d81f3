"""Attention whose scores are large: the exponents of a softmax are differences
of scores, however large the scores are.

Q and K hold small whole numbers (times a power of two), so every product
Q K^T is exact in binary32 and in binary64, and what is compared is the
softmax alone.  Its exponents are then off by
  - half a step of binary32 for each of (x - m) and its product with the scale:
    a term that does not vanish has an exponent of at most 150, so 2^-15 of it;
  - 2^-24 of the scores themselves as long as those are at most 2^12 (in
    exponents of 2), once for either of two maxima: 2^-11 together.
es = 2^-10 covers both as a relative error of P."""
import math

import numpy as np
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ES = 2.0 ** -10
SCALES = [0.5, 300.0, 1e6, 1e8, 1e10, 1e20, 1e30]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def cu(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def whole(gen, low, high, *shape):
    return torch.randint(low, high + 1, shape, generator=gen, device="cuda").to(BF)


def softmax_rows(q, k, v, see, scale):
    """(O, bound, lse) of one head in 64 bits; see [nq, nk].  The scale is the
    binary32 number that the library takes."""
    scale = float(np.float32(scale))
    x = q.double() @ k.double().t().contiguous()
    x = torch.where(see, x, -math.inf)
    m = x.max(1, keepdim=True).values if x.shape[1] else torch.full((x.shape[0], 1), -math.inf, device=x.device)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = torch.exp((x - m) * scale)
    z = p.sum(1, keepdim=True)
    p = p / torch.where(z > 0, z, 1)
    o = p @ v.double()
    lse = torch.where(z > 0, m * scale + z.log(), -math.inf)[:, 0]
    # P and its sum, P's rounding to bf16, O's rounding
    return o, (R.HALF + 2 * ES) * (p @ v.double().abs()) + R.HALF * (1 + R.HALF) * o.abs(), lse


def check_packed(q, k, v, q_lens, k_lens, scale):
    tq, hq, d = q.shape
    tk, hkv = k.shape[:2]
    b = len(q_lens)
    o, lse = torch.full_like(q, 7.0), torch.full((hq, tq), 7.0, device="cuda")
    n = bl.bitlinear_attn_fwd_workspace_bytes(b, tq, tk, hq, hkv, d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    bl.bitlinear_attn_fwd(q, k, v, cu(q_lens), cu(k_lens), b, hq, hkv, d, scale, o, lse, ws=ws)
    for (q0, q1), (k0, k1) in zip(R.spans(q_lens), R.spans(k_lens)):
        see = torch.ones(q1 - q0, k1 - k0, dtype=torch.bool, device="cuda").tril(k1 - k0 - (q1 - q0))
        for h in range(hq):
            g = h // (hq // hkv)
            want, err, wl = softmax_rows(q[q0:q1, h], k[k0:k1, g], v[k0:k1, g], see, scale)
            R.assert_within(o[q0:q1, h], want, err, "O")
            # m scale, the logarithm's sum and the factors ln 2, log2 e: six half steps
            bound = 2 * ES + 6 * R.F32 * torch.where(torch.isinf(wl), 0.0, wl.abs())
            R.assert_within(lse[h, q0:q1], wl, bound, "lse")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("q_lens,k_lens", [
    ([150, 1, 40], [150, 1, 40]),
    ([700], [700]),
    ([5, 70], [3000, 1500]),      # keys shared out between workgroups
    ([90, 3], [30, 200]),         # rows that see no key
])
def test_forward(d, scale, q_lens, k_lens):
    g = torch.Generator(device="cuda").manual_seed(1)
    hq, hkv = 4, 2
    q, k = whole(g, -4, 4, sum(q_lens), hq, d), whole(g, -4, 4, sum(k_lens), hkv, d)
    v = torch.randn(sum(k_lens), hkv, d, generator=g, device="cuda").to(BF)
    check_packed(q, k, v, q_lens, k_lens, scale)


@pytest.mark.parametrize("scale", [1.0, 1e6, 1e30])
def test_forward_of_scores_below_zero(scale):
    """Every score far below zero, and maxima that rise from there to far above."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k = whole(g, 1, 4, 300, 2, 64), whole(g, -4, -1, 300, 1, 64)
    v = torch.randn(300, 1, 64, generator=g, device="cuda").to(BF)
    check_packed(q, k, v, [300], [300], scale)
    up = (torch.arange(300, device="cuda") // 4 - 30).to(BF)[:, None, None].expand(300, 1, 64).contiguous()
    check_packed(q, up, v, [300], [300], scale)


@pytest.mark.parametrize("power", [10, 20, 55])
def test_forward_of_large_values(power):
    """Large rows of Q at an ordinary scale."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = whole(g, -4, 4, 200, 2, 128), whole(g, -4, 4, 200, 1, 128)
    v = torch.randn(200, 1, 128, generator=g, device="cuda").to(BF)
    check_packed((q.float() * 2.0 ** power).to(BF), (k.float() * 2.0 ** power).to(BF), v, [200], [200], 0.125)
