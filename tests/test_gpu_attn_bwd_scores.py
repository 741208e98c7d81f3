"""Gradients of attention with large scores: within the bounds of P's
roundings up to the largest |lse| that the backward takes, and NaN beyond it,
for the rows and keys concerned only.

Scores are exact (whole numbers), as in test_gpu_attn_scores.py.  P = 2^((S -
lse / scale) scale log2 e) is then off by the roundings of lse (three: the
product of the maximum, its sum with the logarithm, the factor ln 2), of its
quotient by the scale and of the two constants (three), and, where the
accumulators start from it, one for each of up to 2 * 8 partial sums of twice
that size: below 48 half steps of binary32 of |lse|."""
import math

import numpy as np
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from test_gpu_attn_scores import cu, whole
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
MOST = 65536.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def gradients(q, k, v, do, q_lens, k_lens, scale):
    tq, hq, d = q.shape
    tk, hkv = k.shape[:2]
    b = len(q_lens)
    o, lse = torch.empty_like(q), torch.empty(hq, tq, device="cuda")
    n = bl.bitlinear_attn_fwd_workspace_bytes(b, tq, tk, hq, hkv, d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    cq, ck = cu(q_lens), cu(k_lens)
    bl.bitlinear_attn_fwd(q, k, v, cq, ck, b, hq, hkv, d, scale, o, lse, ws=ws)
    out = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ws = torch.full((bl.bitlinear_attn_bwd_workspace_bytes(b, tq, tk, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    bl.bitlinear_attn_bwd(q, k, v, o, lse, do, cq, ck, b, hq, hkv, d, scale, *out, ws=ws)
    return out


def check(q, k, v, do, q_lens, k_lens, scale):
    """Every gradient of every row and key; returns how many rows were beyond the limit."""
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    g, scale, beyond = hq // hkv, float(np.float32(scale)), 0
    dq, dk, dv = gradients(q, k, v, do, q_lens, k_lens, scale)
    q, k, v, do = q.double(), k.double(), v.double(), do.double()
    for (q0, q1), (k0, k1) in zip(R.spans(q_lens), R.spans(k_lens)):
        nq, nk = q1 - q0, k1 - k0
        see = torch.ones(nq, nk, dtype=torch.bool, device="cuda").tril(nk - nq)
        for j in range(hkv):
            b, c = k[k0:k1, j], v[k0:k1, j]
            wk, ek, wv, ev = (torch.zeros(nk, d, dtype=torch.float64, device="cuda") for _ in range(4))
            lost = torch.zeros(nk, dtype=torch.bool, device="cuda")
            for h in range(j * g, j * g + g):
                a, w = q[q0:q1, h], do[q0:q1, h]
                x = torch.where(see, scale * (a @ b.t().contiguous()), -math.inf)
                lse = torch.logsumexp(x, 1)
                p = torch.where(see, torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None]), 0.0)
                size = torch.where(torch.isinf(lse), 0.0, lse.abs())[:, None]
                wild = size[:, 0] > MOST
                assert not ((size > MOST * 0.99) & (size < MOST * 1.01)).any(), "rows at the limit itself"
                beyond += int(wild.sum())
                lost |= (see & wild[:, None]).any(0)
                # relative error of P (rows beyond the limit reach no key that is compared: P is 0 there)
                ep = torch.expm1(48 * R.F32 * size.masked_fill(wild[:, None], 0.0)) + 64 * 2 * R.F32
                o, dp = p @ c, w @ c.t().contiguous()
                oe = (R.HALF + 2.0 ** -9) * (p @ c.abs()) + R.HALF * (1 + R.HALF) * o.abs()
                ds = p * (dp - (w * o).sum(1, keepdim=True))
                n32 = (max(nq * g, nk) + 64) * R.F32
                de = (w.abs() * oe).sum(1, keepdim=True) + (d + 8) * R.F32 * (w.abs() @ c.abs().t().contiguous())
                dse = ((1 + ep) * p * de + (R.HALF * (1 + R.HALF) + ep + n32) * ds.abs()) * (1 + R.HALF)
                want, err = scale * (ds @ b), scale * (dse @ b.abs()) * (1 + R.HALF) + R.HALF * (scale * (ds @ b)).abs()
                got = dq[q0:q1, h]
                assert torch.isnan(got[wild]).all(), "rows beyond the limit"
                R.assert_within(got[~wild], want[~wild], err[~wild], "dq")
                wk += scale * (ds.t() @ a)
                ek += scale * (dse.t() @ a.abs()) * (1 + R.HALF)
                wv += p.t() @ w
                ev += ((R.HALF + ep * (1 + R.HALF) + n32) * p).t() @ w.abs() * (1 + R.HALF)
            for got, want, err, n in ((dk, wk, ek, "dk"), (dv, wv, ev, "dv")):
                got = got[k0:k1, j]
                assert torch.isnan(got[lost]).all(), f"{n} of keys that rows beyond the limit see"
                R.assert_within(got[~lost], want[~lost], (err + R.HALF * want.abs())[~lost], n)
    return beyond


def inputs(q_lens, k_lens, hq, hkv, d):
    g = torch.Generator(device="cuda").manual_seed(1)
    tq, tk = sum(q_lens), sum(k_lens)
    return (whole(g, -4, 4, tq, hq, d), whole(g, -4, 4, tk, hkv, d),
            torch.randn(tk, hkv, d, generator=g, device="cuda").to(BF), torch.randn(tq, hq, d, generator=g, device="cuda").to(BF))


LENGTHS = [([100], [100]), ([300, 70], [300, 70]), ([40, 33], [2500, 1500])]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,k_lens", LENGTHS)
@pytest.mark.parametrize("scale", [0.125, 3.0, 40.0, 75.0])
def test_up_to_the_limit(d, q_lens, k_lens, scale):
    assert check(*inputs(q_lens, k_lens, 4, 2, d), q_lens, k_lens, scale) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,k_lens", LENGTHS)
@pytest.mark.parametrize("power", [10, 20, 40])
def test_beyond_the_limit(d, q_lens, k_lens, power):
    """The first 30 rows of the first sequence with one head's scores beyond it."""
    q, k, v, do = inputs(q_lens, k_lens, 4, 2, d)
    q[:30, 1] = (q[:30, 1].float() * 2.0 ** power).to(BF)
    k[:, :, 0] = k[:, :, 0].abs() + 1  # (no row's scores are all zero)
    q[:, :, 0] = q[:, :, 0].abs() + 2.0 ** power * (q[:, :, 0].abs() > 4)
    assert check(q, k, v, do, q_lens, k_lens, 4.0) > 0
