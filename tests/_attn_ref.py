"""Plain 64-bit forms of the attention-side operators, with the error bounds
their roundings allow, for the tests.  Written from the definitions in
include/bitlinear.h; shares nothing with the kernels."""
import math

import torch

HALF = 2.0 ** -8     # half a step of bf16, relative
F32 = 2.0 ** -24     # half a step of binary32, relative


def spans(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def attention(q, k, v, q_lens, k_lens, scale, do=None, do_f32=False):
    """q [tq, hq, d], k and v [tk, hkv, d] (any float type, rows of sequences
    only are read) -> dict of 64-bit results and, under "<name>_err", the
    largest error the kernel's roundings can cause:
      P and dS are rounded to bf16 (HALF of each term), O once more; delta is
      formed from the rounded O; a binary32 dO is rounded to bf16; binary32
      sums of n terms are off by at most n * F32 of their absolute terms, and
      a score error e changes P by a factor exp(e)."""
    q, k, v = q.double(), k.double(), v.double()
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    g = hq // hkv
    z = lambda x: torch.full_like(x, float("nan"))  # noqa: E731
    r = {"o": z(q), "o_err": z(q), "lse": z(q[..., 0].t().contiguous()), "lse_err": z(q[..., 0].t().contiguous())}
    if do is not None:
        do = do.double()
        r |= {"dq": z(q), "dq_err": z(q), "dk": z(k), "dk_err": z(k), "dv": z(v), "dv_err": z(v)}
    dorel = HALF if do_f32 else 0.0
    for (q0, q1), (k0, k1) in zip(spans(q_lens), spans(k_lens)):
        nq, nk = q1 - q0, k1 - k0
        if do is not None and nk:
            for n in ("dk", "dk_err", "dv", "dv_err"):
                r[n][k0:k1] = 0
        if not nq:
            continue
        see = torch.ones(nq, nk, dtype=torch.bool, device=q.device).tril(nk - nq)
        for h in range(hq):
            a, b, c, i = q[q0:q1, h], k[k0:k1, h // g], v[k0:k1, h // g], h
            s = torch.where(see, scale * (a @ b.t()), -math.inf)
            sabs = (scale * (a.abs() @ b.abs().t())).max() if nk else torch.zeros((), dtype=torch.float64)
            es = float(F32 * ((d + 8) * sabs)) * 4 + (nk + 64) * F32 * 2  # relative error of P and of its sum
            empty = ~see.any(1) if nk else torch.ones(nq, dtype=torch.bool, device=q.device)
            lse = torch.logsumexp(s, 1) if nk else torch.full((nq,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.where(see, torch.exp(s - torch.where(empty, 0.0, lse)[:, None]), 0.0)
            o, oabs = p @ c, p @ c.abs()
            oe = (HALF + es) * oabs + HALF * (1 + HALF) * o.abs()
            r["o"][q0:q1, i], r["o_err"][q0:q1, i] = o, oe
            r["lse"][i, q0:q1] = lse
            r["lse_err"][i, q0:q1] = es + 8 * F32 * (1 + torch.where(empty, 0.0, lse).abs() + float(sabs))
            if do is None or not nk:
                if do is not None:
                    r["dq"][q0:q1, i] = r["dq_err"][q0:q1, i] = 0
                continue
            w = do[q0:q1, i]
            wv = w.abs() @ c.abs().t()
            dp = w @ c.t()
            delta = (w * o).sum(1, keepdim=True)
            # delta: O's error, dO's rounding and the binary32 sum
            de = (w.abs() * (1 + dorel) * oe).sum(1, keepdim=True) + (dorel + (d + 8) * F32) * (w * o).abs().sum(1, keepdim=True)
            ds = p * (dp - delta)
            dse = p * (de + (dorel + (d + 8) * F32) * wv) + (HALF + es + HALF * HALF + 4 * F32) * ds.abs()
            dse = dse * (1 + HALF)
            n32 = (max(nq * g, nk) + 64) * F32
            r["dq"][q0:q1, i] = scale * (ds @ b)
            r["dq_err"][q0:q1, i] = scale * ((dse + n32 * ds.abs()) @ b.abs()) * (1 + HALF) + HALF * (scale * (ds @ b)).abs()
            r["dk"][k0:k1, h // g] += scale * (ds.t() @ a)
            r["dk_err"][k0:k1, h // g] += scale * ((dse + n32 * ds.abs()).t() @ a.abs()) * (1 + HALF)
            r["dv"][k0:k1, h // g] += p.t() @ w
            r["dv_err"][k0:k1, h // g] += ((HALF + dorel + HALF * dorel + es + n32) * p).t() @ w.abs() * (1 + HALF)
        if do is not None and nk:
            r["dk_err"][k0:k1] += HALF * r["dk"][k0:k1].abs()
            r["dv_err"][k0:k1] += HALF * r["dv"][k0:k1].abs()
    return r


def assert_within(got, want, err, what):
    """Elementwise |got - want| <= err, infinities equal, where want is not NaN."""
    got = got.double()
    there = ~torch.isnan(want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf & there], want[inf & there]), f"{what}: infinities"
    ok = there & ~inf
    over = (got - want).abs() - err
    bad = ok & ~(over <= 1e-30)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {int(ok.sum())} values off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()}, bound {err[bad][0].item()}")


def rope(x, cos, sin, w, eps):
    """x [t, h, d] -> (y, bound of its error).  cos, sin [t, d/2] 64-bit copies
    of the binary32 table.  binary32 arithmetic: the mean of squares is a tree
    of d terms, its root one instruction of 1 ulp, then three products and a
    sum: fewer than 32 half steps of each term in all; y is rounded once."""
    x = x.double()
    half = x.shape[-1] // 2
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    a, b = x[..., :half], x[..., half:]
    c, s = cos[:, None], sin[:, None]
    y = torch.cat((a * c - b * s, b * c + a * s), -1)
    m = torch.cat((a.abs() + b.abs(),) * 2, -1)
    return y, HALF * (1 + HALF) * y.abs() + 32 * F32 * m


def rope_bwd(x, dy, cos, sin, w, eps):
    """(dx, bound, dw, bound) of `rope` for one side."""
    dy = dy.double()
    half = dy.shape[-1] // 2
    a, b = dy[..., :half], dy[..., half:]
    c, s = cos[:, None], sin[:, None]
    g = torch.cat((a * c + b * s, b * c - a * s), -1)
    gabs = torch.cat((a.abs() + b.abs(),) * 2, -1)
    if w is None:
        return g, HALF * (1 + HALF) * g.abs() + 8 * F32 * gabs, None, None
    x = x.double()
    d = x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    dw = (g * n).sum((0, 1))
    # products good to 32 half steps; each wavefront's binary32 sum has at
    # most rows / 1 terms per lane, bounded here by all rows
    rows = dy.shape[0] * dy.shape[1]
    dwe = ((gabs * n.abs()).sum((0, 1))) * F32 * (32 + min(rows, 4096))
    v = w.double() * g
    vabs = w.double().abs() * gabs
    dx = r * (v - n * (v * n).mean(-1, keepdim=True))
    m = r * (vabs + n.abs() * (vabs * n.abs()).mean(-1, keepdim=True))
    return dx, HALF * (1 + HALF) * dx.abs() + 64 * F32 * m + d * F32 * m, dw, dwe
