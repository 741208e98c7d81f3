"""Feed-forward side of a block in numpy: the formulas in binary64, and the
bit-exact steps (checkpoints, G, U, squared-ReLU gating, the bf16 operands of
the backward) in binary32 as they are defined."""
import numpy as np

U24 = 2.0 ** -24   # half a step of binary32
UBF = 2.0 ** -8    # half a step of bf16
BLOCK = 64
F32 = np.float32


def bf16(x):
    """binary32 values rounded to bf16 (nearest, ties to even), as binary32."""
    b = np.ascontiguousarray(x, dtype=F32).view(np.uint32)
    r = ((b + np.uint32(0x7fff) + ((b >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xffff0000)).view(F32)
    return np.where(np.isnan(x), F32(np.nan), r)


# ------------------------------------------------------------ checkpoints

def ckpt(x):
    """(codes, scales) of binary32 rows; the products are formed in binary64,
    where they are exact, so each code is rounded once."""
    rows, n = x.shape
    nb = -(-n // BLOCK)
    p = np.zeros((rows, nb * BLOCK), F32)
    p[:, :n] = x
    p = p.reshape(rows, nb, BLOCK)
    with np.errstate(all="ignore"):
        a = np.abs(p).max(-1)  # numpy's max keeps a NaN
        bad, small = ~np.isfinite(a), a < F32(2.0 ** -100)
        inv = np.where(bad | small, F32(0), F32(127) / np.where(small, F32(1), a)).astype(F32)
        scale = np.where(bad, F32(np.nan), np.where(small, F32(0), a / F32(127))).astype(F32)
        q = np.rint(p.astype(np.float64) * inv[..., None].astype(np.float64))
    q = np.where(bad[..., None], 0, q)  # codes of a block that comes back as NaN do not matter
    return q.reshape(rows, -1)[:, :n].astype(np.int8), scale


def ckpt_values(codes, scales):
    s = np.repeat(scales, BLOCK, axis=1)[:, :codes.shape[1]]
    return codes.astype(F32) * s


# ---------------------------------------------------------------- the norm

def norm(x, w, b, eps, center):
    """(y, mean, rstd) in binary64."""
    x = x.astype(np.float64)
    mean = x.mean(1) if center else np.zeros(x.shape[0])
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    y = y * (1 if w is None else w) + (0 if b is None else b)
    return y, mean, rstd


def norm_bwd(x, w, mean, rstd, dy, dr, center):
    """(dx, dweight, dbias) in binary64."""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    n = (x - mean[:, None]) * rstd[:, None]
    a = dy * (1 if w is None else w)
    dx = a - n * (a * n).mean(1, keepdims=True)
    if center:
        dx = dx - a.mean(1, keepdims=True)
    dx = dx * rstd[:, None] + (0 if dr is None else dr)
    return dx, (dy * n).sum(0), dy.sum(0)


# -------------------------------------------------------------- the gating

def act(g, kind):
    """act(g) and its derivative in binary64."""
    g = g.astype(np.float64)
    if kind == "relu2":
        r = np.maximum(g, 0)
        return r * r, 2 * r
    z = 1 / (1 + np.exp(-g))
    return g * z, z * (1 + g * (1 - z))


def project(xq, xs, codes, gamma):
    """binary32 outputs of a BitLinear, bit for bit: exact sums, gamma s_t
    rounded once, the product rounded once."""
    acc = xq.astype(np.float64) @ codes.astype(np.float64).T  # exact: below 2^53
    return acc.astype(F32) * (gamma * xs.astype(np.float64)).astype(F32)[:, None]


def relu2_h(g, u):
    r = np.maximum(g, F32(0))
    return bf16((r * r) * u)


def glu_bwd(dh, g, u, kind, xq, xs, codes, gammas):
    """(dX, dW_gate, dW_up) in binary64, each with the sum of its terms' sizes."""
    value, slope = act(g, kind)
    dh, u = dh.astype(np.float64), u.astype(np.float64)
    du, dg = dh * value, dh * u * slope
    x, s = xq.astype(np.float64), xs.astype(np.float64)[:, None]
    c = [m.astype(np.float64) for m in codes]
    dx = dg * gammas[0] @ c[0] + du * gammas[1] @ c[1]
    sizes = np.abs(dg * gammas[0]) @ np.abs(c[0]) + np.abs(du * gammas[1]) @ np.abs(c[1])
    out = [(dx, sizes)]
    for d in (dg, du):
        out.append(((d * s).T @ x, np.abs(d * s).T @ np.abs(x)))
    return out


def relu2_operands(dh, g, u, xs, gammas):
    """The four bf16 operands of squared ReLU's backward, bit for bit: products
    in binary32, each rounded, in the order dh act, (dh u) slope."""
    r = np.maximum(g, F32(0))
    du, dg = dh * (r * r), (dh * u) * (F32(2) * r)
    s = xs[:, None].astype(F32)
    return [bf16(dg * F32(gammas[0])), bf16(du * F32(gammas[1])), bf16(dg * s), bf16(du * s)]
