"""Layer norm on the GPU against its formulas in binary64."""
import numpy as np
import pytest
import torch

import _ffn_ref as R
from _gpu_ffn import TYPES, blocks, dev, empty, host
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
EPS = 1e-5

# Bounds.  A sum over a row adds at most 64 values of a lane one after the other,
# then 6 + 3 levels of a tree: relative to the sum of sizes its error is below
# 73 half steps; with the mean's division and the differences' roundings an
# x - mean is off by at most E = 76 2^-24 (mean|x| + |x|).  That puts the
# variance off by 2 E/sigma + 76 2^-24 of itself, rstd by half of that and 2^-23
# (v_rsq_f32 is good to 1 ulp), so n = (x - mean) rstd is off by at most
#   en = E rstd + |n| (E_max rstd + 40 2^-24).
def norm_bounds(x, mean, rstd):
    x = x.astype(np.float64)
    E = 76 * R.U24 * (np.abs(x).mean(1, keepdims=True) + np.abs(x))
    r = rstd[:, None]
    n = (x - mean[:, None]) * r
    return n, E * r + np.abs(n) * (E.max(1, keepdims=True) * r + 40 * R.U24)


def make(rows, n, x, seed, w=True, b=True):
    rng = np.random.default_rng(seed)
    v = (2 * rng.normal(size=(rows, n)) + 0.5 * rng.normal(size=n)).astype(np.float32)
    v = R.bf16(v) if x == "bf16" else v
    return (rng, v, (1 + 0.2 * rng.normal(size=n)).astype(np.float32) if w else None,
            (0.1 * rng.normal(size=n)).astype(np.float32) if b else None)


def opt(v):
    return None if v is None else dev(v)


def half_step(t):
    return torch.finfo(TYPES[t]).eps / 2


SIZES = [(1, 8), (5, 16), (3, 512), (9, 520), (6, 1024), (5, 1528), (4, 2048), (7, 2560), (3, 2568), (2, 4096), (3, 6144), (2, 6912),
         (3, 8192), (2, 8960), (2, 12288), (3, 16384)]


# more rows than the workgroups that walk over long ones
MANY = [(1543, 4104), (770, 6912), (1541, 8968), (513, 12288)]


@pytest.mark.parametrize("rows,n", SIZES + MANY)
@pytest.mark.parametrize("x,y,center,w,b", [("f32", "bf16", True, True, True), ("bf16", "f32", False, True, False),
                                            ("f32", "f32", True, False, True), ("bf16", "bf16", False, False, False)])
def test_forward(rows, n, x, y, center, w, b):
    rng, v, wt, bs = make(rows, n, x, rows + n, w, b)
    Y, mean, rstd = empty(rows, n, dtype=TYPES[y]), empty(rows), empty(rows)
    bl.bitlinear_layernorm(dev(v, TYPES[x]), rows, n, opt(wt), opt(bs), EPS, center, Y, mean=mean, rstd=rstd)
    ry, rm, rr = R.norm(v, wt, bs, EPS, center)
    nx, en = norm_bounds(v, rm, rr)
    wa = 1 if wt is None else np.abs(wt.astype(np.float64))
    tol = en * wa + 4 * R.U24 * (np.abs(nx) * wa + np.abs(ry)) + half_step(y) * np.abs(ry)
    assert np.all(np.abs(host(Y) - ry) <= tol * 1.01 + 1e-30)
    if center:
        assert np.all(np.abs(host(mean) - rm) <= 76 * R.U24 * np.abs(v).mean(1))
    else:
        assert not host(mean).any()
    E = 76 * R.U24 * (np.abs(v).mean(1) + np.abs(v).max(1))
    assert np.all(np.abs(host(rstd) / rr - 1) <= E * rr + 40 * R.U24)


@pytest.mark.parametrize("rows,n", [s for s in SIZES + MANY if s[1] % 16 == 0])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_forward_keeps_a_checkpoint(rows, n, x):
    _, v, wt, _ = make(rows, n, x, n)
    Y, codes, scales = empty(rows, n, dtype=torch.bfloat16), empty(rows, n, dtype=torch.int8), empty(rows, blocks(n))
    bl.bitlinear_layernorm(dev(v, TYPES[x]), rows, n, dev(wt), None, EPS, False, Y, codes=codes, scales=scales)
    c, s = R.ckpt(v)
    assert np.array_equal(host(codes), c) and np.array_equal(host(scales), s)
    Z = empty(rows, n, dtype=torch.bfloat16)
    bl.bitlinear_layernorm(dev(v, TYPES[x]), rows, n, dev(wt), None, EPS, False, Z)
    assert torch.equal(Y, Z)


BACKWARD = [
    ("f32", "bf16", "f32", True, True, True, True), ("bf16", "f32", "bf16", False, True, False, False),
    ("q8", "bf16", "bf16", True, False, True, True), ("q8", "f32", "f32", False, True, True, False)]


@pytest.mark.parametrize("rows,n,x,dy,dx,center,w,b,res", [
    (*size, *kind) for kind in BACKWARD for size in SIZES + [(600, 64), (2100, 128), (1300, 2576), (700, 8208)]
    if kind[0] != "q8" or size[1] % 16 == 0])  # (a checkpoint's rows are multiples of 16)
def test_backward(rows, n, x, dy, dx, center, w, b, res):
    rng, v, wt, _ = make(rows, n, "f32" if x == "q8" else x, rows + n, w, False)
    _, rm, rr = R.norm(v, None, None, EPS, center)
    mean, rstd = rm.astype(np.float32), rr.astype(np.float32)
    g = rng.normal(size=(rows, n)).astype(np.float32)
    g = R.bf16(g) if dy == "bf16" else g
    dr = None
    if res:
        dr = rng.normal(size=(rows, n)).astype(np.float32)
        dr = R.bf16(dr) if dx == "bf16" else dr
    X, xs, seen = dev(v, TYPES[x]) if x != "q8" else None, None, v
    if x == "q8":
        c, s = R.ckpt(v)
        X, xs, seen = torch.from_numpy(c).cuda(), dev(s), R.ckpt_values(c, s)
    dX, dw, db = empty(rows, n, dtype=TYPES[dx]), empty(n, fill=7.0), empty(n, fill=7.0)
    args = (X, xs, rows, n, opt(wt), dev(mean) if center else None, dev(rstd), dev(g, TYPES[dy]))
    dR = None if dr is None else dev(dr, TYPES[dx])
    ws = torch.empty(bl.bitlinear_layernorm_bwd_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    bl.bitlinear_layernorm_bwd(*args, dX, dw, db if b else None, dR=dR, ws=ws)
    rx, rw, rb = R.norm_bwd(seen, wt, mean.astype(np.float64), rstd.astype(np.float64), g, dr, center)
    # n from the given mean and rstd: two roundings of x - mean (|x| + |mean| at most) and of the product
    nx = (seen.astype(np.float64) - mean[:, None]) * rstd[:, None]
    en = 2 * R.U24 * ((np.abs(seen) + np.abs(mean[:, None])) * rstd[:, None] + np.abs(nx))
    a = np.abs(g.astype(np.float64) * (1 if wt is None else wt))
    # sums over a row: 76 half steps of the sizes, and en in the second
    sa = 76 * R.U24 * a.mean(1, keepdims=True) if center else 0
    sn = 78 * R.U24 * (a * np.abs(nx)).mean(1, keepdims=True) + (a * en).mean(1, keepdims=True)
    tol = np.abs(nx) * sn + en * (a * np.abs(nx)).mean(1, keepdims=True) + sa + 4 * R.U24 * (
        a + a.mean(1, keepdims=True) + np.abs(nx) * (a * np.abs(nx)).mean(1, keepdims=True))
    tol = tol * rstd[:, None] + (half_step(dx) + 2 * R.U24) * np.abs(rx) + (0 if dr is None else R.U24 * np.abs(dr))
    assert np.all(np.abs(host(dX) - rx) <= tol * 1.01 + 1e-30)
    # the parameters: at most ceil(rows / workgroups) + 5 additions in binary32, then binary64 and one rounding
    adds = rows / 256 + 8
    ga = np.abs(g.astype(np.float64))
    assert np.all(np.abs(host(dw) - rw) <= (adds + 1) * R.U24 * (ga * np.abs(nx)).sum(0) + (ga * en).sum(0) + 1e-30)
    if b:
        assert np.all(np.abs(host(db) - rb) <= (adds + 1) * R.U24 * ga.sum(0) + 1e-30)
    else:
        assert (db == 7).all()
    # reruns give the same bits, and dX does not depend on the sums being asked for
    d2, w2 = empty(rows, n, dtype=TYPES[dx]), empty(n)
    bl.bitlinear_layernorm_bwd(*args, d2, w2, None, dR=dR, ws=ws)
    assert torch.equal(dX, d2) and torch.equal(dw, w2)
    bl.bitlinear_layernorm_bwd(*args, d2.zero_(), dR=dR)
    assert torch.equal(dX, d2)


def test_large_mean_and_constant_rows():
    """Differences are formed before squares: a row far from zero keeps its
    variance, a constant row gives bias where eps holds the scale."""
    n = 1024
    v = np.zeros((3, n), np.float32)
    v[0] = 4096 + np.arange(n) % 2
    v[1] = 3
    Y, rstd = empty(3, n), empty(3)
    bl.bitlinear_layernorm(dev(v), 3, n, None, dev(np.full(n, 0.25)), EPS, True, Y, rstd=rstd)
    y = host(Y)
    assert np.all(np.abs(y[0] - 0.25 - np.where(np.arange(n) % 2, 1, -1) / np.sqrt(1 + 4 * EPS)) < 1e-5)
    assert np.array_equal(y[1:], np.full((2, n), 0.25, np.float32))


def test_rows_outside_binary32_are_nan():
    v = np.ones((3, 64), np.float32)
    v[0, 0], v[1, 1] = 1e30, np.nan
    Y = empty(3, 64)
    bl.bitlinear_layernorm(dev(v), 3, 64, None, None, EPS, True, Y)
    assert np.isnan(host(Y)[:2]).all() and not host(Y)[2].any()


def test_strided_rows_and_neighbours():
    wide = torch.randn(7, 3000, device="cuda").bfloat16()
    x = wide[:, 64:64 + 1520]
    Y, Z = empty(9, 1520, dtype=torch.bfloat16, fill=5.0), empty(7, 1520, dtype=torch.bfloat16)
    rstd = empty(7)
    bl.bitlinear_layernorm(x, 7, 1520, None, None, EPS, False, Y[:7], rstd=rstd)
    bl.bitlinear_layernorm(x.contiguous(), 7, 1520, None, None, EPS, False, Z)
    assert torch.equal(Y[:7], Z) and (Y[7:] == 5).all()
    dy = torch.randn(7, 1520, device="cuda")
    d1, d2 = empty(9, 1520, fill=5.0), empty(7, 1520)
    bl.bitlinear_layernorm_bwd(x, None, 7, 1520, None, None, rstd, dy, d1[:7])
    bl.bitlinear_layernorm_bwd(x.contiguous(), None, 7, 1520, None, None, rstd, dy, d2)
    assert torch.equal(d1[:7], d2) and (d1[7:] == 5).all()


def test_no_rows():
    x, Y = empty(0, 64), empty(0, 64)
    bl.bitlinear_layernorm(x, 0, 64, None, None, EPS, False, Y)
    dw, db = empty(64, fill=3.0), empty(64, fill=3.0)
    bl.bitlinear_layernorm_bwd(x, None, 0, 64, None, None, empty(0), Y, x, dw, db)
    assert not dw.any() and not db.any()


def test_refusals_of_tensors():
    x, Y, rstd = empty(4, 64), empty(4, 64), empty(4)
    with pytest.raises(TypeError):
        bl.bitlinear_layernorm(x.double(), 4, 64, None, None, EPS, False, Y)
    with pytest.raises(ValueError):
        bl.bitlinear_layernorm(x, 4, 64, empty(32), None, EPS, False, Y)
    with pytest.raises(ValueError):
        bl.bitlinear_layernorm(x, 4, 64, None, None, EPS, False, Y.cpu())
    with pytest.raises(TypeError):
        bl.bitlinear_layernorm_bwd(x, None, 4, 64, None, None, rstd, Y, empty(4, 64), dR=empty(4, 64, dtype=torch.bfloat16))
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_layernorm_bwd(empty(4, 64, dtype=torch.int8), None, 4, 64, None, None, rstd, Y, empty(4, 64))
