"""Layer norm of rows whose squares leave binary32 at the small end, where only a
tiny eps (or none) stands beside the variance."""
import numpy as np
import pytest
import torch

import _ffn_ref as R
from _gpu_ffn import TYPES, dev, empty, host
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
# one width for each way a row is held: a wavefront, four, workgroups that walk, the longest
SIZES = [(5, 8), (6, 1024), (9, 2560), (3, 4096), (1543, 4104), (3, 8192), (513, 12288), (2, 16384)]


def rows_of(rows, n, x, seed, scale):
    v = (np.random.default_rng(seed).normal(size=(rows, n)) + 0.5).astype(np.float32) * np.float32(scale)
    return R.bf16(v) if x == "bf16" else v


def check(v, x, eps, center):
    rows, n = v.shape
    Y, mean, rstd = empty(rows, n), empty(rows), empty(rows)
    bl.bitlinear_layernorm(dev(v, TYPES[x]), rows, n, None, None, eps, center, Y, mean=mean, rstd=rstd)
    ry, rm, rr = R.norm(v, None, None, float(np.float32(eps)), center)
    # the bounds of rows of ordinary size (a lane's 64 additions and a tree's nine, the mean's and the differences'
    # roundings, v_rsq_f32's ulp): scaling by a power of two changes no rounding
    E = 76 * R.U24 * (np.abs(v.astype("f8")).mean(1, keepdims=True) + np.abs(v))
    r = rr[:, None]
    tol = E * r + np.abs(ry) * (E.max(1, keepdims=True) * r + 45 * R.U24)
    assert np.all(np.abs(host(Y) - ry) <= tol * 1.01)
    assert np.all(np.abs(host(rstd) / rr - 1) <= E.max(1) * rr + 40 * R.U24)


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("x,center", [("f32", True), ("bf16", False), ("f32", False)])
def test_small_rows_without_eps(rows, n, x, center):
    for scale in (1e-17, 1e-19, 3e-20, 1e-23, 1e-34):
        check(rows_of(rows, n, x, n, scale), x, 0.0, center)


@pytest.mark.parametrize("eps", [1e-40, 1e-38, 1e-30])
def test_small_rows_beside_a_small_eps(eps):
    for scale in (1e-15, 1e-19, 1e-20):
        check(rows_of(4, 1024, "f32", 3, scale), "f32", eps, True)


def test_rows_of_different_sizes_side_by_side():
    """In one launch, ordinary rows keep the bits that they have by themselves."""
    for n in (512, 2560, 4104, 16384):
        v = rows_of(1030, n, "f32", n, 1.0)
        small = np.arange(1030) % 3 == 1
        v[small] *= np.float32(2.0 ** -70)
        check(v, "f32", 0.0, True)
        Y, Z = empty(1030, n), empty(int((~small).sum()), n)
        bl.bitlinear_layernorm(dev(v), 1030, n, None, None, 0.0, True, Y)
        bl.bitlinear_layernorm(dev(v[~small]), Z.shape[0], n, None, None, 0.0, True, Z)
        assert torch.equal(Y[torch.from_numpy(~small).cuda()], Z)


def test_backward_of_small_rows():
    n, rows = 1024, 6
    v = rows_of(rows, n, "f32", 9, 1e-23)
    Y, mean, rstd = empty(rows, n), empty(rows), empty(rows)
    bl.bitlinear_layernorm(dev(v), rows, n, None, None, 0.0, True, Y, mean=mean, rstd=rstd)
    dy = (1e-10 * np.random.default_rng(1).normal(size=(rows, n))).astype(np.float32)
    dX = empty(rows, n)
    bl.bitlinear_layernorm_bwd(dev(v), None, rows, n, None, mean, rstd, dev(dy), dX)
    m, r = host(mean).astype("f8"), host(rstd).astype("f8")
    want, _, _ = R.norm_bwd(v, None, m, r, dy, None, True)
    nx = np.abs((v.astype("f8") - m[:, None]) * r[:, None])
    a = np.abs(dy.astype("f8"))
    # as for ordinary rows: 76 and 78 half steps of the sums' sizes, n off by two roundings of x - mean and one of the product
    en = 2 * R.U24 * ((np.abs(v) + np.abs(m[:, None])) * r[:, None] + nx)
    sn = 78 * R.U24 * (a * nx).mean(1, keepdims=True) + (a * en).mean(1, keepdims=True)
    tol = nx * sn + en * (a * nx).mean(1, keepdims=True) + 76 * R.U24 * a.mean(1, keepdims=True)
    tol += 4 * R.U24 * (a + a.mean(1, keepdims=True) + nx * (a * nx).mean(1, keepdims=True))
    assert np.all(np.abs(host(dX) - want) <= (tol * r[:, None] + 3 * R.U24 * np.abs(want)) * 1.01)


def test_constant_rows():
    """Without eps a constant row has no variance: rstd is infinite and the row NaN; with the smallest eps it is zeros."""
    v = np.zeros((4, 256), np.float32)
    v[1], v[2] = 3.0, 1e-30
    Y, rstd = empty(4, 256), empty(4)
    bl.bitlinear_layernorm(dev(v), 4, 256, None, None, 0.0, True, Y, rstd=rstd)
    assert np.isnan(host(Y)).all() and np.isposinf(host(rstd)).all()
    bl.bitlinear_layernorm(dev(v), 4, 256, None, None, 1e-44, True, Y, rstd=rstd)
    eps = float(np.float32(1e-44))
    assert not host(Y).any() and np.all(np.abs(host(rstd) * eps ** 0.5 - 1) <= 4 * R.U24)
