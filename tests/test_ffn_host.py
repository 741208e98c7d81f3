"""Refusals and sizes of the feed-forward side's entry points: arguments are
checked on the host before anything is enqueued, so no GPU is needed."""
import os

import pytest

from sparse_linear_layers_group_amd import bitlinear as bl

A = 4096  # an aligned address, never dereferenced
B = 4100  # 4-byte aligned only
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bl.LIB_PATH):
        from sparse_linear_layers_group_amd import build
        build.build()
    return bl.lib()


def call(f, defaults, kw):
    a = dict(defaults, **kw)
    assert set(a) == set(defaults), set(a) - set(defaults)
    return f(*a.values())


PACK = dict(X=A, x_type=0, x_stride=64, rows=4, n=64, codes=A, scales=A, stream=None)
UNPACK = dict(codes=A, scales=A, rows=4, n=64, Y=A, y_type=0, stream=None)
NORM = dict(X=A, x_type=0, x_stride=64, rows=4, n=64, weight=A, bias=A, eps=1e-6, center=1, Y=A, y_type=1, mean=A, rstd=A,
            codes=A, scales=A, stream=None)
NORM_BWD = dict(X=A, x_type=0, x_scales=None, x_stride=64, rows=4, n=64, weight=A, mean=A, rstd=A, dY=A, dy_type=1, dR=A,
                dX=A, dx_type=0, dweight=A, dbias=A, ws=A, ws_bytes=BIG, stream=None)
GLU = dict(xq=A, x_scale=A, tokens=4, k=256, gate=A, gate_gamma=A, up=A, up_gamma=A, n_out=128, n=6, m=8, act=0, H=A,
           save_type=2, G=A, G_scales=A, U=A, U_scales=A, ws=A, ws_bytes=BIG, stream=None)
GLU_BWD = dict(dH=A, dh_type=0, save_type=2, G=A, G_scales=A, U=A, U_scales=A, xq=A, x_scale=A, gate=A, gate_gamma=A, up=A,
               up_gamma=A, tokens=4, k=256, n_out=128, n=6, m=8, act=0, grad_type=0, dX=A, dW_gate=A, dW_up=A, ws=A,
               ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(x_type=2), bl.BL_EINVAL, "x_type"), (dict(n=8, x_stride=8), bl.BL_ESHAPE, "multiple of 16"),
    (dict(n=0), bl.BL_ESHAPE, "multiple of 16"), (dict(rows=-1), bl.BL_ESHAPE, "rows"),
    (dict(rows=1 << 29), bl.BL_ESHAPE, "blocks"), (dict(x_stride=60), bl.BL_ESHAPE, "x_stride"),
    (dict(x_stride=66), bl.BL_ESHAPE, "x_stride"), (dict(x_type=1, x_stride=68), bl.BL_ESHAPE, "x_stride"),
    (dict(X=None), bl.BL_EINVAL, "X is NULL"), (dict(codes=B), bl.BL_EINVAL, "codes"), (dict(scales=None), bl.BL_EINVAL, "scales")])
def test_pack_refusals(L, kw, status, text):
    assert call(L.bitlinear_ckpt_pack, PACK, kw) == status
    assert text in bl.bitlinear_last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(y_type=2), bl.BL_EINVAL, "y_type"), (dict(n=24), bl.BL_ESHAPE, "multiple of 16"), (dict(rows=-1), bl.BL_ESHAPE, "rows"),
    (dict(codes=None), bl.BL_EINVAL, "codes"), (dict(scales=4097), bl.BL_EINVAL, "scales"), (dict(Y=B), bl.BL_EINVAL, "Y")])
def test_unpack_refusals(L, kw, status, text):
    assert call(L.bitlinear_ckpt_unpack, UNPACK, kw) == status
    assert text in bl.bitlinear_last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(x_type=2), bl.BL_EINVAL, "x_type"), (dict(y_type=3), bl.BL_EINVAL, "y_type"), (dict(n=0), bl.BL_ESHAPE, "n must"),
    (dict(n=60), bl.BL_ESHAPE, "n must"), (dict(n=16392, x_stride=16392), bl.BL_ESHAPE, "n must"),
    (dict(rows=1 << 23), bl.BL_ESHAPE, "rows"), (dict(rows=-1), bl.BL_ESHAPE, "rows"), (dict(eps=-1.0), bl.BL_EINVAL, "eps"),
    (dict(eps=float("nan")), bl.BL_EINVAL, "eps"), (dict(eps=float("inf")), bl.BL_EINVAL, "eps"),
    (dict(codes=None), bl.BL_EINVAL, "both or neither"), (dict(scales=None), bl.BL_EINVAL, "both or neither"),
    (dict(n=72, x_stride=72), bl.BL_ESHAPE, "multiple of 16"), (dict(x_stride=56), bl.BL_ESHAPE, "x_stride"),
    (dict(X=B), bl.BL_EINVAL, "X"), (dict(weight=B), bl.BL_EINVAL, "weight"), (dict(bias=B), bl.BL_EINVAL, "bias"),
    (dict(Y=None), bl.BL_EINVAL, "Y"), (dict(mean=4098), bl.BL_EINVAL, "mean"), (dict(rstd=4098), bl.BL_EINVAL, "rstd")])
def test_norm_refusals(L, kw, status, text):
    assert call(L.bitlinear_layernorm, NORM, kw) == status
    assert text in bl.bitlinear_last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(x_type=3), bl.BL_EINVAL, "x_type"), (dict(dy_type=2), bl.BL_EINVAL, "dy_type"), (dict(dx_type=2), bl.BL_EINVAL, "dx_type"),
    (dict(n=4), bl.BL_ESHAPE, "n must"), (dict(x_type=2, x_scales=A, n=72, x_stride=72), bl.BL_ESHAPE, "multiple of 16"),
    (dict(x_type=2), bl.BL_EINVAL, "x_scales"), (dict(x_type=2, x_scales=A, x_stride=80), bl.BL_ESHAPE, "x_stride"),
    (dict(x_scales=A), bl.BL_EINVAL, "x_scales"), (dict(x_stride=62), bl.BL_ESHAPE, "x_stride"), (dict(rstd=None), bl.BL_EINVAL, "rstd"),
    (dict(dY=None), bl.BL_EINVAL, "dY"), (dict(dR=B), bl.BL_EINVAL, "dR"), (dict(dX=None), bl.BL_EINVAL, "dX"),
    (dict(dweight=B), bl.BL_EINVAL, "dweight"), (dict(dbias=B), bl.BL_EINVAL, "dbias"), (dict(ws=None), bl.BL_EWORKSPACE, "workspace"),
    (dict(ws_bytes=100), bl.BL_EWORKSPACE, "workspace"), (dict(ws=B), bl.BL_EINVAL, "ws"), (dict(rows=1 << 23), bl.BL_ESHAPE, "rows")])
def test_norm_backward_refusals(L, kw, status, text):
    assert call(L.bitlinear_layernorm_bwd, NORM_BWD, kw) == status
    assert text in bl.bitlinear_last_error()


BOTH = [(dict(n=5), bl.BL_EUNSUPPORTED, "5:8"), (dict(k=200), bl.BL_ESHAPE, "k must"), (dict(n_out=192), bl.BL_ESHAPE, "multiple of 128"),
        (dict(n_out=0), bl.BL_ESHAPE, "n_out"), (dict(k=1 << 22), bl.BL_ESHAPE, "2^22"), (dict(act=2), bl.BL_EINVAL, "act"), (dict(tokens=-1), bl.BL_ESHAPE, "tokens"),
        (dict(tokens=1 << 24), bl.BL_ESHAPE, "2^"), (dict(save_type=3), bl.BL_EINVAL, "save_type"), (dict(G=B), bl.BL_EINVAL, "G"),
        (dict(U=None), bl.BL_EINVAL, "U"), (dict(G_scales=None), bl.BL_EINVAL, "G_scales"), (dict(save_type=1), bl.BL_EINVAL, "belong"),
        (dict(xq=B), bl.BL_EINVAL, "xq"), (dict(x_scale=None), bl.BL_EINVAL, "x_scale"), (dict(gate=None), bl.BL_EINVAL, "gate"),
        (dict(up=B), bl.BL_EINVAL, "up"), (dict(gate_gamma=B), bl.BL_EINVAL, "gate_gamma"), (dict(up_gamma=None), bl.BL_EINVAL, "up_gamma")]


@pytest.mark.parametrize("kw,status,text", BOTH + [
    (dict(H=None), bl.BL_EINVAL, "H"), (dict(G=None, U=None), bl.BL_EINVAL, "belong")])
def test_glu_refusals(L, kw, status, text):
    assert call(L.bitlinear_glu, GLU, kw) == status
    assert text in bl.bitlinear_last_error()


@pytest.mark.parametrize("kw,status,text", BOTH + [
    (dict(dH=None), bl.BL_EINVAL, "dH"), (dict(dh_type=2), bl.BL_EINVAL, "dh_type"), (dict(grad_type=2), bl.BL_EINVAL, "grad_type"),
    (dict(dW_up=None), bl.BL_EINVAL, "both or neither"), (dict(dX=B), bl.BL_EINVAL, "dX"), (dict(dW_gate=B), bl.BL_EINVAL, "dW_gate"),
    (dict(ws=None), bl.BL_EWORKSPACE, "workspace"), (dict(ws_bytes=1000), bl.BL_EWORKSPACE, "workspace"), (dict(ws=A + 16), bl.BL_EINVAL, "ws"),
    (dict(tokens=1 << 22), bl.BL_ESHAPE, "2^29"), (dict(n_out=1 << 20, k=1024), bl.BL_ESHAPE, "2^29")])
def test_glu_backward_refusals(L, kw, status, text):
    assert call(L.bitlinear_glu_bwd, GLU_BWD, kw) == status
    assert text in bl.bitlinear_last_error()


def test_empty_calls(L):
    """Nothing to do is no error, whatever the pointers."""
    none = lambda d, *names: {k: None for k in names}  # noqa: E731
    assert call(L.bitlinear_ckpt_pack, PACK, dict(rows=0, **none(PACK, "X", "codes", "scales"))) == bl.BL_OK
    assert call(L.bitlinear_ckpt_unpack, UNPACK, dict(rows=0, **none(UNPACK, "Y", "codes", "scales"))) == bl.BL_OK
    assert call(L.bitlinear_layernorm, NORM, dict(rows=0, X=None, Y=None)) == bl.BL_OK
    assert call(L.bitlinear_layernorm_bwd, NORM_BWD, dict(rows=0, X=None, dweight=None, dbias=None, ws=None)) == bl.BL_OK
    assert call(L.bitlinear_glu, GLU, dict(tokens=0, xq=None, H=None)) == bl.BL_OK
    assert call(L.bitlinear_glu_bwd, GLU_BWD, dict(tokens=0, dX=None, dW_gate=None, dW_up=None, ws=None)) == bl.BL_OK
    assert call(L.bitlinear_glu_bwd, GLU_BWD, dict(dX=None, dW_gate=None, dW_up=None, ws=None)) == bl.BL_OK


def test_workspace_sizes(L):
    assert bl.bitlinear_layernorm_bwd_workspace_bytes(7) == 0 and bl.bitlinear_layernorm_bwd_workspace_bytes(16392) == 0
    assert bl.bitlinear_layernorm_bwd_workspace_bytes(2560) > 0
    assert bl.bitlinear_glu_bwd_workspace_bytes(0, 256, 128) == 0
    assert bl.bitlinear_glu_bwd_workspace_bytes(4, 256, 192) == 0
    assert bl.bitlinear_glu_bwd_workspace_bytes(1 << 22, 256, 128) == 0  # refused by the call as well
    t, k, n = 100, 256, 128  # two operands by rows, two transposed, x_q and the codes transposed
    assert bl.bitlinear_glu_bwd_workspace_bytes(t, k, n) >= 2 * (2 * t * n + 2 * n * 128 + k * 128 + 2 * k * n)
