"""Refusals and sizes of the attention-side entry points, on the host: bad
arguments are named before anything is enqueued (on a host without a GPU a
launch would return BL_EHIP instead)."""
import os

import pytest

from sparse_linear_layers_group_amd import bitlinear as bl

A = 4096  # an aligned, never dereferenced address
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bl.LIB_PATH):
        from sparse_linear_layers_group_amd import build
        build.build()
    return bl.lib()


def rope(L, **kw):
    a = dict(Q=A, K=A, V=A, t=bl.BL_TYPE_F32, qs=512, ks=256, vs=256, n=5, hq=4, hkv=2, d=128, qw=A, kw=A, eps=1e-6,
             table=A, mp=16, pos=A, slots=None, rows=5, Qr=A, Kr=A, Vr=A)
    a.update(kw)
    return L.bitlinear_qk_rope(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(d=96), bl.BL_ESHAPE, "head size"), (dict(hq=5), bl.BL_ESHAPE, "multiple of hkv"),
    (dict(hkv=0), bl.BL_ESHAPE, "hkv"), (dict(t=2), bl.BL_EINVAL, "x_type"), (dict(n=-1), bl.BL_ESHAPE, "tokens"),
    (dict(n=1 << 31), bl.BL_ESHAPE, "tokens"), (dict(qs=508), bl.BL_ESHAPE, "q_stride"),
    (dict(ks=258), bl.BL_ESHAPE, "k_stride"), (dict(vs=128), bl.BL_ESHAPE, "v_stride"),
    (dict(t=bl.BL_TYPE_BF16, qs=516), bl.BL_ESHAPE, "q_stride"), (dict(mp=0), bl.BL_ESHAPE, "max_pos"),
    (dict(kw=None), bl.BL_EINVAL, "both or neither"), (dict(V=None), bl.BL_EINVAL, "both or neither"),
    (dict(eps=-1.0), bl.BL_EINVAL, "eps"), (dict(eps=NAN), bl.BL_EINVAL, "eps"), (dict(eps=INF), bl.BL_EINVAL, "eps"),
    (dict(rows=4), bl.BL_ESHAPE, "kv_rows"), (dict(slots=A, rows=-1), bl.BL_ESHAPE, "kv_rows"),
    (dict(slots=A + 4), bl.BL_EINVAL, "slots"), (dict(Q=None), bl.BL_EINVAL, "Q"), (dict(Q=A + 8), bl.BL_EINVAL, "Q"),
    (dict(table=A + 8), bl.BL_EINVAL, "table"), (dict(pos=None), bl.BL_EINVAL, "pos"),
    (dict(Kr=A + 2), bl.BL_EINVAL, "Kr"), (dict(qw=A + 4), bl.BL_EINVAL, "q_weight"),
])
def test_qk_rope_refuses(L, bad, status, word):
    assert rope(L, **bad) == status
    assert word in bl.bitlinear_last_error()


def test_no_tokens_is_no_work(L):
    assert rope(L, n=0, Q=None, K=None, V=None, Qr=None, Kr=None, Vr=None, table=None, pos=None) == bl.BL_OK


def rope_bwd(L, **kw):
    a = dict(Q=A, K=A, t=bl.BL_TYPE_BF16, qs=512, ks=256, n=5, hq=4, hkv=2, d=128, qw=A, kw=A, eps=1e-6, table=A, mp=16,
             pos=A, dQr=A, dKr=A, dQ=A, dK=A, gq=A, gk=A, ws=A, wn=bl.bitlinear_qk_rope_bwd_workspace_bytes(128))
    a.update(kw)
    return L.bitlinear_qk_rope_bwd(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(d=32), bl.BL_ESHAPE, "head size"), (dict(t=-1), bl.BL_EINVAL, "x_type"), (dict(gq=None), bl.BL_EINVAL, "dq_weight"),
    (dict(ws=None), bl.BL_EWORKSPACE, "workspace"), (dict(wn=100), bl.BL_EWORKSPACE, "workspace"),
    (dict(Q=None), bl.BL_EINVAL, "Q"), (dict(qs=100), bl.BL_ESHAPE, "q_stride"), (dict(dQr=None), bl.BL_EINVAL, "dQr"),
    (dict(dK=A + 8), bl.BL_EINVAL, "dK"), (dict(kw=None), bl.BL_EINVAL, "both or neither"),
    (dict(qw=None, kw=None, Q=None, K=None, ws=None, wn=0, dQ=None), bl.BL_EINVAL, "dQ"),
])
def test_qk_rope_bwd_refuses(L, bad, status, word):
    assert rope_bwd(L, **bad) == status
    assert word in bl.bitlinear_last_error()


def test_rope_table_refuses(L):
    f = L.bitlinear_rope_table
    assert f(0, 64, 1e4, A, None) == bl.BL_ESHAPE
    assert f(16, 80, 1e4, A, None) == bl.BL_ESHAPE
    assert f(16, 64, 0.0, A, None) == bl.BL_EINVAL
    assert f(16, 64, NAN, A, None) == bl.BL_EINVAL
    assert f(16, 64, 1e4, None, None) == bl.BL_EINVAL


ATTN_BAD = [
    (dict(d=256), bl.BL_ESHAPE, "head size"), (dict(hq=3), bl.BL_ESHAPE, "multiple of hkv"),
    (dict(b=0), bl.BL_ESHAPE, "batch"), (dict(b=65536), bl.BL_ESHAPE, "batch"), (dict(tq=-1), bl.BL_ESHAPE, "total_q"),
    (dict(tk=1 << 31), bl.BL_ESHAPE, "total_k"), (dict(tq=(1 << 31) - 1, hq=4096, hkv=4096, qs=4096 * 128), bl.BL_ESHAPE, "too many"),
    (dict(scale=0.0), bl.BL_EINVAL, "scale"), (dict(scale=-1.0), bl.BL_EINVAL, "scale"), (dict(scale=NAN), bl.BL_EINVAL, "scale"),
    (dict(scale=INF), bl.BL_EINVAL, "scale"), (dict(qs=511), bl.BL_ESHAPE, "q_stride"), (dict(ks=248), bl.BL_ESHAPE, "k_stride"),
    (dict(vs=1 << 22), bl.BL_ESHAPE, "v_stride"), (dict(Q=A + 8), bl.BL_EINVAL, "Q"), (dict(K=None), bl.BL_EINVAL, "K"),
    (dict(V=None), bl.BL_EINVAL, "V"), (dict(cq=None), bl.BL_EINVAL, "cu_q"), (dict(ck=A + 2), bl.BL_EINVAL, "cu_k"),
    (dict(O=None), bl.BL_EINVAL, "O"),
]


def attn_fwd(L, **kw):
    a = dict(Q=A, K=A, V=A, qs=512, ks=256, vs=256, cq=A, ck=A, b=2, tq=10, tk=12, hq=4, hkv=2, d=128, scale=0.1, O=A,
             lse=A, ws=A, wn=1 << 30)
    a.update(kw)
    return L.bitlinear_attn_fwd(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", ATTN_BAD + [(dict(lse=A + 2), bl.BL_EINVAL, "lse")])
def test_attn_fwd_refuses(L, bad, status, word):
    assert attn_fwd(L, **bad) == status
    assert word in bl.bitlinear_last_error()


def test_attn_fwd_without_rows(L):
    assert attn_fwd(L, tq=0, Q=None, K=None, V=None, O=None, ws=None, wn=0) == bl.BL_OK


def attn_bwd(L, **kw):
    a = dict(Q=A, K=A, V=A, qs=512, ks=256, vs=256, O=A, lse=A, dO=A, t=bl.BL_TYPE_F32, cq=A, ck=A, b=2, tq=10, tk=12, hq=4,
             hkv=2, d=128, scale=0.1, dQ=A, dK=A, dV=A, ws=A, wn=bl.bitlinear_attn_bwd_workspace_bytes(2, 10, 12, 4, 2, 128))
    a.update(kw)
    return L.bitlinear_attn_bwd(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", ATTN_BAD + [
    (dict(lse=None), bl.BL_EINVAL, "lse"), (dict(dO=None), bl.BL_EINVAL, "dO"), (dict(t=5), bl.BL_EINVAL, "do_type"),
    (dict(dQ=A + 8), bl.BL_EINVAL, "dQ"), (dict(dK=None), bl.BL_EINVAL, "dK"), (dict(dV=None), bl.BL_EINVAL, "dV"),
    (dict(ws=None), bl.BL_EWORKSPACE, "workspace"), (dict(wn=64), bl.BL_EWORKSPACE, "workspace"),
    (dict(ws=A + 64), bl.BL_EINVAL, "ws"),
])
def test_attn_bwd_refuses(L, bad, status, word):
    assert attn_bwd(L, **bad) == status
    assert word in bl.bitlinear_last_error()


def cache(L, **kw):
    a = dict(Q=A, qs=512, K=A, V=A, rows=640, pages=A, mp=10, page=64, lens=A, tree=A, b=2, t=4, hq=4, hkv=2, d=128, scale=0.1,
             O=A, ws=A, wn=bl.bitlinear_attn_cache_workspace_bytes(2, 4, 4, 2, 128))
    a.update(kw)
    return L.bitlinear_attn_cache(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(d=120), bl.BL_ESHAPE, "head size"), (dict(b=0), bl.BL_ESHAPE, "batch"), (dict(t=0), bl.BL_ESHAPE, "draft"),
    (dict(t=65), bl.BL_ESHAPE, "draft"), (dict(page=8), bl.BL_ESHAPE, "page"), (dict(page=40), bl.BL_ESHAPE, "page"),
    (dict(mp=0), bl.BL_ESHAPE, "max_pages"), (dict(mp=1 << 26), bl.BL_ESHAPE, "max_pages"),
    (dict(b=65535, mp=1 << 15), bl.BL_ESHAPE, "tiles"), (dict(rows=-1), bl.BL_ESHAPE, "cache_rows"),
    (dict(rows=1 << 31), bl.BL_ESHAPE, "cache_rows"), (dict(scale=NAN), bl.BL_EINVAL, "scale"),
    (dict(qs=504), bl.BL_ESHAPE, "q_stride"), (dict(Q=None), bl.BL_EINVAL, "Q"), (dict(K=A + 8), bl.BL_EINVAL, "K"),
    (dict(V=None), bl.BL_EINVAL, "V"), (dict(pages=None), bl.BL_EINVAL, "pages"), (dict(lens=A + 1), bl.BL_EINVAL, "lens"),
    (dict(tree=A + 4), bl.BL_EINVAL, "tree"), (dict(O=None), bl.BL_EINVAL, "O"), (dict(ws=None), bl.BL_EWORKSPACE, "workspace"),
    (dict(wn=1000), bl.BL_EWORKSPACE, "workspace"),
])
def test_attn_cache_refuses(L, bad, status, word):
    assert cache(L, **bad) == status
    assert word in bl.bitlinear_last_error()


def test_workspace_sizes_of_refused_shapes_are_zero(L):
    assert bl.bitlinear_qk_rope_bwd_workspace_bytes(100) == 0
    assert bl.bitlinear_attn_bwd_workspace_bytes(1, 10, 10, 3, 2, 128) == 0
    assert bl.bitlinear_attn_fwd_workspace_bytes(0, 10, 10, 4, 2, 128) == 0
    assert bl.bitlinear_attn_cache_workspace_bytes(1, 65, 4, 2, 128) == 0


def test_more_workgroups_than_a_launch_holds(L):
    """2^32 threads: refused by size, not left to the launch."""
    assert rope(L, n=(1 << 26) - 3, rows=(1 << 26) - 3) == bl.BL_ESHAPE
    assert "too many head rows" in bl.bitlinear_last_error()
    assert rope_bwd(L, n=1 << 26, qw=None, kw=None) == bl.BL_ESHAPE
    assert L.bitlinear_rope_table(1 << 26, 128, 1e4, A, None) == bl.BL_ESHAPE
    assert "max_pos" in bl.bitlinear_last_error()
    for f in (attn_fwd, attn_bwd):
        for bad in (dict(b=65535, hq=256, hkv=1, qs=256 * 128), dict(b=65535, hq=128, hkv=128, qs=128 * 128),
                    dict(tq=1 << 30, hq=2, hkv=1), dict(tk=1 << 29, hq=1, hkv=1)):
            assert f(L, **bad) == bl.BL_ESHAPE
            assert "too many rows" in bl.bitlinear_last_error()
    assert cache(L, b=1 << 15, t=16, hq=32, hkv=16, mp=1) == bl.BL_ESHAPE
    assert "2^24" in bl.bitlinear_last_error()
    assert cache(L, b=1 << 15, t=64, hq=32, hkv=16, mp=1) == bl.BL_ESHAPE
    assert "2^26" in bl.bitlinear_last_error()


@pytest.mark.parametrize("scale,status", [(9e-31, bl.BL_EINVAL), (1.1e30, bl.BL_EINVAL), (1e-45, bl.BL_EINVAL)])
def test_scales_that_leave_binary32(L, scale, status):
    for f in (attn_fwd, attn_bwd, cache):
        assert f(L, scale=scale) == status
        assert "scale" in bl.bitlinear_last_error()
