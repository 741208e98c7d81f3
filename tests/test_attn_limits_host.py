"""Limits of bitlinear_attn_cache near 2^31, on the host: the kernels count a
call's rows and tiles in 32 bits and round both up, so what they could not
count has to be refused."""
import os

import pytest
import torch

from sparse_linear_layers_group_amd import bitlinear as bl

A = 4096  # an aligned, never dereferenced address
MOST = (1 << 31) - 1024


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bl.LIB_PATH):
        from sparse_linear_layers_group_amd import build
        build.build()
    return bl.lib()


def cache(L, batch, draft, hq, hkv, d, max_pages, page):
    n = bl.bitlinear_attn_cache_workspace_bytes(batch, draft, hq, hkv, d)
    return L.bitlinear_attn_cache(A, hq * d, A, A, 1 << 20, A, max_pages, page, A, None, batch, draft, hq, hkv, d, 0.1,
                                  A, A, n, None)


def places(batch, draft, hq, hkv, rows):
    """Tiles of the whole call as the host counts them: 32 rows each, 8 more for every unit."""
    return batch * (-(-rows // 32) + 8) * hkv * -(-(draft * hq // hkv) // 32)


def ranges_end(batch, draft, hq, hkv, d, rows):
    """The largest number the kernels form of a call whose sequences are all
    `rows` long: all units' tiles plus the workgroups less one, which the
    number of tiles in a workgroup's range is made from."""
    wide = draft * hq // hkv > 32
    tile = 64 if wide else 32
    blocks = -(-(draft * hq // hkv) // 32)
    per = -(-blocks // -(-blocks // 4)) if wide else 1
    tiles = batch * ((rows + tile - 1) // tile + 6) * hkv * -(-blocks // per)
    return tiles + (256 if d == 128 else 512) - 1


# (the first: four sequences of 2147483360 rows, 8 + 8 heads of 64: 2147483552 tiles, 511 more wrap)
@pytest.mark.parametrize("batch,draft,hq,hkv,d,max_pages,page", [
    (4, 1, 8, 8, 64, 2147483360 // 16, 16),
    (4, 1, 8, 8, 128, 2147483360 // 16, 16),
    (32, 1, 2, 1, 64, 2147483392 // 32, 32),
    (1, 1, 1, 1, 64, ((1 << 31) - 16) // 16, 16),    # rows that cannot be rounded up to a tile
    (1, 1, 1, 1, 128, ((1 << 31) - 64) // 64, 64),
    (1, 33, 1, 1, 128, ((1 << 31) - 1008) // 16, 16),
])
def test_refuses_what_32_bits_do_not_hold(L, batch, draft, hq, hkv, d, max_pages, page):
    rows = max_pages * page
    assert rows > MOST or ranges_end(batch, draft, hq, hkv, d, rows) > (1 << 31) - 1 \
        or places(batch, draft, hq, hkv, rows) > MOST
    assert cache(L, batch, draft, hq, hkv, d, max_pages, page) == bl.BL_ESHAPE
    assert "max_pages" in bl.bitlinear_last_error() or "tiles" in bl.bitlinear_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the stand-in addresses must not reach a GPU")
@pytest.mark.parametrize("batch,draft,hq,hkv,d,page", [
    (1, 1, 1, 1, 64, 16), (1, 1, 1, 1, 128, 1024), (4, 1, 8, 8, 64, 16), (32, 1, 2, 1, 64, 32), (3, 64, 20, 5, 128, 16),
    (1, 64, 64, 1, 64, 16),
])
def test_takes_the_largest_that_they_hold(L, batch, draft, hq, hkv, d, page):
    """One page less than the first refused call passes the checks (a launch
    without a GPU fails), and every number the kernels form stays below 2^31."""
    low, high = 1, (1 << 31) // page
    while high - low > 1:
        mid = (low + high) // 2
        if cache(L, batch, draft, hq, hkv, d, mid, page) == bl.BL_ESHAPE:
            high = mid
        else:
            low = mid
    assert cache(L, batch, draft, hq, hkv, d, low, page) == bl.BL_EHIP
    rows = low * page
    assert rows + 4 * 64 < 1 << 31 and ranges_end(batch, draft, hq, hkv, d, rows) < 1 << 31
    assert (low + 1) * page > MOST or places(batch, draft, hq, hkv, (low + 1) * page) > MOST
