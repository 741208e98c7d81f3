"""The norm's backward with more rows than its workgroups take at once, for every
width of row it has a variant for, and a last round that is not full."""
import pytest

import test_gpu_norm as N

pytestmark = pytest.mark.gpu
# 256 workgroups at most, of 8 (up to 1536 values), 4, 2 and 1 rows
SIZES = [(2101, 512), (4103, 1024), (2101, 1536), (1037, 2048), (1037, 2560), (519, 4096), (1101, 6144), (601, 8208),
         (601, 12288), (601, 16384), (259, 12304)]


@pytest.mark.parametrize("rows,n,x,dy,dx,center,w,b,res", [(*size, *kind) for kind in N.BACKWARD for size in SIZES])
def test_backward(rows, n, x, dy, dx, center, w, b, res):
    N.test_backward(rows, n, x, dy, dx, center, w, b, res)
