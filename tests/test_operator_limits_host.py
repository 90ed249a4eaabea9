"""Row counts that layer norm and its gradients take and refuse, on the host.  Each call
that passes the size checks has a misaligned output, so that none is ever launched."""
import ctypes

import pytest

import adaptive_residual_gradient_amd as A
from test_operators_host import MISALIGNED, OK, TOO_LARGE, norm_back, norm_call


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not A.LIB_PATH.exists():
        from adaptive_residual_gradient_amd import _build
        _build.build()


@pytest.mark.parametrize("rows,cols,forward,backward", [
    (1 << 26, 4, MISALIGNED, MISALIGNED),             # bounded grids step over any number of rows
    ((1 << 32) - 1, 64, MISALIGNED, MISALIGNED),
    (1 << 32, 1, TOO_LARGE, TOO_LARGE),
    ((1 << 22) - 1, 16384, MISALIGNED, MISALIGNED),
    (1 << 22, 8192, MISALIGNED, MISALIGNED),
    (1 << 22, 8193, MISALIGNED, TOO_LARGE),           # one workgroup of 1024 threads a row
    (5_000_000, 8193, MISALIGNED, TOO_LARGE),
    (1 << 22, 16385, TOO_LARGE, TOO_LARGE),
    ((1 << 22) - 1, 65536, MISALIGNED, MISALIGNED),
])
def test_layer_norm_rows(rows, cols, forward, backward):
    assert norm_call(rows=rows, cols=cols, xs=cols, ys=cols, y=0x30002) == forward
    assert norm_back(rows=rows, cols=cols, ds=cols, xs=cols, dxs=cols, dx=0x40002) == backward
    n = ctypes.c_uint64()
    st = A.lib().adacomp_layer_norm_workspace_bytes(rows, cols, ctypes.byref(n))
    assert st == (TOO_LARGE if backward == TOO_LARGE else OK)
