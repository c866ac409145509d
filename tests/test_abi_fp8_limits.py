"""CPU checks of the FP8 products' largest sizes (every call stops before any device
work; the pointers are stand-ins that are never read)."""
import ctypes as C

import pytest

from tests.test_abi_fp8_gated_norm import SHAPE, f8, f8t, vp

INT_MAX = 2 ** 31 - 1
MOST = INT_MAX - 511   # a tile's rows past the end are counted too


@pytest.mark.parametrize("m,n", [(MOST + 1, 8), (INT_MAX, 8), (8, MOST + 1), (8, INT_MAX), (INT_MAX + 1, 8), (8, INT_MAX + 1)])
def test_products_refuse_rows_that_int32_tiles_cannot_count(lib, m, n):
    a, w = f8(m, 32), f8t(n, 32)
    assert lib.mxq_gemm(C.byref(a), C.byref(w), None, None, 0, None, 0, None, vp(64), n, n, None, 0, None) == SHAPE
    assert lib.mxq_gemm_mixed(C.byref(a), C.byref(w), 1, vp(64), None, 0, None, 0, None, vp(64), n, n, None, 0, None) == SHAPE


def test_grouped_products_refuse_columns_that_int32_tiles_cannot_count(lib):
    for n in (2 ** 31 - 384, 2 ** 31 - 128):   # multiples of 128 past 2**31 - 512
        a, w = f8(8, 32), f8t(n, 32)
        assert lib.mxq_gemm_grouped(C.byref(a), C.byref(w), 1, vp(64), None, vp(64), n, None) == SHAPE
