"""CPU: the number of rows that the operators on grouped rows accept.  A group of n rows is cut into
nt tiles of 16 to 128 rows, and n + nt has to stay below 2^31 in the kernels' 32-bit arithmetic."""
import ctypes

import pytest

from fp4_weight_only_nvfp4_gb300 import _lib

F = ctypes.c_void_p(0x10000)  # a fake device pointer: no call below may use it
ODD = ctypes.c_void_p(0x10001)  # an accepted size is told that it is misaligned, and nothing is launched
MOST = 2 ** 31 - 2 ** 27 - 1


@pytest.fixture(scope="module")
def L():
    from fp4_weight_only_nvfp4_gb300 import build
    build.build()
    return _lib.lib()


def test_the_tiles_of_the_largest_group_fit_32_bits():
    for tile in (16, 64, 128):
        assert MOST + (MOST + tile - 1) // tile + 128 < 2 ** 31


@pytest.mark.parametrize("rows", [MOST + 1, 2 ** 31 - 2, 2 ** 31 - 1])
def test_more_rows_are_refused(L, rows):
    n = ctypes.c_size_t(0)
    assert L.vt_fp4_group_workspace_bytes(MOST, 4, ctypes.byref(n)) == 0
    assert L.vt_fp4_group_workspace_bytes(rows, 4, ctypes.byref(n)) == _lib.VT_ERR_INVALID_ARG
    assert L.vt_fp4_group_rows(ODD, rows, 4, F, F, F, 1 << 30, None) == _lib.VT_ERR_INVALID_ARG
    assert L.vt_fp4_moe_route(ODD, 0, rows, 16, 16, 1, 0, None, 1, 1.0, F, F, F, F, F, 1 << 30,
                              None) == _lib.VT_ERR_INVALID_ARG
    assert L.vt_fp4_moe_route(ODD, 0, (rows + 7) // 8, 16, 16, 8, 0, None, 1, 1.0, F, F, F, F, F, 1 << 30,
                              None) == _lib.VT_ERR_INVALID_ARG
    assert L.vt_fp4_lora_add(ODD, rows, 8, 8, F, F, F, None, 1, 8, 8, F, F, F, 8, F, 8,
                             None) == _lib.VT_ERR_INVALID_ARG
    assert L.vt_fp4_lora_add(ODD, MOST, 8, 8, F, F, F, None, 1, 8, 8, F, F, F, 8, F, 8,
                             None) == _lib.VT_ERR_MISALIGNED
