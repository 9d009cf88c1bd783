"""The attention's workspace is as large as its call needs."""
import ctypes

import numpy as np
import pytest
import torch

from fp4_weight_only_nvfp4_gb300 import _lib
import fp4_weight_only_nvfp4_gb300 as vt

A0 = 0x10000                      # fake device addresses: no call below may use them
F = ctypes.c_void_p(A0)


def _view(dim, heads=4):
    return ctypes.byref(_lib.KvCacheView(A0, 4, heads * 16 * dim * 9 // 8, 16, heads, dim, A0, A0))


def _bytes(T, B, q_heads, dim):
    from fp4_weight_only_nvfp4_gb300 import build
    build.build()
    n = ctypes.c_size_t(0)
    assert _lib.lib().vt_fp4_attention_workspace_bytes(_view(dim), T, B, q_heads, ctypes.byref(n)) == _lib.VT_OK
    return n.value


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_calls_of_few_rows_need_no_room_for_tiles(dim):
    few, many = _bytes(0, 1, 4, dim), _bytes(2 ** 20, 1, 4, dim)
    assert 10 * few < many
    for q_heads, T in ((4, 32), (8, 16), (24, 5), (128, 1)):
        assert _bytes(T, 1, q_heads, dim) == few and _bytes(T + 1, 1, q_heads, dim) == many
    assert _bytes(1, 1, 256, dim) == many  # 64 heads a key/value head: a single row with starts is a tile
    for T in (0, 1, 33, 2 ** 24):          # the number of sequences counts for nothing
        assert _bytes(T, 0, 4, dim) == _bytes(T, 2 ** 24, 4, dim)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_workspace_that_is_too_small_is_refused(dim):
    few, many = _bytes(0, 1, 32, dim), _bytes(100, 1, 32, dim)
    ld = 32 * dim

    def call(T, starts, n):
        return _lib.lib().vt_fp4_paged_attention(_view(dim), T, F, 32, ld, F, 3, F, starts, T, 0.1, 0, None, F, ld, F, n, None)

    for T, starts, n in ((100, F, many - 1), (100, F, few), (5, F, few), (4, F, few - 1), (100, None, few - 1)):
        assert call(T, starts, n) == _lib.VT_ERR_INVALID_ARG
        assert b"bytes" in _lib.lib().vt_fp4_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_calls_with_the_smallest_workspace_write_nothing_behind_it(D):
    from test_gpu_paged_attention import Case
    rng = np.random.default_rng(D)
    for rows, T in ((None, 0), ([4, 1, 3], 8), ([40, 1, 30], 71)):
        c = Case(rng, [700, 3000, 900], 8, 2, D, 16, rows=rows)
        n = vt.attention_workspace(T, 3, 8, c.cache).numel()
        room = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        ws = room[:n]
        ws[:4096].zero_()
        want = c.run()
        for _ in range(3):
            assert torch.equal(c.run(workspace=ws), want)
        assert (room[n:] == 0x5A).all() and vt.workspace_status(ws) == 0
