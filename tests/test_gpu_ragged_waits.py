"""GPU: the bounded waits of the ragged products, without a GPU fault.  A wait that runs out sets
VT_ERR_TIMEOUT in the workspace's status word, the call returns, and the next call on the same
workspace is right.  The waits run out because the weight producer stops, or, where it pauses for
about as long as the limit, while the copies that they wait for land: threads of one team are
then answered differently, with copies and products under way."""
import time

import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from fp4_weight_only_nvfp4_gb300 import _lib
from rows_helpers import acts, group64, random_weight

pytestmark = pytest.mark.gpu

# M, topk, E, N, K of a call of each kernel variant on 152 SMs
ONE_TILE = (12, 2, 8, 256, 1024)         # a weight row tile per item
TWO_TILES = (60, 4, 200, 300, 512)       # two, 64-row token tiles, an odd last row tile
MANY_ROWS = (700, 2, 16, 1400, 1024)     # 128-row token tiles, rows written in group order first
GATHERED = (2100, 8, 64, 640, 544)       # 128-row token tiles, rows gathered by the product


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _call(size, fmt, silu):
    M, topk, E, N, K = size
    rng = np.random.default_rng(M + fmt)
    parts = [random_weight(rng, fmt, E, N // 2 if silu else N, K) for _ in range(2 if silu else 1)]
    parts = [(_dev(c), _dev(s), g) for c, s, g in parts]
    W = vt.PackedWeight.grouped_gate_up(*parts, fmt, E, N // 2, K) if silu else \
        vt.PackedWeight.grouped(*parts[0], fmt, E, N, K)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
    order, offsets = group64(ids, E)
    groups = vt.RowGroups(_dev(ids), _dev(order), _dev(offsets))
    x, ws = acts(rng, M, K).cuda(), W.ragged_workspace(M, topk)
    f = vt.w4a16_gemm_ragged_silu_mul if silu else vt.w4a16_gemm_ragged
    return lambda **opts: f(x, W, groups, workspace=ws, opts=opts or None), ws


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("size", [ONE_TILE, TWO_TILES, MANY_ROWS, GATHERED])
def test_a_call_whose_weights_stop_arriving_returns(size, fmt, silu):
    call, ws = _call(size, fmt, silu)
    want = call()
    torch.cuda.synchronize()
    for steps in (1, 2, size[4] // 64):
        t0 = time.perf_counter()
        call(withhold_weights=steps, wait_limit_us=20000)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 1.5
        assert vt.workspace_status(ws) == _lib.VT_ERR_TIMEOUT
        assert vt.workspace_status(ws) == _lib.VT_OK  # reading cleared it
        assert torch.equal(call(), want)
        assert vt.workspace_status(ws) == _lib.VT_OK


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("size", [ONE_TILE, TWO_TILES, MANY_ROWS, GATHERED])
def test_a_call_whose_waits_run_out_as_the_weights_arrive_returns(size, silu):
    call, ws = _call(size, vt.NVFP4, silu)
    want = call()
    torch.cuda.synchronize()
    seen = set()
    for step in (1, 3):
        for limit in range(600, 1150, 10):
            t0 = time.perf_counter()
            got = call(withhold_weights=-step, wait_limit_us=limit)
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 1.0
            status = vt.workspace_status(ws)
            assert status in (_lib.VT_OK, _lib.VT_ERR_TIMEOUT)
            assert status != _lib.VT_OK or torch.equal(got, want)
            seen.add(status)
        assert torch.equal(call(), want)
        assert vt.workspace_status(ws) == _lib.VT_OK
    assert seen == {_lib.VT_OK, _lib.VT_ERR_TIMEOUT}


def test_only_the_wait_options_are_taken():
    call, _ = _call(ONE_TILE, vt.NVFP4, False)
    for opts in (dict(grid=4), dict(stages=3), dict(warps=4), dict(force_path=1), dict(wait_limit_us=-1),
                 dict(withhold_weights=-2 ** 31)):
        with pytest.raises(_lib.VtError, match="wait_limit_us"):
            call(**opts)
    with pytest.raises(TypeError):
        call(wait_limit=5)
