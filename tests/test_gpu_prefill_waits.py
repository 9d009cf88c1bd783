"""GPU: the tile kernel's bounded waits running out as the copies that they wait for land.  The
producer starts a millisecond late and the limit lies around that, so that lanes, warps and CTAs of
one call are answered differently; every call returns, and the next one is right."""
import time

import pytest
import torch

import synth
import fp4_weight_only_nvfp4_gb300 as vt
from fp4_weight_only_nvfp4_gb300 import _lib
from gpu_helpers import bf16_dev, make_acts, make_weight, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("M,N,K", [(40, 640, 2048), (300, 5000, 128), (700, 9000, 512)])
def test_waits_that_run_out_as_the_copies_land(fmt, M, N, K):
    codes, scales, G = make_weight(fmt, synth.tensor_id(81, fmt, N), N, K)
    W = vt.PackedWeight.from_codes(to_dev(codes), to_dev(scales), G, fmt, N, K)
    A = bf16_dev(make_acts(synth.tensor_id(81, fmt, M, 2), M, K))
    ws = W.new_workspace(M)
    want = vt.w4a16_gemm(A, W, workspace=ws, opts={"force_path": 2})
    torch.cuda.synchronize()
    seen = set()
    for limit in range(700, 1200, 10):
        t0 = time.perf_counter()
        got = vt.w4a16_gemm(A, W, workspace=ws,
                            opts={"force_path": 2, "withhold_weights": -1, "wait_limit_us": limit})
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 1.0
        status = vt.workspace_status(ws)
        assert status in (_lib.VT_OK, _lib.VT_ERR_TIMEOUT)
        assert status != _lib.VT_OK or torch.equal(got, want)
        seen.add(status)
        assert torch.equal(vt.w4a16_gemm(A, W, workspace=ws, opts={"force_path": 2}), want)
        assert vt.workspace_status(ws) == _lib.VT_OK
    assert seen == {_lib.VT_OK, _lib.VT_ERR_TIMEOUT}
