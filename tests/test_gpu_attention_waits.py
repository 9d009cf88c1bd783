"""GPU: the bounded waits of the attention of chunks, without a GPU fault.  A wait that runs out sets VT_ERR_TIMEOUT in
the workspace's status word and the call returns; once the workspace's first bytes are zeros again the next call is right.
The waits run out because the warps that load the keys stop, or pause for about as long as the limit, so that some waits
are answered and others not, with products and parts under way."""
import time

import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from fp4_weight_only_nvfp4_gb300 import _lib
from fp4_weight_only_nvfp4_gb300.layer import CLEARED
from layer_helpers import gpu
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu

# sequences' keys and rows: pairs of row tiles; single ones, whose blocks go to both groups; tiles that CTAs share;
# rows for both kernels
SHAPES = [([1500, 700], [1400, 600]), ([400] * 30, [30] * 30), ([9000], [200]), ([900, 2000, 64], [800, 2, 1])]


@pytest.fixture(autouse=True)
def _defaults():
    yield
    torch.cuda.synchronize()
    assert _lib.lib().vt_fp4_attention_test_hooks(0, 0) == _lib.VT_OK


def _hooks(limit, withhold):
    assert _lib.lib().vt_fp4_attention_test_hooks(limit, withhold) == _lib.VT_OK


def _call(shape, D):
    rng = np.random.default_rng(D + len(shape[0]))
    c = Case(rng, shape[0], 8, 2, D, 16, rows=shape[1])
    q, tables, lens, starts = c.q.cuda(), gpu(c.tables), gpu(c.lens), gpu(c.starts)
    ws = vt.attention_workspace(q.shape[0], len(shape[0]), 8, c.cache)
    return lambda: vt.paged_attention(q, c.cache, tables, lens, starts, workspace=ws), ws


def _again(call, ws, want):
    assert vt.workspace_status(ws) == _lib.VT_OK  # reading cleared it
    ws[:CLEARED].zero_()
    assert torch.equal(call(), want)
    assert vt.workspace_status(ws) == _lib.VT_OK


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_call_whose_keys_stop_arriving_returns(D, shape):
    call, ws = _call(SHAPES[shape], D)
    want = call()
    torch.cuda.synchronize()
    for block in (1, 2):
        _hooks(20000, block)
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 1.5
        assert vt.workspace_status(ws) == _lib.VT_ERR_TIMEOUT
        _hooks(0, 0)
        _again(call, ws, want)


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_call_whose_waits_run_out_as_the_keys_arrive_returns(D, shape):
    call, ws = _call(SHAPES[shape], D)
    want = call()
    torch.cuda.synchronize()
    for block in (1, 2):
        for limit in range(600, 1150, 25):
            _hooks(limit, -block)
            t0 = time.perf_counter()
            got = call()
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 1.0
            _hooks(0, 0)
            status = vt.workspace_status(ws)
            assert status in (_lib.VT_OK, _lib.VT_ERR_TIMEOUT)
            if status == _lib.VT_OK:
                assert torch.equal(got, want)
            else:
                ws[:CLEARED].zero_()
    _again(call, ws, want)


def test_rows_of_the_other_kernel_are_right_all_the_same():
    """A call of single rows has none of these waits; of one with both, the sequences of few rows are written."""
    rng = np.random.default_rng(5)
    one, both = Case(rng, [300, 40], 8, 2, 128, 16), Case(rng, [900, 300], 8, 2, 128, 16, rows=[800, 2])
    want = one.run(), both.run()
    ws = vt.attention_workspace(802, 2, 8, one.cache)
    _hooks(20000, 1)
    assert torch.equal(one.run(workspace=ws), want[0])
    assert vt.workspace_status(ws) == _lib.VT_OK
    assert torch.equal(both.run(workspace=ws)[800:], want[1][800:])
    assert vt.workspace_status(ws) == _lib.VT_ERR_TIMEOUT
