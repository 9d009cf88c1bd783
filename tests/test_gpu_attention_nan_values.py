"""GPU: NaN scales among the values of chunks of rows, where the rows of one warp see different keys."""
import numpy as np
import pytest

from layer_helpers import attention, gpu
from rows_helpers import assert_close, f64
from test_gpu_paged_attention import Case

import torch

pytestmark = pytest.mark.gpu


def _check(c, window, runs=1):
    ref, err = attention(f64(c.q), *c.kv(), c.tables, c.lens, c.starts, c.page, c.D ** -0.5, window)
    lost = np.isnan(ref)
    got = c.run(window=window)
    assert np.array_equal(np.isnan(f64(got)), lost)
    assert_close(f64(got)[~lost], ref[~lost], err[~lost])
    for _ in range(runs - 1):
        assert torch.equal(c.run(window=window).nan_to_num(), got.nan_to_num())
    return lost


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (6, 2), (16, 1)])
def test_rows_of_a_warp_that_see_it_and_rows_that_do_not(Hq, Hkv, D):
    """The token stands in the middle of a warp's rows, at both borders of their windows and behind the last."""
    rng = np.random.default_rng(D + Hq)
    c = Case(rng, [170, 300, 77], Hq, Hkv, D, 16, rows=[150, 43, 77])
    vs = c.raw[3]
    for b, j, h, g in ((0, 85, 0, 1), (0, 20, Hkv - 1, 0), (1, 280, 0, D // 16 - 1), (1, 3, 0, 2), (2, 76, Hkv - 1, 3), (2, 0, 0, 0)):
        vs[c.slots(b)[j], h, g] = 0x7F
    c.cache.put(gpu(np.arange(c.pages * c.page)), *(gpu(a) for a in c.raw))
    for window in (0, 1, 17, 64, 200):
        lost = _check(c, window, 5)
        assert lost.any() and not lost.all()
