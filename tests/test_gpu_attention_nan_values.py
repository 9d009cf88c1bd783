"""GPU: NaN scales among the values of chunks of rows, where the rows of one warp see different keys."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from layer_helpers import attention, gpu
from rows_helpers import assert_close, f64
from test_gpu_paged_attention import Case

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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 700, 1500])
def test_in_blocks_that_every_row_sees_and_at_the_borders(window, D):
    """Tiles cut into several segments: tokens in blocks that all rows see, in those at either border, on both sides of the
    limits between them, on a page that stands in the table twice and on one that is left out."""
    rng = np.random.default_rng(D + window)
    c = Case(rng, [4000, 1900], 4, 2, D, 32, rows=[300, 45])
    c.tables[0, 70], c.tables[0, 90] = -1, c.tables[0, 60]
    where = [(0, j, j % 2, j % (D // 16)) for j in (0, 127, 128, 60 * 32 + 7, 2200, 2440, 3000, 3199, 3200, 3583, 3584, 3699, 3700, 3712, 3999)]
    where += [(1, j, 0, 1) for j in (3, 400, 1855, 1899)]
    for b, j, h, g in where:
        page = c.tables[b, j // 32]
        if page >= 0:
            c.raw[3][page * 32 + j % 32, h, g] = 0xFF
    c.cache.put(gpu(np.arange(c.pages * c.page)), *(gpu(a) for a in c.raw))
    lost = _check(c, window, 3)
    assert lost.any() and not lost.all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_value_is_one(D):
    rng = np.random.default_rng(D)
    c = Case(rng, [1500, 700], 4, 2, D, 16, rows=[200, 700])
    c.raw[3][:] = 0x7F
    c.cache.put(gpu(np.arange(c.pages * c.page)), *(gpu(a) for a in c.raw))
    assert c.run().isnan().all() and c.run(window=300).isnan().all()


def test_one_far_back_costs_no_search_through_the_sequence():
    """The time with a NaN near the start of a long context is that without one (a search of the rows' keys one by one
    takes tens of times as long, and for contexts of millions the seconds after which the waits give up)."""
    D, heads, keys, rows, page = 64, 8, 200000, 1024, 64
    g = torch.full((heads,), 1.0, device="cuda")
    pages = keys // page
    cache = vt.KVCache.empty(pages, page, heads, D, g, g.clone())
    cache.data.fill_(0x38)  # codes 8 and 3 (0 and 1.5), scales of 1
    q = torch.randn(rows, heads, D, device="cuda").bfloat16()
    tables = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ws = vt.attention_workspace(rows, 1, heads, cache)
    clock = lambda: torch.cuda.Event(enable_timing=True)

    def run():
        best = float("inf")
        for _ in range(4):
            a, b = clock(), clock()
            a.record()
            out = vt.paged_attention(q, cache, tables, i32(keys), i32(0, rows), workspace=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        assert vt.workspace_status(ws) == 0
        return out, best

    want, plain = run()
    slots = torch.tensor([5], device="cuda")
    raw = cache.get(slots)
    raw[3][0, :, 1] = 0x7F
    cache.put(slots, *raw)
    got, poisoned = run()
    print(f"{plain:.2f} ms, with a NaN {poisoned:.2f} ms")
    assert got[:, :, 16:32].isnan().all()
    assert torch.equal(got[:, :, :16], want[:, :, :16]) and torch.equal(got[:, :, 32:], want[:, :, 32:])
    assert poisoned < 3 * plain
