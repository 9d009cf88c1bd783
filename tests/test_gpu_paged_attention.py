"""GPU: causal attention over the paged NVFP4 cache, against fp64."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from layer_helpers import F, attention, gpu, random_tokens, values
from rows_helpers import acts, assert_close, f64

pytestmark = pytest.mark.gpu


class Case:
    """A cache of random tokens and sequences of the given lengths on shuffled pages."""

    def __init__(self, rng, lens, Hq, Hkv, D, page, rows=None, spare=2):
        self.rng, self.Hq, self.Hkv, self.D, self.page = rng, Hq, Hkv, D, page
        self.lens = np.array(lens, dtype=np.int32)
        need = [-(-max(n, 0) // page) for n in lens]
        self.pages = sum(need) + spare
        g = lambda: torch.from_numpy(rng.uniform(0.01, 0.03, Hkv).astype(F)).cuda()
        self.cache = vt.KVCache.empty(self.pages, page, Hkv, D, g(), g())
        self.cache.data.fill_(0xFF)  # unused places hold NaN scales
        self.tables = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
        order, at = rng.permutation(self.pages), 0
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            at += n
        slots = np.concatenate([self.slots(b) for b in range(len(lens))] + [np.zeros(0, dtype=np.int64)])
        self.raw = random_tokens(rng, self.pages * page, Hkv, D)
        if slots.size:
            self.cache.put(gpu(slots), *(gpu(a[slots]) for a in self.raw))
        if rows is None:
            self.starts, T = None, len(lens)
        else:
            self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
            T = int(self.starts[-1])
        self.q = acts(rng, T, Hq, D)

    def slots(self, b):
        j = np.arange(max(int(self.lens[b]), 0))
        return self.tables[b][j // self.page].astype(np.int64) * self.page + j % self.page

    def kv(self):
        kc, ks, vc, vs = self.raw
        wide = lambda t: f64(t)[None, :, None]
        return values(kc, ks, wide(self.cache.k_scale)), values(vc, vs, wide(self.cache.v_scale))

    def run(self, **kw):
        more = {} if self.starts is None else {"starts": gpu(self.starts)}
        return vt.paged_attention(self.q.cuda(), self.cache, gpu(self.tables), gpu(self.lens), **more, **kw)

    def check(self, scale=None, window=0, sinks=None):
        got = self.run(scale=scale, window=window, sinks=None if sinks is None else gpu(sinks))
        ref, err = attention(f64(self.q), *self.kv(), self.tables, self.lens, self.starts, self.page,
                             self.D ** -0.5 if scale is None else scale, window, sinks)
        assert_close(got, ref, err)
        return got


HEADS = [(1, 1), (8, 1), (4, 4), (6, 2), (14, 2), (16, 1), (24, 2), (64, 1), (5, 5), (33, 3)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_one_row_per_sequence(Hq, Hkv, D):
    rng = np.random.default_rng(Hq * 300 + D)
    Case(rng, [1, 77, 0, 16, 300, 33], Hq, Hkv, D, 16 << (Hq % 3)).check()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 256), (128, 16), (256, 64)])
@pytest.mark.parametrize("lens", [[0], [1], [15, 16, 17], [63, 64, 65, 127, 128, 129], [0, 0, 5, 0], [2000], [1] * 90])
def test_lengths(lens, D, page):
    rng = np.random.default_rng(len(lens) + D)
    Case(rng, lens, 4, 2, D, page).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_rows_of_a_prompt(Hq, Hkv, D):
    rng = np.random.default_rng(Hq * 301 + D)
    Case(rng, [50, 40, 7, 150], Hq, Hkv, D, 16 << (Hq % 3), rows=[1, 40, 0, 70]).check()


@pytest.mark.parametrize("D,page", [(64, 32), (128, 64), (256, 16)])
@pytest.mark.parametrize("lens,rows", [([1], [1]), ([300], [300]), ([0, 3], [0, 3]), ([129, 400, 5], [129, 2, 5]),
                                       ([1000], [3]), ([128, 128], [128, 64]), ([520, 130], [17, 130])])
def test_chunks(lens, rows, D, page):
    rng = np.random.default_rng(sum(lens) + D)
    Case(rng, lens, 8, 2, D, page, rows=rows).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 100, 129, 5000])
def test_windows_and_sinks(window, D):
    rng = np.random.default_rng(window + D)
    sinks = rng.standard_normal(8).astype(F)
    sinks[2], sinks[3] = -np.inf, 30.0
    Case(rng, [1, 64, 200, 333, 0], 8, 2, D, 16).check(window=window, sinks=sinks)
    Case(rng, [150, 64, 290], 8, 2, D, 32, rows=[150, 5, 130]).check(window=window, sinks=sinks)


@pytest.mark.parametrize("rows", [None, [3, 40, 9]])
def test_more_rows_than_keys_and_rows_behind_the_last(rows):
    """Rows that see no key are zeros; rows of no sequence are left as they were."""
    rng = np.random.default_rng(9)
    c = Case(rng, [10, 20, 0], 4, 2, 64, 16, rows=rows)
    if rows is None:
        c.check(sinks=np.ones(4, dtype=F))
        return
    c.check()
    c.check(sinks=np.ones(4, dtype=F), window=3)
    T = c.q.shape[0]
    wide = torch.full((T + 5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.cat([c.q, torch.full((5, 4, 64), float("nan"), dtype=torch.bfloat16)]).cuda()
    vt.paged_attention(q, c.cache, gpu(c.tables), gpu(c.lens), starts=gpu(c.starts), out=wide)
    assert torch.equal(wide[:T], c.run()) and (wide[T:] == 7).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [None, [70, 3, 130]])
def test_not_a_number_in_keys_values_and_queries(rows, D):
    """A NaN scale of a key makes the rows that see it NaN, one of a value the 16 columns it scales
    of those rows; rows that do not see the token keep their numbers."""
    rng = np.random.default_rng(D)
    c = Case(rng, [90, 200, 130], 6, 2, D, 16, rows=rows)
    kc, ks, vc, vs = c.raw
    first = lambda j, b: c.slots(b)[j]
    vs[first(60, 0), 1, 2], vs[first(150, 1), 0, 0], vs[first(199, 1), 0, 3] = 0x7F, 0xFF, 0x7F
    vs[first(129, 2), 1, 1], ks[first(128, 2), 0, 1], ks[first(5, 0), 0, 0] = 0x7F, 0x7F, 0xFF
    everything = np.arange(c.pages * c.page)
    c.cache.put(gpu(everything), *(gpu(a) for a in c.raw))
    c.q[-1, 5, 3] = float("nan")
    for window in (0, 20):
        got = f64(c.run(window=window))
        ref, err = attention(f64(c.q), *c.kv(), c.tables, c.lens, c.starts, c.page, D ** -0.5, window)
        lost = np.isnan(ref)
        assert lost.any() and np.array_equal(np.isnan(got), lost)
        assert_close(got[~lost], ref[~lost], err[~lost])


@pytest.mark.parametrize("rows", [None, [2, 60]])
def test_large_and_small_scores(rows):
    """Scores of thousands, of one sign, and q from tiny to huge: the largest score alone counts."""
    rng = np.random.default_rng(11)
    for size in (1e-30, 1e-4, 300.0):
        c = Case(rng, [100, 190], 4, 2, 128, 16, rows=rows)
        c.q *= size
        c.check(scale=1.0 if size < 1 else 0.3)
    c = Case(rng, [100, 190], 4, 2, 128, 16, rows=rows)
    c.q *= 1e30
    got = f64(c.run(scale=1e-30))
    assert np.isfinite(got).all()
    c.check(scale=-0.1e-30)
    c.check(scale=0.0)


@pytest.mark.parametrize("rows", [None, [2, 60]])
def test_pages_outside_the_cache_are_left_out(rows):
    rng = np.random.default_rng(12)
    c = Case(rng, [100, 190], 4, 2, 128, 16, rows=rows)
    c.tables[0, 2], c.tables[1, 0], c.tables[1, 11] = -7, c.pages, 2 ** 31 - 1
    c.check()
    c.tables[1, :] = -1
    c.check()
    assert (c.run()[-1] == 0).all()


@pytest.mark.parametrize("rows", [None, [2, 60]])
def test_lens_beyond_the_table_and_below_zero(rows):
    rng = np.random.default_rng(13)
    c = Case(rng, [96, 192], 4, 2, 64, 16, rows=rows)
    keep = c.lens.copy()
    want = c.run()
    c.tables = np.ascontiguousarray(c.tables)
    c.lens = np.array([keep[0], 2 ** 31 - 1], dtype=np.int32)  # the table holds 192 for the second
    got = c.run()
    assert torch.equal(got, want)
    c.lens = np.array([-5, -2 ** 31], dtype=np.int32)
    assert (c.run() == 0).all()


def test_starts_out_of_range_touch_nothing_else():
    rng = np.random.default_rng(14)
    c = Case(rng, [96, 192, 50], 4, 2, 64, 16, rows=[5, 6, 7])
    q = c.q.cuda()
    wide = torch.full((18 + 40, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for s in ([0, 5, 11, 2 ** 31 - 1], [-2 ** 31, 5, 11, 18], [18, 11, 5, 0], [0, 40, 3, 18], [-1, -1, -1, -1],
              [2 ** 31 - 1] * 4):
        vt.paged_attention(q, c.cache, gpu(c.tables), gpu(c.lens), starts=gpu(np.array(s, dtype=np.int32)), out=wide[20:38])
        assert (wide[:20] == 7).all() and (wide[38:] == 7).all()


@pytest.mark.parametrize("rows", [None, [2, 60]])
def test_strides_another_stream_and_the_same_workspace_again(rows):
    rng = np.random.default_rng(15)
    c = Case(rng, [100, 190], 4, 2, 128, 16, rows=rows)
    T = c.q.shape[0]
    want = c.run()
    qkv = torch.full((T, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, :4] = c.q.cuda()
    out = torch.full((T, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    more = {} if rows is None else {"starts": gpu(c.starts)}
    ws = vt.attention_workspace(T, 2, 4, c.cache)
    tables, lens = gpu(c.tables), gpu(c.lens)
    vt.paged_attention(qkv[:, :4], c.cache, tables, lens, out=out[:, 1:5], workspace=ws, **more)
    assert torch.equal(out[:, 1:5], want) and (out[:, 0] == 7).all() and (out[:, 5] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = vt.paged_attention(qkv[:, :4], c.cache, tables, lens, workspace=ws, stream=side, **more)
    side.synchronize()
    assert torch.equal(got, want)
    assert vt.workspace_status(ws) == 0


@pytest.mark.parametrize("rows", [None, [2, 60]])
def test_a_captured_call_follows_lens_and_tables(rows):
    rng = np.random.default_rng(16)
    c = Case(rng, [100, 190], 4, 2, 128, 16, rows=rows)
    more = {} if rows is None else {"starts": gpu(c.starts)}
    q, tables, lens = c.q.cuda(), gpu(c.tables), gpu(c.lens)
    out, ws = torch.empty_like(q), vt.attention_workspace(q.shape[0], 2, 4, c.cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.paged_attention(q, c.cache, tables, lens, out=out, workspace=ws, **more)
    for n in ([100, 190], [64, 3], [100, 77]):
        c.lens = np.array(n, dtype=np.int32)
        c.q = acts(rng, *c.q.shape)
        lens.copy_(gpu(c.lens)), q.copy_(c.q)
        graph.replay()
        assert torch.equal(out, c.run())


@pytest.mark.parametrize("D,Hq,Hkv,lens,rows", [(128, 8, 1, [40000], None), (256, 6, 1, [30000], [5]),
                                               (64, 16, 2, [20001, 5, 9000], [40, 1, 3])])
def test_long_sequences(D, Hq, Hkv, lens, rows):
    rng = np.random.default_rng(D)
    Case(rng, lens, Hq, Hkv, D, 64, rows=rows).check()


def test_two_runs_are_bit_for_bit_alike():
    rng = np.random.default_rng(17)
    for rows in (None, [30, 200, 1]):
        c = Case(rng, [3000, 500, 9000], 8, 2, 128, 16, rows=rows)
        want = c.run()
        for _ in range(5):
            assert torch.equal(c.run(), want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_short_calls_again_and_again(D):
    """Tiles of two or three blocks shared between CTAs, many times over: a part handed on too early
    shows in some runs only."""
    rng = np.random.default_rng(D + 1)
    c = Case(rng, [50, 40, 7, 150], 64, 1, D, 16, rows=[1, 40, 0, 70])
    want = c.check()
    for _ in range(60):
        assert torch.equal(c.run(), want)


def test_two_graphs_share_a_workspace():
    """Replayed one after another in a stream: single rows, and chunks of few and of many rows."""
    rng = np.random.default_rng(18)
    one, many = Case(rng, [300, 40, 1000], 8, 2, 128, 16), Case(rng, [300, 40, 1000], 8, 2, 128, 16, rows=[5, 1, 200])
    ws = vt.attention_workspace(206, 3, 8, one.cache)
    calls = []
    for c in (one, many):
        q, tables, lens = c.q.cuda(), gpu(c.tables), gpu(c.lens)
        more = {} if c.starts is None else {"starts": gpu(c.starts)}
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            vt.paged_attention(q, c.cache, tables, lens, out=out, workspace=ws, **more)
        calls.append((graph, out, c.run(), (q, tables, lens, more)))
    for _ in range(4):
        for graph, out, want, _ in calls:
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
    assert vt.workspace_status(ws) == 0


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(19)
    cases = [Case(rng, [3000, 40, 5000], 8, 2, 128, 16), Case(rng, [3000, 400, 1000], 8, 2, 128, 16, rows=[5, 300, 200])]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    held = [(c.q.cuda(), gpu(c.tables), gpu(c.lens), {} if c.starts is None else {"starts": gpu(c.starts)},
             vt.attention_workspace(c.q.shape[0], 3, 8, c.cache)) for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s, (q, tables, lens, more, ws) in zip(cases, streams, held):
            got.append(vt.paged_attention(q, c.cache, tables, lens, workspace=ws, stream=s, **more))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_a_set_with_limits_of_their_own(D):
    """Few rows of several heads share a set of columns: windows and NaN values that only some of them see."""
    rng = np.random.default_rng(D + 7)
    c = Case(rng, [70, 33, 200, 5], 6, 2, D, 16, rows=[3, 5, 4, 5])
    vs = c.raw[3]
    vs[c.slots(0)[68], 0, 1] = vs[c.slots(1)[32], 1, 0] = vs[c.slots(2)[198], 1, D // 16 - 1] = vs[c.slots(3)[0], 0, 2] = 0x7F
    c.cache.put(gpu(np.arange(c.pages * c.page)), *(gpu(a) for a in c.raw))
    for window in (0, 1, 2, 30):
        got = f64(c.run(window=window))
        ref, err = attention(f64(c.q), *c.kv(), c.tables, c.lens, c.starts, c.page, D ** -0.5, window)
        lost = np.isnan(ref)
        assert lost.any() and np.array_equal(np.isnan(got), lost)
        assert_close(got[~lost], ref[~lost], err[~lost])


def test_more_sequences_than_threads():
    """The line of a thousand short sequences, some of them empty, takes several rounds of the prologue."""
    rng = np.random.default_rng(20)
    lens = rng.integers(0, 40, 1300).tolist()
    Case(rng, lens, 2, 1, 64, 16).check()
    rows = [min(n, int(r)) for n, r in zip(lens, rng.integers(0, 60, 1300))]
    Case(rng, lens, 2, 1, 64, 16, rows=rows).check()


@pytest.mark.parametrize("rows", [None, [3, 70, 9]])
def test_the_output_in_the_place_of_q(rows):
    rng = np.random.default_rng(21)
    c = Case(rng, [3000, 400, 9], 8, 2, 128, 16, rows=rows)
    want, q = c.run(), c.q.cuda()
    more = {} if rows is None else {"starts": gpu(c.starts)}
    for _ in range(10):
        q.copy_(c.q)
        assert vt.paged_attention(q, c.cache, gpu(c.tables), gpu(c.lens), out=q, **more) is q
        assert torch.equal(q, want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [None, [2, 70, 5]])
def test_infinities_in_queries_and_sinks(rows, D):
    """An infinity in q makes its row and head NaN (or a product 0 * inf does), one in the sinks the head;
    what stands beside them keeps its numbers."""
    rng = np.random.default_rng(D + 2)
    c = Case(rng, [100, 190, 40], 6, 2, D, 16, rows=rows)
    T = c.q.shape[0]
    c.q[1, 2, 5], c.q[T - 1, 0, 1], c.q[0, 4, 0] = float("inf"), -float("inf"), float("nan")
    sinks = np.array([0.5, -np.inf, 1.0, np.inf, -2.0, np.nan], dtype=F)
    got = f64(c.run(sinks=gpu(sinks)))
    ref, err = attention(f64(c.q), *c.kv(), c.tables, c.lens, c.starts, c.page, D ** -0.5, 0, sinks)
    lost = np.zeros(got.shape, dtype=bool)
    lost[1, 2] = lost[T - 1, 0] = lost[0, 4] = True
    lost[:, 3] = lost[:, 5] = True
    assert np.isnan(got[lost]).all() and not np.isnan(got[~lost]).any()
    assert_close(got[~lost], ref[~lost], err[~lost])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [None, [2, 70, 5]])
def test_pages_and_rows_more_than_32_bits_apart(rows, D):
    """Pages 2^32 bytes apart and rows of q and out whose offsets pass 2^32 elements give what dense ones do."""
    rng = np.random.default_rng(D + 3)
    c = Case(rng, [40, 75, 17], 8, 1, D, 32, rows=rows, spare=0)
    want = c.run()
    n = c.cache.data.shape[1]
    room = torch.empty(((c.pages - 1) << 32) + n, dtype=torch.uint8, device="cuda")
    far = room.as_strided((c.pages, n), (1 << 32, 1))
    far.copy_(c.cache.data)
    c.cache = vt.KVCache(far, c.page, 1, D, c.cache.k_scale, c.cache.v_scale)
    assert torch.equal(c.run(), want)
    T = c.q.shape[0]
    ld = ((1 << 33) // T + 7) // 8 * 8
    wide = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    q, out = wide[:, :8 * D].unflatten(1, (8, D)), wide[:, 8 * D:16 * D].unflatten(1, (8, D))
    q.copy_(c.q)
    more = {} if rows is None else {"starts": gpu(c.starts)}
    vt.paged_attention(q, c.cache, gpu(c.tables), gpu(c.lens), out=out, **more)
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [None, [3, 60, 40]])
def test_sequences_that_share_pages(rows):
    """A prefix in common: the same pages in several tables, and twice in one."""
    rng = np.random.default_rng(22)
    c = Case(rng, [100, 190, 130], 8, 2, 128, 16, rows=rows)
    c.tables[1, :4] = c.tables[2, :4] = c.tables[0, :4]
    c.tables[2, 5] = c.tables[2, 4]
    c.check()
    c.check(window=50)
