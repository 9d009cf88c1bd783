"""GPU: the paged NVFP4 cache, bit for bit against the formulas in fp32."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from layer_helpers import F, gpu, head_norm, quantise, random_tokens, rotate, values
from rows_helpers import acts

pytestmark = pytest.mark.gpu


def _cache(rng, pages, page, heads, D, fill=0xA5):
    g = lambda: torch.from_numpy(rng.uniform(0.002, 0.006, heads).astype(F)).cuda()
    c = vt.KVCache.empty(pages, page, heads, D, g(), g())
    c.data.fill_(fill)
    return c


def _f32(t):
    return t.float().cpu().numpy()


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F)).to(torch.bfloat16)


def _expect(cache, q, k, v, slots, positions, table, qn, kn, eps, interleaved, raw):
    """raw (the cache's tokens before) after the append, and q."""
    q, k, v = (None if t is None else _f32(t) for t in (q, k, v))
    if kn is not None:
        q, k = None if q is None else head_norm(q, _f32(qn), eps), head_norm(k, _f32(kn), eps)
    if table is not None:
        cos, sin = np.split(_f32(table)[positions], 2, axis=1)
        q, k = (None if t is None else rotate(t, cos, sin, interleaved) for t in (q, k))
    raw = [a.copy() for a in raw]
    there = (slots >= 0) & (slots < cache.pages * cache.page_size)
    for i, (x, g) in enumerate(((k, cache.k_scale), (v, cache.v_scale))):
        codes, scales = quantise(x, _f32(g)[None, :, None])
        raw[2 * i][slots[there]], raw[2 * i + 1][slots[there]] = codes[there], scales[there]
    return raw, q


@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot,norm,fp32,interleaved", [
    (1, 8, 8, 64, 16, 64, False, False, False), (1, 1, 1, 128, 16, 0, False, False, False),
    (37, 32, 8, 128, 16, 128, True, False, False), (5, 6, 2, 256, 64, 64, True, True, False),
    (130, 7, 7, 64, 32, 16, True, False, True), (33, 16, 1, 128, 128, 64, False, False, True),
    (64, 24, 4, 256, 256, 256, True, True, True), (1000, 5, 1, 64, 16, 32, True, True, False),
    (3, 0, 3, 128, 16, 128, True, False, False), (17, 0, 2, 256, 32, 0, False, False, False)])
def test_append(T, Hq, Hkv, D, page, rot, norm, fp32, interleaved):
    rng = np.random.default_rng(T + D + rot)
    pages = -(-T // page) + 2
    cache = _cache(rng, pages, page, Hkv, D)
    everything = torch.arange(pages * page, device="cuda")
    before = [t.cpu().numpy() for t in cache.get(everything)]
    qkv = acts(rng, T, Hq + 2 * Hkv, D) * 2
    q, k, v = (t if t.shape[1] else None for t in qkv.split([Hq, Hkv, Hkv], 1))
    w = lambda: (1 + 0.3 * torch.from_numpy(rng.standard_normal(D).astype(F))).to(torch.float32 if fp32 else torch.bfloat16)
    qn, kn = (w() if Hq else None, w()) if norm else (None, None)
    slots = rng.permutation(pages * page)[:T]
    if T > 2:
        slots[1], slots[T // 2] = -1, pages * page + 3
    positions = rng.integers(0, 500, T)
    table = vt.rope_table(500, rot, 1000.0) if rot else None
    on = lambda t: None if t is None else t.cuda()
    dev = qkv.cuda()
    dq, dk, dv = dev.split([Hq, Hkv, Hkv], 1)
    got = vt.kv_append(dq if Hq else None, dk, dv, cache, gpu(slots), gpu(positions.astype(np.int32)) if rot else None,
                       table, on(qn), on(kn), eps=1e-5, interleaved=interleaved)
    raw, want = _expect(cache, q, k, v, slots, positions, table, qn, kn, 1e-5, interleaved, before)
    for a, b in zip(cache.get(everything), raw):
        assert np.array_equal(a.cpu().numpy(), b)
    if Hq:
        assert torch.equal(got.cpu(), _bf16(want))
    else:
        assert got is None
    kk, vv = vt.kv_read(cache, gpu(slots))
    there = (slots >= 0) & (slots < pages * page)
    for x, c, s, g in ((kk, raw[0], raw[1], cache.k_scale), (vv, raw[2], raw[3], cache.v_scale)):
        # E2M1 * E4M3 is exact; one rounding to fp32, then to bf16
        ref = _bf16(values(c, s, 1.0)[np.where(there, slots, 0)].astype(F) * _f32(g)[None, :, None])
        ref[torch.from_numpy(~there)] = 0
        assert torch.equal(x.cpu(), ref)


def test_append_in_place_and_one_row_of_any_stride():
    rng = np.random.default_rng(3)
    cache = _cache(rng, 4, 16, 2, 128)
    x = acts(rng, 9, 8, 128).cuda()
    q, k, v = x.split([4, 2, 2], 1)
    slots = torch.arange(9, device="cuda")
    pos, table = torch.arange(9, dtype=torch.int32, device="cuda"), vt.rope_table(16, 128)
    want = vt.kv_append(q, k, v, cache, slots, pos, table)
    kept = x[:, 4:].clone()
    assert vt.kv_append(q, k, v, cache, slots, pos, table, out=q) is q
    assert torch.equal(q, want) and torch.equal(x[:, 4:], kept)
    one = acts(rng, 1, 8, 128).cuda()
    odd = torch.zeros(1, 8 * 128 + 8, dtype=torch.bfloat16, device="cuda")[:, :1024].unflatten(1, (8, 128))
    odd.copy_(one)
    a = vt.kv_append(*one.split([4, 2, 2], 1), cache, slots[:1])
    b = vt.kv_append(*odd.split([4, 2, 2], 1), cache, slots[:1])
    assert torch.equal(a, b)


def test_values_that_are_not_finite_zero_or_huge():
    rng = np.random.default_rng(4)
    D, cache = 64, _cache(rng, 2, 16, 1, 64)
    k, v = acts(rng, 6, 1, D), acts(rng, 6, 1, D)
    k[0, 0, 3], k[1, 0, 63], v[2, 0, 17] = float("nan"), float("inf"), -float("inf")
    k[3] = 0
    k[4] *= 1e30
    v[5] *= 1e-30
    slots = np.arange(6)
    before = [t.cpu().numpy() for t in cache.get(torch.arange(32, device="cuda"))]
    vt.kv_append(None, k.cuda(), v.cuda(), cache, gpu(slots))
    raw, _ = _expect(cache, None, k, v, slots, None, None, None, None, 0, False, before)
    got = cache.get(torch.arange(32, device="cuda"))
    for a, b in zip(got, raw):
        assert np.array_equal(a.cpu().numpy(), b)
    assert got[1][0, 0, 0] == 0x7F and got[1][1, 0, 3] == 0x7F and got[3][2, 0, 1] == 0x7F
    kk, vv = vt.kv_read(cache, gpu(slots))
    assert kk[0, 0, :16].isnan().all() and not kk[0, 0, 16:].isnan().any() and vv[2, 0, 16:32].isnan().all()


def test_positions_outside_the_table_give_nan():
    rng = np.random.default_rng(5)
    cache = _cache(rng, 2, 16, 1, 128)
    x = acts(rng, 4, 3, 128).cuda()
    pos = torch.tensor([0, -1, 8, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        q = vt.kv_append(*x.split([1, 1, 1], 1), cache, torch.arange(4, device="cuda"), pos, vt.rope_table(8, 64),
                         interleaved=interleaved)
        k, v = vt.kv_read(cache, torch.arange(4, device="cuda"))
        assert not q[0].isnan().any() and not v.isnan().any()
        for t in (q, k):
            assert t[1:, :, :64].isnan().all() and not t[1:, :, 64:].isnan().any()


@pytest.mark.parametrize("D,page,heads", [(64, 16, 3), (128, 64, 2), (256, 256, 1)])
def test_put_and_get(D, page, heads):
    rng = np.random.default_rng(D)
    pages = 3
    cache = _cache(rng, pages, page, heads, D, 0)
    T = pages * page // 2
    raw = random_tokens(rng, T, heads, D)
    slots = rng.permutation(pages * page)[:T]
    slots[0], slots[1] = -1, pages * page
    cache.put(gpu(slots), *(gpu(a) for a in raw))
    got = cache.get(torch.arange(pages * page, device="cuda"))
    for a, b in zip(got, raw):
        want = np.zeros(a.shape, dtype=np.uint8)
        want[slots[2:]] = b[2:]
        assert np.array_equal(a.cpu().numpy(), want)
    far = cache.get(torch.tensor([-1, pages * page, 2 ** 40, -2 ** 63, 2 ** 63 - 1], device="cuda"))
    assert not any(t.any() for t in far)


def test_pages_of_several_layers_in_one_buffer():
    """Strided pages: what lies between them is not touched."""
    rng = np.random.default_rng(6)
    pages, page, heads, D, layers = 4, 32, 2, 128, 3
    n = vt.KVCache.page_bytes(page, heads, D)
    data = torch.full((pages, layers, n), 0x5A, dtype=torch.uint8, device="cuda")
    one = _cache(rng, pages, page, heads, D, 0x5A)
    cache = vt.KVCache(data[:, 1], page, heads, D, one.k_scale, one.v_scale)
    x = acts(rng, 70, 2 * heads, D).cuda()
    slots = gpu(rng.permutation(pages * page)[:70])
    for c in (cache, one):
        vt.kv_append(None, *x.split([heads, heads], 1), c, slots)
    assert torch.equal(data[:, 1], one.data)
    assert (data[:, 0] == 0x5A).all() and (data[:, 2] == 0x5A).all()
    for a, b in zip(vt.kv_read(cache, slots), vt.kv_read(one, slots)):
        assert torch.equal(a, b)


def test_no_tokens():
    rng = np.random.default_rng(7)
    cache = _cache(rng, 1, 16, 1, 64)
    none = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert vt.kv_append(none, none, none, cache, slots).shape == (0, 1, 64)
    assert vt.kv_append(None, none, none, cache, slots) is None
    assert vt.kv_read(cache, slots)[0].shape == (0, 1, 64)
    assert (cache.data == 0xA5).all()


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(8)
    cache, other = _cache(rng, 8, 16, 2, 128), _cache(np.random.default_rng(8), 8, 16, 2, 128)
    x = acts(rng, 40, 6, 128).cuda()
    slots = torch.arange(40, device="cuda") + 3
    want = vt.kv_append(*x.split([2, 2, 2], 1), cache, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    vt.kv_append(*x.split([2, 2, 2], 1), other, slots, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.data, other.data)
    other.data.zero_()
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.kv_append(*x.split([2, 2, 2], 1), other, slots, out=out)
    x.mul_(-0.5)
    graph.replay()
    want = vt.kv_append(*x.split([2, 2, 2], 1), cache, slots)
    everything = torch.arange(40, device="cuda") + 3
    assert torch.equal(out, want)
    for a, b in zip(other.get(everything), cache.get(everything)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_and_rows_more_than_32_bits_apart(D):
    rng = np.random.default_rng(D + 9)
    pages, page, heads, T = 4, 16, 2, 9
    one = _cache(rng, pages, page, heads, D)
    n = one.data.shape[1]
    room = torch.empty(((pages - 1) << 32) + n, dtype=torch.uint8, device="cuda")
    far = room.as_strided((pages, n), (1 << 32, 1))
    far.copy_(one.data)
    cache = vt.KVCache(far, page, heads, D, one.k_scale, one.v_scale)
    wide = torch.empty((T, 1 << 30), dtype=torch.bfloat16, device="cuda")
    x = acts(rng, T, 4 * heads, D).cuda()
    q, k, v = x.split([2 * heads, heads, heads], 1)
    rows = wide[:, :6 * heads * D].unflatten(1, (6 * heads, D))
    rows[:, :4 * heads] = x
    slots = gpu(rng.permutation(pages * page)[:T])
    want = vt.kv_append(q, k, v, one, slots)
    got = vt.kv_append(rows[:, :2 * heads], rows[:, 2 * heads:3 * heads], rows[:, 3 * heads:4 * heads], cache, slots,
                       out=rows[:, 4 * heads:])
    assert torch.equal(got, want) and torch.equal(far, one.data)
    for a, b in zip(vt.kv_read(cache, slots), vt.kv_read(one, slots)):
        assert torch.equal(a, b)
    for a, b in zip(cache.get(slots), one.get(slots)):
        assert torch.equal(a, b)
    raw = [t.flip(0).contiguous() for t in one.get(slots)]
    cache.put(slots, *raw), one.put(slots, *raw)
    assert torch.equal(far, one.data)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -8, 0.0037, 1e-20, 1e20, 3e-37, 2.0 ** -126])
def test_codes_on_and_beside_their_borders(g, D):
    """Quotients that fall on the borders between codes (globals that are powers of two), and globals from the
    smallest normal number on."""
    rng = np.random.default_rng(D)
    T, H = 500, 3
    gs = torch.full((H,), g, dtype=torch.float32, device="cuda")
    cache = vt.KVCache.empty(-(-T // 16), 16, H, D, gs, gs)
    k = _bf16(rng.standard_normal((T, H, D)) * np.exp(rng.uniform(-6, 6, (T, H, 1))) * min(g * 100, 1e30))
    v = _bf16(rng.integers(-60, 61, (T, H, D)) / 8 * g)
    slots = torch.arange(T, device="cuda")
    vt.kv_append(None, k.cuda(), v.cuda(), cache, slots)
    kc, ks, vc, vs = (t.cpu().numpy() for t in cache.get(slots))
    for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
        want = quantise(_f32(x), F(g))
        assert np.array_equal(codes, want[0]) and np.array_equal(scales, want[1])
