"""GPU: low-rank adapters of many requests beside a shared projection, against fp64."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import acts, assert_close, f64, random_weight, weight64

pytestmark = pytest.mark.gpu


def _adapters(rng, L, R, K, N, ranks=None):
    A, B = acts(rng, L, R, K), acts(rng, L, N, R)
    scale = torch.from_numpy(rng.uniform(-1, 2, L).astype(np.float32))
    ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32)
    return A, B, scale, ranks


def _ref(x, y, ids, A, B, scale, ranks):
    """y + s B (A x) in fp64 and the bound on its fp32 evaluation: v = A x is held to 2^-16 at
    least (fp32, or two bf16 terms), both sums to n * 2^-23 of their absolute values."""
    L, R, K = A.shape
    out, err = f64(y).copy(), np.zeros(y.shape)
    for m, a in enumerate(ids):
        if 0 <= a < L:
            r = R if ranks is None else min(max(int(ranks[a]), 0), R)
            Aa, Ba, s = f64(A[a, :r]), f64(B[a, :, :r]), float(scale[a])
            v, va = Aa @ f64(x[m]), np.abs(Aa) @ np.abs(f64(x[m]))
            out[m] += s * (Ba @ v)
            err[m] = abs(s) * (np.abs(Ba) @ ((K * 2.0 ** -23 + r * 2.0 ** -23) * va + 2.0 ** -15 * np.abs(v)))
    return out, err + 2.0 ** -20 * np.abs(f64(y))


def _run(x, y, ids, A, B, scale, ranks, **kw):
    ad = vt.LoraAdapters(A.cuda(), B.cuda(), scale.cuda(), None if ranks is None else ranks.cuda())
    groups = vt.group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), A.shape[0])
    return vt.lora_add(x.cuda(), ad, groups, y.cuda(), **kw)


@pytest.mark.parametrize("M,L,R,K,N", [
    (1, 1, 1, 1, 1), (1, 4, 16, 512, 384), (1, 2, 8, 4096, 130), (3, 2, 5, 33, 17), (16, 16, 16, 256, 256),
    (17, 3, 64, 1000, 321), (96, 64, 32, 640, 512), (130, 2, 128, 264, 200), (700, 3, 24, 520, 328),
    (1025, 1, 16, 128, 96), (64, 1, 100, 4100, 1031)])
def test_adapters(M, L, R, K, N):
    rng = np.random.default_rng(M + K)
    A, B, scale, _ = _adapters(rng, L, R, K, N)
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = rng.integers(0, L, M)
    out = _run(x, y, ids, A, B, scale, None)
    assert_close(out, *_ref(x, y, ids, A, B, scale, None))


def test_ranks_missing_adapters_and_unused_storage():
    rng = np.random.default_rng(2)
    M, L, R, K, N = 90, 6, 32, 320, 264
    ranks = [32, 1, 0, 17, 99, -3]  # clamped to [0, R]
    A, B, scale, ranks = _adapters(rng, L, R, K, N, ranks)
    for a in range(L):  # what lies past an adapter's rank is not read as numbers
        r = min(max(int(ranks[a]), 0), R)
        A[a, r:], B[a, :, r:] = float("nan"), float("inf")
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = rng.integers(-2, L + 2, M)
    out = _run(x, y, ids, A, B, scale, ranks)
    assert_close(out, *_ref(x, y, ids, A, B, scale, ranks))
    none = torch.from_numpy((ids < 0) | (ids >= L))
    assert torch.equal(out.cpu()[none], y[none])


@pytest.mark.parametrize("R", [24, 64, 128])
@pytest.mark.parametrize("M", [1, 4])
def test_few_rows_with_ranks_and_unused_storage(M, R):
    rng = np.random.default_rng(R + M)
    L, K, N = 4, 2056, 1032
    A, B, scale, ranks = _adapters(rng, L, R, K, N, [R - 8, 3, 17, R])
    for a in range(L):
        A[a, ranks[a]:], B[a, :, ranks[a]:] = float("nan"), float("inf")
    x, y = acts(rng, M, K), acts(rng, M, N)
    for first in range(L):
        ids = (first + np.arange(M)) % L
        out = _run(x, y, ids, A, B, scale, ranks)
        assert_close(out, *_ref(x, y, ids, A, B, scale, ranks))


@pytest.mark.parametrize("K,N,padx,pady", [(128, 128, 0, 0), (128, 128, 8, 8), (129, 127, 1, 1),
                                           (132, 130, 4, 2), (136, 133, 3, 5)])
def test_strides_in_place_and_canaries(K, N, padx, pady):
    rng = np.random.default_rng(K + padx)
    M, L, R = 41, 3, 16
    A, B, scale, _ = _adapters(rng, L, R, K, N)
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = rng.integers(-1, L, M)
    ref = _ref(x, y, ids, A, B, scale, None)
    xw = torch.full((M, K + 2 * padx), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:, padx:padx + K] = x.cuda()
    yw = torch.full((M + 2, N + 2 * pady), 5.0, dtype=torch.bfloat16, device="cuda")
    yv = yw[1:-1, pady:pady + N]
    yv.copy_(y.cuda())
    ad = vt.LoraAdapters(A.cuda(), B.cuda(), scale.cuda())
    groups = vt.group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), L)
    xv = xw[:, padx:padx + K]
    out = vt.lora_add(xv, ad, groups, yv)          # into a new tensor
    assert_close(out, *ref)
    r = vt.lora_add(xv, ad, groups, yv, out=yv)    # in place
    assert r is yv and torch.equal(yv, out)
    keep = yw.clone()
    keep[1:-1, pady:pady + N] = 5.0
    assert torch.all(keep == 5.0)


def test_beside_a_packed_projection_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(7)
    N, K, M, L, R = 192, 256, 12, 5, 8
    c, s, g = random_weight(rng, vt.NVFP4, 1, N, K)
    W = vt.PackedWeight.from_codes(torch.from_numpy(c[0]).cuda(), torch.from_numpy(s[0]).cuda(), g[0],
                                   vt.NVFP4, N, K)
    w64 = weight64(vt.NVFP4, c[0], s[0], g[0])
    A, B, scale, _ = _adapters(rng, L, R, K, N)
    ad = vt.LoraAdapters(A.cuda(), B.cuda(), scale.cuda())
    ids = rng.integers(-1, L, M)
    groups = vt.group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), L)
    ws = W.new_workspace(M)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        vt.w4a16_gemm(x, W, out=y, workspace=ws, stream=stream)
        vt.lora_add(x, ad, groups, y, out=y, stream=stream)

    def check(xh):
        torch.cuda.synchronize()
        base = torch.from_numpy(f64(xh) @ w64.T)
        ref, err = _ref(xh, base, ids, A, B, scale, None)
        # the projection's own rounding to bf16 and fp32 sum come first
        err = err + 2.0 ** -8 * np.abs(base.numpy()) + K * 2.0 ** -22 * (np.abs(f64(xh)) @ np.abs(w64).T)
        assert_close(y, ref, err)

    side = torch.cuda.Stream()
    xh = acts(rng, M, K)
    x.copy_(xh)
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    check(xh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        xh = acts(rng, M, K)
        x.copy_(xh)
        graph.replay()
        check(xh)


def test_infinite_inputs_stay_in_their_rows():
    rng = np.random.default_rng(9)
    M, L, R, K, N = 20, 2, 16, 128, 64
    A, B, scale, _ = _adapters(rng, L, R, K, N)
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = np.arange(M) % L
    x[3, 5], x[4, 7], y[6, 2] = float("nan"), float("inf"), float("inf")
    out = f64(_run(x, y, ids, A, B, scale, None))
    assert np.isnan(out[3]).all() and not np.isfinite(out[4]).any()
    assert out[6, 2] == np.inf and np.isfinite(np.delete(out[6], 2)).all()
    fine = [m for m in range(M) if m not in (3, 4, 6)]
    ref, err = _ref(x[fine], y[fine], ids[fine], A, B, scale, None)
    assert_close(out[fine], ref, err)


def test_repeats_are_bit_equal():
    rng = np.random.default_rng(10)
    M, L, R, K, N = 300, 2, 16, 512, 256
    A, B, scale, _ = _adapters(rng, L, R, K, N)
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = np.array([0] * 200 + [1] * 100)
    a = _run(x, y, ids, A, B, scale, None)
    assert torch.equal(a, _run(x, y, ids, A, B, scale, None))


@pytest.mark.parametrize("M,L,R,K,N", [
    (1, 2, 16, 512, 1027), (2, 1, 64, 264, 513), (50, 9, 32, 256, 130), (90, 6, 64, 136, 1285),
    (90, 30, 128, 128, 301), (1025, 2, 32, 128, 131), (400, 2, 64, 256, 333), (300, 1, 128, 72, 259)])
def test_outputs_of_any_width_and_place(M, L, R, K, N):
    """Columns, row strides and bases of y and out that are not whole 16-byte pieces, apart and in
    place; what lies around them stays."""
    rng = np.random.default_rng(N)
    A, B, scale, _ = _adapters(rng, L, R, K, N)
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = rng.integers(-1, L, M)
    ref, err = _ref(x, y, ids, A, B, scale, None)
    assert_close(_run(x, y, ids, A, B, scale, None), ref, err)
    for pad, first in ((1, 0), (3, 1), (2, 2), (8, 5)):
        wide_y = torch.full((M, N + pad + first), 9.0, dtype=torch.bfloat16, device="cuda")
        wide_o = torch.full((M, N + 2 * pad + first), 7.0, dtype=torch.bfloat16, device="cuda")
        sy, so = wide_y[:, first:first + N], wide_o[:, first:first + N]
        sy.copy_(y)
        _run(x, sy, ids, A, B, scale, None, out=so)
        assert_close(so, ref, err)
        assert (wide_o[:, :first] == 7).all() and (wide_o[:, first + N:] == 7).all()
        _run(x, sy, ids, A, B, scale, None, out=sy)  # in place
        assert torch.equal(sy, so)
        assert (wide_y[:, :first] == 9).all() and (wide_y[:, first + N:] == 9).all()
