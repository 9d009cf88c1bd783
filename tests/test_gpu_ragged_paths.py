"""GPU: every kernel variant of the ragged products through every form of call, just below and above
the sizes at which the variant changes, against fp64; each call's status is read."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import (BF16, acts, assert_close, f64, group64, products64, random_weight,
                          silu_mul64, weight64)

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _plain(rng, fmt, E, N, K, wide):
    c, s, g = random_weight(rng, fmt, E, N, K, wide)
    return vt.PackedWeight.grouped(_dev(c), _dev(s), g, fmt, E, N, K), \
        [weight64(fmt, c[e], s[e], g[e]) for e in range(E)]


def _paired(rng, fmt, E, I, K, wide):
    a, b = random_weight(rng, fmt, E, I, K, wide), random_weight(rng, fmt, E, I, K, wide)
    W = vt.PackedWeight.grouped_gate_up(*((_dev(c), _dev(s), g) for c, s, g in (a, b)), fmt, E, I, K)
    return W, [[weight64(fmt, c[e], s[e], g[e]) for e in range(E)] for c, s, g in (a, b)]


def _groups(rng, M, topk, E):
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
    weights = rng.random((M, topk)).astype(np.float32)
    order, offsets = group64(ids, E)
    return vt.RowGroups(_dev(ids), _dev(order), _dev(offsets), _dev(weights)), order, offsets, weights


# 24 experts of 796 rows: 7 row tiles, the last one short and without a partner.  152 SMs take two
# row tiles per item from 22 of these experts on, 128-row token tiles from 64 rows per expert on, and
# gathering loaders from more than 2^23 gathered values on (topk > 1).
E, N, K = 24, 796, 544
SIZES = {"one row tile": (2, 8, 64), "two": (150, 8, 64), "64 rows per expert less 8": (191, 8, 64),
         "64 rows per expert": (192, 8, 128), "2^23 values less 2304": (1927, 8, 128),
         "2^23 values and 2048": (1928, 8, 128), "one slot each": (1600, 1, 128)}


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4", "wide mxfp4"])
@pytest.mark.parametrize("size", list(SIZES))
def test_plain_products_and_their_sum(kind, size):
    M, topk, tokens = SIZES[size]
    fmt, wide = (vt.NVFP4 if kind == "nvfp4" else vt.MXFP4), kind.startswith("wide")
    rng = np.random.default_rng(M)
    W, ws = _plain(rng, fmt, E, N, K, wide)
    groups, order, offsets, weights = _groups(rng, M, topk, E)
    space = W.ragged_workspace(M, topk)
    x, xg = acts(rng, M, K), acts(rng, M * topk, K)
    run = lambda a, **kw: f64(vt.w4a16_gemm_ragged(a.cuda(), W, groups, workspace=space, **kw))
    gathered, scattered = run(x), run(x, scatter=True)
    assert W.stats()["m_tile"] == tokens
    assert np.array_equal(scattered[order], gathered)
    grouped = run(xg, gather=False)
    y = f64(vt.w4a16_gemm_ragged_combine(xg.cuda(), W, groups, workspace=space))
    assert vt.workspace_status(space) == 0
    ref, err = np.zeros((M, N)), np.zeros((M, N))
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        assert_close(gathered[i], *products64(f64(x[order[i] // topk]), ws[e]), what=e)
        d, derr = products64(f64(xg[i]), ws[e])
        assert_close(grouped[i], d, derr, what=e)
        m, j = order[i] // topk, order[i] % topk
        w = weights[m, j][:, None].astype(np.float64)
        ref[m] += w * d  # (an expert serves a token once)
        err[m] += w * (derr + (BF16 + topk * 2.0 ** -22) * (np.abs(d) + derr))
    assert_close(y, ref, err)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4", "wide mxfp4"])
@pytest.mark.parametrize("size", list(SIZES))
def test_silu_mul_gathered_and_grouped(kind, size):
    M, topk, tokens = SIZES[size]
    fmt, wide = (vt.NVFP4 if kind == "nvfp4" else vt.MXFP4), kind.startswith("wide")
    rng = np.random.default_rng(M + 1)
    W, (wg, wu) = _paired(rng, fmt, E, N // 2, K, wide)
    groups, order, offsets, _ = _groups(rng, M, topk, E)
    space = W.ragged_workspace(M, topk)
    x, xg = acts(rng, M, K), acts(rng, M * topk, K)
    gathered = f64(vt.w4a16_gemm_ragged_silu_mul(x.cuda(), W, groups, workspace=space))
    assert W.stats()["m_tile"] == tokens
    grouped = f64(vt.w4a16_gemm_ragged_silu_mul(xg.cuda(), W, groups, workspace=space, gather=False))
    assert vt.workspace_status(space) == 0
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        assert_close(gathered[i], *silu_mul64(f64(x[order[i] // topk]), wg[e], wu[e]), what=e)
        assert_close(grouped[i], *silu_mul64(f64(xg[i]), wg[e], wu[e]), what=e)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4", "wide mxfp4"])
@pytest.mark.parametrize("K", [1024, 1056, 2048, 2080, 4128])
def test_rows_longer_than_the_conversion_holds(kind, K):
    fmt, wide = (vt.NVFP4 if kind == "nvfp4" else vt.MXFP4), kind.startswith("wide")
    rng = np.random.default_rng(K)
    M, topk, E, N = 30, 2, 5, 72
    W, ws = _plain(rng, fmt, E, N, K, wide)
    groups, order, offsets, _ = _groups(rng, M, topk, E)
    x, space = acts(rng, M, K), W.ragged_workspace(M, topk)
    x[:, K - 3] *= 64  # the row's largest value is among the last
    y = f64(vt.w4a16_gemm_ragged(x.cuda(), W, groups, workspace=space))
    assert vt.workspace_status(space) == 0
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        assert_close(y[i], *products64(f64(x[order[i] // topk]), ws[e]), what=e)


@pytest.mark.parametrize("M,topk,E,N,K", [(6, 2, 4, 136, 96), (700, 4, 16, 1400, 224)])
def test_the_sum_reports_pairs_and_offsets_out_of_range(M, topk, E, N, K):
    """They are not followed: nothing beside the output is written, tokens of no such pair are right."""
    rng = np.random.default_rng(M)
    W, _ = _plain(rng, vt.NVFP4, E, N, K, False)
    groups, order, offsets, _ = _groups(rng, M, topk, E)
    h, space = acts(rng, M * topk, K).cuda(), W.ragged_workspace(M, topk)
    want = vt.w4a16_gemm_ragged_combine(h, W, groups, workspace=space)
    assert vt.workspace_status(space) == 0
    wild = order.copy()
    at = rng.choice(M * topk, 4, replace=False)
    wild[at] = [-1, M * topk, 2 ** 31 - 1, -2 ** 31]
    full = torch.full((M + 2, N + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[1:-1, 3:3 + N]
    for o, f in ((wild, offsets), (order, np.where(np.arange(E + 1) == E // 2, M * topk + 9, offsets)),
                 (order, np.where(np.arange(E + 1) == 1, -5, offsets))):
        bad = vt.RowGroups(groups.ids, _dev(o), _dev(f.astype(np.int32)), groups.weights)
        vt.w4a16_gemm_ragged_combine(h, W, bad, out=out, workspace=space)
        assert vt.workspace_status(space) == 6
        if o is wild:
            right = np.setdiff1d(np.arange(M), order[at] // topk)
            assert torch.equal(out[_dev(right)], want[_dev(right)])
        keep = full.clone()
        keep[1:-1, 3:3 + N] = 7.0
        assert torch.all(keep == 7.0)
