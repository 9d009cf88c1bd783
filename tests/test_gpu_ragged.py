"""GPU: the ragged expert products, their epilogues and the block that chains them, against
fp64 forms of the definitions, at the sizes and routings where they can go wrong."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from fp4_weight_only_nvfp4_gb300 import _lib
from rows_helpers import (BF16, acts, assert_close, f64, group64, products64, random_weight,
                          silu_mul64, weight64)

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _plain(rng, fmt, E, N, K, wide=False):
    c, s, g = random_weight(rng, fmt, E, N, K, wide)
    return vt.PackedWeight.grouped(_dev(c), _dev(s), g, fmt, E, N, K), \
        [weight64(fmt, c[e], s[e], g[e]) for e in range(E)]


def _paired(rng, fmt, E, I, K, wide=False):
    a, b = random_weight(rng, fmt, E, I, K, wide), random_weight(rng, fmt, E, I, K, wide)
    b = (b[0], b[1], [2 * x for x in b[2]] if fmt == 0 else b[2])
    W = vt.PackedWeight.grouped_gate_up(*((_dev(c), _dev(s), g) for c, s, g in (a, b)), fmt, E, I, K)
    return W, [[weight64(fmt, c[e], s[e], g[e]) for e in range(E)] for c, s, g in (a, b)]


def _groups(ids, E, weights=None):
    order, offsets = group64(ids, E)
    return vt.RowGroups(_dev(ids.astype(np.int32)), _dev(order), _dev(offsets),
                        None if weights is None else _dev(weights.astype(np.float32))), order, offsets


def _ids(rng, M, topk, E):
    return np.stack([rng.permutation(E)[:topk] for _ in range(M)]).astype(np.int32) if M \
        else np.zeros((0, topk), np.int32)


def _counts_ids(counts):
    """topk = 1 ids giving expert e counts[e] rows, dealt out in turn."""
    left, ids = list(counts), []
    while sum(left):
        for e in range(len(left)):
            if left[e]:
                left[e] -= 1
                ids.append(e)
    return np.array(ids, np.int32).reshape(-1, 1)


def _ref(x, ws, order, offsets, topk, gather):
    """Outputs in group order and their error bounds."""
    n = int(offsets[-1])
    out, err = np.zeros((len(order), ws[0].shape[0])), np.zeros((len(order), ws[0].shape[0]))
    for e, w in enumerate(ws):
        i = np.arange(offsets[e], offsets[e + 1])
        rows = order[i] // topk if gather else i
        out[i], err[i] = products64(x[rows], w)
    return out[:n], err[:n]


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("M,topk,E,N,K", [
    (1, 1, 1, 1, 32), (1, 2, 4, 128, 64), (2, 8, 16, 257, 96), (5, 3, 7, 130, 224), (40, 4, 8, 300, 512),
    (33, 8, 60, 96, 1056), (300, 2, 5, 384, 160)])
def test_products(fmt, M, topk, E, N, K):
    rng = np.random.default_rng(M * 31 + N)
    W, ws = _plain(rng, fmt, E, N, K)
    ids = _ids(rng, M, topk, E)
    groups, order, offsets = _groups(ids, E)
    x = acts(rng, M, K)
    y = vt.w4a16_gemm_ragged(x.cuda(), W, groups)
    ref, err = _ref(f64(x), ws, order, offsets, topk, True)
    assert_close(y, ref, err)
    # pair order out, grouped rows in
    xg = acts(rng, M * topk, K)
    y = vt.w4a16_gemm_ragged(xg.cuda(), W, groups, gather=False, scatter=True)
    ref, err = _ref(f64(xg), ws, order, offsets, topk, False)
    assert_close(f64(y)[order], ref, err)
    y = vt.w4a16_gemm_ragged(x.cuda(), W, groups, scatter=True)
    assert_close(f64(y)[order], *_ref(f64(x), ws, order, offsets, topk, True))
    assert vt.workspace_status(W.ragged_workspace(0, 1)) == 0


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
def test_group_sizes_around_every_tile_edge(fmt):
    counts = [1, 7, 8, 9, 15, 16, 17, 0, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 0, 255, 256, 257,
              500, 513, 0]
    rng = np.random.default_rng(11)
    E, N, K = len(counts), 200, 192
    W, ws = _plain(rng, fmt, E, N, K)
    ids = _counts_ids(counts)
    groups, order, offsets = _groups(ids, E)
    x = acts(rng, len(ids), K)
    y = vt.w4a16_gemm_ragged(x.cuda(), W, groups)
    assert_close(y, *_ref(f64(x), ws, order, offsets, 1, True))


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("M,topk,E,I,K", [(1, 1, 1, 1, 32), (1, 8, 12, 96, 256), (3, 2, 5, 65, 64),
                                          (50, 4, 9, 130, 416), (400, 2, 3, 192, 128),
                                          (1100, 1, 2, 100, 96)])
def test_silu_mul(fmt, M, topk, E, I, K):
    rng = np.random.default_rng(M + I)
    W, (wg, wu) = _paired(rng, fmt, E, I, K)
    ids = _ids(rng, M, topk, E)
    groups, order, offsets = _groups(ids, E)
    x = acts(rng, M, K)
    h = vt.w4a16_gemm_ragged_silu_mul(x.cuda(), W, groups)
    ref, err = np.zeros((M * topk, I)), np.zeros((M * topk, I))
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        ref[i], err[i] = silu_mul64(f64(x)[order[i] // topk], wg[e], wu[e])
    assert_close(h, ref, err)


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("M,topk,E,N,K", [(1, 1, 1, 3, 32), (1, 8, 12, 256, 96), (2, 3, 5, 131, 64),
                                          (70, 4, 9, 130, 224), (513, 2, 3, 256, 128)])
def test_combine(fmt, M, topk, E, N, K):
    rng = np.random.default_rng(M + N)
    W, ws = _plain(rng, fmt, E, N, K)
    ids = _ids(rng, M, topk, E)
    if M > 1:  # a slot in no group, with a weight that must not count; a token with none
        ids[1, 0], ids[M // 2, :] = -1, E
    weights = rng.random((M, topk)).astype(np.float32)
    groups, order, offsets = _groups(ids, E, weights)
    h = acts(rng, M * topk, K)
    ws_ = W.ragged_workspace(M, topk)
    ws_[256:] = 0x7F  # scratch of an earlier call: not zero
    y = vt.w4a16_gemm_ragged_combine(h.cuda(), W, groups, workspace=ws_)
    d, derr = _ref(f64(h), ws, order, offsets, topk, False)
    ref, err = np.zeros((M, N)), np.zeros((M, N))
    for i, p in enumerate(order[:offsets[-1]]):
        w = float(weights[p // topk, p % topk])
        ref[p // topk] += w * d[i]
        # each pair's output may be rounded to bf16 before the fp32 sum
        err[p // topk] += w * (derr[i] + (BF16 + topk * 2.0 ** -22) * (np.abs(d[i]) + derr[i]))
    assert_close(y, ref, err)
    assert vt.workspace_status(ws_) == 0


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("M,topk,E,N,K,wide", [
    (60, 4, 200, 300, 96, False),      # enough groups for two weight row tiles per item, an odd one last
    (500, 3, 170, 128, 352, True),     # a single row tile; mixed operand types
    (2100, 8, 64, 640, 544, True)])    # more gathered rows than are written in group order first
def test_many_items(fmt, M, topk, E, N, K, wide):
    rng = np.random.default_rng(M)
    wide = wide and fmt == vt.MXFP4
    W, ws = _plain(rng, fmt, E, N, K, wide)
    Wp, (wg, wu) = _paired(rng, fmt, E, N // 2 - 3, K, wide)
    ids = _ids(rng, M, topk, E)
    groups, order, offsets = _groups(ids, E)
    x = acts(rng, M, K)
    ref, err = _ref(f64(x), ws, order, offsets, topk, True)
    assert_close(vt.w4a16_gemm_ragged(x.cuda(), W, groups), ref, err)
    assert_close(f64(vt.w4a16_gemm_ragged(x.cuda(), W, groups, scatter=True))[order], ref, err)
    h = f64(vt.w4a16_gemm_ragged_silu_mul(x.cuda(), Wp, groups))
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        assert_close(h[i], *silu_mul64(f64(x)[order[i] // topk], wg[e], wu[e]))


def test_wide_mx_scales():
    rng = np.random.default_rng(3)
    E, N, K, M = 3, 140, 256, 37
    W, ws = _plain(rng, vt.MXFP4, E, N, K, wide=True)
    groups, order, offsets = _groups(_ids(rng, M, 2, E), E)
    x = acts(rng, M, K)
    assert_close(vt.w4a16_gemm_ragged(x.cuda(), W, groups), *_ref(f64(x), ws, order, offsets, 2, True))
    Wp, (wg, wu) = _paired(rng, vt.MXFP4, E, 70, K, wide=True)
    h = f64(vt.w4a16_gemm_ragged_silu_mul(x.cuda(), Wp, groups))
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        assert_close(h[i], *silu_mul64(f64(x)[order[i] // 2], wg[e], wu[e]))


def test_activations_of_every_magnitude():
    """Rows at the ends of bf16's range, and one row's NaN and infinity staying its own."""
    rng = np.random.default_rng(8)
    E, N, K, M = 2, 128, 128, 24
    W, ws = _plain(rng, vt.NVFP4, E, N, K)
    groups, order, offsets = _groups(_ids(rng, M, 1, E), E)
    x = acts(rng, M, K).float()
    x[3] *= 2.0 ** 100
    x[4] *= 2.0 ** -100
    x[5] = 0
    x[6, 10] = float("nan")
    x[7, 11] = float("inf")
    x = x.to(torch.bfloat16)
    y = f64(vt.w4a16_gemm_ragged(x.cuda(), W, groups, scatter=True))
    assert np.isnan(y[6]).all()
    assert not np.isfinite(y[7][[n for n in range(N) if ws[int(groups.ids[7])][n, 11] != 0]]).any()
    fine = [m for m in range(M) if m not in (6, 7)]
    for m in fine:
        ref, err = products64(f64(x)[m:m + 1], ws[int(groups.ids[m])])
        assert_close(y[m:m + 1], ref, err)
    assert not y[5].any()


def test_plain_weight_serves_one_group():
    rng = np.random.default_rng(4)
    N, K, M = 100, 96, 50
    c, s, g = random_weight(rng, vt.NVFP4, 1, N, K)
    W = vt.PackedWeight.from_codes(_dev(c[0]), _dev(s[0]), g[0], vt.NVFP4, N, K)
    ids = np.where(np.arange(M) % 3 == 0, -1, 0).astype(np.int32).reshape(-1, 1)
    groups, order, offsets = _groups(ids, 1)
    x = acts(rng, M, K)
    y = vt.w4a16_gemm_ragged(x.cuda(), W, groups)
    assert_close(f64(y)[:offsets[-1]], *_ref(f64(x), [weight64(0, c[0], s[0], g[0])], order, offsets, 1, True))


def test_only_the_outputs_are_written():
    """Strided operands; rows of pairs in no group and the columns beside the output keep
    what they held."""
    rng = np.random.default_rng(6)
    E, K, M, topk = 4, 64, 30, 3
    for N in (128, 97):
        W, ws = _plain(rng, vt.NVFP4, E, N, K)
        ids = _ids(rng, M, topk, E)
        ids[::4] = -1
        groups, order, offsets = _groups(ids, E)
        for pad in (0, 1, 8):
            xw = torch.full((M, K + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
            x = acts(rng, M, K)
            xw[:, 8:8 + K] = x.cuda()
            full = torch.full((M * topk + 2, N + 2 * pad + 3), 7.0, dtype=torch.bfloat16, device="cuda")
            out = full[1:-1, pad:pad + N]
            for scatter in (False, True):
                full.fill_(7.0)
                vt.w4a16_gemm_ragged(xw[:, 8:8 + K], W, groups, out=out, scatter=scatter)
                n = int(offsets[-1])
                rows = order[:n] if scatter else np.arange(n)
                assert_close(f64(out)[rows], *_ref(f64(x), ws, order, offsets, topk, True))
                keep = full.clone()
                keep[1:-1, pad:pad + N][torch.from_numpy(rows.astype(np.int64)).cuda()] = 7.0
                assert torch.all(keep == 7.0)


def test_block_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(9)
    E, I, H, M, topk = 8, 96, 160, 21, 2
    Wgu, (wg, wu) = _paired(rng, vt.NVFP4, E, I, H)
    Wd, wd = _plain(rng, vt.NVFP4, E, H, I)
    ws = Wd.ragged_workspace(M, topk)
    gws = vt.group_workspace(M, topk, E, "cuda")
    groups = vt.RowGroups.empty(M, topk, E, "cuda", weights=True)
    x = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(M, E, device="cuda")
    h = torch.empty(M * topk, I, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")

    def block(stream=None):
        vt.moe_route(logits, topk, out=groups, workspace=gws, stream=stream)
        vt.moe_ffn(x, Wgu, Wd, groups, out=out, h=h, workspace=ws, stream=stream)

    def check(xh, lh):
        torch.cuda.synchronize()
        ids, w = f64(groups.ids).astype(int), f64(groups.weights)
        assert np.array_equal(ids, np.argsort(-lh.double().numpy(), axis=1, kind="stable")[:, :topk])
        ref, err = np.zeros((M, H)), np.zeros((M, H))
        for m in range(M):
            for j in range(topk):
                hh, herr = silu_mul64(f64(xh)[m:m + 1], wg[ids[m, j]], wu[ids[m, j]])
                herr = herr + BF16 * (np.abs(hh) + herr)       # h is bf16
                d, derr = products64(hh, wd[ids[m, j]])
                derr = derr + herr @ np.abs(wd[ids[m, j]]).T
                ref[m] += w[m, j] * d[0]
                err[m] += w[m, j] * (derr[0] + (BF16 + topk * 2.0 ** -22) * (np.abs(d[0]) + derr[0]))
        assert_close(out, ref, err)

    side = torch.cuda.Stream()
    xh, lh = acts(rng, M, H), torch.randn(M, E)
    x.copy_(xh), logits.copy_(lh)
    side.wait_stream(torch.cuda.current_stream())
    block(side)
    side.synchronize()
    check(xh, lh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for _ in range(2):
        xh, lh = acts(rng, M, H), torch.randn(M, E)
        x.copy_(xh), logits.copy_(lh)
        graph.replay()
        check(xh, lh)
    assert vt.workspace_status(ws) == 0


def test_repeats_are_bit_equal():
    rng = np.random.default_rng(10)
    E, N, K = 3, 256, 512
    W, _ = _plain(rng, vt.NVFP4, E, N, K)
    x = acts(rng, 400, K).cuda()
    ids = np.array([1] * 300 + [0] * 60 + [2] * 40, np.int32).reshape(-1, 1)
    groups, _, _ = _groups(ids, E)
    a = vt.w4a16_gemm_ragged(x, W, groups, scatter=True)
    b = vt.w4a16_gemm_ragged(x, W, groups, scatter=True)
    assert torch.equal(a, b)


def test_paired_grouped_weight_unpacks_to_its_sources():
    rng = np.random.default_rng(12)
    for fmt in (vt.NVFP4, vt.MXFP4):
        E, I, K = 3, 70, 96
        a, b = random_weight(rng, fmt, E, I, K), random_weight(rng, fmt, E, I, K)
        W = vt.PackedWeight.grouped_gate_up(*((_dev(c), _dev(s), g) for c, s, g in (a, b)), fmt, E, I, K)
        codes, scales = W.unpack()
        assert np.array_equal(codes.cpu().numpy().reshape(E, 2 * I, -1), np.concatenate([a[0], b[0]], 1))
        assert np.array_equal(scales.cpu().numpy().reshape(E, 2 * I, -1), np.concatenate([a[1], b[1]], 1))


def test_wrong_shapes_are_refused():
    rng = np.random.default_rng(13)
    E, N, K, M, topk = 4, 64, 64, 6, 2
    W, _ = _plain(rng, vt.NVFP4, E, N, K)
    Wp, _ = _paired(rng, vt.NVFP4, E, 32, K)
    groups, _, _ = _groups(_ids(rng, M, topk, E), E)
    other, _, _ = _groups(_ids(rng, M, topk, E), E + 1)
    x = acts(rng, M, K).cuda()
    with pytest.raises(ValueError, match="experts"):
        vt.w4a16_gemm_ragged(x, W, other)
    with pytest.raises(ValueError, match="A must be"):
        vt.w4a16_gemm_ragged(x[:-1], W, groups)
    with pytest.raises(ValueError, match="A must be"):
        vt.w4a16_gemm_ragged(x, W, groups, gather=False)
    with pytest.raises(ValueError, match="out must be"):
        vt.w4a16_gemm_ragged(x, W, groups, out=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="weights"):
        vt.w4a16_gemm_ragged_combine(acts(rng, M * topk, K).cuda(), W, groups)
    with pytest.raises(_lib.VtError, match="paired"):
        vt.w4a16_gemm_ragged_silu_mul(x, W, groups)
    with pytest.raises(_lib.VtError, match="paired"):
        vt.w4a16_gemm_ragged(x, Wp, groups)
    with pytest.raises(_lib.VtError, match="MISALIGNED"):
        vt.w4a16_gemm_ragged(torch.zeros(M, K + 4, dtype=torch.bfloat16, device="cuda")[:, :K], W, groups)
    gw, _, _ = _groups(_ids(rng, M, topk, E), E, np.ones((M, topk)))
    with pytest.raises(_lib.VtError, match="workspace holds"):
        vt.w4a16_gemm_ragged_combine(acts(rng, M * topk, K).cuda(), W, gw,
                                     workspace=W.ragged_workspace(0, 1))
    with pytest.raises(_lib.VtError, match="plain grouped"):
        vt.w4a16_gemm_ragged_combine(acts(rng, M * topk, K).cuda(), Wp, gw)


def test_more_token_tiles_than_the_lookup_table_holds():
    rng = np.random.default_rng(14)
    E, N, K = 1024, 72, 32
    counts = [1] * 600 + [40000] + [3] * (E - 601)
    W, ws = _plain(rng, vt.NVFP4, E, N, K)
    ids = np.repeat(np.arange(E, dtype=np.int32), counts).reshape(-1, 1)
    groups, order, offsets = _groups(ids, E)
    x = acts(rng, len(ids), K)
    assert_close(vt.w4a16_gemm_ragged(x.cuda(), W, groups), *_ref(f64(x), ws, order, offsets, 1, True))


def test_smallest_mx_scales():
    """Scale byte 0 (2^-127) beside scales near 1, and rows that hold nothing else."""
    rng = np.random.default_rng(15)
    E, N, K, M = 2, 130, 96, 20
    c, s, g = random_weight(rng, vt.MXFP4, E, N, K)
    s[:, ::2, 1] = 0
    s[:, 1::4] = 0
    W = vt.PackedWeight.grouped(_dev(c), _dev(s), g, vt.MXFP4, E, N, K)
    ws = [weight64(vt.MXFP4, c[e], s[e]) for e in range(E)]
    groups, order, offsets = _groups(_ids(rng, M, 1, E), E)
    x = acts(rng, M, K)
    assert_close(vt.w4a16_gemm_ragged(x.cuda(), W, groups), *_ref(f64(x), ws, order, offsets, 1, True))


@pytest.mark.parametrize("M,topk,E,N,K", [(6, 2, 4, 136, 96), (2100, 8, 64, 320, 544)])
def test_pairs_out_of_range_are_reported_and_not_followed(M, topk, E, N, K):
    rng = np.random.default_rng(M)
    W, ws = _plain(rng, vt.NVFP4, E, N, K)
    groups, order, offsets = _groups(_ids(rng, M, topk, E), E)
    x, xg = acts(rng, M, K), acts(rng, M * topk, K)
    wild = order.copy()
    at = rng.choice(M * topk, 4, replace=False)
    wild[at] = [-1, M * topk, 2 ** 31 - 1, -2 ** 31]
    bad = vt.RowGroups(groups.ids, _dev(wild), groups.offsets)
    right = np.setdiff1d(np.arange(M * topk), at)
    for gather, scatter in ((True, False), (True, True), (False, True)):
        ws_ = W.ragged_workspace(M, topk)
        out = torch.zeros(M * topk, N, dtype=torch.bfloat16, device="cuda")
        a = x if gather else xg
        vt.w4a16_gemm_ragged(a.cuda(), W, bad, out=out, workspace=ws_, gather=gather, scatter=scatter)
        assert vt.workspace_status(ws_) == 6
        ref, err = _ref(f64(a), ws, order, offsets, topk, gather)
        got = f64(out)[order] if scatter else f64(out)
        assert_close(got[right], ref[right], err[right])
        if scatter:
            assert not got[at].any()  # no such row


@pytest.mark.parametrize("change", [lambda o, P: o.__setitem__(1, P + 5), lambda o, P: o.__setitem__(2, -3),
                                    lambda o, P: o.__setitem__(3, 0), lambda o, P: o.fill(2 ** 31 - 1)])
def test_offsets_out_of_range_are_reported(change):
    rng = np.random.default_rng(17)
    M, topk, E, N, K = 50, 2, 6, 136, 96
    W, _ = _plain(rng, vt.NVFP4, E, N, K)
    groups, order, offsets = _groups(_ids(rng, M, topk, E), E)
    wild = offsets.copy()
    change(wild, M * topk)
    ws = W.ragged_workspace(M, topk)
    guard = torch.full((M * topk + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    vt.w4a16_gemm_ragged(acts(rng, M, K).cuda(), W, vt.RowGroups(groups.ids, groups.order, _dev(wild)),
                         out=guard[1:-1], workspace=ws)
    assert vt.workspace_status(ws) == 6
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
