"""GPU: what the calls on grouped rows accept, refuse and report."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from fp4_weight_only_nvfp4_gb300 import _lib
from rows_helpers import acts, group64, random_weight

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _grouped(rng, E, N, K):
    c, s, g = random_weight(rng, vt.NVFP4, E, N, K)
    return vt.PackedWeight.grouped(_dev(c), _dev(s), g, vt.NVFP4, E, N, K)


def _paired(rng, E, I, K):
    parts = [random_weight(rng, vt.NVFP4, E, I, K) for _ in range(2)]
    return vt.PackedWeight.grouped_gate_up(*((_dev(c), _dev(s), g) for c, s, g in parts), vt.NVFP4, E, I, K)


def _groups(rng, M, topk, E):
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
    order, offsets = group64(ids, E)
    return vt.RowGroups(_dev(ids), _dev(order), _dev(offsets), torch.rand(M, topk, device="cuda"))


def test_groups_out_has_the_shape_of_ids():
    ids = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for M, topk in ((4, 2), (8, 1), (1, 8)):
        with pytest.raises(ValueError, match="shape"):
            vt.group_rows(ids, 3, out=vt.RowGroups.empty(M, topk, 3, "cuda"))
        with pytest.raises(ValueError, match="shape"):
            vt.group_rows(ids, 3, out=vt.RowGroups.empty(M, topk, 3, "cuda", weights=True))
    out = vt.RowGroups.empty(2, 4, 3, "cuda")
    assert vt.group_rows(ids, 3, out=out) is out
    flat = vt.RowGroups.empty(8, 1, 3, "cuda")
    assert vt.group_rows(ids.view(8), 3, out=flat) is flat  # [M] and [M, 1] are one shape


def test_a_plain_gemm_names_the_entry_that_serves_a_grouped_weight():
    rng = np.random.default_rng(1)
    Wp, W = _paired(rng, 3, 64, 64), _grouped(rng, 3, 64, 64)
    x = acts(rng, 2, 64).cuda()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for call, kw in ((vt.w4a16_gemm, dict(workspace=ws)), (vt.w4a16_gemm_silu_mul, dict(workspace=ws)),
                     (vt.w4a16_gemm_noalloc, {})):
        with pytest.raises(_lib.VtError, match="vt_fp4_w4a16_gemm_ragged") as err:
            call(x, Wp, **kw)
        assert "_moe" not in str(err.value)
    with pytest.raises(_lib.VtError, match="vt_fp4_w4a16_gemm_moe"):
        vt.w4a16_gemm(x, W, workspace=ws)


def test_stats_report_the_ragged_calls():
    rng = np.random.default_rng(2)
    E, N, K = 4, 300, 64
    W, Wp = _grouped(rng, E, N, K), _paired(rng, E, N // 2, K)
    M, topk = 6, 2
    g = _groups(rng, M, topk, E)
    vt.w4a16_gemm_ragged(acts(rng, M, K).cuda(), W, g)
    s = W.stats()
    assert (s["path"], s["calls"], s["launches"], s["m_tile"], s["stage_k_tiles"]) == (4, 1, 2, 64, 1)
    assert s["grid"] >= 1 and s["items"] >= 4 * 3 and s["warps_per_cta"] == 28
    vt.w4a16_gemm_ragged_combine(acts(rng, M * topk, K).cuda(), W, g)
    s = W.stats()
    assert (s["path"], s["calls"], s["launches"]) == (4, 2, 3)
    vt.w4a16_gemm_ragged_silu_mul(acts(rng, M, K).cuda(), Wp, g)
    assert (Wp.stats()["path"], Wp.stats()["calls"], Wp.stats()["launches"]) == (4, 1, 2)
    big = _groups(rng, 4000, 1, E)
    W2 = _grouped(rng, E, 128 * 40, K)
    vt.w4a16_gemm_ragged(acts(rng, 4000, K).cuda(), W2, big)
    assert W2.stats()["m_tile"] == 128
    none = vt.RowGroups(torch.zeros(0, 2, dtype=torch.int32, device="cuda"),
                        torch.zeros(0, dtype=torch.int32, device="cuda"),
                        torch.zeros(E + 1, dtype=torch.int32, device="cuda"))
    vt.w4a16_gemm_ragged(acts(rng, 1, K).cuda()[:0], W, none)
    assert W.stats()["calls"] == 2  # no pair, no call recorded


def test_a_single_row_may_have_any_row_stride():
    rng = np.random.default_rng(3)
    E, N, K = 3, 72, 64
    W, g = _grouped(rng, E, N, K), _groups(rng, 1, 1, E)
    x = acts(rng, 1, K).cuda()
    wide = torch.zeros(1, K + 5, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = x
    view = wide[:, :K]
    assert view.stride(0) % 8
    want = vt.w4a16_gemm_ragged(x, W, g)
    assert torch.equal(vt.w4a16_gemm_ragged(view, W, g), want)
    assert torch.equal(vt.w4a16_gemm_ragged(view, W, g, gather=False), want)
    assert torch.equal(vt.w4a16_gemm_ragged_combine(view, W, g), vt.w4a16_gemm_ragged_combine(x, W, g))


def test_calls_without_a_workspace_on_memory_used_before():
    """What an earlier tensor left in the memory of a workspace changes nothing."""
    rng = np.random.default_rng(4)
    E, I, H, M, topk = 6, 96, 160, 50, 3
    Wgu, Wd = _paired(rng, E, I, H), _grouped(rng, E, H, I)
    x, logits = acts(rng, M, H).cuda(), torch.randn(M, E, device="cuda")
    zeroed = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
    routes = vt.moe_route(logits, topk, workspace=zeroed(1 << 20))
    want = vt.moe_ffn(x, Wgu, Wd, routes, workspace=zeroed(1 << 22))
    for byte in (0x7F, 0xFF, 0x01):
        used = [torch.full((n,), byte, dtype=torch.uint8, device="cuda") for n in [1 << 12, 1 << 17, 1 << 21, 1 << 24] * 3]
        torch.cuda.synchronize()
        del used
        r = vt.moe_route(logits, topk)
        assert torch.equal(r.order, routes.order) and torch.equal(r.offsets, routes.offsets)
        g = vt.group_rows(r.ids, E)
        assert torch.equal(g.order, routes.order) and torch.equal(g.offsets, routes.offsets)
        assert torch.equal(vt.moe_ffn(x, Wgu, Wd, r), want)
        ws = vt.moe_ffn_workspace(Wgu, Wd, M, topk)
        assert torch.equal(vt.moe_ffn(x, Wgu, Wd, r, workspace=ws), want)
        assert vt.workspace_status(ws) == 0
