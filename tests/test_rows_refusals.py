"""CPU: the entry points on grouped rows check sizes, options, pointers, alignment and workspace
before any CUDA call, and the binding refuses tensors the kernels cannot be handed."""
import ctypes

import pytest
import torch

from fp4_weight_only_nvfp4_gb300 import _lib
import fp4_weight_only_nvfp4_gb300 as vt

F = ctypes.c_void_p(0x10000)      # a fake device pointer: no call below may use it
ODD = ctypes.c_void_p(0x10001)
INV, MIS = _lib.VT_ERR_INVALID_ARG, _lib.VT_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    from fp4_weight_only_nvfp4_gb300 import build
    build.build()
    return _lib.lib()


def test_group_workspace_and_rows(L):
    n = ctypes.c_size_t(0)
    for pairs, E in ((-1, 4), (4, 0), (4, 1025), (2 ** 31, 4)):
        assert L.vt_fp4_group_workspace_bytes(pairs, E, ctypes.byref(n)) == INV
    assert L.vt_fp4_group_workspace_bytes(4, 4, None) == INV
    assert L.vt_fp4_group_workspace_bytes(1000, 128, ctypes.byref(n)) == 0 and n.value > 0
    big = n.value
    g = L.vt_fp4_group_rows
    assert g(F, 8, 0, F, F, F, big, None) == INV
    assert g(None, 8, 4, F, F, F, big, None) == INV
    assert g(F, 8, 4, None, F, F, big, None) == INV
    assert g(F, 8, 4, F, None, F, big, None) == INV
    assert g(F, 8, 4, F, F, None, big, None) == INV
    assert g(F, 1000, 128, F, F, F, big - 1, None) == INV
    assert g(F, 8, 4, F, F, ODD, big, None) == MIS
    assert g(ODD, 8, 4, F, F, F, big, None) == MIS


def _route(L, logits=F, bf16=0, M=4, ld=16, E=16, topk=2, scoring=0, bias=None, renorm=1, scale=1.0,
           ids=F, w=F, order=F, offsets=F, ws=F, n=1 << 24):
    return L.vt_fp4_moe_route(logits, bf16, M, ld, E, topk, scoring, bias, renorm, scale, ids, w,
                              order, offsets, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), INV), (dict(ids=None), INV), (dict(w=None), INV), (dict(order=None), INV),
    (dict(offsets=None), INV), (dict(ws=None), INV), (dict(M=-1), INV), (dict(E=0), INV),
    (dict(E=1025, ld=1025), INV), (dict(topk=0), INV), (dict(topk=33, E=64, ld=64), INV),
    (dict(topk=17), INV), (dict(ld=15), INV), (dict(scoring=2), INV), (dict(bf16=2), INV),
    (dict(bias=F), INV), (dict(scale=float("nan")), INV), (dict(n=64), INV), (dict(ws=ODD), MIS),
    (dict(logits=ODD), MIS), (dict(logits=ctypes.c_void_p(0x10002)), MIS), (dict(w=ODD), MIS)])
def test_route(L, kw, want):
    assert _route(L, **kw) == want
    assert L.vt_fp4_last_error()


def test_ragged_needs_a_weight(L):
    n = ctypes.c_size_t(0)
    assert L.vt_fp4_ragged_workspace_bytes(None, 4, 2, ctypes.byref(n)) == INV
    assert L.vt_fp4_w4a16_gemm_ragged(F, 64, None, F, F, 8, 2, 1, F, 64, F, 1 << 20, None) == INV
    assert L.vt_fp4_w4a16_gemm_ragged_combine(F, 64, None, F, F, F, F, 4, 2, F, 64, F, 1 << 20,
                                              None) == INV


def test_prepack_grouped_gate_up(L):
    h = ctypes.c_void_p(0x1234)
    p = L.vt_fp4_prepack_grouped_gate_up
    ok = [F, F, F, F, F, F]
    assert p(*ok, 0, 2, 64, 64, F, 1 << 24, None, None) == INV
    for i in range(6):
        a = list(ok)
        a[i] = None
        assert p(*a, 0, 2, 64, 64, F, 1 << 24, None, ctypes.byref(h)) == INV
        assert h.value in (None, 0)
    for E, I, K, n in ((0, 64, 64, 1 << 24), (2, 0, 64, 1 << 24), (2, -5, 64, 1 << 24),
                       (2, 64, 24, 1 << 24), (2, 64, 64, 100)):
        assert p(*ok, 0, E, I, K, F, n, None, ctypes.byref(h)) == INV


def _lora(L, x=F, M=4, ldx=64, K=64, A=F, B=F, scale=F, ranks=None, La=2, R=8, N=32, order=F,
          offsets=F, y=F, ldy=32, out=ctypes.c_void_p(0x20000), ldo=32):
    return L.vt_fp4_lora_add(x, M, ldx, K, A, B, scale, ranks, La, R, N, order, offsets, y, ldy, out,
                             ldo, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(A=None), INV), (dict(B=None), INV), (dict(scale=None), INV),
    (dict(order=None), INV), (dict(offsets=None), INV), (dict(y=None), INV), (dict(out=None), INV),
    (dict(M=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(La=0), INV), (dict(La=1025), INV),
    (dict(R=0), INV), (dict(R=129), INV), (dict(ldx=63), INV), (dict(ldy=31), INV),
    (dict(ldo=31), INV), (dict(x=ODD), MIS), (dict(out=ODD), MIS), (dict(scale=ODD), MIS),
    (dict(out=F, ldo=40), INV), (dict(M=0), 0)])
def test_lora(L, kw, want):
    assert _lora(L, **kw) == want


def test_binding_refuses_host_and_misshaped_tensors():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vt.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="CUDA"):
        vt.group_rows(torch.zeros(4, **i32), 2)
    with pytest.raises(ValueError, match="CUDA"):
        vt.RowGroups(torch.zeros(4, 2, **i32), torch.zeros(8, **i32), torch.zeros(5, **i32))
    with pytest.raises(ValueError, match="ids must be"):
        vt.RowGroups(torch.zeros(4, 2), torch.zeros(8, **i32), torch.zeros(5, **i32))
    with pytest.raises(ValueError, match="A must be"):
        vt.LoraAdapters(torch.zeros(4, 8), torch.zeros(2, 6, 4), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        vt.LoraAdapters(torch.zeros(2, 4, 8, dtype=torch.bfloat16),
                        torch.zeros(2, 6, 4, dtype=torch.bfloat16), torch.zeros(2))


def test_public_names():
    for name in ("moe_route", "group_rows", "RowGroups", "w4a16_gemm_ragged", "moe_ffn",
                 "w4a16_gemm_ragged_silu_mul", "w4a16_gemm_ragged_combine", "lora_add", "LoraAdapters"):
        assert name in vt.__all__
