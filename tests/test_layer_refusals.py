"""CPU: the cache, its attention and the norms check sizes, pointers, alignment and workspace before any
CUDA call, and the binding refuses tensors the kernels cannot be handed."""
import ctypes

import pytest
import torch

from fp4_weight_only_nvfp4_gb300 import _lib
import fp4_weight_only_nvfp4_gb300 as vt

A0 = 0x10000                      # fake device addresses: no call below may use them
F, ODD, OFF8 = ctypes.c_void_p(A0), ctypes.c_void_p(A0 + 1), ctypes.c_void_p(A0 + 8)
OK, INV, UNS, MIS = _lib.VT_OK, _lib.VT_ERR_INVALID_ARG, _lib.VT_ERR_UNSUPPORTED, _lib.VT_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    from fp4_weight_only_nvfp4_gb300 import build
    build.build()
    return _lib.lib()


def _view(data=A0, pages=4, stride=4 * 2304, page_size=16, heads=4, dim=128, ks=A0, vs=A0):
    return _lib.KvCacheView(data, pages, stride, page_size, heads, dim, ks, vs)


def test_page_bytes(L):
    assert vt.KVCache.page_bytes(16, 1, 64) == 16 * 64 * 9 // 8
    assert vt.KVCache.page_bytes(64, 8, 128) == 8 * 64 * 128 * 9 // 8
    assert vt.KVCache.page_bytes(256, 2, 256) == 2 * 256 * 256 * 9 // 8
    n = ctypes.c_size_t(0)
    for args, want in (((15, 1, 64), INV), ((0, 1, 64), INV), ((512, 1, 64), INV), ((16, 0, 64), INV),
                       ((16, 1025, 64), INV), ((16, 1, 96), UNS), ((16, 1, 512), UNS)):
        assert L.vt_fp4_kv_page_bytes(*args, ctypes.byref(n)) == want
    assert L.vt_fp4_kv_page_bytes(16, 1, 64, None) == INV


@pytest.mark.parametrize("kw,want", [
    (dict(data=None), INV), (dict(pages=0), INV), (dict(pages=2 ** 27), INV), (dict(stride=4 * 2304 - 128), INV),
    (dict(stride=2 ** 33), INV), (dict(page_size=24), INV), (dict(heads=0), INV), (dict(dim=80), UNS), (dict(ks=None), INV),
    (dict(vs=None), INV), (dict(data=A0 + 64), MIS), (dict(stride=4 * 2304 + 64), MIS), (dict(ks=A0 + 2), MIS)])
def test_a_cache_is_checked_by_every_call(L, kw, want):
    v = ctypes.byref(_view(**kw))
    n = ctypes.c_size_t(0)
    assert L.vt_fp4_kv_read(v, 1, F, F, F, None) == want
    assert L.vt_fp4_kv_put(v, 1, F, F, F, F, F, None) == want
    assert L.vt_fp4_kv_get(v, 1, F, F, F, F, F, None) == want
    assert L.vt_fp4_attention_workspace_bytes(v, 1, 1, 4, ctypes.byref(n)) == want
    assert _append(L, cache=v) == want
    assert _attend(L, cache=v) == want
    assert L.vt_fp4_last_error()


def _append(L, cache=None, T=2, q=F, heads=8, ldq=1024, k=F, ldk=512, v=F, ldv=512, slots=F, positions=F,
            table=F, rows=10, rot=128, inter=0, qn=F, kn=F, fp32=0, eps=1e-6, out=ctypes.c_void_p(0x90000), ldo=1024):
    return L.vt_fp4_kv_append(cache or ctypes.byref(_view()), T, q, heads, ldq, k, ldk, v, ldv, slots, positions,
                              table, rows, rot, inter, qn, kn, fp32, eps, out, ldo, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(T=2 ** 24 + 1), INV), (dict(heads=6), INV), (dict(heads=4 * 65, ldq=2 ** 20), INV),
    (dict(heads=0), INV), (dict(q=None), INV), (dict(q=None, heads=0, qn=None), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(out=None), INV), (dict(slots=None), INV), (dict(positions=None), INV), (dict(table=None), INV), (dict(rows=0), INV),
    (dict(rot=8), INV), (dict(rot=144), INV), (dict(rot=-16), INV), (dict(rot=0), INV), (dict(inter=2), INV),
    (dict(fp32=2), INV), (dict(qn=None), INV), (dict(kn=None), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(ldq=1016), INV), (dict(ldk=504), INV), (dict(ldv=504), INV), (dict(ldo=1000), INV), (dict(ldk=516), MIS),
    (dict(out=F, ldo=2048), INV), (dict(q=OFF8), MIS), (dict(v=ODD), MIS), (dict(table=OFF8), MIS), (dict(qn=OFF8), MIS),
    (dict(slots=ctypes.c_void_p(A0 + 4)), MIS), (dict(positions=ODD), MIS), (dict(T=0), OK)])
def test_append(L, kw, want):
    assert _append(L, **kw) == want


def test_moves(L):
    v = ctypes.byref(_view())
    assert L.vt_fp4_kv_read(v, 0, None, None, None, None) == OK
    for args, want in (((-1, F, F, F), INV), ((1, None, F, F), INV), ((1, F, None, F), INV), ((1, F, F, None), INV),
                       ((1, F, OFF8, F), MIS), ((1, ODD, F, F), MIS)):
        assert L.vt_fp4_kv_read(v, *args, None) == want
    for i in range(5):
        a = [F] * 5
        a[i] = None
        assert L.vt_fp4_kv_put(v, 1, *a, None) == INV and L.vt_fp4_kv_get(v, 1, *a, None) == INV
    assert L.vt_fp4_kv_put(v, 1, F, ODD, F, F, F, None) == MIS
    assert L.vt_fp4_kv_read(None, 1, F, F, F, None) == INV


def _attend(L, cache=None, T=2, q=F, heads=8, ldq=1024, tables=F, ldt=3, lens=F, starts=None, B=2, scale=0.1, window=0,
            sinks=None, out=F, ldo=1024, ws=F, n=1 << 30):
    return L.vt_fp4_paged_attention(cache or ctypes.byref(_view()), T, q, heads, ldq, tables, ldt, lens, starts, B, scale,
                                    window, sinks, out, ldo, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(B=3), INV), (dict(B=2 ** 24 + 1, starts=F), INV), (dict(heads=7), INV), (dict(heads=260, ldq=2 ** 20), INV),
    (dict(ldt=0), INV), (dict(ldt=2 ** 27), INV), (dict(ldt=2 ** 26 + 1), INV), (dict(scale=float("inf")), INV), (dict(window=-1), INV), (dict(q=None), INV),
    (dict(out=None), INV), (dict(tables=None), INV), (dict(lens=None), INV), (dict(ws=None), INV), (dict(n=100), INV),
    (dict(ldq=1016), INV), (dict(ldo=1020), INV), (dict(ldo=1032), INV), (dict(ldo=1028), MIS), (dict(q=OFF8), MIS), (dict(ws=ctypes.c_void_p(A0 + 128)), MIS),
    (dict(tables=ODD), MIS), (dict(starts=ODD), MIS), (dict(sinks=ODD), MIS), (dict(T=0, B=0), OK), (dict(T=0, starts=F), OK)])
def test_attention(L, kw, want):
    assert _attend(L, **kw) == want


def test_attention_workspace(L):
    v, n = ctypes.byref(_view()), ctypes.c_size_t(0)
    for args in ((-1, 1, 4), (1, -1, 4), (2 ** 24 + 1, 1, 4), (1, 1, 6), (1, 1, 0)):
        assert L.vt_fp4_attention_workspace_bytes(v, *args, ctypes.byref(n)) == INV
    assert L.vt_fp4_attention_workspace_bytes(v, 1, 1, 4, None) == INV
    assert L.vt_fp4_attention_workspace_bytes(v, 1, 1, 4, ctypes.byref(n)) == OK and n.value >= 4096


def _norm(L, x=F, T=2, H=64, ldx=64, r=F, ldr=64, r32=0, pw=F, g=F, ldg=64, scale=1.0, w=F, w32=0, eps=1e-6,
          h=ctypes.c_void_p(0x20000), ldh=64, y=ctypes.c_void_p(0x30000), ldy=64):
    return L.vt_fp4_residual_norm(x, T, H, ldx, r, ldr, r32, pw, g, ldg, scale, w, w32, eps, h, ldh, y, ldy, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(H=16385), INV), (dict(r32=2), INV), (dict(w32=-1), INV), (dict(scale=float("nan")), INV),
    (dict(eps=-1e-6), INV), (dict(r=None), INV), (dict(h=None), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV),
    (dict(ldx=63), INV), (dict(ldy=63), INV), (dict(ldr=63), INV), (dict(ldh=63), INV), (dict(ldg=63), INV), (dict(x=ODD), MIS),
    (dict(r=ctypes.c_void_p(A0 + 2), r32=1), MIS), (dict(w=ctypes.c_void_p(A0 + 2), w32=1), MIS), (dict(h=F, ldh=72), INV),
    (dict(y=F, ldy=72), INV), (dict(T=0), OK)])
def test_norm(L, kw, want):
    assert _norm(L, **kw) == want


def test_the_cache_structure_has_the_headers_layout():
    assert [(f, getattr(_lib.KvCacheView, f).offset) for f, _ in _lib.KvCacheView._fields_] == [
        ("data", 0), ("pages", 8), ("page_stride", 16), ("page_size", 24), ("heads", 32), ("head_dim", 40),
        ("k_scale", 48), ("v_scale", 56)]


def test_binding_refuses_host_and_misshaped_tensors(L):
    g = torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        vt.KVCache.empty(2, 16, 2, 64, g, g)
    with pytest.raises(ValueError, match="data must be"):
        vt.KVCache(torch.zeros(2, 100, dtype=torch.uint8), 16, 2, 64, g, g)
    with pytest.raises(vt.VtError, match="page_size"):
        vt.KVCache.empty(2, 20, 2, 64, g, g)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        vt.residual_norm(x, x, x[0])
    for rot in (0, 8, 24):
        with pytest.raises(ValueError, match="rot"):
            vt.rope_table(4, rot)


def test_rope_table_is_taken_in_fp64():
    t = vt.rope_table(70000, 64, 1e6, device="cpu")
    assert t.shape == (70000, 64) and t.dtype == torch.float32
    i, p = 3, 69999
    a = torch.tensor(p * 1e6 ** (-2 * i / 64), dtype=torch.float64)
    assert abs(t[p, i].double() - a.cos()) < 2.0 ** -23 and abs(t[p, 32 + i].double() - a.sin()) < 2.0 ** -23


def test_public_names():
    for name in ("KVCache", "rope_table", "kv_append", "kv_read", "paged_attention", "attention_workspace", "residual_norm"):
        assert name in vt.__all__ and hasattr(vt, name)
