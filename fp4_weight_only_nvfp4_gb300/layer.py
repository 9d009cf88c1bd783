"""What a decoder layer runs between its products: the paged NVFP4 cache of keys and values, the
attention over it, and the norms around the blocks (the entry points of include/vt_fp4.h from
vt_fp4_kv_page_bytes to vt_fp4_residual_norm).  Argument checks and marshalling only."""
from __future__ import annotations

import ctypes

import torch

from ._lib import KvCacheView, check, lib
from .rows import _empty, _made_on, _need, _raw, _rows, _workspace

CLEARED = 4096  # bytes of an attention workspace that start as zeros
_BF16, _F32 = torch.bfloat16, torch.float32


def _on(t, name, gpu):
    """gpu is a CUDA device's number, which no tensor of another kind returns as its own."""
    if t.get_device() != gpu:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{gpu} (got {t.device})")


def _heads(t, name, rows, heads, dim, gpu):
    """A bf16 [rows, heads, dim] tensor whose heads stand side by side; returns its row stride."""
    if t.dtype is not _BF16 or t.shape != (rows, heads, dim):
        raise ValueError(f"{name} must be a bf16 [{rows}, {heads}, {dim}] tensor")
    ld, between, inner = t.stride()
    if inner != 1 or (between != dim and heads > 1):
        raise ValueError(f"the heads of a row of {name} must stand side by side")
    _on(t, name, gpu)
    if rows <= 1:
        return heads * dim
    if ld < heads * dim:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld


def _vector(t, name, dtype, n, gpu):
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape [{n}]")
    _on(t, name, gpu)
    return t.data_ptr()


def _weights(a, a_name, b, b_name, n, gpu):
    """Two weights [n], either of which may be None, both bf16 or both fp32: (pointers, 1 if fp32)."""
    if a is None and b is None:
        return 0, 0, 0
    kind = (b if a is None else a).dtype
    if kind is not _BF16 and kind is not _F32:
        raise ValueError(f"{a_name} and {b_name} must be bf16 or fp32")
    return (0 if a is None else _vector(a, a_name, kind, n, gpu), 0 if b is None else _vector(b, b_name, kind, n, gpu),
            int(kind is _F32))


class KVCache:
    """Keys and values of pages * page_size tokens in NVFP4: E2M1 codes, an E4M3 scale per 16 of a
    head's head_dim, and one fp32 global per head (k_scale, v_scale; CUDA [heads]).  Slot p is token p %
    page_size of page p // page_size.  data: uint8 [pages, page bytes], rows contiguous (a view
    of a cache of several layers has a larger stride); its inner order is the kernels' own: put,
    get and kv_read convert."""

    def __init__(self, data: torch.Tensor, page_size: int, heads: int, head_dim: int,
                 k_scale: torch.Tensor, v_scale: torch.Tensor):
        n = self.page_bytes(page_size, heads, head_dim)
        if data.dtype != torch.uint8 or data.dim() != 2 or data.shape[1] != n or data.stride(1) != 1:
            raise ValueError(f"data must be a uint8 [pages, {n}] tensor with unit inner stride")
        if not data.is_cuda:
            raise ValueError(f"data must be a CUDA tensor (got {data.device})")
        self.pages, self.page_size, self.heads, self.head_dim = data.shape[0], page_size, heads, head_dim
        self.device, self.gpu = data.device, data.get_device()
        if self.pages > 1 and data.stride(0) < n:
            raise ValueError("data must not have overlapping pages")
        _need(k_scale, "k_scale", _F32, (heads,), self.device)
        _need(v_scale, "v_scale", _F32, (heads,), self.device)
        self.data, self.k_scale, self.v_scale = data, k_scale, v_scale
        stride = data.stride(0) if self.pages > 1 else n
        self._view = KvCacheView(data.data_ptr(), self.pages, stride, page_size, heads, head_dim,
                                 k_scale.data_ptr(), v_scale.data_ptr())
        self.view = ctypes.byref(self._view)

    @staticmethod
    def page_bytes(page_size: int, heads: int, head_dim: int) -> int:
        out = ctypes.c_size_t(0)
        check(lib().vt_fp4_kv_page_bytes(page_size, heads, head_dim, ctypes.byref(out)),
              "vt_fp4_kv_page_bytes")
        return out.value

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, k_scale: torch.Tensor,
              v_scale: torch.Tensor) -> "KVCache":
        """A cache of its own memory, uncleared, on the GPU of its globals."""
        data = torch.empty((pages, cls.page_bytes(page_size, heads, head_dim)), dtype=torch.uint8,
                           device=k_scale.device)
        return cls(data, page_size, heads, head_dim, k_scale, v_scale)

    def _tokens(self, T, lead):
        return [torch.empty((T, self.heads, self.head_dim // n), dtype=torch.uint8, device=lead.device)
                for n in (2, 16, 2, 16)]

    def _slots(self, slots):
        if slots.dim() != 1:
            raise ValueError("slots must be an int64 tensor [T]")
        return _vector(slots, "slots", torch.int64, slots.shape[0], self.gpu)

    def put(self, slots: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor,
            v_codes: torch.Tensor, v_scales: torch.Tensor, stream=None) -> None:
        """Writes raw tokens: codes uint8 [T, heads, head_dim / 2] (low nibble = even), E4M3 bytes uint8 [T,
        heads, head_dim / 16].  Slots are distinct; those outside the cache are skipped."""
        sp, T = self._slots(slots), slots.shape[0]
        for t, name, n in ((k_codes, "k_codes", 2), (k_scales, "k_scales", 16), (v_codes, "v_codes", 2),
                           (v_scales, "v_scales", 16)):
            _need(t, name, torch.uint8, (T, self.heads, self.head_dim // n), self.device)
        check(lib().vt_fp4_kv_put(self.view, T, sp, k_codes.data_ptr(), k_scales.data_ptr(),
                                  v_codes.data_ptr(), v_scales.data_ptr(), _raw(stream, self.gpu)),
              "vt_fp4_kv_put")

    def get(self, slots: torch.Tensor, stream=None):
        """(k_codes, k_scales, v_codes, v_scales) of tokens, as put takes them; zeros for slots
        outside the cache."""
        sp, T = self._slots(slots), slots.shape[0]
        with _made_on(stream):
            out = self._tokens(T, slots)
        check(lib().vt_fp4_kv_get(self.view, T, sp, *(t.data_ptr() for t in out), _raw(stream, self.gpu)),
              "vt_fp4_kv_get")
        return tuple(out)


def rope_table(positions: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotation's table for kv_append: fp32 [positions, rot], rot / 2 cosines and rot / 2 sines of
    position * base^(-2i / rot), the angles taken in fp64."""
    if positions < 1 or rot < 16 or rot % 16:
        raise ValueError("positions must be at least 1, rot a positive multiple of 16")
    half = rot // 2
    step = base ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * step
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: KVCache, slots: torch.Tensor,
              positions: torch.Tensor | None = None, table: torch.Tensor | None = None,
              q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, eps: float = 1e-6,
              interleaved: bool = False, out: torch.Tensor | None = None, stream=None):
    """Appends T tokens to the cache at their slots (int64 [T]; outside the cache: skipped) and
    returns q as the attention takes it.  q bf16 [T, q_heads, D] (or None), k, v bf16 [T, heads, D]:
    the heads of a row side by side, any row stride that is a multiple of 8, so views of one projection's output will
    do.  q_norm, k_norm [D] (bf16 or fp32): per-head norms first; positions int32 [T] and table
    (rope_table): then the rotation.  out may be q.  See vt_fp4_kv_append in include/vt_fp4.h."""
    T, D, gpu = k.shape[0], cache.head_dim, cache.gpu
    ldk, ldv = _heads(k, "k", T, cache.heads, D, gpu), _heads(v, "v", T, cache.heads, D, gpu)
    sp = _vector(slots, "slots", torch.int64, T, gpu)
    if (positions is None) != (table is None):
        raise ValueError("positions and table go together")
    rot = rows = pp = tp = 0
    if table is not None:
        if table.dim() != 2:
            raise ValueError("table must be fp32 [positions, rot]")
        rows, rot = table.shape
        if table.dtype is not _F32 or not table.is_contiguous():
            raise ValueError("table must be a contiguous fp32 tensor [positions, rot]")
        _on(table, "table", gpu)
        pp, tp = _vector(positions, "positions", torch.int32, T, gpu), table.data_ptr()
    qn, kn, fp32 = _weights(q_norm, "q_norm", k_norm, "k_norm", D, gpu)
    heads = ldq = ldo = qp = op = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be a bf16 [{T}, q_heads, {D}] tensor")
        heads = q.shape[1]
        ldq = _heads(q, "q", T, heads, D, gpu)
        if out is None:
            out = _empty((T, heads, D), _BF16, cache.device, stream)
        ldo = _heads(out, "out", T, heads, D, gpu)
        qp, op = q.data_ptr(), out.data_ptr()
        if T == 0:
            return out
    elif out is not None:
        raise ValueError("without q there is no out")
    check(lib().vt_fp4_kv_append(cache.view, T, qp, heads, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, sp, pp,
                                 tp, rows, rot, int(interleaved), qn, kn, fp32, eps, op, ldo,
                                 _raw(stream, gpu)), "vt_fp4_kv_append")
    return out


def kv_read(cache: KVCache, slots: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None,
            stream=None):
    """The values of tokens: (k, v) bf16 [T, heads, D]; zeros for slots outside the cache."""
    sp, shape = cache._slots(slots), (slots.shape[0], cache.heads, cache.head_dim)
    if out is None:
        out = _empty(shape, _BF16, cache.device, stream), _empty(shape, _BF16, cache.device, stream)
    else:
        for t, name in zip(out, ("k", "v")):
            _need(t, name, _BF16, shape, cache.device)
    check(lib().vt_fp4_kv_read(cache.view, shape[0], sp, out[0].data_ptr(), out[1].data_ptr(),
                               _raw(stream, cache.gpu)), "vt_fp4_kv_read")
    return out


def attention_workspace(T_max: int, B_max: int, q_heads: int, cache: KVCache) -> torch.Tensor:
    """A workspace for paged_attention of up to T_max rows of q_heads heads and B_max sequences; T_max = 0 for
    calls without starts, whatever their rows."""
    n = ctypes.c_size_t(0)
    check(lib().vt_fp4_attention_workspace_bytes(cache.view, T_max, B_max, q_heads, ctypes.byref(n)),
          "vt_fp4_attention_workspace_bytes")
    ws = torch.empty(n.value, dtype=torch.uint8, device=cache.device)
    ws[:CLEARED].zero_()
    return ws


def paged_attention(q: torch.Tensor, cache: KVCache, tables: torch.Tensor, lens: torch.Tensor,
                    starts: torch.Tensor | None = None, scale: float | None = None, window: int = 0,
                    sinks: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of q (bf16 [T, q_heads, D]) over the cache, whose last keys are the rows'
    own: out bf16 [T, q_heads, D].  tables int32 [B, pages]: each sequence's pages, lens int32 [B]:
    its keys.  starts int32 [B + 1]: its rows are starts[b] to starts[b + 1] of q (None: one each).
    scale: D ** -0.5 by default; window: the number of latest keys a row sees (0: all); sinks fp32
    [q_heads].  out may be q.  See vt_fp4_paged_attention in include/vt_fp4.h."""
    if q.dim() != 3:
        raise ValueError("q must be a bf16 [T, q_heads, head_dim] tensor")
    T, heads, D = q.shape
    gpu = cache.gpu
    if tables.dim() != 2:
        raise ValueError("tables must be int32 [B, pages]")
    B, ldt = tables.shape
    if tables.dtype is not torch.int32 or not tables.is_contiguous() or tables.get_device() != gpu:
        raise ValueError(f"tables must be a contiguous int32 CUDA tensor on cuda:{gpu}")
    ldq = _heads(q, "q", T, heads, cache.head_dim, gpu)
    lp = _vector(lens, "lens", torch.int32, B, gpu)
    sp = 0 if starts is None else _vector(starts, "starts", torch.int32, B + 1, gpu)
    kp = 0 if sinks is None else _vector(sinks, "sinks", _F32, heads, gpu)
    if out is None:
        out = _empty((T, heads, D), _BF16, cache.device, stream)
    ldo = _heads(out, "out", T, heads, D, gpu)
    if workspace is None:
        with _made_on(stream):
            workspace = attention_workspace(0 if starts is None else T, B, heads, cache)
    wp, wn = _workspace(workspace, gpu)
    check(lib().vt_fp4_paged_attention(cache.view, T, q.data_ptr(), heads, ldq, tables.data_ptr(), ldt, lp, sp, B,
                                       D ** -0.5 if scale is None else scale, window, kp, out.data_ptr(),
                                       ldo, wp, wn, _raw(stream, gpu)), "vt_fp4_paged_attention")
    return out


def _matrix(t, name, dtype, rows, cols, gpu):
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if dtype is _BF16:
        return _rows(t, name, rows, cols, gpu)
    if t.shape != (rows, cols) or (t.stride(1) != 1 and cols > 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{name} must be a [{rows}, {cols}] tensor with unit inner stride")
    _on(t, name, gpu)
    return t.stride(0) if rows > 1 else cols


def residual_norm(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor,
                  post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  scale: float = 1.0, eps: float = 1e-6, out=None, stream=None):
    """(h, y): h = residual + scale * gate * a with a = x or norm(x) * post_weight, and y = norm(h)
    * weight.  x bf16 [T, H]; residual bf16 or fp32 [T, H], h of its type (None: h = scale * gate * a is
    not kept); gate bf16 [T, H] or [H]; weights [H], bf16 or fp32.  out: (h, y), which may be
    residual and x.  See vt_fp4_residual_norm in include/vt_fp4.h."""
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a bf16 CUDA [T, H] tensor")
    (T, H), gpu = x.shape, x.get_device()
    ldx = _rows(x, "x", T, H, gpu)
    wp, pw, fp32 = _weights(weight, "weight", post_weight, "post_weight", H, gpu)
    gp = ldg = 0
    if gate is not None:
        gp = gate.data_ptr()
        if gate.dim() == 1:
            _vector(gate, "gate", _BF16, H, gpu)
        else:
            ldg = _rows(gate, "gate", T, H, gpu)
    kind = _BF16 if residual is None else residual.dtype
    if kind not in (_BF16, _F32):
        raise ValueError("residual must be bf16 or fp32")
    if out is None:
        out = (None if residual is None else _empty((T, H), kind, x.device, stream),
               _empty((T, H), _BF16, x.device, stream))
    h, y = out
    if (h is None) != (residual is None):
        raise ValueError("residual and h go together")
    ldr = ldh = rp = hp = 0
    if residual is not None:
        ldr, ldh = _matrix(residual, "residual", kind, T, H, gpu), _matrix(h, "h", kind, T, H, gpu)
        rp, hp = residual.data_ptr(), h.data_ptr()
    ldy = _rows(y, "y", T, H, gpu)
    check(lib().vt_fp4_residual_norm(x.data_ptr(), T, H, ldx, rp, ldr, int(kind is _F32), pw, gp, ldg, scale, wp,
                                     fp32, eps, hp, ldh, y.data_ptr(), ldy, _raw(stream, gpu)),
          "vt_fp4_residual_norm")
    return h, y
