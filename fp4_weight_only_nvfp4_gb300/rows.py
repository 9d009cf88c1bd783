"""Operators on rows grouped by an index chosen on the device: the mixture-of-experts router,
the experts' ragged products, and low-rank adapters (the entry points of include/vt_fp4.h from
vt_fp4_group_rows to vt_fp4_lora_add).  Argument checks and marshalling only."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import GemmOpts, check, lib

SCORING = {"softmax": 0, "sigmoid": 1}
GATHER, SCATTER, SILU_MUL = 1, 2, 4


# (a torch without CUDA has neither, and no tensor that gets as far as their use)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_BF16 = torch.bfloat16


def _raw(stream, gpu):
    """The handle of the call's stream.  The kernels launch on the current GPU: the operands (on GPU
    number gpu) and the stream must be its own."""
    if _current_device() != gpu:
        raise ValueError(f"the operands are on cuda:{gpu}, the current GPU is cuda:{_current_device()}")
    if stream is None:
        return _current_stream(gpu)
    if getattr(stream, "device_index", gpu) != gpu:
        raise ValueError(f"the stream must be on cuda:{gpu}")
    return stream.cuda_stream


def _made_on(stream):
    """Buffers made for a call belong to the stream it runs on: they are zeroed there, and the
    allocator hands them out again in that stream's order."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _made_on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need(t, name, dtype, shape, device):
    """A contiguous tensor of this type and shape on this GPU."""
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device} (got {t.device})")


def _rows(t, name, rows, cols, gpu):
    """A bf16 matrix with unit inner stride on GPU number gpu; returns its row stride (one row: its
    columns)."""
    if t.dtype is not _BF16 or t.shape != (rows, cols):
        raise ValueError(f"{name} must be a bf16 [{rows}, {cols}] tensor with unit inner stride")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must be a bf16 [{rows}, {cols}] tensor with unit inner stride")
    if t.get_device() != gpu or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{gpu} (got {t.device})")
    if rows <= 1:  # no second row for the stride to lead to
        return cols
    if ld < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld


def _workspace(ws, gpu):
    if ws.dtype is not torch.uint8 or not ws.is_contiguous() or ws.get_device() != gpu \
            or not ws.is_cuda:
        raise ValueError(f"workspace must be a contiguous uint8 CUDA tensor on cuda:{gpu}")
    return ws.data_ptr(), ws.numel()


class RowGroups:
    """(token, slot) pairs grouped by an index.  ids int32 [M, topk] (or [M], topk = 1), order
    int32 [M * topk], offsets int32 [E + 1]: group e holds the pairs order[offsets[e]:offsets[e
    + 1]], pair p being slot p % topk of token p // topk; pairs whose id is outside [0, E) come
    last.  weights: fp32 [M, topk] where a router made them."""

    def __init__(self, ids: torch.Tensor, order: torch.Tensor, offsets: torch.Tensor,
                 weights: torch.Tensor | None = None):
        if ids.dim() not in (1, 2):
            raise ValueError("ids must be [M, topk] or [M]")
        self.M, self.topk = ids.shape[0], (ids.shape[1] if ids.dim() == 2 else 1)
        self.E, self.pairs = offsets.numel() - 1, ids.numel()
        dev = self.device = ids.device
        self.gpu = ids.get_device()
        _need(ids, "ids", torch.int32, tuple(ids.shape), dev)
        _need(order, "order", torch.int32, (self.pairs,), dev)
        _need(offsets, "offsets", torch.int32, (self.E + 1,), dev)
        if weights is not None:
            _need(weights, "weights", torch.float32, (self.M, self.topk), dev)
        self.ids, self.order, self.offsets, self.weights = ids, order, offsets, weights

    @classmethod
    def empty(cls, M: int, topk: int, E: int, device, weights: bool = False) -> "RowGroups":
        """Uninitialised buffers for moe_route (weights=True) or group_rows to fill."""
        ids = torch.empty((M, topk), dtype=torch.int32, device=device)
        return cls(ids, torch.empty(M * topk, dtype=torch.int32, device=device),
                   torch.empty(E + 1, dtype=torch.int32, device=device),
                   torch.empty((M, topk), dtype=torch.float32, device=device) if weights else None)


def group_workspace(M_max: int, topk: int, E: int, device) -> torch.Tensor:
    """A workspace for moe_route and group_rows of up to M_max tokens of topk pairs."""
    out = ctypes.c_size_t(0)
    check(lib().vt_fp4_group_workspace_bytes(M_max * topk, E, ctypes.byref(out)),
          "vt_fp4_group_workspace_bytes")
    return torch.empty(out.value, dtype=torch.uint8, device=device)


def status_workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace of which only the status word (its first 256 bytes) is cleared: the rest is
    scratch, 185 MB for 4096 tokens of 8 pairs on 2048 columns, that every call writes first."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def group_rows(ids: torch.Tensor, E: int, out: RowGroups | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> RowGroups:
    """Groups the pairs of ids (int32 [M] or [M, topk]; outside [0, E): in no group).  out: of the
    same [M, topk]; it takes ids as its own, and its weights, if any, stay the caller's business."""
    if ids.dtype != torch.int32 or ids.dim() not in (1, 2) or not ids.is_contiguous() \
            or not ids.is_cuda:
        raise ValueError("ids must be a contiguous int32 CUDA tensor [M] or [M, topk]")
    dev, gpu = ids.device, ids.get_device()
    shape = (ids.shape[0], ids.shape[1] if ids.dim() == 2 else 1)
    if out is None:
        out = RowGroups(ids, _empty(ids.numel(), torch.int32, dev, stream),
                        _empty(E + 1, torch.int32, dev, stream))
    elif out.E != E or (out.M, out.topk) != shape or out.device != dev:
        raise ValueError("out does not have the shape of ids and E")
    else:
        out.ids = ids
    if workspace is None:
        with _made_on(stream):
            workspace = group_workspace(ids.numel(), 1, E, dev)
    wp, wn = _workspace(workspace, gpu)
    check(lib().vt_fp4_group_rows(ids.data_ptr(), ids.numel(), E, out.order.data_ptr(),
                                  out.offsets.data_ptr(), wp, wn, _raw(stream, gpu)),
          "vt_fp4_group_rows")
    return out


def moe_route(logits: torch.Tensor, topk: int, scoring: str = "softmax",
              bias: torch.Tensor | None = None, renormalize: bool = True, scale: float = 1.0,
              out: RowGroups | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> RowGroups:
    """The router: per token (row of logits, fp32 or bf16 [M, E]) the topk experts of largest
    score, ties to the lowest index, with their weights, grouped by expert.  An expert masked
    by a logit of -inf is never chosen (id -1, weight 0).  See vt_fp4_moe_route in
    include/vt_fp4.h."""
    if logits.dtype not in (torch.float32, torch.bfloat16) or logits.dim() != 2 \
            or (logits.shape[1] > 1 and logits.stride(1) != 1) or not logits.is_cuda:
        raise ValueError("logits must be an fp32 or bf16 CUDA [M, E] tensor with unit inner stride")
    if scoring not in SCORING:
        raise ValueError(f"scoring must be one of {sorted(SCORING)}")
    M, E = logits.shape
    dev, gpu = logits.device, logits.get_device()
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,), dev)
    if out is None:
        with _made_on(stream):
            out = RowGroups.empty(M, topk, E, dev, weights=True)
    elif (out.M, out.topk, out.E, out.gpu) != (M, topk, E, gpu) or out.weights is None:
        raise ValueError("out must be RowGroups.empty(M, topk, E, device, weights=True)")
    if workspace is None:
        with _made_on(stream):
            workspace = group_workspace(M, topk, E, dev)
    wp, wn = _workspace(workspace, gpu)
    ld = logits.stride(0) if M > 1 else max(logits.stride(0), E)
    check(lib().vt_fp4_moe_route(logits.data_ptr(), int(logits.dtype == torch.bfloat16), M, ld, E,
                                 topk, SCORING[scoring], bias.data_ptr() if bias is not None else 0,
                                 int(renormalize), scale, out.ids.data_ptr(),
                                 out.weights.data_ptr(), out.order.data_ptr(),
                                 out.offsets.data_ptr(), wp, wn, _raw(stream, gpu)),
          "vt_fp4_moe_route")
    return out


def _check_groups(W, groups):
    E = getattr(W, "E", 1)
    if groups.E != E:
        raise ValueError(f"the groups are of {groups.E} indices, the weight has {E} experts")
    gpu = W.packed.get_device()
    if groups.gpu != gpu:
        raise ValueError(f"groups must be on {W.packed.device}")
    return gpu


def _options(opts):
    unknown = set(opts) - {name for name, _ in GemmOpts._fields_}
    if unknown:
        raise TypeError(f"unknown options {sorted(unknown)}")
    return ctypes.byref(GemmOpts(**opts))


def _ragged(A, W, groups, out, workspace, stream, flags, cols, opts=None):
    gpu = _check_groups(W, groups)
    lda = _rows(A, "A", groups.M if flags & GATHER else groups.pairs, W.K, gpu)
    if out is None:
        out = _empty((groups.pairs, cols), _BF16, A.device, stream)
    ldc = _rows(out, "out", groups.pairs, cols, gpu)
    if workspace is None:
        with _made_on(stream):
            workspace = W.ragged_workspace(groups.M, groups.topk)
    wp, wn = _workspace(workspace, gpu)
    check(lib().vt_fp4_w4a16_gemm_ragged_ex(A.data_ptr(), lda, W.handle, groups.order.data_ptr(),
                                            groups.offsets.data_ptr(), groups.pairs, groups.topk,
                                            flags, out.data_ptr(), ldc, wp, wn,
                                            _raw(stream, gpu),
                                            _options(opts) if opts else None),
          "vt_fp4_w4a16_gemm_ragged")
    return out


def w4a16_gemm_ragged(A: torch.Tensor, W, groups: RowGroups, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None, gather: bool = True,
                      scatter: bool = False, opts: dict | None = None) -> torch.Tensor:
    """Every grouped pair's row times its expert's weight, for any number of pairs: out
    [pairs, N] (bf16).  gather: A holds one row per token, else one row per pair in group order.
    scatter: pair p's output is row p, else the rows are in group order.  Rows of pairs in no
    group are not written.  opts: wait_limit_us, withhold_weights.  See vt_fp4_w4a16_gemm_ragged
    and vt_fp4_w4a16_gemm_ragged_ex in include/vt_fp4.h."""
    return _ragged(A, W, groups, out, workspace, stream,
                   (GATHER if gather else 0) | (SCATTER if scatter else 0), W.N, opts)


def w4a16_gemm_ragged_silu_mul(A: torch.Tensor, W, groups: RowGroups,
                               out: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None,
                               gather: bool = True, opts: dict | None = None) -> torch.Tensor:
    """The experts' gate and up products with silu(gate) * up as the output: out [pairs, I]
    (bf16), rows in group order, for a weight from PackedWeight.grouped_gate_up."""
    return _ragged(A, W, groups, out, workspace, stream, SILU_MUL | (GATHER if gather else 0),
                   W.N // 2, opts)


def w4a16_gemm_ragged_combine(A: torch.Tensor, W, groups: RowGroups,
                              out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The experts' second products (A [pairs, K], rows in group order) and each token's sum of
    them by groups.weights: out [M, N] (bf16).  The products are rounded to bf16 first, as
    w4a16_gemm_ragged writes them; the sum is fp32.  Pairs in no group count as zero."""
    gpu = _check_groups(W, groups)
    if groups.weights is None:
        raise ValueError("the groups hold no weights")
    lda = _rows(A, "A", groups.pairs, W.K, gpu)
    if out is None:
        out = _empty((groups.M, W.N), _BF16, A.device, stream)
    ldc = _rows(out, "out", groups.M, W.N, gpu)
    if workspace is None:
        with _made_on(stream):
            workspace = W.ragged_workspace(groups.M, groups.topk)
    wp, wn = _workspace(workspace, gpu)
    check(lib().vt_fp4_w4a16_gemm_ragged_combine(
        A.data_ptr(), lda, W.handle, groups.ids.data_ptr(), groups.order.data_ptr(),
        groups.offsets.data_ptr(), groups.weights.data_ptr(), groups.M, groups.topk,
        out.data_ptr(), ldc, wp, wn, _raw(stream, gpu)), "vt_fp4_w4a16_gemm_ragged_combine")
    return out


def moe_ffn_workspace(W_gate_up, W_down, M_max: int, topk: int) -> torch.Tensor:
    """A workspace for moe_ffn of up to M_max tokens of topk pairs each: one that serves the ragged
    products on either weight."""
    n = max(W.ragged_workspace_bytes(M_max, topk) for W in (W_gate_up, W_down))
    return status_workspace(n, W_down.packed.device)


def moe_ffn(x: torch.Tensor, W_gate_up, W_down, groups: RowGroups, out: torch.Tensor | None = None,
            h: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """A mixture-of-experts feed-forward block for any number of tokens: x [M, H] through the
    chosen experts' gate_up (silu(gate) * up) and down weights, summed by the router's weights
    into out [M, H].  h: optional bf16 [pairs, I] buffer of the inner activations; workspace:
    moe_ffn_workspace(W_gate_up, W_down, M_max, topk)."""
    # what the second product would refuse after the first is under way
    gpu = _check_groups(W_down, groups)
    if groups.weights is None:
        raise ValueError("the groups hold no weights")
    if W_gate_up.N != 2 * W_down.K:
        raise ValueError(f"W_down must take the {W_gate_up.N // 2} columns of gate and up (it takes {W_down.K})")
    if out is not None:
        _rows(out, "out", groups.M, W_down.N, gpu)
    if workspace is None:
        with _made_on(stream):
            workspace = moe_ffn_workspace(W_gate_up, W_down, groups.M, groups.topk)
    h = w4a16_gemm_ragged_silu_mul(x, W_gate_up, groups, out=h, workspace=workspace, stream=stream)
    return w4a16_gemm_ragged_combine(h, W_down, groups, out=out, workspace=workspace, stream=stream)


class LoraAdapters:
    """L low-rank adapters beside one projection: A bf16 [L, R, K], B bf16 [L, N, R], scale fp32
    [L], ranks int32 [L] (the rank in use of each, at most R; None: R)."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 ranks: torch.Tensor | None = None):
        if A.dim() != 3 or B.dim() != 3:
            raise ValueError("A must be [L, R, K] and B [L, N, R]")
        self.L, self.R, self.K = A.shape
        self.N = B.shape[1]
        dev = self.device = A.device
        _need(A, "A", torch.bfloat16, tuple(A.shape), dev)
        _need(B, "B", torch.bfloat16, (self.L, self.N, self.R), dev)
        _need(scale, "scale", torch.float32, (self.L,), dev)
        if ranks is not None:
            _need(ranks, "ranks", torch.int32, (self.L,), dev)
        self.A, self.B, self.scale, self.ranks = A, B, scale, ranks
        self.gpu = A.get_device()


def lora_add(x: torch.Tensor, adapters: LoraAdapters, groups: RowGroups, y: torch.Tensor,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out = y + scale_a * B_a (A_a x) for every row's adapter a (groups of the rows' adapter
    ids, topk = 1; rows in no group keep y).  y: the shared projection's output; out may be y."""
    ad = adapters
    if groups.topk != 1 or groups.E != ad.L:
        raise ValueError("groups must hold one id of [0, L) per row")
    gpu, M = ad.gpu, groups.M
    if groups.gpu != gpu:
        raise ValueError(f"groups must be on {ad.device}")
    ldx, ldy = _rows(x, "x", M, ad.K, gpu), _rows(y, "y", M, ad.N, gpu)
    if out is None:
        out = _empty((M, ad.N), _BF16, ad.device, stream)
    ldo = _rows(out, "out", M, ad.N, gpu)
    check(lib().vt_fp4_lora_add(x.data_ptr(), M, ldx, ad.K, ad.A.data_ptr(), ad.B.data_ptr(),
                                ad.scale.data_ptr(), 0 if ad.ranks is None else ad.ranks.data_ptr(),
                                ad.L, ad.R, ad.N, groups.order.data_ptr(),
                                groups.offsets.data_ptr(), y.data_ptr(), ldy, out.data_ptr(), ldo,
                                _raw(stream, gpu)), "vt_fp4_lora_add")
    return out
