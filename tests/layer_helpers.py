"""Plain forms of the cache, its attention and the norms, written from their definitions, and the
error bounds their tests use.

Bounds (elementwise, derived from the arithmetic, before any run):
  rounding to bf16 moves a value by at most 2^-8 of it, to f16 by at most 2^-11;
  an fp32 sum of n terms, in any order and with truncating adders, is off by at most n 2^-23 of the
  sum of their absolute values; fp32 exp2, division and square root are good to a few units of
  2^-24: 2^-20 covers them.
Attention: a score s = scale q.k is off by ds = (D + 8) 2^-23 scale sum |q k| (q held in f16 times a power
  of two is exact but for values below 2^-28 of the largest: 2^-39 of it, under one of the D units),
  so p = exp(s - m) is off by a factor 2 max ds (its own and the maximum's); p in f16 by 2^-11, and by
  2^-24 of the largest p where it is subnormal; the sums by n 2^-23.  The output is a ratio of two
  such sums: err = (2^-11 + 4 max ds + 2 n 2^-23 + 2^-18) sum p |v| / sum p + n 2^-24 max |v| / sum p,
  column by column."""
from __future__ import annotations

import numpy as np
import torch

from rows_helpers import E2M1, e4m3

F = np.float32


def quantise(x, g):
    """x fp32 [..., D], g fp32 broadcast against [..., 1]: (codes [..., D/2], scale bytes [...,
    D/16]), every operation rounded to fp32."""
    v = x.reshape(*x.shape[:-1], -1, 16)
    g = np.broadcast_to(g, x.shape[:-1] + (1,))[..., None].astype(F)
    bad = ~np.isfinite(v).all(-1, keepdims=True)
    with np.errstate(all="ignore"):
        top = np.where(bad, F(0), np.abs(v).max(-1, keepdims=True)).astype(F)
        t = (top / (F(6) * g)).astype(F)
    grid = e4m3(np.arange(127, dtype=np.uint8))  # finite, ascending
    t = np.minimum(t, 448).astype(np.float64)
    lo = np.searchsorted(grid, t, side="right") - 1
    hi = np.minimum(lo + 1, 126)
    up = (t - grid[lo] > grid[hi] - t) | ((t - grid[lo] == grid[hi] - t) & (lo % 2 == 1))
    byte = np.where(up, hi, lo).astype(np.uint8)
    unit = (grid[byte].astype(F) * g).astype(F)
    with np.errstate(all="ignore"):
        q = np.abs((v / unit).astype(F)).astype(np.float64)
    mag = E2M1[:8]
    c = np.zeros(v.shape, dtype=np.uint8)
    for i, border in enumerate((mag[1:] + mag[:-1]) / 2):  # halfway: to the even code
        c = np.where((q > border) | ((q == border) & (i % 2 == 1)), np.uint8(i + 1), c)
    c = np.where(bad | (grid[byte] == 0), np.uint8(0), c)
    c = np.where((v < 0) & (c > 0), c + 8, c).astype(np.uint8).reshape(x.shape)
    byte = np.where(bad, np.uint8(0x7F), byte)[..., 0]
    return c[..., 0::2] | (c[..., 1::2] << 4), byte


def values(codes, scales, g):
    """fp64 values of codes [..., D/2], scale bytes [..., D/16], globals broadcast against [..., 1]."""
    x = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    x[..., 0::2], x[..., 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    s = e4m3(scales)
    s = np.where((scales & 0x7F) == 0x7F, np.nan, s)
    return x * np.repeat(s, 16, axis=-1) * g


def head_norm(x, w, eps):
    ss = (x.astype(np.float64) ** 2).sum(-1, keepdims=True).astype(F)
    r = F(1) / np.sqrt(ss / F(x.shape[-1]) + F(eps))
    return (x * r).astype(F) * w.astype(F)


def rotate(x, cos, sin, interleaved):
    """cos, sin fp32 [T, half] against x fp32 [T, heads, D]."""
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    y = x.copy()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ra, rb = (a * c).astype(F) - (b * s).astype(F), (b * c).astype(F) + (a * s).astype(F)
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ra, rb
    else:
        y[..., :half], y[..., half:2 * half] = ra, rb
    return y


def attention(q, k, v, tables, lens, starts, page, scale, window=0, sinks=None, pages=None):
    """q fp64 [T, Hq, D]; k, v fp64 [slots, Hkv, D] by slot -> (out, err) [T, Hq, D]; rows of no
    sequence are NaN."""
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    pages = k.shape[0] // page if pages is None else pages
    out, err = np.full(q.shape, np.nan), np.zeros(q.shape)
    for b in range(len(lens)):
        r0, r1 = (b, b + 1) if starts is None else (starts[b], starts[b + 1])
        n = int(min(max(lens[b], 0), tables.shape[1] * page))
        j = np.arange(n)
        on = tables[b][j // page]
        there = (on >= 0) & (on < pages)
        slot = np.where(there, on, 0).astype(np.int64) * page + j % page
        for t in range(r0, r1):
            pos = n - (r1 - r0) + (t - r0)
            see = there & (j <= pos)
            if window:
                see &= j > pos - window
            for h in range(Hq):
                if not see.any():
                    out[t, h] = 0
                    continue
                K, V = k[slot[see], h // group], v[slot[see], h // group]
                with np.errstate(all="ignore"):
                    s = scale * (K @ q[t, h])
                    ds = (D + 8) * 2.0 ** -23 * abs(scale) * (np.abs(K) @ np.abs(q[t, h])).max()
                    m = s.max() if sinks is None else max(s.max(), sinks[h])
                    p = np.exp(s - m)
                    total = p.sum() + (0 if sinks is None else np.exp(sinks[h] - m))
                    out[t, h] = p @ V / total
                    m_count = int(see.sum())
                    rel = 2.0 ** -11 + 4 * ds + 2 * m_count * 2.0 ** -23 + 2.0 ** -18
                    err[t, h] = rel * (p @ np.abs(V)) / total + m_count * 2.0 ** -24 * np.abs(V).max(0) / total
    return out, err


def random_tokens(rng, slots, heads, D):
    """Raw tokens with every code and scales over several binades: (k_codes, k_scales, v_codes,
    v_scales) uint8."""
    c = lambda: rng.integers(0, 256, (slots, heads, D // 2), dtype=np.uint8)
    s = lambda: rng.integers(0x20, 0x48, (slots, heads, D // 16), dtype=np.uint8)
    return c(), s(), c(), s()


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()
