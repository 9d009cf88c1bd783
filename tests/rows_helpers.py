"""Plain fp64 forms of the operators on grouped rows, written from their definitions, and the
error bounds their tests use.

Bounds (elementwise, derived from the arithmetic, before any run):
  rounding a value v to bf16 (8 significant bits, ties to even) moves it by at most 2^-8 |v|;
  an fp32 sum of K exact products a_k w_k, in any order and with truncating adders, is off by at
  most K * 2^-23 * sum_k |a_k w_k|;
  fp32 expf, division and products are good to a few units of 2^-24: 2^-20 covers them."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
BF16 = 2.0 ** -8
GROUP = {0: 16, 1: 32}


def e4m3(b: np.ndarray) -> np.ndarray:
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, np.exp2(e - 7.0) * (1 + m / 8))
    return np.where(b >= 128, -v, v)


def weight64(fmt, codes, scales, glob=1.0):
    """One weight in fp64: codes [N, K/2], scales [N, K/g]."""
    n, half = codes.shape
    w = np.empty((n, half * 2))
    w[:, 0::2], w[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    unit = e4m3(scales) * glob if fmt == 0 else np.exp2(scales.astype(np.float64) - 127)
    return w * np.repeat(unit, GROUP[fmt], axis=1)


def random_weight(rng, fmt, E, N, K, wide=False):
    """Codes of every value, scales over several binades: codes [E, N, K/2], scales, globals."""
    codes = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
    if fmt == 0:
        scales = rng.integers(0x10, 0x58, size=(E, N, K // 16), dtype=np.uint8)
        glob = [float(np.float32(0.004 * (1 + e % 3))) for e in range(E)]
    else:
        scales = rng.integers(116, 124, size=(E, N, K // 32), dtype=np.uint8)
        if wide:  # spans more exponents than the packed re-encoding holds
            scales[:, ::3, 0] = 80
        glob = [1.0] * E
    return codes, scales, glob


def acts(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def group64(ids, E):
    """order, offsets from the definition."""
    flat = ids.reshape(-1)
    inside = (flat >= 0) & (flat < E)
    order = [i for e in range(E) for i in np.nonzero(flat == e)[0]] + list(np.nonzero(~inside)[0])
    counts = [int((flat == e).sum()) for e in range(E)]
    return np.array(order, dtype=np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def silu64(g):
    return g / (1 + np.exp(-g))


def products64(x, w):
    """(x . w^T, the bound on an fp32 evaluation's error) in fp64."""
    return x @ w.T, x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def silu_mul64(x, wg, wu):
    """(silu(g) * u, error bound before the final rounding); |silu'| <= 1.1."""
    g, dg = products64(x, wg)
    u, du = products64(x, wu)
    h = silu64(g) * u
    return h, 1.1 * dg * np.abs(u) + np.abs(silu64(g)) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(h)


def assert_close(got, ref, err, what=""):
    """|got - ref| <= err + the final rounding to bf16 of a value within err of ref."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bound = err + BF16 * (np.abs(ref) + err) + 2.0 ** -133
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], bound[bad][:4])
