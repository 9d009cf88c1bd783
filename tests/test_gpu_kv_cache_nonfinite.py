"""GPU: per-head norms of heads that hold an inf or NaN.  A warp takes four heads of 64 or two of 128 at a time:
the others of the token stay bit for bit those of the formulas."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from layer_helpers import F, gpu
from rows_helpers import acts
from test_gpu_kv_cache import _bf16, _cache, _expect

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _check(D, Hq, Hkv, T, rot, interleaved, fp32, bad):
    """bad: (token, head of the row, column, value)."""
    rng = np.random.default_rng(D + T + rot)
    cache = _cache(rng, -(-T // 16) + 1, 16, Hkv, D)
    x = acts(rng, T, Hq + 2 * Hkv, D)
    for t, h, d, value in bad:
        x[t, h, d] = value
    q, k, v = (t if t.shape[1] else None for t in x.split([Hq, Hkv, Hkv], 1))
    w = lambda: (1 + 0.3 * torch.from_numpy(rng.standard_normal(D).astype(F))).to(torch.float32 if fp32 else torch.bfloat16)
    qn, kn = w() if Hq else None, w()
    slots, positions = rng.permutation(cache.pages * 16)[:T], rng.integers(0, 90, T)
    table = vt.rope_table(90, rot, 1000.0) if rot else None
    everything = torch.arange(cache.pages * 16, device="cuda")
    before = [t.cpu().numpy() for t in cache.get(everything)]
    on = lambda t: None if t is None else t.cuda()
    got = vt.kv_append(on(q), k.cuda(), v.cuda(), cache, gpu(slots), gpu(positions.astype(np.int32)) if rot else None, table,
                       on(qn), on(kn), eps=1e-5, interleaved=interleaved)
    with np.errstate(invalid="ignore"):
        raw, want = _expect(cache, q, k, v, slots, positions, table, qn, kn, 1e-5, interleaved, before)
    for a, b in zip(cache.get(everything), raw):
        assert np.array_equal(a.cpu().numpy(), b)
    if Hq:
        got, want = got.cpu(), _bf16(want)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
    return raw


@pytest.mark.parametrize("rot,interleaved", [(0, False), (32, False), (64, True)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_head_that_is_not_finite(D, rot, interleaved):
    Hq, Hkv = 6, 2
    for h in range(Hq + 2 * Hkv):
        bad = [(0, h, 3, INF), (1, h, D - 1, -INF), (2, h, D // 2, NAN)]
        _check(D, Hq, Hkv, 4, rot, interleaved, h % 2 == 0, bad)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_heads_of_every_kind_in_one_warp(D):
    """Finite, infinite and NaN heads beside one another, none finite, and warps that take several steps of a token."""
    for T, Hq, Hkv in ((5, 8, 4), (3, 0, 3), (700, 32, 8)):
        rng = np.random.default_rng(T)
        heads = Hq + 2 * Hkv
        bad = [(int(t), int(h), int(rng.integers(D)), (INF, -INF, NAN)[int(rng.integers(3))])
               for t in range(min(T, 40)) for h in rng.permutation(heads)[:rng.integers(1, heads + 1)]]
        bad += [(0, h, 1, NAN if h % 2 else INF) for h in range(heads)]
        raw = _check(D, Hq, Hkv, T, 16, False, False, bad)
        assert (raw[1] == 0x7F).any() and (raw[3] == 0x7F).any()
