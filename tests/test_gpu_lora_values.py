"""GPU: infinities, values at the ends of fp32 and bit patterns in the low-rank adapters.  The
expected values are the definition's, out = y + s * B (A x) over an adapter's own ranks, evaluated in
fp64 with IEEE infinities."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import acts, f64

pytestmark = pytest.mark.gpu


def _run(x, y, ids, A, B, scale, ranks=None, **kw):
    ad = vt.LoraAdapters(A.cuda(), B.cuda(), scale.cuda(),
                         None if ranks is None else torch.tensor(ranks, dtype=torch.int32).cuda())
    groups = vt.group_rows(torch.from_numpy(np.asarray(ids, np.int32)).cuda(), A.shape[0])
    return vt.lora_add(x.cuda(), ad, groups, y.cuda(), **kw)


@pytest.mark.parametrize("M,K,N", [(1, 64, 40), (9, 256, 129), (130, 72, 264), (9, 33, 17)])
@pytest.mark.parametrize("R,ranks", [(1, None), (5, None), (17, None), (24, None), (40, [40, 3]),
                                     (64, [50, 1]), (100, None)])
def test_an_infinite_activation_meets_its_adapters_own_ranks_only(M, K, N, R, ranks):
    """A, B and the scale positive: an infinite x makes every v, and so every column, +Inf."""
    rng = np.random.default_rng(R + N)
    A, B = acts(rng, 2, R, K).abs() + 0.25, acts(rng, 2, N, R).abs() + 0.25
    scale = torch.tensor([0.5, 2.0])
    x, y = acts(rng, M, K), acts(rng, M, N)
    ids = np.arange(M) % 2
    rows = [0] if M == 1 else [0, 3, M - 1]
    for m in rows:
        x[m, (7 * m) % K] = float("inf")
    out = f64(_run(x, y, ids, A, B, scale, ranks))
    assert (out[rows] == np.inf).all()
    assert np.isfinite(np.delete(out, rows, 0)).all()


@pytest.mark.parametrize("R", [1, 16])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_finite_v_beyond_the_largest_bf16(R, sign):
    """v = 2^128 (1 - 2^-10), an fp32 number that rounds to infinity in bf16; B = 2^-100."""
    K, N = 8, 24
    x, A = torch.zeros(2, K), torch.zeros(1, R, K)
    x[:, 0], x[:, 1] = 255 / 128 * 2.0 ** 63, 2.0 ** 63
    A[0, R - 1, 0], A[0, R - 1, 1] = sign * 2.0 ** 64, sign * 3 * 2.0 ** 55
    B = torch.zeros(1, N, R)
    B[0, :, R - 1] = 2.0 ** -100
    bf = torch.bfloat16
    out = f64(_run(x.to(bf), torch.zeros(2, N, dtype=bf), [0, 0], A.to(bf), B.to(bf), torch.ones(1)))
    want = sign * 2.0 ** 28 * (1 - 2.0 ** -10)
    assert (np.abs(out - want) <= 2.0 ** -8 * abs(want)).all(), out


@pytest.mark.parametrize("M,R", [(1, 1), (5, 16), (70, 24)])
def test_an_infinite_entry_of_b(M, R):
    """B[n][r] = Inf makes column n infinite with v_r's sign, whether or not v_r is a bf16 number."""
    rng = np.random.default_rng(R)
    K, N = 64, 40
    A, B, scale = acts(rng, 1, R, K), acts(rng, 1, N, R), torch.ones(1)
    x, y = acts(rng, M, K), acts(rng, M, N)
    x[0] = 0
    x[0, 0], A[0, :, 0] = 1.0, torch.arange(1, R + 1).to(torch.bfloat16)  # small integers: v exact in bf16
    B[0, 3, R - 1], B[0, 30, 0] = float("inf"), float("-inf")
    out = f64(_run(x, y, np.zeros(M), A, B, scale))
    v = f64(x) @ f64(A[0]).T
    assert (v[:, [0, R - 1]] != 0).all()
    assert np.array_equal(out[:, 3], np.sign(v[:, R - 1]) * np.inf)
    assert np.array_equal(out[:, 30], -np.sign(v[:, 0]) * np.inf)
    assert np.isfinite(np.delete(out, [3, 30], 1)).all()


def test_an_infinite_v_meets_an_infinite_entry_of_b():
    K, N, bf = 16, 24, torch.bfloat16
    A, B = torch.ones(1, 1, K, dtype=bf), torch.ones(1, N, 1, dtype=bf)
    x, y = torch.ones(2, K, dtype=bf), torch.zeros(2, N, dtype=bf)
    x[0, 2], B[0, 5, 0], B[0, 6, 0] = float("inf"), float("inf"), float("-inf")
    out = f64(_run(x, y, [0, 0], A, B, torch.ones(1)))
    assert (out[:, 5] == np.inf).all() and (out[:, 6] == -np.inf).all()
    assert (np.delete(out[0], [5, 6]) == np.inf).all() and (np.delete(out[1], [5, 6]) == K).all()


@pytest.mark.parametrize("N", [64, 77])
def test_rows_without_an_adapter_keep_every_bit(N):
    """-0, subnormals and NaNs of any payload, for rows in no group and for an adapter of rank 0."""
    rng = np.random.default_rng(N)
    M, K, L, R = 40, 32, 3, 8
    A, B, scale = acts(rng, L, R, K), acts(rng, L, N, R), torch.ones(L)
    bits = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, size=(M, N)).astype(np.int16))
    bits[:, :6] = torch.tensor([-32768, 0, 0x7FC1, 0x7F81, 1, -32767], dtype=torch.int16)
    x, y = acts(rng, M, K), bits.view(torch.bfloat16)
    ids = np.arange(M) % 4 - 1                          # -1, 0, 1, 2
    out = _run(x, y, ids, A, B, scale, [8, 0, -2]).cpu().view(torch.int16)
    kept = torch.from_numpy(ids != 0)
    assert torch.equal(out[kept], bits[kept])
