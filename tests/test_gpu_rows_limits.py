"""GPU: the router and the adapters at the ends of their ranges: up to 1024 experts and adapters,
biases that are infinite or NaN, groups that hold values out of range."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import acts, assert_close, f64, group64

pytestmark = pytest.mark.gpu


def _lora64(x, y, ids, A, B, scale):
    """y + s B (A x) and the bound on its evaluation (v to 2^-16, the sums to n 2^-23)."""
    out, err = f64(y).copy(), 2.0 ** -20 * np.abs(f64(y))
    K, R = A.shape[2], A.shape[1]
    for m, a in enumerate(ids):
        if 0 <= a < A.shape[0]:
            Aa, Ba, s = f64(A[a]), f64(B[a]), float(scale[a])
            v, va = Aa @ f64(x[m]), np.abs(Aa) @ np.abs(f64(x[m]))
            out[m] += s * (Ba @ v)
            err[m] += abs(s) * (np.abs(Ba) @ ((K + R) * 2.0 ** -23 * va + 2.0 ** -15 * np.abs(v)))
    return out, err


def _case(rng, M, L, R, K, N):
    A, B = acts(rng, L, R, K), acts(rng, L, N, R)
    scale = torch.from_numpy(rng.uniform(0.5, 2, L).astype(np.float32))
    return acts(rng, M, K), acts(rng, M, N), A, B, scale, vt.LoraAdapters(A.cuda(), B.cuda(), scale.cuda())


@pytest.mark.parametrize("M,L,R,K,N", [(1, 1024, 8, 64, 72), (300, 1024, 8, 64, 72), (1500, 700, 16, 40, 33),
                                       (70000, 1024, 8, 16, 8)])
def test_a_thousand_adapters(M, L, R, K, N):
    rng = np.random.default_rng(M)
    x, y, A, B, scale, ad = _case(rng, M, L, R, K, N)
    ids = rng.integers(-1, L, M)
    ids[0] = L - 1
    groups = vt.group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), L)
    out = vt.lora_add(x.cuda(), ad, groups, y.cuda())
    some = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 400)]))
    t = torch.from_numpy(some)
    assert_close(out.cpu()[t], *_lora64(x[t], y[t], ids[some], A, B, scale))


@pytest.mark.parametrize("M", [40, 600])
def test_adapters_do_not_follow_groups_out_of_range(M):
    rng = np.random.default_rng(M)
    L, R, K, N = 4, 8, 64, 40
    x, y, A, B, scale, ad = _case(rng, M, L, R, K, N)
    ids = rng.integers(-1, L, M)
    order, offsets = group64(ids, L)
    ref, err = _lora64(x, y, ids, A, B, scale)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).cuda()
    full = torch.full((M + 2, N + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[1:-1, 3:3 + N]
    wild = order.copy()
    at = rng.choice(M, 4, replace=False)
    wild[at] = [-1, M, 2 ** 31 - 1, -2 ** 31]
    for o, f in ((wild, offsets), (order, np.where(np.arange(L + 1) == 2, M + 9, offsets)),
                 (order, np.where(np.arange(L + 1) == 1, -5, offsets)), (order, np.full(L + 1, 2 ** 31 - 1)),
                 (order, np.full(L + 1, -2 ** 31))):
        out.fill_(7.0)
        groups = vt.RowGroups(dev(ids), dev(o), dev(f))
        vt.lora_add(x.cuda(), ad, groups, y.cuda(), out=out)
        if o is wild:
            right = np.setdiff1d(np.arange(M), order[at])
            assert_close(f64(out)[right], ref[right], err[right])
            assert (out[dev(order[at]).long()] == 7).all()
        keep = full.clone()
        keep[1:-1, 3:3 + N] = 7.0
        assert torch.all(keep == 7.0)


@pytest.mark.parametrize("M,E,topk", [(5, 300, 6), (90, 1024, 32), (2000, 257, 8)])
def test_sigmoid_router_of_many_experts(M, E, topk):
    """Scores a step of 2^-11 apart in another order for every token."""
    rng = np.random.default_rng(E)
    perm = np.stack([rng.permutation(E) for _ in range(M)])
    p = (perm + 512) / 2048.0
    logits = np.log(p / (1 - p)).astype(np.float32)
    want = np.argsort(-perm, axis=1)[:, :topk]
    w = np.take_along_axis(1 / (1 + np.exp(-logits.astype(np.float64))), want, 1)
    order, offsets = group64(want.astype(np.int32), E)
    for bias in (None, torch.full((E,), 0.25, device="cuda")):
        r = vt.moe_route(torch.from_numpy(logits).cuda(), topk, scoring="sigmoid", bias=bias, renormalize=False)
        assert np.array_equal(r.ids.cpu().numpy(), want)
        assert np.all(np.abs(f64(r.weights) - w) <= 2.0 ** -20 * w)
        assert np.array_equal(r.order.cpu().numpy(), order)
        assert np.array_equal(r.offsets.cpu().numpy(), offsets)


@pytest.mark.parametrize("E", [20, 200, 600])
def test_biases_that_are_infinite_or_nan(E):
    """-Inf: never chosen; +Inf and NaN: chosen first (NaN before Inf); the weights are the sigmoids'."""
    rng = np.random.default_rng(E)
    logits = torch.from_numpy(rng.standard_normal((9, E)).astype(np.float32))
    bias = torch.full((E,), -float("inf"))
    bias[3], bias[7], bias[E - 1], bias[5] = float("inf"), 0.0, float("nan"), 10.0
    r = vt.moe_route(logits.cuda(), 6, scoring="sigmoid", bias=bias.cuda())
    assert r.ids.tolist() == [[E - 1, 3, 5, 7, -1, -1]] * 9
    p = torch.sigmoid(logits.double())[:, [E - 1, 3, 5, 7]]
    got = r.weights.double().cpu()
    assert torch.allclose(got[:, :4], p / p.sum(1, keepdim=True), rtol=2e-6, atol=0)
    assert not got[:, 4:].any()
    bias[:] = -float("inf")
    r = vt.moe_route(logits.cuda(), 6, scoring="sigmoid", bias=bias.cuda())
    assert (r.ids == -1).all() and not r.weights.any() and not r.offsets.any()
