"""GPU: the router's choice, its weights and the grouping of rows by an index, against the
definitions in fp64 (the choice and the grouping exactly)."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import group64

pytestmark = pytest.mark.gpu


def _route64(logits, topk, scoring="softmax", bias=None, renormalize=True, scale=1.0):
    """ids and weights by the definition; logits fp64 [M, E].  The score of a sigmoid router is
    taken in fp32 as the operator defines it; the tests keep biased scores well apart."""
    M, E = logits.shape
    ids = np.full((M, topk), -1, dtype=np.int32)
    w = np.zeros((M, topk))
    for m in range(M):
        l = logits[m]
        live = l != -np.inf
        if scoring == "softmax":
            p = np.where(live, np.exp(l - l[live].max()), 0.0) if live.any() else np.zeros(E)
            p = p / p.sum() if live.any() else p
            score = l
        else:
            p = 1 / (1 + np.exp(-l))
            score = p + (0 if bias is None else bias)
        rank = sorted((e for e in range(E) if live[e]), key=lambda e: (-score[e], e))[:topk]
        v = p[rank]
        if renormalize and len(rank):
            v = v / v.sum()
        ids[m, :len(rank)], w[m, :len(rank)] = rank, v * scale
    return ids, w


def _check(r, ids, w, E):
    torch.cuda.synchronize()
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    # expf, one division each by the sum: a few units of 2^-24; 2^-19 leaves room for the sum's
    assert np.all(np.abs(r.weights.double().cpu().numpy() - w) <= 2.0 ** -19 * np.abs(w) + 1e-30)
    order, offsets = group64(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)


@pytest.mark.parametrize("M,E,topk", [(1, 1, 1), (1, 8, 2), (1, 128, 8), (3, 60, 4), (5, 33, 32),
                                      (31, 7, 7), (33, 1024, 8), (257, 128, 8), (700, 160, 6),
                                      (2049, 128, 8), (5000, 16, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_softmax_router(M, E, topk, dtype):
    g = torch.Generator().manual_seed(M * 7 + E)
    # bf16 logits repeat: equal ones go to the lowest index
    logits = (2 * torch.randn(M, E, generator=g)).to(dtype)
    r = vt.moe_route(logits.cuda(), topk)
    _check(r, *_route64(logits.double().numpy(), topk), E)


@pytest.mark.parametrize("renormalize,scale", [(True, 2.5), (False, 1.0), (False, 0.5)])
def test_weights_options(renormalize, scale):
    logits = torch.randn(65, 48, generator=torch.Generator().manual_seed(1))
    for scoring in ("softmax", "sigmoid"):
        r = vt.moe_route(logits.cuda(), 5, scoring=scoring, renormalize=renormalize, scale=scale)
        _check(r, *_route64(logits.double().numpy(), 5, scoring, None, renormalize, scale), 48)


def test_sigmoid_router_with_a_bias_that_changes_the_choice():
    rng = np.random.default_rng(5)
    M, E = 40, 32
    # scores a step of 1/64 apart after the bias, in another order for every token
    perm = np.stack([rng.permutation(E) for _ in range(M)])
    bias = rng.permutation(E) / 16.0
    logits = np.log((perm + 1) / 64.0) - np.log1p(-(perm + 1) / 64.0) + 1e-3 * rng.random((M, E))
    logits = torch.from_numpy(logits.astype(np.float32))
    b = torch.from_numpy(bias.astype(np.float32))
    r = vt.moe_route(logits.cuda(), 6, scoring="sigmoid", bias=b.cuda())
    ids, w = _route64(logits.double().numpy(), 6, "sigmoid", bias)
    assert not np.array_equal(ids, _route64(logits.double().numpy(), 6, "sigmoid")[0])
    _check(r, ids, w, E)


def test_masked_experts_and_empty_rows():
    E, topk = 20, 4
    logits = torch.randn(6, E, generator=torch.Generator().manual_seed(2))
    logits[0] = -float("inf")                       # nothing left
    logits[1, 3:] = -float("inf")                   # three left, four wanted
    logits[2, ::2] = -float("inf")
    logits[3] = torch.finfo(torch.float32).min      # the lowest number is a number: a tie
    logits[4, :] = 0.0
    logits[4, 1::2] = -0.0                          # equal to 0
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            r = vt.moe_route(logits.cuda(), topk, scoring=scoring, renormalize=renormalize)
            ids, w = _route64(logits.double().numpy(), topk, scoring, None, renormalize)
            if scoring == "sigmoid":
                # sigmoid(lowest) is 0: nothing to divide by
                keep = [0, 1, 2, 4, 5]
                torch.cuda.synchronize()
                assert np.array_equal(r.ids.cpu().numpy(), ids)
                assert np.allclose(r.weights.double().cpu().numpy()[keep], w[keep], rtol=2e-6, atol=0)
            else:
                _check(r, ids, w, E)
            assert r.ids[0].tolist() == [-1] * topk and r.weights[0].abs().sum().item() == 0


def test_nan_counts_as_largest():
    logits = torch.zeros(2, 9)
    logits[0, 5] = float("nan")
    r = vt.moe_route(logits.cuda(), 2)
    assert r.ids.tolist() == [[5, 0], [0, 1]]
    assert torch.isnan(r.weights[0, 0]) and torch.equal(r.weights[1].cpu(), torch.tensor([.5, .5]))


def test_strided_logits_and_reused_buffers():
    E, topk = 24, 3
    ws = vt.group_workspace(600, topk, E, "cuda")
    for M in (600, 1, 33, 0, 512):
        wide = torch.randn(M, E + 7, generator=torch.Generator().manual_seed(M))
        out = vt.RowGroups.empty(M, topk, E, "cuda", weights=True)
        r = vt.moe_route(wide.cuda()[:, 3:3 + E], topk, out=out, workspace=ws)
        assert r is out
        ids, w = _route64(wide[:, 3:3 + E].double().numpy(), topk)
        _check(r, ids, w, E)


@pytest.mark.parametrize("M,topk,E", [(0, 1, 3), (1, 1, 1), (1, 4, 9), (130, 8, 128), (4097, 2, 1024),
                                      (3000, 8, 5), (20011, 1, 64), (70000, 1, 3)])
def test_group_rows(M, topk, E):
    rng = np.random.default_rng(M + E)
    ids = rng.integers(-2, E + 2, size=(M, topk)).astype(np.int32)  # some in no group
    if M > 100:
        ids[M // 3:M // 2] = E // 2                                 # one heavy group
    r = vt.group_rows(torch.from_numpy(ids).cuda(), E)
    order, offsets = group64(ids, E)
    torch.cuda.synchronize()
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)


def test_grouping_on_another_stream_and_in_a_graph():
    E, topk, M = 64, 4, 900
    logits = torch.empty(M, E, device="cuda")
    ws = vt.group_workspace(M, topk, E, "cuda")
    out = vt.RowGroups.empty(M, topk, E, "cuda", weights=True)
    side = torch.cuda.Stream()
    host = [torch.randn(M, E, generator=torch.Generator().manual_seed(s)) for s in range(3)]
    logits.copy_(host[0])
    side.wait_stream(torch.cuda.current_stream())
    vt.moe_route(logits, topk, out=out, workspace=ws, stream=side)
    side.synchronize()
    _check(out, *_route64(host[0].double().numpy(), topk), E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.moe_route(logits, topk, out=out, workspace=ws)
    for h in host[1:]:
        logits.copy_(h)
        graph.replay()
        _check(out, *_route64(h.double().numpy(), topk), E)
