"""GPU: the weighted sum of the experts' products is the sum of what the plain ragged product
writes (bf16), in fp32 and slot order, rounded once more."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import BF16, acts, f64, group64, random_weight

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("fmt", [vt.NVFP4, vt.MXFP4])
@pytest.mark.parametrize("M,topk,E,N,K", [
    (1, 1, 1, 3, 32), (3, 9, 12, 130, 64), (2, 32, 40, 264, 96), (70, 17, 33, 96, 160), (60, 4, 200, 300, 96),
    (700, 8, 16, 1400, 224)])
def test_the_sum_is_of_the_products_as_they_are_written(fmt, M, topk, E, N, K):
    rng = np.random.default_rng(M + N)
    c, s, g = random_weight(rng, fmt, E, N, K)
    W = vt.PackedWeight.grouped(_dev(c), _dev(s), g, fmt, E, N, K)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
    if topk > 1:  # slots in no group (weights that must not count), a token with none
        ids[:, topk // 2], ids[M // 2] = -1, E + 3
    weights = (rng.random((M, topk)) - 0.25).astype(np.float32)
    order, offsets = group64(ids, E)
    groups = vt.RowGroups(_dev(ids), _dev(order), _dev(offsets), _dev(weights))
    h, ws = acts(rng, M * topk, K).cuda(), W.ragged_workspace(M, topk)
    d = torch.zeros(M * topk, N, dtype=torch.bfloat16, device="cuda")
    vt.w4a16_gemm_ragged(h, W, groups, out=d, workspace=ws, gather=False, scatter=True)
    terms = f64(d).reshape(M, topk, N) * weights[:, :, None].astype(np.float64)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    y = f64(vt.w4a16_gemm_ragged_combine(h, W, groups, workspace=ws))
    # topk fp32 multiply-adds, then one rounding to bf16
    assert (np.abs(y - want) <= (topk * 2.0 ** -23) * size + BF16 * np.abs(want) + 2.0 ** -133).all()
    assert vt.workspace_status(ws) == 0
