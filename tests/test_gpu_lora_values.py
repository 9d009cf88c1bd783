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
