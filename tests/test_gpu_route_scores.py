"""GPU: the sigmoid router's choice where fp32 sigmoids of different logits are equal."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,E,topk", [(1, 8, 3), (40, 64, 8), (70, 300, 5)])
@pytest.mark.parametrize("base,step", [(17.0, 0.125), (-200.0, 0.5), (9.0, 2.0 ** -17)])
def test_without_a_bias_the_larger_logit_is_chosen(M, E, topk, base, step):
    """The sigmoid grows with the logit, so the choice is the logits' own order; sigmoids of
    these round to a few numbers (or one) in fp32."""
    rng = np.random.default_rng(E)
    perm = np.stack([rng.permutation(E) for _ in range(M)])
    logits = (base + step * perm).astype(np.float32)
    assert all(len(set(row)) == E for row in logits)
    r = vt.moe_route(torch.from_numpy(logits).cuda(), topk, scoring="sigmoid")
    want = np.argsort(-logits.astype(np.float64), axis=1, kind="stable")[:, :topk]
    assert np.array_equal(r.ids.cpu().numpy(), want)
