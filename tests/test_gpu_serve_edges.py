"""Ends of the routing and of the adapters: where memory ends, whose bits depend on what,
and bits that the small pieces of sums hold.  Oracle and tolerances as in
tests/test_gpu_route.py and tests/test_gpu_lora.py, or derived at the test."""
import numpy as np
import pytest

from tests import _gpu as G
from tests import test_gpu_route as R

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,experts,topk,groups,topk_groups", [(1 << 21, 2, 2, 1, 1), (2048, 2, 2, 1, 1),
                                                               (1 << 20, 4, 1, 4, 2), (1 << 19, 8, 3, 2, 1),
                                                               (1 << 18, 16, 5, 8, 3)])
def test_route_logits_that_end_with_their_memory(t, experts, topk, groups, topk_groups, scoring):
    """Balanced scores of fewer allowed experts than the lists of choices hold: the lanes
    past the choices hold no expert, and read no logit of one.  16 MB (16 KB in one case)
    of logits, behind which their memory ends."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(experts)
    rule = R.rule_of(experts, topk, rng.standard_normal(experts) * 0.1, scoring=scoring, groups=groups,
                     topk_groups=topk_groups)
    l = (rng.standard_normal((400, experts)) * 1.5).astype(np.float32)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    buf = torch.zeros((t, experts), device=G.dev())
    buf[-400:] = G.to_dev(l)
    ids, w = X.exl3_route_topk(buf, rule)
    R.check(ids[-400:], w[-400:], l, rule)
