"""A softmax with an infinite logit that is not chosen: its scores are NaN, the index chooses, and the weights are NaN."""
import numpy as np
import pytest

from tests.gpu_util import qlib
from tests.test_route_by_gpu import compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("t", [1, 3, 40, 200])
def test_infinite_logits_behind_the_chosen(t, renormalise):
    q = qlib()
    rng = np.random.default_rng(t)
    lg = rng.standard_normal((t, 96)).astype(np.float32)
    lg[::2, 90] = np.inf
    lg[::3, 5] = -np.inf
    bias = 0.1 * rng.standard_normal(96)
    for kw in (dict(bias=bias), dict(bias=bias, groups=8, topk_groups=2), dict(groups=8, topk_groups=2, group_best=2), dict()):
        compare(q, lg, 6, score="softmax", renormalise=renormalise, **kw)
