"""Groups valued by the sum of two experts whose values have opposite signs: the sum is small and the error of its summands is
not.  The choice is that of 64-bit scores."""
import numpy as np
import pytest

from tests.gpu_util import qlib
from tests.test_route_by_gpu import compare

pytestmark = pytest.mark.gpu


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [2.0, 50.0, 256.0, 1000.0])
def test_near_groups_of_opposite_values(size, score):
    """Two groups of two, their sums 1e-7 to 1e-4 apart; biases of +size and -size."""
    q = qlib()
    rng = np.random.default_rng(int(size))
    t = 6000
    a, b, c = rng.uniform(-1.5, 1.5, (3, t))
    apart = np.exp(rng.uniform(np.log(1e-7), np.log(1e-4), t)) * rng.choice([-1.0, 1.0], t)
    if score == "sigmoid":
        last = sigmoid(a) + sigmoid(b) - sigmoid(c) + apart
        keep = (last > 0.02) & (last < 0.98)
        last = np.where(keep, last, 0.5)
        d = np.log(last / (1.0 - last))
    else:  # the scores are exp over one sum
        last = np.exp(a) + np.exp(b) - np.exp(c) + apart
        keep = last > 0.02
        d = np.log(np.where(keep, last, 1.0))
    lg = np.stack([a, b, c, d], 1).astype(np.float32)[keep]
    assert len(lg) > 2000
    bias = np.array([size, -size, size, -size], np.float32)
    compare(q, lg, 2, bias=bias, tables=False, score=score, groups=2, topk_groups=1, group_best=2)


@pytest.mark.parametrize("size", [50.0, 256.0])
def test_many_groups_of_opposite_values(size):
    q = qlib()
    rng = np.random.default_rng(int(size) + 1)
    e = 64
    base = rng.uniform(-1.0, 1.0, (600, 2))
    lg = np.repeat(base[:, None], 32, 1)
    lg[..., 0] += 1e-5 * rng.standard_normal((600, 32))  # groups' sums some 1e-6 apart
    bias = np.tile(np.array([size, -size], np.float32), 32)
    compare(q, lg.reshape(600, e), 8, bias=bias, tables=False, score="sigmoid", groups=32, topk_groups=12, group_best=2)


def test_summands_at_the_ends_of_the_range():
    """3e38 and -3e38: the sum of their magnitudes passes fp32's range, their sum does not."""
    q = qlib()
    rng = np.random.default_rng(9)
    lg = rng.standard_normal((50, 16)).astype(np.float32)
    bias = np.tile(np.array([3e38, -3e38, -np.inf, -np.inf], np.float32), 4)
    compare(q, lg, 4, bias=bias, tables=False, score="sigmoid", groups=4, topk_groups=2, group_best=2)
    bias = np.tile(np.array([3e38, 3e38, 0.0, 0.0], np.float32), 4)
    bias[4:6] = 2e38
    compare(q, lg, 4, bias=bias, tables=False, score="sigmoid", groups=4, topk_groups=2, group_best=2)
