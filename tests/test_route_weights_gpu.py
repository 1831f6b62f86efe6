"""Weights of a softmax over all experts (no renormalising) in fp32, against 64 bits.

u = 2^-24.  expf is within 1 ulp (2 u) and takes the rounding of its argument (u times its size).  A lane adds up to 16 terms in pairs (4
roundings), the warp 32 lanes (5); 1 / sum, the product with it and with the factor round once each."""
import numpy as np
import pytest
import torch

from tests.gpu_util import qlib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def errors(q, lg, k, bias=None, scale=1.0):
    """(relative errors of the weights in u, the chosen logits' distances from the largest)."""
    rule = q.RouteRule("softmax", bias=bias, renormalise=False, scale=scale)
    ids, w, _ = q.route(torch.from_numpy(lg).cuda(), k, rule=rule)
    ids, w = ids.cpu().numpy().astype(np.int64), w.cpu().numpy().astype(np.float64)
    far = lg.max(1, keepdims=True).astype(np.float64) - lg
    s = np.exp(-far)
    want = scale * np.take_along_axis(s / s.sum(1, keepdims=True), ids, 1)
    return np.abs(w - want) / want / U, np.take_along_axis(far, ids, 1)


@pytest.mark.parametrize("t,e,k", [(1, 512, 10), (64, 512, 16), (5001, 160, 6), (2000, 512, 10), (300, 96, 4), (9, 33, 8)])
@pytest.mark.parametrize("biased", [False, True])
def test_random_logits(t, e, k, biased):
    """The mean distance that enters the sum is at most log e (6.3): 2 + 6.3 + 9 for the sum, 2 + distance for the term, 3 after."""
    q = qlib()
    rng = np.random.default_rng(t + e)
    bias = torch.from_numpy((0.2 * rng.standard_normal(e)).astype(np.float32)).cuda() if biased else None
    off, far = errors(q, (1.5 * rng.standard_normal((t, e))).astype(np.float32), k, bias, 2.5)
    assert np.all(off <= 22.4 + far), off.max()


def test_one_large_term_among_many_small_ones():
    """The largest term is 1 and exact; the others, 2 u off, are less than a seventh of the sum: 0.3 + 9 + 2."""
    q = qlib()
    for d in np.linspace(8.0, 8.95, 400):
        lg = np.full((1, 512), -d, np.float32)
        lg[0, 3] = 0.0
        off, _ = errors(q, lg, 1)
        assert off.max() <= 11.3, (d, off.max())


def test_scores_below_every_number():
    """Renormalised weights are of exact scores: e^-800 and e^-801 are in the proportion of e to 1.  Each term 2 u and its argument's
    rounding (none: whole numbers), the sum 5 u, a division, the factor: 10 u."""
    q = qlib()
    lg = torch.full((3, 40), -2000.0, device="cuda")
    lg[:, 7], lg[:, 9] = -800.0, -801.0
    want = 2.5 * np.array([1.0 / (1.0 + np.exp(-1.0)), 1.0 / (1.0 + np.exp(1.0))])
    # by sigmoid, and by a softmax whose largest logit is in a group that a bias leaves out
    groups = lg.clone()
    groups[:, 30] = 100.0
    bias = torch.zeros(40, device="cuda")
    bias[20:] = -4.0
    for ids, w, _ in (q.route(lg, 2, rule=q.RouteRule("sigmoid", scale=2.5)),
                      q.route(groups, 2, rule=q.RouteRule("softmax", bias=bias, groups=2, topk_groups=1, group_best=1, scale=2.5))):
        w = w.cpu().numpy().astype(np.float64)
        if int(ids[0, 0]) == 7:
            assert ids.tolist() == [[7, 9]] * 3 and np.all(np.abs(w - want) <= 10 * U * want)
        else:  # the softmax's scores are 0 in 64 bits: the index decides, and the weights are those of the chosen logits
            assert ids.tolist() == [[0, 1]] * 3 and np.all(np.abs(w - 1.25) <= 10 * U * 1.25)
    lg.fill_(float("-inf"))
    assert torch.isnan(q.route(lg, 2, rule=q.RouteRule("sigmoid"))[1]).all()
