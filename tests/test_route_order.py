"""The oracle's order of experts whose scores 64 bits cannot tell apart, and of a softmax with NaN logits (no GPU)."""
import numpy as np
import pytest

from oracle import layer as ol


def test_saturated_sigmoids_without_a_bias_go_by_their_logits():
    lg = np.array([[40.0, 50.0, -3.0, 45.0, 50.0]], np.float32)
    assert len(set(1.0 / (1.0 + np.exp(-lg[0, [0, 1, 3]].astype(np.float64))))) == 1
    assert ol.route_by(lg, 4, "sigmoid")[0].tolist() == [[1, 4, 3, 0]]
    # with a bias the scores in 64 bits are meant, and equal values go by the index
    assert ol.route_by(lg, 4, "sigmoid", bias=np.zeros(5, np.float32))[0].tolist() == [[0, 1, 3, 4]]


@pytest.mark.parametrize("score,lg,want", [
    ("sigmoid", [-900.0, 99.0, -800.0, 98.0, 100.0, -850.0], [4, 1, 5, 0]),  # 99, 98 and 100 are all 1, -900 and -850 are 0
    ("softmax", [-900.0, -1.0, -800.0, -2.0, 0.0, -950.0], [4, 1, 0, 5])])
def test_groups_of_equal_scores_go_by_their_logits(score, lg, want):
    assert ol.route_by(np.array([lg], np.float32), 4, score, groups=3, topk_groups=2, group_best=1)[0].tolist() == [want]


def test_a_nan_logit_adds_nothing_to_a_softmax():
    lg = np.array([[1.0, np.nan, 0.0, 2.0]], np.float32)
    ids, w = ol.route_by(lg, 4, "softmax", renormalise=False)
    want = np.exp([2.0, 1.0, 0.0]) / np.exp([2.0, 1.0, 0.0]).sum()
    assert ids.tolist() == [[3, 0, 2, 1]] and np.allclose(w[0, :3], want) and np.isnan(w[0, 3])


def test_a_group_without_numbers_is_as_minus_infinity():
    lg = np.array([[np.nan, np.nan, -np.inf, -np.inf, 0.0, 1.0]], np.float32)
    assert ol.route_by(lg, 4, "sigmoid", groups=3, topk_groups=2, group_best=1)[0].tolist() == [[5, 4, 0, 1]]
