"""The oracle of the norm, the adapters and the routing by a rule, against closed forms and library sorts (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import layer as ol


def test_norm_of_a_constant_row_is_the_weight():
    w = np.array([1.0, -2.0, 0.5, 3.0])
    h, y = ol.rms_norm(np.full((2, 4), [[3.0], [-0.25]]), None, w, 0.0, 1.0)
    assert np.allclose(y, [w + 1.0, -(w + 1.0)], rtol=1e-15, atol=0)


def test_norm_adds_the_residual_in_bf16():
    h, _ = ol.rms_norm([[1.0, 2.0]], [[2.0 ** -8, 2.0 ** -6]], [1.0, 1.0], 1e-6, 0.0)
    want = (torch.tensor([[1.0, 2.0]]).bfloat16() + torch.tensor([[2.0 ** -8, 2.0 ** -6]]).bfloat16()).double().numpy()
    assert np.array_equal(h, want) and h[0, 0] == 1.0  # a tie goes to the even neighbour


def test_quantised_groups_reach_448():
    y = np.random.default_rng(0).standard_normal((3, 100))
    q, s = ol.quantise(y, 32)
    assert s.shape == (3, 4)
    for i in range(4):
        assert np.allclose(np.max(np.abs(q[:, 32 * i:32 * i + 32]), axis=1), 448.0, rtol=1e-15)
    assert np.array_equal(ol.quantise(np.zeros((1, 5)), 0)[1], [[2.0 ** -100]])
    q, s = ol.quantise(np.array([[np.inf, 7.0, np.nan, -np.inf]]), 0)
    assert s[0, 0] == 7.0 / 448 and q[0, 1] == 448.0 and np.isinf(q[0, 0])


def test_lora_is_two_products_a_row():
    rng = np.random.default_rng(1)
    a, b = rng.standard_normal((2, 4, 6)), rng.standard_normal((2, 5, 4))
    x, y = rng.standard_normal((3, 6)), rng.standard_normal((3, 5))
    out, _, _ = ol.lora([1, -1, 0], x, y, a, b, [0.5, 2.0], [4, 3])
    assert np.allclose(out[0], y[0] + 2.0 * (b[1, :, :3] @ a[1, :3]) @ x[0])
    assert np.array_equal(out[1], y[1])
    assert np.allclose(out[2], y[2] + 0.5 * (b[0] @ a[0]) @ x[2])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_by_without_bias_is_a_sort_of_the_logits(score):
    lg = np.random.default_rng(2).standard_normal((20, 48)).astype(np.float32)
    ids, w = ol.route_by(lg, 5, score, renormalise=False, scale=3.0)
    t = torch.from_numpy(lg).double()
    s = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    top = s.topk(5, 1)
    assert np.array_equal(ids, top.indices.numpy()) and np.allclose(w, 3.0 * top.values.numpy(), rtol=1e-14)
    ids2, w2 = ol.route_by(lg, 5, score)
    assert np.array_equal(ids, ids2) and np.allclose(w2.sum(1), 1.0)


def test_route_by_groups_and_bias():
    # groups {0,1}, {2,3}, {4,5}; the bias moves the choice and not the weights
    lg = np.log(np.array([[0.5, 0.1, 0.3, 0.25, 0.45, 0.05]]) / (1 - np.array([[0.5, 0.1, 0.3, 0.25, 0.45, 0.05]]))).astype(np.float32)
    ids, w = ol.route_by(lg, 2, "sigmoid", groups=3, topk_groups=1, group_best=1, renormalise=False)
    assert ids.tolist() == [[0, 1]]
    ids, w = ol.route_by(lg, 2, "sigmoid", groups=3, topk_groups=1, group_best=2, bias=np.array([-0.2, 0, 0, 0, 0, 0]), renormalise=False)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, [[0.3, 0.25]], atol=1e-7)
    ids, _ = ol.route_by(np.zeros((1, 6)), 3, "sigmoid", groups=3, topk_groups=2, group_best=2)
    assert ids.tolist() == [[0, 1, 2]]  # ties to the lower index
    ids, w = ol.route_by(np.array([[np.nan, 1.0, -np.inf, 0.0]]), 4, "softmax", renormalise=False)
    assert ids.tolist() == [[1, 3, 2, 0]] and w[0, 2] == 0.0 and np.isnan(w[0, 3]) and np.isclose(w[0, :3].sum(), 1.0)
