"""The sublayer's oracle at the edges of its definitions, against closed forms."""

import numpy as np

from oracle import sublayer as ref

INF = np.inf


def test_a_masked_expert_comes_last_whatever_its_bias():
    z = np.array([[0.0, -1.0, -INF, -2.0], [-INF, -INF, 3.0, -INF], [-INF] * 4])
    bias = np.array([0.0, 0.0, 0.9, 0.0])
    for score in ("softmax", "sigmoid"):
        ids, weights, *_ = ref.route(z, 4, bias=bias, score=score)
        assert ids.tolist() == [[0, 1, 3, 2], [2, 0, 1, 3], [0, 1, 2, 3]]
        assert (weights[0, 3], weights[1, 1:].tolist(), weights[2].tolist()) == (0.0, [0.0] * 3, [0.0] * 4)


def test_masked_experts_add_nothing_to_a_group():
    # three groups: one masked under a large bias, one with a single expert left, one of two weaker experts
    z = np.array([[-INF, -INF, 2.0, -INF, -3.0, -3.0]])
    bias = np.array([9.0, 9.0, -0.1, 9.0, -0.1, -0.1])
    kw = dict(bias=bias, groups=3, score="sigmoid")
    assert ref.route(z, 1, top_groups=1, **kw)[0].tolist() == [[2]]
    assert ref.route(z, 3, top_groups=2, **kw)[0].tolist() == [[2, 4, 5]]
    assert ref.route(z, 2, top_groups=1, **kw)[0].tolist() == [[2, 3]]


def test_the_gradient_of_saturated_sigmoids():
    # s (1 - s) = e / (1 + e)^2 with e = exp(-|l|)
    z = np.concatenate([np.linspace(8, 60, 14), np.linspace(-8, -60, 14)])[None]
    e = np.exp(-np.abs(z[0]))
    got = ref.route_backward(z, np.arange(28)[None], np.ones((1, 28)), "sigmoid", False, 2.0)[0]
    assert np.all(np.abs(got - 2 * e / (1 + e) ** 2) <= 1e-14 * got)
