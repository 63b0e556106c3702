"""The plain forms at their ends, by values worked out by hand."""
import numpy as np

from oracle import dense as D

INF = np.inf


def test_an_infinite_temperature():
    x = np.array([[1.0, INF, 3.0, INF, -INF], [2.0, 1.0, 2.0, -3.0, -INF]])
    for u, want in ((0.0, [1, 0]), (0.6, [3, 1]), (1.0, [3, 3])):
        ids, lp, kept = D.sample(x, np.array([u, u]), np.array([INF, INF]))
        assert ids.tolist() == want and kept.tolist() == [4, 4]
        assert np.allclose(lp, [-np.log(2), -np.log(4)])
    _, _, kept = D.sample(x, np.array([0.5, 0.5]), np.array([INF, INF]), min_p=np.array([1.0, 1.0]))
    assert kept.tolist() == [2, 4]


def test_a_minimal_probability_above_one_keeps_the_first():
    ids, lp, kept = D.sample(np.zeros((1, 5)), np.array([0.9]), min_p=np.array([2.0]))
    assert ids.tolist() == [0] and kept.tolist() == [1] and lp[0] == 0


def test_uniforms_of_one_give_the_last_with_weight():
    x = np.array([[0.0, -3.0, -3.0, -3.0, -1e5], [-3.0, 0.0, -3.0, -3.0, -4.0]])
    ids, _, kept = D.sample(x, np.array([1.0, 7.0]))
    assert ids.tolist() == [3, 4] and kept.tolist() == [5, 5]
    ids, _, kept = D.sample(x, np.array([1.0, 7.0]), top_k=np.array([3, 3]))
    assert ids.tolist() == [2, 2] and kept.tolist() == [3, 3]
    ids, _, kept = D.sample(np.array([[0.0, -36.0, -34.0]]), np.array([1.0]))   # half a unit: 2^-51 = e^-35.35
    assert ids.tolist() == [2] and kept.tolist() == [3]


def test_routing_with_infinite_logits_and_a_bias():
    x = np.array([[0.0, INF, 1.0, 2.0], [INF, 0.0, INF, -INF]])
    bias = np.array([0.1, 0.2, 0.3, -0.1])
    with np.errstate(invalid="ignore"):
        ids = D.route_grouped(x, 4, 1, 1, bias=bias)[0]              # keys .1 1.2 .3 -.1; .6 .2 .8
        assert ids.tolist() == [[1, 2, 0, 3], [2, 0, 1, -1]]
        ids = D.route_grouped(x, 2, 2, 1, bias=bias)[0]
        assert ids.tolist() == [[1, 0], [2, -1]]
        bias[1] = -INF
        assert D.route_grouped(x, 2, 1, 1, bias=bias)[0].tolist() == [[2, 0], [2, 0]]
