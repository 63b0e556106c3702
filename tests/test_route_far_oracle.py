"""The 64-bit routing weights where the chosen lie far below the best logit
or below fp32's smallest score."""
import numpy as np

from oracle import serving as S


def test_softmax_of_the_chosen_however_far_below():
    for gap in (1.0, 100.0, 700.0, 800.0, 1e30):
        x = np.array([[0.0, -gap, -gap, -2 * gap]])
        ids, w, *_ = S.route(x, 2, bias=np.array([-9.0, 0.0, 0.0, 0.0]))
        assert ids.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]]
    _, w, *_ = S.route(np.array([[300.0, -600.0, -601.0]]), 2, bias=np.array([-9.0, 0.0, -1e-9]))
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]], rtol=1e-15)


def test_sigmoid_scores_that_are_zero_in_fp32():
    x = np.array([[-103.0, -104.5], [-104.5, -105.0], [-np.inf, -200.0], [-60.0, -61.0]])
    ids, w, *_ = S.route(x, 2, "sigmoid")
    assert np.allclose(w[[0, 3]], [[1 / (1 + np.exp(-d)), 1 / (1 + np.exp(d))] for d in (1.5, 1.0)])
    assert (w[1:3] == 0).all() and ids.tolist() == [[0, 1], [0, 1], [1, -1], [0, 1]]
    assert (S.route(x, 2, "sigmoid", renorm=False)[1][:2] > 0).all()
