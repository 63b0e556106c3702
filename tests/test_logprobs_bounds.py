"""The error bounds that log probabilities are held to, on the CPU: fp32 forms
that take the difference from the maximum first stay inside, forms that round
at the size of the logits or of the wrong base do not."""
import numpy as np
import pytest

from oracle import serving as S

F32 = np.float32
LOG2E, LN2 = F32(1.44269504088896340736), F32(0.69314718055994530942)


def _rows(shift, sigma=3.0, t=4, v=20000, seed=0):
    rng = np.random.default_rng([seed, v])
    return (rng.standard_normal((t, v)) * sigma + shift).astype(F32)


def difference_first(x):
    """(log probabilities, entropy) in fp32, the exponents relative to the maximum."""
    m = x.max(axis=1, keepdims=True)
    e = np.maximum((x - m) * LOG2E, F32(-300))
    p = np.exp2(e)
    z, u = p.sum(axis=1, dtype=F32), (e * p).sum(axis=1, dtype=F32)
    ln_z = np.log2(z) * LN2
    return (x - m) - ln_z[:, None], ln_z - LN2 * (u / z)


def product_first(x):
    """The same with x log2 e rounded at the size of the logits."""
    m = x.max(axis=1, keepdims=True)
    e = x * LOG2E - m * LOG2E
    p = np.exp2(e)
    z, u = p.sum(axis=1, dtype=F32), (e * p).sum(axis=1, dtype=F32)
    lse = np.log2(z)[:, None] * LN2 + m
    return x - lse, (np.log2(z) - u / z) * LN2


def terms_of_the_wrong_base(x):
    lp, h = difference_first(x)
    m = x.max(axis=1, keepdims=True)
    e = (x - m).astype(np.float64)
    p = np.exp(e)
    return lp, (np.log(p.sum(1)) - 0.6932 * (e * p).sum(1) / p.sum(1)).astype(F32)   # ln 2 once too often


def eight_bits(x):
    """Exponents rounded to bf16."""
    m = x.max(axis=1, keepdims=True)
    e = (x - m) * LOG2E
    e = ((e.view(np.uint32) + 0x8000) & 0xFFFF0000).view(F32)
    z = np.exp2(e).sum(axis=1, dtype=F32)
    return (x - m) - (np.log2(z) * LN2)[:, None], difference_first(x)[1]


def _outside(form, x):
    """Whether the form leaves the bounds: (log probabilities, entropy); the
    bounds of the parity tests, relative to 1 + the value, and the plain ones."""
    lp, h = form(x)
    exact = x.astype(np.float64)
    top = exact.max(axis=1, keepdims=True)
    want = (exact - top) - np.log(np.exp(exact - top).sum(axis=1, keepdims=True))
    want_h = -(np.exp(want) * want).sum(axis=1)
    tol, (err, err_h) = S.logprobs_tolerance(x, want_h), S.logprobs_errors(x)
    off, off_h = np.abs(lp - want), np.abs(h - want_h)
    return ((off > tol[:, None] * (1 + np.abs(want))).any() or (off_h > tol * (1 + want_h)).any(),
            (off > err[:, None] + S.EPS32 * np.abs(want)).any() or (off_h > err_h).any())


@pytest.mark.parametrize("shift", [0.0, -1000.0, 500.0, 30000.0, 1e6, -1e6])
@pytest.mark.parametrize("sigma", [1e-3, 1.0, 3.0, 100.0, 1e4])
def test_differences_first_stay_inside(shift, sigma):
    assert _outside(difference_first, _rows(shift, sigma)) == (False, False)


@pytest.mark.parametrize("shift", [30000.0, -30000.0, 1e6])
def test_products_first_do_not(shift):
    assert _outside(product_first, _rows(shift)) == (True, True)


def test_products_first_next_to_zero():
    assert _outside(product_first, _rows(-1000.0))[1] and not _outside(product_first, _rows(0.0))[1]


@pytest.mark.parametrize("form", [terms_of_the_wrong_base, eight_bits])
@pytest.mark.parametrize("shift", [0.0, 30000.0])
def test_other_mistakes_do_not(form, shift):
    assert _outside(form, _rows(shift)) == (True, True)


def test_rows_without_a_distribution():
    x = np.zeros((4, 300), F32)
    x[0], x[1, 3], x[2, 5] = -np.inf, np.nan, np.inf
    err, err_h = S.logprobs_errors(x)
    assert np.isfinite(err).all() and np.isfinite(err_h).all()
    assert np.isfinite(S.logprobs_tolerance(x, np.array([0.0, np.nan, np.nan, 1.0]))).all()
