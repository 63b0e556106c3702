"""GPU parity of the products grouped by more than 256 experts, whose offsets
take several passes: every kernel, runs that end at a pass's edge, and all
slots with one expert of any pass."""
import numpy as np
import pytest

from test_gpu_experts import F, _check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e", [257, 512, 700])
@pytest.mark.parametrize("avg", [1, 6, 12])
@pytest.mark.parametrize("fmt,act", [("block", "swiglu"), ("mx", "none"), ("row", "swiglu")])
def test_uneven_groups(F, e, avg, fmt, act):  # noqa: F811
    rng = np.random.default_rng(e + avg)
    _check(F, list(rng.multinomial(avg * e, rng.dirichlet(np.ones(e)))), 64, 128, fmt, act, slots=avg * e + 3)


def test_dense_groups(F):  # noqa: F811
    rng = np.random.default_rng(5)
    sizes = rng.multinomial(120 * 260, np.full(260, 1 / 260))
    _check(F, list(sizes), 64, 128, "block", "swiglu")
    _check(F, list(sizes), 40, 80, "row")


@pytest.mark.parametrize("at", [0, 255, 256, 511, 512, 599])
@pytest.mark.parametrize("count", [1, 40, 700])
def test_one_expert_takes_all(F, at, count):  # noqa: F811
    _check(F, [count if i == at else 0 for i in range(600)], 64, 128, "block", "swiglu", x_rows=count)


@pytest.mark.parametrize("edge", [256, 512])
def test_short_mx_rows_and_odd_halves(F, edge):  # noqa: F811
    """The simple kernel, with slots on both sides of a pass's edge."""
    sizes = [0] * 600
    for i, c in ((edge - 2, 3), (edge - 1, 17), (edge, 16), (edge + 1, 1), (599, 20)):
        sizes[i] += c
    _check(F, sizes, 32, 64, "mx")
    _check(F, sizes, 10, 144, "block", "swiglu")
