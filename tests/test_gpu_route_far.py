"""GPU routing weights where the chosen experts lie far below the row's best
(a selection bias chooses) or far below zero (sigmoid scores near and below
fp32's smallest number): the weights are ratios of the chosen scores, however
small those are."""
import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu

# An exponential's argument is one fp32 difference d (rounded by 2^-24 |d|),
# the exponential and the divisions are good to 2 units of 2^-23 each, the sum
# of up to 16 terms adds a rounding for each.
EPS32 = 2.0 ** -23


def tolerance(x, k):
    return (np.ptp(x) + k + 8) * EPS32


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _route(F, x, bias, k, **kw):
    r = F.fp8w_route_experts(x, k, bias=bias, **kw)
    torch.cuda.synchronize()
    return r.ids.cpu().numpy(), r.weights.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("gap", [5, 60, 88, 90, 96, 103, 104, 120, 200, 1000, 3e38])
@pytest.mark.parametrize("e,k", [(3, 2), (60, 6), (128, 16), (200, 17), (256, 8), (300, 8), (1024, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t", [3, 40])
def test_softmax_of_the_chosen_below_the_best(F, gap, e, k, dtype, t):
    """The best logit is barred by its bias, and the others lie `gap` below."""
    g = torch.Generator(device="cuda").manual_seed(e + k)
    x = (torch.randn(t, e, generator=g, device=dev()) - gap).to(dtype)
    x[:, e // 2] = 0.5
    bias = torch.zeros(e, device=dev())
    bias[e // 2] = -5.0
    bias[torch.randperm(e, generator=g, device=dev())[:k]] += torch.arange(1, k + 1, device=dev()).float()
    bias[e // 2] = -5.0
    ids, w = _route(F, x, bias, k)
    named = np.flatnonzero(bias.cpu().numpy() > 0)             # their biases decide: a score is at most 1
    xs = x.float().cpu().numpy().astype(np.float64)
    for r in range(t):
        assert (ids[r] >= 0).all()
        if gap >= 60:                                         # and nothing, beside the barred one's
            assert np.isin(named, ids[r]).all()
        c = xs[r, ids[r]]
        p = np.exp(c - c.max())
        p /= p.sum()
        assert (np.abs(w[r] - p) <= tolerance(c, k) * p + 1e-37).all(), (r, w[r], p)


def test_softmax_with_a_bias_as_in_the_definition(F):
    x = torch.tensor([[200.0, 0.0, -1.0, -2.0], [0.0, -120.0, -119.0, -400.0]], device=dev())
    ids, w = _route(F, x, torch.tensor([-5.0, 0.0, 0.0, 0.0], device=dev()), 2)
    assert ids.tolist() == [[1, 2], [2, 1]]
    assert np.abs(w - [[0.7310585786, 0.2689414214]] * 2).max() < 1e-6
    # without renorm they are parts of the whole row's sum: nothing, in fp32
    _, w = _route(F, x, torch.tensor([-5.0, 0.0, 0.0, 0.0], device=dev()), 2, renorm=False)
    assert (w == 0).all()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("e,k", [(4, 2), (40, 16), (200, 20), (300, 4)])
def test_sigmoid_scores_next_to_the_smallest_number(F, e, k, bias):
    """Ratios of scores from e^-80 down to where fp32 has none left."""
    g = torch.Generator(device="cuda").manual_seed(e)
    far = torch.tensor([0.0, -30.0, -80.0, -86.0, -88.0, -89.0, -91.0, -95.0, -98.0, -101.0], device=dev())
    x = far[:, None] - torch.rand(10, e, generator=g, device=dev()) * 2
    x[0, 0] = x[5, 1] = 3.0                                  # one score of ordinary size among small ones
    b = torch.rand(e, generator=g, device=dev()) if bias else None
    ids, w = _route(F, x, b, k, score="sigmoid")
    xs = x.cpu().numpy().astype(np.float64)
    for r in range(len(xs)):
        c = xs[r, ids[r]]
        p = 1 / (1 + np.exp(-c))
        p /= p.sum()
        assert (np.abs(w[r] - p) <= tolerance(c, k) * p + 1e-37).all(), (r, w[r], p)


def test_sigmoid_scores_below_the_smallest_number(F):
    """A score below fp32's smallest number is zero, and zeros have no ratio;
    beside a larger one it counts by its definition."""
    x = torch.tensor([[-104.5, -105.0, -300.0], [-103.0, -104.5, -300.0], [-np.inf, -200.0, -201.0]], device=dev())
    _, w = _route(F, x, None, 2, score="sigmoid")
    assert (w[[0, 2]] == 0).all()
    assert np.abs(w[1] - [0.8175744762, 0.1824255238]).max() < 1e-6
    _, w = _route(F, x, None, 2, score="sigmoid", renorm=False)
    assert (w <= 1e-44).all() and (w >= 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k", [(9, 6), (70, 20), (300, 5)])
def test_barred_experts(F, score, e, k):
    """A bias of -inf or NaN bars an expert; its score stays in softmax's sum."""
    from oracle import serving as S
    g = torch.Generator(device="cuda").manual_seed(e)
    x = torch.randn(35, e, generator=g, device=dev())
    bias = torch.randn(e, generator=g, device=dev())
    bias[torch.randperm(e, generator=g, device=dev())[:e // 2]] = -np.inf
    bias[e - 1], bias[3] = float("nan"), float("inf")
    for renorm in (True, False):
        r = F.fp8w_route_experts(x, k, score=score, bias=bias, renorm=renorm)
        torch.cuda.synchronize()
        want = S.route(x.cpu().numpy(), k, score, bias.cpu().numpy(), renorm)
        for got, w in zip((r.ids, r.slots, r.rows, r.offsets), (want[0], *want[2:])):
            assert np.array_equal(got.cpu().numpy(), w)
        assert (np.abs(r.weights.cpu().numpy() - want[1]) <= (8 + e + k + 8) * EPS32 * want[1] + 1e-37).all()
    left = int((bias > -np.inf).sum())
    assert (r.ids[:, :left] >= 0).all() and (r.ids[:, left:] == -1).all()
