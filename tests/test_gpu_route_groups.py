"""GPU parity of expert routing within the best groups against the 64-bit
form: group counts and sizes that divide the lanes and ones that do not, both
ratings, ties, masks, batches on both sides of the group of tokens."""
import numpy as np
import pytest
import torch

from oracle import dense as D
from gpu_util import dev

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _check(F, x, k, groups, top, by="max", score="softmax", bias=None, renorm=True, scale=1.0):
    """Weights within 40 roundings of fp32: exponentials, sums of up to 64
    terms in four steps and a division, of arguments no larger than 30."""
    r = F.fp8w_route_experts(x, k, score, None if bias is None else torch.from_numpy(bias).to(dev()), renorm, scale,
                             groups=groups, top_groups=top, group_score=by)
    torch.cuda.synchronize()
    ids, w, slots, rows, offsets = D.route_grouped(x.double().cpu().numpy(), k, groups, top, by, score, bias, renorm, scale)
    for got, want in ((r.ids, ids), (r.slots, slots), (r.rows, rows), (r.offsets, offsets)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert (np.abs(r.weights.double().cpu().numpy() - w) <= 40 * 2.0 ** -24 * w + 2.0 ** -140).all()
    return r


def _logits(t, e, dtype=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 977 + t * 31 + e)
    return (torch.randn(t, e, generator=g, device=dev()) * 1.5).to(dtype)


SHAPES = [(4, 2, 1), (8, 8, 3), (16, 4, 2), (24, 3, 2), (60, 5, 2), (60, 60, 9), (64, 16, 5), (96, 12, 4), (128, 8, 4), (160, 8, 3),
          (250, 5, 2), (256, 8, 4), (256, 16, 3), (256, 2, 1), (384, 3, 1), (510, 17, 6), (512, 64, 10), (640, 10, 3), (1024, 33 - 1, 7),
          (1020, 34, 9), (1024, 2, 1), (1014, 39, 11)]


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("shape", SHAPES)
def test_groups(F, shape, by):
    e, groups, top = shape
    k = min(6, top * (e // groups))
    rng = np.random.default_rng(e)
    bias = (0.3 * rng.standard_normal(e)).astype(np.float32)
    for t in (1, 5, 40):
        _check(F, _logits(t, e), k, groups, top, by, "softmax")
        _check(F, _logits(t, e, BF16), k, groups, top, by, "sigmoid", bias)
    _check(F, _logits(33, e), k, groups, top, by, "softmax", bias, renorm=False, scale=2.5)
    _check(F, _logits(33, e), k, groups, top, by, "sigmoid", renorm=False)


@pytest.mark.parametrize("by", ["max", "top2"])
def test_many_choices(F, by):
    _check(F, _logits(50, 256), 64, 8, 4, by)
    _check(F, _logits(50, 256), 17, 16, 2, by, "sigmoid")
    _check(F, _logits(9, 1024), 64, 4, 1, by)


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties(F, by, score):
    x = torch.randint(-2, 2, (70, 48), device=dev()).float()
    x[0], x[1, ::2] = 0.0, -0.0
    _check(F, x, 5, 6, 2, by, score)
    _check(F, x, 5, 6, 2, by, score, np.zeros(48, np.float32))


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
def test_masks(F, by, biased):
    x = _logits(40, 32)
    x[0] = -np.inf
    x[1, :24] = -np.inf                                    # one group left, of three that may be open
    x[2, ::8] = -np.inf
    x[3, 1::2], x[3, 4:8] = float("nan"), -np.inf
    x[4], x[4, 9] = -np.inf, -80.0
    x[5] = torch.finfo(F32).min
    bias = None
    if biased:
        bias = np.zeros(32, np.float32)
        bias[3], bias[10], bias[20] = -np.inf, np.nan, 5.0
    for k in (1, 4, 8):
        _check(F, x, k, 8, 3, by, "sigmoid", bias)
        _check(F, x, k, 4, 1, by, "softmax", bias)


def test_best_logit_in_a_shut_group(F):
    """Weights of the chosen alone, far below the row's best."""
    x = torch.full((3, 8), -200.0, device=dev())
    x[:, 0], x[:, 4], x[:, 5] = 10.0, 1.0, 0.5
    bias = np.array([0, -9, -9, -9, 0, 0, 0, 0], np.float32)
    r = _check(F, x, 2, 2, 1, "top2", "sigmoid", bias)
    assert (r.ids.cpu() == torch.tensor([4, 5])).all()
    bias = np.array([-9] * 4 + [0, 0, 0, 0], np.float32)
    x[:, 4], x[:, 5] = -150.0, -151.0
    _check(F, x, 2, 2, 1, "max", "softmax", bias)


def test_all_groups_open_is_the_plain_choice(F):
    x = _logits(45, 96)
    want = F.fp8w_route_experts(x, 7)
    for kw in (dict(groups=8), dict(groups=8, top_groups=8, group_score="top2"), dict(groups=1)):
        assert all(torch.equal(a, b) for a, b in zip(want, F.fp8w_route_experts(x, 7, **kw)))


def test_refusals(F):
    x = _logits(4, 32)
    for bad in (dict(groups=5), dict(groups=8, top_groups=9), dict(groups=8, top_groups=0), dict(groups=16, top_groups=1, top_k=3)):
        with pytest.raises(F.Fp8wError):
            F.fp8w_route_experts(x, **{"top_k": 2, **bad})
    with pytest.raises(ValueError):
        F.fp8w_route_experts(x, 2, groups=4, top_groups=2, group_score="mean")


def test_repeatable_on_another_stream_and_in_a_graph(F):
    for t in (7, 90):
        x = _logits(t, 64)
        kw = dict(groups=8, top_groups=3, group_score="top2")
        want = [v.clone() for v in F.fp8w_route_experts(x, 4, **kw)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = F.fp8w_route_experts(x, 4, **kw, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        buf = [torch.empty_like(v) for v in want]
        ws = torch.empty(max(F.lib().fp8w_route_experts_workspace_bytes(t, 64), 4), dtype=torch.uint8, device=dev())
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            F.fp8w_route_experts(x, 4, "softmax", None, True, 1.0, *buf, workspace=ws, **kw)
        for i in range(3):
            x.copy_(_logits(t, 64, seed=i + 1))
            for b in buf:
                b.fill_(-1)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(buf, F.fp8w_route_experts(x, 4, **kw))), i


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [3, 40])
def test_an_infinite_logit_opens_its_group(F, by, score, t):
    """The choice is defined, the weights are not."""
    x = _logits(t, 64)
    x[0, 41], x[1, 3] = np.inf, np.inf
    x[1, 60:62] = np.inf
    r = F.fp8w_route_experts(x, 4, score, groups=8, top_groups=2, group_score=by)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ids = D.route_grouped(x.double().cpu().numpy(), 4, 8, 2, by, score)[0]
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert 41 in ids[0]
