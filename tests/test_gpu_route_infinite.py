"""Routing with logits of +inf under a selection bias, with groups and without:
an infinite logit's softmax score is one (shared among the infinite ones), the
others' zero, and the choice is by score and bias as ever.  The weights of
such a token are unspecified."""
import numpy as np
import pytest
import torch

from oracle import dense as D
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [4, 40])
@pytest.mark.parametrize("e,groups,top,by", [(64, 1, 1, "max"), (64, 8, 2, "max"), (64, 8, 2, "top2"), (128, 1, 1, "max"),
                                             (256, 1, 1, "max"), (256, 8, 4, "top2"), (640, 1, 1, "max"), (640, 10, 3, "top2")])
def test_infinite_logits_under_a_bias(F, e, groups, top, by, t, score):
    g = torch.Generator(device="cuda").manual_seed(e + t)
    x = torch.randn(t, e, generator=g, device=dev()) * 1.5
    x[0, 41] = np.inf
    x[1, 3] = x[1, 20] = x[1, 60] = np.inf
    x[2, 7] = np.inf                                       # one that the bias bars
    x[3], x[3, 50] = -np.inf, np.inf
    bias = (0.1 * np.random.default_rng(e).standard_normal(e)).astype(np.float32)
    bias[7] = -np.inf
    r = F.fp8w_route_experts(x, 4, score, torch.from_numpy(bias).to(dev()), groups=groups, top_groups=top, group_score=by)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ids, _, slots, rows, offsets = D.route_grouped(x.double().cpu().numpy(), 4, groups, top, by, score, bias)
    assert (score == "sigmoid" or (ids[0] == 41).any()) and ids[3].tolist() == [50, -1, -1, -1] and not (ids == 7).any()
    for got, want in ((r.ids, ids), (r.slots, slots), (r.rows, rows), (r.offsets, offsets)):
        assert np.array_equal(got.cpu().numpy(), want)
