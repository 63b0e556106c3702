"""GPU log probabilities and entropies within the bounds that their roundings
leave, wherever the logits lie: shifted far from zero, spread wide and
narrow, one row or a chip full, with and without alternatives."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from gpu_util import dev
from test_gpu_logprobs import F, _logits  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,v", [(3, 700), (4, 20000), (2, 151936), (600, 9000)])
@pytest.mark.parametrize("shift", [0.0, -1000.0, 500.0, 30000.0, 1e6, -1e6])
@pytest.mark.parametrize("sigma", [1e-3, 3.0, 100.0])
@pytest.mark.parametrize("top", [0, 5])
def test_bounds(F, t, v, shift, sigma, top):  # noqa: F811
    x = _logits(t, v, torch.float32, scale=sigma) + shift
    targets = torch.arange(t, device=dev(), dtype=torch.int32) * 37 % v
    r = F.fp8w_logprobs(x, targets, top)
    torch.cuda.synchronize()
    keep = slice(0, 24)                                      # of many rows some, for the 64-bit form's sake
    xs = x[keep].cpu().numpy()
    lp, ent, ids, best = S.logprobs(xs, targets[keep].cpu().numpy(), top)
    err, err_h = S.logprobs_errors(xs)
    assert np.array_equal(r.top_ids[keep].cpu().numpy(), ids)
    for got, want in ((r.logprob[keep], lp), (r.top_logprobs[keep], best)):
        e = err if want.ndim == 1 else err[:, None]
        assert (np.abs(got.cpu().numpy() - want) <= e + S.EPS32 * np.abs(want)).all()
    assert (np.abs(r.entropy[keep].cpu().numpy() - ent) <= err_h).all()
