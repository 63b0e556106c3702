"""Drawn tokens at the ends of what may be drawn: random numbers of 1 and more,
crowds of tokens whose bins are divided, vocabularies whose sums are rounded by
more than a random number's last place, minimal probabilities of 1 and more,
and an infinite temperature."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_sample import BF16, F32, F, _check  # noqa: F401

pytestmark = pytest.mark.gpu


def _crowds(v):
    """More tokens in a bin than a list holds, which is not the first bin: of
    different values and of one, with a token far below and without, and two
    crowds."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = -3 + 1e-3 * torch.randn(5, v, generator=g, device=dev())
    x[2] = -3.0
    x[3, ::2] -= 2.0
    x[4, ::2] = -3.0
    x[4, 1::2] = -4.0
    x[:, v // 3] = 0.0
    x[0, 5] = x[2, v - 1] = x[3, 0] = -200.0
    return x


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [7000, 60000])
@pytest.mark.parametrize("u", [1 - 2.0 ** -24, 1.0, 1.5, float("inf")])
def test_the_end_of_a_crowd(F, u, v, dtype):
    x = _crowds(v).to(dtype)
    for k in (dict(), dict(top_k=v - 1), dict(top_k=v - 2), dict(top_k=v // 2 + 1), dict(top_k=v // 2), dict(top_p=0.999),
              dict(min_p=0.04), dict(min_p=1e-3), dict(temperature=2.0), dict(temperature=0.5, top_k=v - 1, top_p=0.9999),
              dict(top_k=v - 1, min_p=1e-3), dict(top_k=100), dict(temperature=0.0)):
        _check(F, x, u=u, **k)


@pytest.mark.parametrize("v", [1 << 20, 1 << 22, 1 << 24])
@pytest.mark.parametrize("u", [1 - 2.0 ** -24, 1.0])
def test_never_past_what_is_kept(F, u, v):
    """Sums of so many are known to 2^-27 ... 2^-19, so the last but a few may
    be drawn in the last one's place; never one that was not kept."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = -3 + 1e-3 * torch.randn(3, v, generator=g, device=dev())
    x[1] = -3.0
    x[:, 9], x[2, 11] = 0.0, -200.0
    token = torch.arange(v, device=dev())
    for top_k in (None, v - 1, v - 2, v // 2):
        k = None if top_k is None else torch.full((3,), top_k, dtype=torch.int32, device=dev())
        r = F.fp8w_sample(x, torch.full((3,), u, device=dev()), top_k=k)
        assert (r.kept == (v if top_k is None else top_k)).all()
        for i in range(3):
            t = int(r.tokens[i])
            assert 0 <= t < v
            rank = int((x[i] > x[i, t]).sum()) + int(((x[i] == x[i, t]) & (token < t)).sum())
            room = 2.0 ** -19 * v + 1                                # what the sums leave open, in tokens of one weight
            end = int(r.kept[i]) - (1 if i == 2 and top_k is None else 0)   # the token far below has no weight
            assert rank < end and (rank == end - 1 if u == 1 else rank >= end - 1 - room), (i, rank, end)


@pytest.mark.parametrize("v", [40, 7000, 60000])
def test_a_minimal_probability_of_one_and_above(F, v):
    """Of one the first and its equals, above the first alone."""
    x = torch.zeros(3, v, device=dev())
    x[1] = -torch.arange(v, device=dev()).remainder(3).float()
    x[2, :5] = -np.inf
    for low in (1.0, 1.0 + 2.0 ** -23, 2.0, float("inf")):
        for k in (dict(), dict(top_k=7), dict(top_p=0.5), dict(temperature=3.0), dict(temperature=float("inf"))):
            _check(F, x, u=0.7 if "top_p" not in k else 0.3, min_p=low, **k)
    x[2, v - 2:] = np.inf
    _check(F, x, u=0.75, min_p=2.0)


@pytest.mark.parametrize("v", [40, 7000, 60000])
def test_an_infinite_temperature(F, v):
    """All tokens weigh the same, but beside a logit of +inf no finite one has weight."""
    x = torch.randn(4, v, generator=torch.Generator(device="cuda").manual_seed(v), device=dev())
    x[1, 5:9] = -np.inf
    x[2, 7], x[2, v - 3] = np.inf, np.inf
    x[3] = torch.finfo(F32).max
    x[3, 3] = np.inf
    for k in (dict(), dict(min_p=1.0), dict(min_p=0.5), dict(top_p=0.5), dict(top_k=6), dict(top_k=6, top_p=0.9, min_p=1e-3)):
        for u in (0.0, 0.3, 0.99, 1.0):
            _check(F, x, u=u, temperature=float("inf"), **k)
            _check(F, x, u=u, temperature=3e38, **k)


@pytest.mark.parametrize("v", [1, 900, 5000, 9000, 20000, 40000, 70000, 151936, 300000, 600000, 1 << 20, 1 << 21, 1 << 22])
def test_the_only_token_left_has_log_probability_zero(F, v):
    """Whatever the fixed point of its weight."""
    x = torch.randn(3, v, generator=torch.Generator(device="cuda").manual_seed(v), device=dev())
    x[:, v // 2] = 9.0
    u = torch.tensor([0.0, 0.4, 0.9], device=dev())
    full = lambda value, dtype=F32: torch.full((3,), value, dtype=dtype, device=dev())   # noqa: E731
    for k in (dict(temperature=full(0.0)), dict(top_k=full(1, torch.int32)), dict(top_p=full(1e-9)), dict(min_p=full(0.9)),
              dict(min_p=full(2.0)), dict(temperature=full(0.01), top_k=full(1, torch.int32))):
        r = F.fp8w_sample(x, u, **k)
        assert (r.tokens == v // 2).all() and (r.kept == 1).all() and (r.logprob == 0).all(), (k, r)


@pytest.mark.parametrize("v", [50, 4096, 4097, 9000, 70000])
def test_the_last_token_with_weight(F, v):
    """Weights below half a unit are zero: such tokens are kept, and never drawn."""
    x = -torch.arange(v, device=dev()).remainder(997).float() / 4 - 1
    x = torch.stack([x, x / 2, x * 8])
    x[:, 0] = 0.0
    for u in (1.0, 3.0):
        for k in (dict(), dict(top_k=v - 3), dict(top_k=40), dict(temperature=0.3), dict(temperature=5.0), dict(min_p=1e-18), dict(min_p=1e-9)):
            _check(F, x, u=u, **k)
