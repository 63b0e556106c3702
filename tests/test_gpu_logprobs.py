"""GPU parity of token log probabilities, entropy and top alternatives
against the 64-bit form: segment and vector edges, unaligned rows, ties,
masks down to nothing, values out of range, NaN and infinities."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _check(F, x, top, targets="random", seed=0, **kw):
    t, v = x.shape
    rng = np.random.default_rng([seed, t, v])
    tg = rng.integers(0, v, t).astype(np.int32) if isinstance(targets, str) else targets
    r = F.fp8w_logprobs(x, None if tg is None else torch.from_numpy(tg).to(dev()), top, **kw)
    torch.cuda.synchronize()
    xs = x.float().cpu().numpy()
    lp, ent, ids, best = S.logprobs(xs, tg, top)
    tol = S.logprobs_tolerance(xs, ent)
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)

    def near(got, want, tol):
        got = got.cpu().numpy().astype(np.float64)
        same = (got == want) | (np.isnan(got) & np.isnan(want))      # infinities and NaN exactly
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(got - want) <= tol * (1 + np.abs(want)))
        assert ok.all(), (got[~ok][:4], want[~ok][:4], np.argwhere(~ok)[:4])
    near(r.entropy, ent, tol)
    near(r.top_logprobs, best, tol[:, None])
    if tg is not None:
        near(r.logprob, lp, tol)
    return r


def _logits(t, v, dtype=torch.bfloat16, scale=3.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + t * 31 + v)
    return (torch.randn(t, v, generator=g, device=dev()) * scale).to(dtype)


@pytest.mark.parametrize("v", [1, 2, 7, 8, 9, 63, 64, 65, 1000, 1023, 1024, 1025, 8191, 8192, 8193, 16384, 32001, 50257])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_vocabulary_edges(F, v, dtype):
    _check(F, _logits(3, v, dtype), min(v, 5))


@pytest.mark.parametrize("top", [0, 1, 2, 20, 63, 64])
@pytest.mark.parametrize("t", [1, 5, 600])
def test_alternatives(F, top, t):
    _check(F, _logits(t, 3001), top)
    _check(F, _logits(min(t, 3), 40000, torch.float32), top)


@pytest.mark.parametrize("pad", [1, 3, 8, 61])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_rows(F, pad, dtype):
    wide = _logits(6, 9000 + pad, dtype)
    _check(F, wide[:, pad:], 4)
    _check(F, wide[:, :9000], 4)
    _check(F, wide[2:3, pad:], 4)


@pytest.mark.parametrize("v", [100, 9000, 70000])
def test_ties_go_to_the_lower_token(F, v):
    x = torch.zeros(5, v, device=dev())
    x[1] = torch.randint(-1, 2, (v,), device=dev()).float()
    x[2, ::2] = -0.0                                        # equal to +0
    x[3] = -torch.arange(v, device=dev()).remainder(7).float()
    x[4] = torch.finfo(torch.float32).min
    _check(F, x, 64)
    _check(F, x[:4].to(torch.bfloat16), 64)


@pytest.mark.parametrize("rising", [True, False])
def test_sorted_rows(F, rising):
    """Every step of a rising row beats all before it."""
    x = torch.linspace(-20, 20, 60000, device=dev())
    x = x if rising else x.flip(0)
    _check(F, x[None].contiguous(), 50)
    _check(F, x[None].expand(520, -1).contiguous()[:, :20000].contiguous(), 50)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [50, 9000, 40000])
def test_masks(F, v, dtype):
    x = _logits(7, v, dtype)
    x[0] = -np.inf                                          # nothing left
    x[1], x[1, v - 1] = -np.inf, 2.5                        # one token
    x[2, v // 3:] = -np.inf                                 # the end
    x[3, :v - 3] = -np.inf                                  # all but three: fewer than the alternatives
    x[4, torch.rand(v, device=dev()) < 0.9] = -np.inf
    x[5] = torch.finfo(dtype).min                           # the lowest value everywhere is no mask
    x[6], x[6, 4] = torch.finfo(dtype).min, 0.0
    _check(F, x, 8)
    _check(F, x, 8, targets=np.full(7, v - 1, np.int32))


@pytest.mark.parametrize("t", [6, 700])
def test_nan_and_infinity_spoil_their_row_only(F, t):
    x = _logits(t, 9000)
    x[1, 8999], x[2, 0], x[3, 4000] = float("nan"), float("inf"), float("-nan")
    x[4, :] = float("nan")
    r = _check(F, x, 6)
    assert torch.isnan(r.entropy[1:5]).all() and torch.isfinite(r.entropy[[0, 5]]).all()


def test_targets_outside_are_not_followed(F):
    tg = np.array([-1, 500, 2**31 - 1, -2**31, 0, 499], np.int32)
    r = _check(F, _logits(6, 500), 3, targets=tg)
    assert torch.isnan(r.logprob[:4]).all() and torch.isfinite(r.logprob[4:]).all()
    r = _check(F, _logits(6, 500), 3, targets=None)
    assert r.logprob is None


@pytest.mark.parametrize("shift", [-1000.0, 500.0, 30000.0])
def test_logits_far_from_zero(F, shift):
    _check(F, _logits(4, 20000, torch.float32) + shift, 5)


def test_wide_spread(F):
    _check(F, _logits(4, 20000, torch.float32, scale=1e4), 5)
    _check(F, _logits(4, 20000, torch.bfloat16, scale=1e-3), 5)
    _check(F, _logits(4, 3000, torch.float32, scale=1e37), 5)


def test_no_rows(F):
    r = F.fp8w_logprobs(torch.empty(0, 50, device=dev()), torch.empty(0, dtype=torch.int32, device=dev()), 3)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 3)


def test_lm_head_rows(F):
    _check(F, _logits(4, 151936), 20)


def test_repeatable_on_another_stream_and_in_a_graph(F):
    x = _logits(4, 40000)
    tg = torch.arange(4, dtype=torch.int32, device=dev())
    want = [v.clone() for v in F.fp8w_logprobs(x, tg, 10)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.fp8w_logprobs(x, tg, 10, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = [torch.empty_like(v) for v in want]
    ws = torch.empty(F.lib().fp8w_logprobs_workspace_bytes(4, 40000, 10), dtype=torch.uint8, device=dev())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp8w_logprobs(x, tg, 10, *buf, workspace=ws)
    for i in range(3):
        x.copy_(_logits(4, 40000, seed=i + 1))
        for b in buf:
            b.fill_(-1)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(buf, F.fp8w_logprobs(x, tg, 10))), i
