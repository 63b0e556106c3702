"""GPU parity of drawn tokens against the extended-precision form: every filter
alone and together, vocabulary edges, ties beyond a list's room, masks down to
nothing, values and settings out of range, streams and graphs.  Tokens and
counts have to be equal."""
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


def _check(F, x, u=None, seed=0, **settings):
    """Settings: numpy arrays, or single values for every row."""
    t, v = x.shape
    rng = np.random.default_rng([seed, t, v])
    u = rng.random(t, np.float32) if u is None else np.broadcast_to(np.asarray(u, np.float32), t)
    k = {n: None if s is None else np.ascontiguousarray(np.broadcast_to(np.asarray(s, np.int32 if n == "top_k" else np.float32), t))
         for n, s in settings.items()}
    r = F.fp8w_sample(x, torch.tensor(u).to(dev()), **{n: None if s is None else torch.from_numpy(s).to(dev()) for n, s in k.items()})
    torch.cuda.synchronize()
    ids, lp, kept = D.sample(x.double().cpu().numpy(), u, **k)
    got = r.tokens.cpu().numpy(), r.logprob.double().cpu().numpy(), r.kept.cpu().numpy()
    bad = np.flatnonzero((got[0] != ids) | (got[2] != kept))
    assert not len(bad), (len(bad), [(int(b), got[0][b], ids[b], got[2][b], kept[b], {n: s[b] for n, s in k.items() if s is not None}, u[b]) for b in bad[:3]])
    same = got[1] == lp
    with np.errstate(invalid="ignore"):
        assert (same | (np.abs(got[1] - lp) <= D.sample_tolerance(lp, v))).all(), (got[1], lp)
    return r


def _logits(t, v, dtype=BF16, scale=2.5, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + t * 31 + v)
    return (torch.randn(t, v, generator=g, device=dev()) * scale).to(dtype)


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=5), dict(top_k=900), dict(top_k=3000), dict(top_p=0.9), dict(top_p=0.999),
           dict(min_p=0.05), dict(min_p=1e-6), dict(temperature=1.3, top_k=40, top_p=0.95), dict(temperature=2.0, top_p=0.8, min_p=0.01),
           dict(top_k=2500, top_p=0.99, min_p=1e-4), dict(temperature=0.0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("i", range(len(FILTERS)))
def test_filters(F, i, dtype):
    _check(F, _logits(9, 5000, dtype), **FILTERS[i])
    _check(F, _logits(3, 40001, dtype), **FILTERS[i])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [1, 2, 3, 7, 8, 9, 63, 64, 65, 1000, 1023, 1024, 1025, 2047, 2049, 8191, 8193, 16385, 33000])
def test_vocabulary_edges(F, v, dtype):
    x = _logits(6, v, dtype)
    _check(F, x)
    _check(F, x, top_p=0.7, min_p=0.001)
    _check(F, x, top_k=3)


@pytest.mark.parametrize("t", [1, 2, 63, 64, 65, 300, 700])
def test_rows_with_settings_of_their_own(F, t):
    rng = np.random.default_rng(t)

    def among(*v):
        return np.array(v)[rng.integers(0, len(v), t)]
    for dtype, v in ((BF16, 9000), (F32, 3001)):
        _check(F, _logits(t, v, dtype), temperature=among(0.0, 0.3, 1.0, 1.7), top_k=among(0, 1, 30, 700, 1500, 10**6),
               top_p=among(1.0, 0.95, 0.5, 0.01), min_p=among(0.0, 0.0, 0.02, 0.3))


@pytest.mark.parametrize("pad", [1, 3, 8, 61])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unaligned_rows(F, pad, dtype):
    wide = _logits(6, 9000 + pad, dtype)
    wide[:, 4000] = 30.0
    _check(F, wide[:, pad:], top_p=0.9)
    _check(F, wide[:, :9000], temperature=3.0)
    _check(F, wide[2:3, pad:], top_k=50)


@pytest.mark.parametrize("v", [8, 1024, 1500, 5000, 40000])
def test_ties(F, v):
    """All equal, few values, and equal up to zero's sign: lower tokens first,
    and borders that are met exactly take no more."""
    x = torch.zeros(6, v, device=dev())
    x[1] = torch.randint(0, 3, (v,), device=dev()).float() * np.log(2.0)
    x[2, ::2] = -0.0
    x[3] = 5.0
    x[4] = -torch.arange(v, device=dev()).remainder(7).float()
    x[5] = torch.finfo(F32).min
    u = np.array([0.0, 0.5, 0.25, 0.999999, 0.7, 0.125], np.float32)
    for k in (dict(), dict(top_k=max(v // 2, 1)), dict(top_p=0.25), dict(top_p=0.5, top_k=max(v // 4, 1)), dict(min_p=1.0),
              dict(min_p=0.25, top_p=0.75), dict(temperature=1e-3), dict(temperature=1e6, top_p=0.5)):
        _check(F, x[[0, 2, 3, 5]], u=u[[0, 2, 3, 5]], **k)
        _check(F, x, u=u + np.float32(0.0001), **k) if "top_p" not in k else None
    _check(F, x[:5].to(BF16), top_p=0.3)


@pytest.mark.parametrize("v", [3000, 50000])
def test_tight_bunches(F, v):
    """More tokens in a bin than a list holds, of different values."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn(4, v, generator=g, device=dev()) * 1e-4
    x[1] += 100.0
    x[1, 7], x[2, 9] = -1e30, 50.0
    x[3] *= 1e-30
    for k in (dict(), dict(top_k=v // 2), dict(top_p=0.6), dict(min_p=0.9999), dict(min_p=1.0), dict(top_k=v - 10, top_p=0.9, min_p=0.5),
              dict(temperature=1e4), dict(temperature=1e-5), dict(top_k=20)):
        _check(F, x, **k)
        _check(F, x.to(BF16), **k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [50, 9000, 40000])
def test_masks(F, v, dtype):
    x = _logits(8, v, dtype)
    x[0] = -np.inf                                          # nothing left
    x[1], x[1, v - 1] = -np.inf, 2.5                        # one token
    x[2, v // 3:] = -np.inf                                 # the end
    x[3, :v - 3] = -np.inf                                  # all but three
    x[4, torch.rand(v, device=dev()) < 0.9] = -np.inf
    x[5] = torch.finfo(dtype).min                           # the lowest value everywhere is no mask
    x[6], x[6, 4] = torch.finfo(dtype).min, 0.0
    x[7, ::3] = float("nan")                                # NaN is one
    for k in FILTERS:
        _check(F, x, **k)
    r = _check(F, x, temperature=0.0)
    assert r.tokens[0] == -1 and r.kept[0] == 0 and r.logprob[0] == -np.inf


def test_infinite_logits(F):
    x = _logits(4, 3000, F32)
    x[0, 77] = np.inf
    x[1, 5:2000:5] = np.inf
    x[2] = np.inf
    x[3, 0], x[3, 9] = np.inf, -np.inf
    for k in (dict(), dict(top_p=0.5), dict(top_k=10), dict(min_p=0.5), dict(temperature=0.0), dict(temperature=0.1, top_p=0.999)):
        _check(F, x, **k)


@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1.0, 1.5, -1.0, float("nan"), float("inf"), -float("inf")])
def test_uniforms_at_and_past_their_ends(F, u):
    x = _logits(5, 4000)
    for k in (dict(), dict(top_k=7), dict(top_p=0.5)):
        _check(F, x, u=u, **k)


def test_settings_out_of_range(F):
    x, nan, inf = _logits(7, 6000), np.nan, np.inf
    _check(F, x, temperature=[nan, -1.0, inf, 1e-38, 1e38, 1e-45, -0.0])
    _check(F, x, top_k=[-1, 0, 6000, 6001, 2**31 - 1, -2**31, 1])
    _check(F, x, top_p=[nan, -1.0, 0.0, 1.0, 2.0, inf, 1e-30])
    _check(F, x, min_p=[nan, -1.0, 0.0, 1.0, 2.0, inf, 1e-45])
    _check(F, x, temperature=[inf, inf, 1e-3, 1e3, 5, 5, 5], top_p=[0.5, 1.0, 0.5, 0.5, 0.99999, 1e-9, 0.3],
           min_p=[0.1, 0.999, 0.1, 0.999, 0, 0, 1e-20])


@pytest.mark.parametrize("shift", [-1000.0, 500.0, 30000.0])
def test_logits_far_from_zero(F, shift):
    _check(F, _logits(4, 20000, F32) + shift, top_p=0.9)
    _check(F, _logits(4, 20000, F32) + shift)


def test_wide_spread(F):
    for k in (dict(), dict(top_p=0.9), dict(top_k=2000)):
        _check(F, _logits(4, 20000, F32, scale=1e4), **k)
        _check(F, _logits(4, 20000, BF16, scale=1e-3), **k)
        _check(F, _logits(4, 3000, F32, scale=1e37), **k)


def test_optional_outputs_and_refusals(F):
    x = _logits(3, 700)
    u = torch.rand(3, device=dev())
    want = F.fp8w_sample(x, u)
    ids = torch.empty(3, dtype=torch.int32, device=dev())
    st = F.lib().fp8w_sample(x.data_ptr(), 0, 700, 3, 700, u.data_ptr(), None, None, None, None, ids.data_ptr(), None, None, None, 0,
                             torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == F.OK and torch.equal(ids, want.tokens)
    for bad in (dict(uniforms=u[:2]), dict(uniforms=u.double()), dict(uniforms=None), dict(temperature=u[:2]), dict(top_k=u),
                dict(tokens=u), dict(kept=ids[:2]), dict(logits=x.half())):
        with pytest.raises((ValueError, TypeError)):
            F.fp8w_sample(**{"logits": x, "uniforms": u, **bad})


def test_no_rows(F):
    r = F.fp8w_sample(torch.empty(0, 50, device=dev()), torch.empty(0, device=dev()))
    assert r.tokens.shape == (0,)


def test_lm_head_rows(F):
    x = _logits(4, 151936)
    x[0, 100:130] += 14.0
    for k in (dict(), dict(top_k=50, top_p=0.95), dict(top_p=0.9), dict(min_p=0.02), dict(temperature=0.0)):
        _check(F, x, **k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("i", range(len(FILTERS)))
def test_long_rows(F, i, dtype):
    """Rows of which pieces are taken at once."""
    _check(F, _logits(3, 70001, dtype), **FILTERS[i])


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_rows_unaligned_and_masked(F, pad, dtype):
    wide = _logits(5, 60000 + pad, dtype)
    wide[0, 30000:] = -np.inf
    wide[1] = -np.inf
    wide[2] = -np.inf
    wide[2, [pad, 59999]] = 1.0
    wide[3, ::3] = float("nan")
    for k in FILTERS[::2]:
        _check(F, wide[:, pad:], **k)
        _check(F, wide[:, :60000], **k)


@pytest.mark.parametrize("t", [20, 349, 350])
def test_long_rows_with_settings_of_their_own(F, t):
    rng = np.random.default_rng(t)

    def among(*v):
        return np.array(v)[rng.integers(0, len(v), t)]
    _check(F, _logits(t, 49152), temperature=among(0.0, 0.3, 1.0, 1.7), top_k=among(0, 1, 30, 700, 1500, 10**6),
           top_p=among(1.0, 0.95, 0.5, 0.01), min_p=among(0.0, 0.0, 0.02, 0.3))


@pytest.mark.parametrize("v", [262144, 262145, 300000, 600000, 1 << 21])
def test_more_tokens_than_a_count_of_18_bits(F, v):
    """All in one bin, all equal, and spread: a bin's sums stay within their part of its word."""
    x = torch.zeros(4, v, device=dev())
    x[1] = torch.randn(v, generator=torch.Generator(device="cuda").manual_seed(v), device=dev()) * 1e-4
    x[1, 5], x[1, 6] = 1.0, -60.0                          # bins of a wide range, one of which has nearly all
    x[2] = -30.0
    x[2, -1] = 0.0
    x[3] = _logits(1, v, F32)[0]
    for k in (dict(), dict(top_p=0.6), dict(top_k=v // 2), dict(min_p=0.3), dict(top_k=40, top_p=0.9)):
        _check(F, x, u=np.array([0.3, 0.6, 0.999, 0.42], np.float32), **k)


def test_rows_beyond_4_gib(F):
    """The last row starts past 2^32 bytes."""
    stride = (1 << 30) + 64
    try:
        wide = torch.empty(2 * stride + 60000, dtype=BF16, device=dev())
    except torch.OutOfMemoryError:
        pytest.skip("needs 4 GiB")
    x = torch.as_strided(wide, (3, 60000), (stride, 1))
    x.copy_(_logits(3, 60000))
    _check(F, x, top_p=0.9)
    _check(F, x[:, :7001], top_k=30)


def test_shares_follow_the_probabilities(F):
    """20000 evenly spaced numbers give every token its share of them, off by one at most."""
    x = _logits(1, 40, F32, scale=1.0)
    n = 20000
    u = (torch.arange(n, device=dev(), dtype=torch.float64) + 0.5).div(n).float()
    r = F.fp8w_sample(x.expand(n, 40).contiguous(), u)
    share = torch.bincount(r.tokens.long(), minlength=40).double() / n
    p = torch.softmax(x[0].double(), 0)
    assert (share - p).abs().max() <= 1.01 / n


@pytest.mark.parametrize("v", [40000, 70000])
def test_repeatable_on_another_stream_and_in_a_graph(F, v):
    x, u = _logits(5, v), torch.rand(5, device=dev())
    k = dict(temperature=torch.full((5,), 0.8, device=dev()), top_p=torch.full((5,), 0.9, device=dev()))
    want = [v.clone() for v in F.fp8w_sample(x, u, **k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.fp8w_sample(x, u, **k, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = [torch.empty_like(v) for v in want]
    ws = torch.empty(max(F.lib().fp8w_sample_workspace_bytes(5, v), 16), dtype=torch.uint8, device=dev())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp8w_sample(x, u, **k, tokens=buf[0], logprob=buf[1], kept=buf[2], workspace=ws)
    for i in range(4):
        x.copy_(_logits(5, v, seed=i + 1))
        u.copy_(torch.rand(5, device=dev()))
        for b in buf:
            b.fill_(-7)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(buf, F.fp8w_sample(x, u, **k))), i
