"""The plain forms of the product with its epilogue, of sampling and of routing
in groups (``oracle/dense.py``) against torch on the CPU, planted mistakes
that these checks must catch, and the refusals of the entry points, which need
no GPU."""
import types

import numpy as np
import pytest
import torch

import oracle
from oracle import dense as D
from fp8_block_scaled_02_amd import workloads as W


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"])
def test_linear_against_torch(act):
    codes, scales = oracle.quantize_format(W.gaussian_weight(3, 0, 40, 160), "block")
    x = W.activation(3, 35, 160)
    rng = np.random.default_rng(1)
    n_out = 20 if act in D.GATED else 40
    bias, residual = rng.standard_normal(40), rng.standard_normal((35, n_out))
    y, err = D.linear(x, codes, scales, "block", bias, act, residual)
    w = codes.reshape(-1)
    w = torch.from_numpy(w).view(torch.float8_e4m3fn).double().view(40, 160)
    w = w * torch.from_numpy(scales).double().repeat_interleave(128, 0)[:40].repeat_interleave(128, 1)[:, :160]
    v = torch.from_numpy(oracle.bf16_to_f32(x)).double() @ w.T + torch.from_numpy(bias)
    f = torch.nn.functional
    g, u = v.chunk(2, 1)
    want = {"none": lambda: v, "silu": lambda: f.silu(v), "gelu": lambda: f.gelu(v), "relu": lambda: f.relu(v),
            "gelu_tanh": lambda: f.gelu(v, approximate="tanh"), "swiglu": lambda: f.silu(g) * u,
            "geglu": lambda: f.gelu(g, approximate="tanh") * u}[act]().numpy() + residual
    assert np.allclose(y, want, rtol=1e-12, atol=1e-13) and (err > 0).all() and err.max() < 1e-2


def _settings(t, seed):
    rng = np.random.default_rng(seed)

    def of(values, dtype=np.float32):
        return np.array(values, dtype)[rng.integers(0, len(values), t)]
    return dict(uniforms=rng.random(t, np.float32), temperature=of([0.5, 1, 2]), top_k=of([0, 3, 10, 500], np.int32),
                top_p=of([1.0, 0.9, 0.3]), min_p=of([0.0, 0.05, 0.4]))


def test_sample_against_torch():
    """By probabilities: masks of the tokens each filter leaves, then the place of u."""
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(60, 80, generator=g) * 3).bfloat16().double()
    x[::7, 5:30] = -np.inf
    k = _settings(60, 3)
    tokens, logprob, kept = D.sample(x.numpy(), **k)
    for r in range(60):
        p = torch.softmax(x[r] / float(k["temperature"][r]), 0)
        v, order = torch.sort(p, descending=True, stable=True)
        v = v[v > 0]
        if k["top_k"][r] > 0:
            v = v[:int(k["top_k"][r])]
        v = v / v.sum()
        keep = torch.ones(len(v), dtype=torch.bool)
        if k["top_p"][r] < 1:
            keep &= v.cumsum(0) - v < float(k["top_p"][r])
        if k["min_p"][r] > 0:
            keep &= v >= float(k["min_p"][r]) * v[0]
        keep[0] = True
        v = v[keep] / v[keep].sum()
        j = int((v.cumsum(0) <= float(k["uniforms"][r])).sum())
        assert kept[r] == len(v) and tokens[r] == order[j] and abs(logprob[r] - float(torch.log(v[j]))) < 1e-11


def test_sample_edges():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 2.0, 2.0, -inf, nan], [-inf] * 4 + [nan], [inf, 0.0, inf, 1.0, -inf]])
    three = lambda *v: np.array(v, np.float64)   # noqa: E731
    ids, lp, kept = D.sample(x, three(0.99, 0.5, 0.5), three(0.0, 1.0, 1.0))
    assert ids.tolist() == [1, -1, 2] and kept.tolist() == [1, 0, 4] and lp[0] == 0 and lp[1] == -inf
    assert np.isclose(lp[2], -np.log(2))
    ids, lp, kept = D.sample(x[[0, 0, 0]], three(0.0, 0.5, 0.999), top_k=np.array([2, 2, 2]))
    assert ids.tolist() == [1, 2, 2] and kept.tolist() == [2, 2, 2]
    ids, _, kept = D.sample(x[[0, 0, 0]], three(1.0, -1.0, nan), top_p=three(1.0, 0.0, 0.2))
    assert ids.tolist() == [0, 1, 1] and kept.tolist() == [3, 1, 1]
    flat = np.zeros((3, 8))
    _, _, kept = D.sample(flat, three(0, 0, 0), top_p=three(0.25, 0.3, 2.0))
    assert kept.tolist() == [2, 3, 8]                              # a border met exactly takes no more
    _, _, kept = D.sample(x[[0, 0, 0]], three(0, 0, 0), min_p=three(1.0, 2.0, nan))
    assert kept.tolist() == [2, 1, 3]
    ids, lp, kept = D.sample(x[[0, 2, 0]], three(0.9, 0.9, 0.9), three(inf, 1e-30, nan))
    assert kept.tolist() == [3, 4, 1] and ids.tolist() == [0, 2, 1]


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_grouped_against_torch(by, score, biased):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(50, 24, generator=g).double()
    x[:, 12] = x[:, 3]                                             # ties over groups
    bias = torch.randn(24, generator=g).double() if biased else None
    ids, w, slots, rows, offsets = D.route_grouped(x.numpy(), 3, 6, 2, by, score, None if bias is None else bias.numpy())
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    key = p if bias is None else p + bias
    part = key.view(50, 6, 4)
    rating = part.amax(2) if by == "max" else part.topk(2, 2).values.sum(2)
    best = torch.sort(rating, dim=1, descending=True, stable=True).indices[:, :2]
    shut = torch.ones(50, 6, dtype=torch.bool).scatter_(1, best, False).repeat_interleave(4, 1)
    want = torch.sort(key.masked_fill(shut, -np.inf), dim=1, descending=True, stable=True).indices[:, :3]
    assert np.array_equal(ids, want.numpy())
    tw = p.gather(1, want)
    assert np.allclose(w, (tw / tw.sum(1, keepdim=True)).numpy(), rtol=1e-13)
    order = np.argsort(ids.reshape(-1), kind="stable")
    assert np.array_equal(rows, order // 3) and np.array_equal(slots.reshape(-1)[order], np.arange(150))
    assert np.array_equal(np.diff(offsets), np.bincount(ids.reshape(-1), minlength=24))


def test_route_grouped_masks():
    inf = np.inf
    x = np.array([[5.0, -inf, 1.0, 1.5, -inf, -inf], [-inf] * 6, [-inf, -inf, -inf, -inf, 0.0, np.nan]])
    ids, w, *_ = D.route_grouped(x, 2, 3, 1, "top2", "sigmoid")
    assert ids.tolist() == [[3, 2], [-1, -1], [4, -1]]             # one live expert counts once
    ids, *_ = D.route_grouped(x, 2, 3, 1)
    assert ids.tolist() == [[0, -1], [-1, -1], [4, -1]]
    ids, *_ = D.route_grouped(x, 4, 3, 2)
    assert ids.tolist() == [[0, 3, 2, -1], [-1] * 4, [4, -1, -1, -1]]


@pytest.mark.parametrize("old,new", [
    ("v = v + bias", "v = v"),
    ("y = s * u", "y = g * u"),
    ("0.044715 * v ** 3", "0.044715 * v ** 2"),
    ("z = -v * math.sqrt(0.5)", "z = v * math.sqrt(0.5)"),
    ("y = y + residual", "y = y - residual"),
    ("g, eg, u, eu = v[:, :h], err[:, :h], v[:, h:], err[:, h:]", "u, eu, g, eg = v[:, :h], err[:, :h], v[:, h:], err[:, h:]"),
    ("np.argsort(-x, kind=\"stable\")", "np.argsort(x, kind=\"stable\")[::-1]"),       # ties to the higher token
    ("before < np.longdouble", "before <= np.longdouble"),                              # one more at an exact border
    ("* upto[n - 1])", "* upto[-1])"),                                                  # the nucleus of all tokens
    ("scaled >= math.log", "scaled > math.log"),
    ("upto[:stop] <= goal", "upto[:stop] < goal"),
    ("stop = max(stop, 1)", "pass"),
    ("np.log(upto[stop - 1])", "np.log(upto[-1])"),
    ("key=lambda g: (-rating[g], g)", "key=lambda g: (-rating[g], -g)"),
    ("best[:2].sum()", "best.sum()"),
    ("value = p if bias is None and by == \"top2\" else key", "value = key"),
    ("live &= np.isin(parts, best)", "pass"),
])
def test_planted_mistakes_are_caught(old, new, monkeypatch):
    text = open(D.__file__).read()
    assert text.count(old) == 1
    broken = types.ModuleType("oracle.dense_broken")
    broken.__package__ = "oracle"
    exec(compile(text.replace(old, new), "dense_broken", "exec"), broken.__dict__)
    monkeypatch.setitem(globals(), "D", broken)
    checks = [lambda a=a: test_linear_against_torch(a) for a in ("none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu")]
    checks += [test_sample_against_torch, test_sample_edges, test_route_grouped_masks]
    checks += [lambda b=b, s=s, z=z: test_route_grouped_against_torch(b, s, z) for b in ("max", "top2")
               for s in ("softmax", "sigmoid") for z in (False, True)]
    caught = 0
    with np.errstate(all="ignore"):
        for check in checks:
            try:
                check()
            except (AssertionError, IndexError, ValueError):
                caught += 1
    assert caught


# -------------------------------------------------------------- refusals --

A, B, C, E, G, H, I = (0x10000000 * i for i in range(1, 8))   # never dereferenced


@pytest.fixture(scope="module")
def L():
    import fp8_block_scaled_02_amd as F
    return F.lib()


def test_linear_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(x=A, xs=64, m=8, codes=B, scales=C, fmt=0, n=32, k=64, bias=E, bd=0, act=0, res=G, rs=32, y=H, yd=0, ys=32,
             ws=I, wn=1 << 40):
        return L.fp8w_linear(x, xs, m, codes, scales, fmt, n, k, bias, bd, act, res, rs, y, yd, ys, ws, wn, None)
    for name in ("x", "codes", "scales", "y"):
        assert call(**{name: None}) == F.ERR_NULL, name
    for bad in (dict(fmt=5), dict(fmt=-1), dict(act=7), dict(act=-1), dict(bd=2), dict(yd=2)):
        assert call(**bad) == F.ERR_UNSUPPORTED, bad
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(n=33, act=1), dict(n=33, act=6, res=None), dict(xs=56), dict(ys=31),
                dict(rs=31), dict(xs=1 << 31), dict(xs=(1 << 28) + 8), dict(ys=1 << 31), dict(rs=1 << 31), dict(m=(1 << 30) + 1),
                dict(n=(1 << 28) + 1, ys=1 << 29, rs=1 << 29), dict(k=(1 << 28) + 16, xs=1 << 29),
                dict(m=1 << 30, n=1 << 28, ys=1 << 28, res=None, x=1 << 62, y=1 << 61)):
        assert call(**bad) == F.ERR_SHAPE, bad
    for bad in (dict(k=72, xs=72), dict(xs=68), dict(x=A + 8), dict(codes=B + 8), dict(scales=C + 2), dict(bias=E + 1),
                dict(bias=E + 2, bd=1), dict(res=G + 1), dict(y=H + 1), dict(y=H + 2, yd=1)):
        assert call(**bad) == F.ERR_ALIGN, bad
    for bad in (dict(y=A + 32), dict(y=B + 32 * 64 - 2), dict(y=C), dict(y=E), dict(y=G + 2), dict(y=G, yd=1),
                dict(y=G, ys=40), dict(y=A + 7 * 1024 + 126, xs=512)):
        assert call(**bad) == F.ERR_OVERLAP, bad
    assert call(m=0, x=None, y=None) == F.OK                        # nothing to do, nothing launched
    size = L.fp8w_linear_workspace_bytes
    for bad in ((0, 32, 64, 0, 0), (-1, 32, 64, 0, 0), (8, 0, 64, 0, 0), (8, 32, 8, 0, 0), (8, 32, 64, 5, 0), (8, 32, 64, 0, 7),
                (8, 33, 64, 0, 1)):
        assert size(*bad) == 0, bad


def test_linear_workspace_refusals(L):
    """Of a shape that takes one, if there is any."""
    import fp8_block_scaled_02_amd as F
    shape = (64, 2048, 8192)
    need = L.fp8w_linear_workspace_bytes(*shape, 0, 0)
    if need == 0:
        pytest.skip("these sizes need no workspace")

    def call(ws=I, wn=need, y=H):
        m, n, k = shape
        return L.fp8w_linear(A, k, m, B, C, 0, n, k, None, 0, 0, None, 0, y, 0, n, ws, wn, None)
    assert call(ws=None) == F.ERR_NULL and call(wn=need - 1) == F.ERR_SHAPE and call(ws=I + 8) == F.ERR_ALIGN
    assert call(y=I + need - 2) == F.ERR_OVERLAP and call(ws=B + 1024) == F.ERR_OVERLAP


def test_sample_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(logits=A, dtype=0, stride=100, t=4, v=100, u=B, temp=None, k=None, p=None, low=None, ids=C, lp=E, kept=G, ws=H,
             wn=1 << 40):
        return L.fp8w_sample(logits, dtype, stride, t, v, u, temp, k, p, low, ids, lp, kept, ws, wn, None)
    for name in ("logits", "u", "ids"):
        assert call(**{name: None}) == F.ERR_NULL, name
    assert call(dtype=2) == F.ERR_UNSUPPORTED
    for bad in (dict(t=-1), dict(v=0), dict(stride=99), dict(v=(1 << 24) + 1, stride=1 << 25), dict(stride=1 << 31),
                dict(t=1 << 30, u=1 << 50, ids=1 << 51, lp=1 << 52, kept=1 << 53, ws=1 << 54)):
        assert call(**bad) == F.ERR_SHAPE, bad
    for bad in (dict(logits=A + 1), dict(logits=A + 2, dtype=1), dict(u=B + 2), dict(temp=I + 1), dict(k=I + 2), dict(p=I + 3),
                dict(low=I + 1), dict(ids=C + 2), dict(lp=E + 1), dict(kept=G + 2)):
        assert call(**bad) == F.ERR_ALIGN, bad
    for bad in (dict(ids=A + 796), dict(ids=B), dict(lp=C + 12), dict(kept=E), dict(temp=C), dict(k=E + 4), dict(p=G),
                dict(low=G + 12)):
        assert call(**bad) == F.ERR_OVERLAP, bad
    assert call(t=0, logits=None, u=None, ids=None) == F.OK
    need = L.fp8w_sample_workspace_bytes(4, 151936)
    if need:
        big = dict(v=151936, stride=151936)
        assert call(ws=None, **big) == F.ERR_NULL and call(wn=need - 1, **big) == F.ERR_SHAPE
        assert call(ws=H + 8, **big) == F.ERR_ALIGN and call(ws=A + 16, **big) == F.ERR_OVERLAP


def test_route_grouped_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(t=4, e=16, k=2, groups=4, top=2, by=0):
        return L.fp8w_route_experts_grouped(A, 1, e, t, e, k, 0, None, groups, top, by, 1, 1.0, B, C, E, G, H, I, 1 << 20, None)
    assert call(by=2) == F.ERR_UNSUPPORTED and call(by=-1) == F.ERR_UNSUPPORTED
    for bad in (dict(groups=0), dict(groups=3), dict(groups=32), dict(top=0), dict(top=5), dict(k=9, top=2), dict(groups=-4),
                dict(e=130, groups=65, top=1, k=1)):
        assert call(**bad) == F.ERR_SHAPE, bad


def test_binding_refuses_before_the_library():
    import fp8_block_scaled_02_amd as F
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 1)
    with pytest.raises(ValueError):
        F.fp8w_linear(x, codes, scales)                              # CPU tensors
    with pytest.raises(ValueError):
        F.fp8w_sample(x, torch.zeros(2))
    with pytest.raises(TypeError):
        F.fp8w_linear([1.0], codes, scales)
