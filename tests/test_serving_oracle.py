"""The 64-bit forms of the routing, experts, combine and log probability
operators (``oracle/serving.py``) against torch on the CPU, and planted
mistakes that these checks must catch; then the refusals of the library's
entry points, which need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S
from fp8_block_scaled_02_amd import workloads as W


def _route_by_torch(x, k, score, bias, renorm):
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    key = x if bias is None else p + bias
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    return ids.numpy(), (w / w.sum(1, keepdim=True) if renorm else w).numpy()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_against_torch(score, biased, renorm):
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-6, 6, (40, 24), generator=g).double() / 4   # many ties
    bias = torch.randn(24, generator=g).double() if biased else None
    ids, w, slots, rows, offsets = S.route(x.numpy(), 5, score, None if bias is None else bias.numpy(), renorm)
    ti, tw = _route_by_torch(x, 5, score, bias, renorm)
    assert np.array_equal(ids, ti) and np.abs(w - tw).max() < 1e-14
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(rows, order // 5)
    assert np.array_equal(slots.reshape(-1)[order], np.arange(200))
    assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=24))]))


def test_route_masked_experts():
    x = np.full((3, 4), -np.inf)
    x[1, 2], x[2, :] = 1.0, [0.0, np.nan, 2.0, -np.inf]
    ids, w, slots, rows, offsets = S.route(x, 3)
    assert ids.tolist() == [[-1, -1, -1], [2, -1, -1], [2, 0, -1]]
    assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0] and abs(w[2].sum() - 1) < 1e-15
    assert slots.tolist() == [[-1, -1, -1], [1, -1, -1], [2, 0, -1]]
    assert rows.tolist() == [2, 1, 2] + [-1] * 6 and offsets.tolist() == [0, 1, 1, 3, 3]


@pytest.mark.parametrize("fmt", sorted(oracle.FORMATS))
def test_experts_against_dequantized_matmul(fmt):
    codes, scales, deq = [], [], []
    for e in range(3):
        c, s = oracle.quantize_format(W.gaussian_weight(7, e, 34, 160), fmt)
        codes.append(c), scales.append(s)
        eye = np.eye(160, dtype=np.float32)
        deq.append(oracle.gemv_format_f64(W._to_bf16(eye[:32]), c, s, fmt)[0])   # 32 columns of the weight
    x = W.activation(7, 5, 160)
    x[:, 32:] = 0                                                                # so that those decide
    rows, offsets = np.array([4, 0, 9, 1, 4, 3]), np.array([0, 2, 2, 5])
    y, b = S.gemm_experts(x, np.stack(codes), np.stack(scales), offsets, rows, fmt)
    xf = oracle.bf16_to_f32(x).astype(np.float64)
    for i, (e, r) in enumerate([(0, 4), (0, 0), (2, None), (2, 1), (2, 4)]):
        want = np.zeros(34) if r is None else xf[r, :32] @ deq[e]
        assert np.allclose(y[i], want, rtol=1e-12, atol=1e-14) and (b[i] >= np.abs(want) - 1e-12).all()
    assert np.isnan(y[5]).all()


def test_swiglu_and_combine_against_torch():
    rng = np.random.default_rng(2)
    y = rng.standard_normal((7, 12)) * 3
    t = torch.from_numpy(y)
    out, _ = S.swiglu(y, np.zeros_like(y))
    assert np.allclose(out, (torch.nn.functional.silu(t[:, :6]) * t[:, 6:]).numpy(), rtol=1e-13)
    slots = np.array([[0, 6], [-1, 3], [7, -1]])
    w = rng.random((3, 2)).astype(np.float32)
    out, bound = S.combine(y, w, slots)
    assert np.allclose(out, [w[0, 0] * y[0] + w[0, 1] * y[6], w[1, 1] * y[3], 0 * y[0]], rtol=1e-13)
    assert (bound >= np.abs(out) - 1e-15).all()


def test_logprobs_against_torch():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(6, 300, generator=g) * 4).bfloat16().double()
    x[1, ::2] = -np.inf
    x[2] = 1.5
    x[3] = -np.inf
    x[4, 7] = np.nan
    targets = np.array([5, 4, 299, 0, 1, -1])
    lp, ent, ids, best = S.logprobs(x.numpy(), targets, 9)
    ok = [0, 1, 2, 5]
    ref = torch.log_softmax(x[ok], 1)
    assert np.allclose(lp[[0, 1, 2]], [ref[0, 5], ref[1, 4], ref[2, 299]], atol=1e-12) and np.isnan(lp[[4, 5]]).all()
    cat = torch.distributions.Categorical(logits=torch.where(x[ok].isinf(), torch.tensor(-1e30).double(), x[ok]))
    assert np.allclose(ent[ok], cat.entropy().numpy(), atol=1e-12)
    want = torch.sort(x[ok], dim=1, descending=True, stable=True)
    assert np.array_equal(ids[ok], want.indices[:, :9].numpy())
    assert np.allclose(best[ok], ref.gather(1, want.indices[:, :9]).numpy(), atol=1e-12)
    assert lp[3] == -np.inf and ent[3] == 0 and ids[3].tolist() == list(range(9))
    assert np.isnan(ent[4]) and 7 not in ids[4]


@pytest.mark.parametrize("old,new", [
    ("(-key[i], i)", "(-key[i], -i)"),                       # ties to the higher expert
    ("p + np.asarray(bias, np.float64)", "p"),               # the bias dropped
    ("w[r] /= p[order].sum()", "pass"),                      # not renormalized
    ("sorted((ids[r, j], r, j)", "sorted((ids[r, j], -r, j)"),   # tokens of an expert in reverse
    ("offsets[i + 1] += 1", "offsets[i] += 1"),              # offsets shifted
    ("g / (1.0 + np.exp(-g))", "g / (1.0 + np.exp(g))"),     # the gate's sign
    ("g, u = y[:, :h], y[:, h:]", "u, g = y[:, :h], y[:, h:]"),   # the halves swapped
    ("0 <= slots[r, j] < len(y)", "slots[r, j] < len(y)"),   # a choice not made read as the last row
    ("np.argsort(-rank, kind=\"stable\")", "np.argsort(rank, kind=\"stable\")[::-1]"),   # ties to the higher token
    ("np.where(p > 0, logp, 0.0)", "logp"),                  # 0 * inf in a masked entropy
])
def test_planted_mistakes_are_caught(old, new, monkeypatch):
    """Each mistake, planted in a copy of the plain forms, fails a check above."""
    import types
    text = open(S.__file__).read()
    assert text.count(old) == 1
    broken = types.ModuleType("oracle.serving_broken")
    broken.__package__ = "oracle"
    exec(compile(text.replace(old, new), "serving_broken", "exec"), broken.__dict__)
    monkeypatch.setitem(globals(), "S", broken)
    checks = [lambda s=s, b=b, r=r: test_route_against_torch(s, b, r) for s in ("softmax", "sigmoid")
              for b in (False, True) for r in (False, True)]
    checks += [test_route_masked_experts, test_swiglu_and_combine_against_torch, test_logprobs_against_torch]
    caught = 0
    with np.errstate(all="ignore"):
        for check in checks:
            try:
                check()
            except (AssertionError, IndexError):
                caught += 1
    assert caught


# -------------------------------------------------------------- refusals --

A, B, C, D, E, G, H = (0x1000000 * i for i in range(1, 8))   # never dereferenced


@pytest.fixture(scope="module")
def L():
    import fp8_block_scaled_02_amd as F
    return F.lib()


def test_route_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(logits=A, dtype=1, stride=16, t=4, e=16, k=2, score=0, bias=None, ids=B, w=C, slots=D, rows=E, off=G,
             ws=H, ws_n=1 << 20):
        return L.fp8w_route_experts(logits, dtype, stride, t, e, k, score, bias, 1, 1.0, ids, w, slots, rows, off,
                                    ws, ws_n, None)
    for name in ("logits", "ids", "w", "slots", "rows", "off"):
        assert call(**{name: None}) == F.ERR_NULL, name
    assert call(dtype=2) == F.ERR_UNSUPPORTED and call(score=2) == F.ERR_UNSUPPORTED
    for bad in (dict(t=-1), dict(e=0), dict(e=1025, stride=1025), dict(k=0), dict(k=17), dict(stride=15),
                dict(e=256, stride=256, k=65), dict(t=1 << 31)):
        assert call(**bad) == F.ERR_SHAPE, bad
    assert call(t=33, ws=None) == F.ERR_NULL
    assert L.fp8w_route_experts_workspace_bytes(32, 60) == 0
    need = L.fp8w_route_experts_workspace_bytes(33, 61)
    assert need == 2 * 64
    assert call(t=33, e=61, stride=61, ws_n=need - 1) == F.ERR_SHAPE
    for bad in (dict(logits=A + 2), dict(logits=A + 1, dtype=0), dict(bias=H + 2), dict(ids=B + 2), dict(off=G + 1)):
        assert call(**bad) == F.ERR_ALIGN, bad
    assert call(ids=A + 64) == F.ERR_OVERLAP and call(w=B + 8) == F.ERR_OVERLAP
    assert call(t=33, ws=G + 8) == F.ERR_OVERLAP and call(bias=D) == F.ERR_OVERLAP
    assert call(stride=1 << 10, slots=A + 4096 * 3 + 60) == F.ERR_OVERLAP      # the last row's last logit


def test_gemm_experts_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(x=A, x_rows=8, rows=B, off=C, e=4, slots=16, codes=D, scales=E, fmt=0, n=32, k=64, act=0, y=G):
        return L.fp8w_gemm_experts(x, x_rows, rows, off, e, slots, codes, scales, fmt, n, k, act, y, None)
    for name in ("x", "off", "codes", "scales", "y"):
        assert call(**{name: None}) == F.ERR_NULL, name
    assert call(fmt=5) == F.ERR_UNSUPPORTED and call(act=2) == F.ERR_UNSUPPORTED
    for bad in (dict(n=0), dict(k=8), dict(e=0), dict(slots=-1), dict(x_rows=0), dict(rows=None), dict(n=33, act=1),
                dict(n=1 << 31), dict(e=1 << 30, n=1 << 20, k=1 << 20)):
        assert call(**bad) == F.ERR_SHAPE, bad
    for bad in (dict(k=72), dict(x=A + 8), dict(codes=D + 8), dict(scales=E + 2), dict(y=G + 4), dict(rows=B + 2),
                dict(off=C + 2)):
        assert call(**bad) == F.ERR_ALIGN, bad
    for bad in (dict(y=A + 64), dict(y=B + 8), dict(y=C - 8), dict(y=D + 4 * 32 * 64 - 8), dict(y=E)):
        assert call(**bad) == F.ERR_OVERLAP, bad
    assert call(slots=0, x=None, y=None, x_rows=0) == F.OK                     # nothing to do, nothing launched


def test_gemm_experts_limits(L):
    """Sizes whose tiles would step past 32 bits."""
    import fp8_block_scaled_02_amd as F

    def call(e=1, slots=16, n=32, k=64, x_rows=8):
        return L.fp8w_gemm_experts(A, x_rows, B, C, e, slots, D, E, 0, n, k, 0, G, None)
    for bad in (dict(n=(1 << 28) + 1), dict(k=(1 << 28) + 16), dict(e=(1 << 28) + 1), dict(slots=(1 << 30) + 1)):
        assert call(**bad) == F.ERR_SHAPE, bad


def test_combine_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(y=A, slot_rows=16, w=B, slots=C, t=4, k=2, n=32, out=D):
        return L.fp8w_combine_experts(y, slot_rows, w, slots, t, k, n, out, None)
    for name in ("y", "w", "slots", "out"):
        assert call(**{name: None}) == F.ERR_NULL, name
    for bad in (dict(t=-1), dict(k=0), dict(k=65), dict(n=0), dict(slot_rows=-1), dict(t=1 << 26, k=64)):
        assert call(**bad) == F.ERR_SHAPE, bad
    for bad in (dict(y=A + 1), dict(w=B + 2), dict(slots=C + 1), dict(out=D + 1)):
        assert call(**bad) == F.ERR_ALIGN, bad
    for bad in (dict(out=A + 64), dict(out=B), dict(out=C)):
        assert call(**bad) == F.ERR_OVERLAP, bad
    assert call(t=0, w=None, slots=None, out=None) == F.OK


def test_logprobs_refusals(L):
    import fp8_block_scaled_02_amd as F

    def call(logits=A, dtype=0, stride=100, t=4, v=100, targets=B, top=3, lp=C, ent=D, ids=E, best=G, ws=H,
             ws_n=1 << 24):
        return L.fp8w_logprobs(logits, dtype, stride, t, v, targets, top, lp, ent, ids, best, ws, ws_n, None)
    for name in ("logits", "targets", "lp", "ids", "best"):
        assert call(**{name: None}) == F.ERR_NULL, name
    assert call(dtype=3) == F.ERR_UNSUPPORTED
    for bad in (dict(t=-1), dict(v=0), dict(top=-1), dict(top=65), dict(v=2, top=3), dict(stride=99),
                dict(v=(1 << 31) - 1, stride=(1 << 31) - 1)):
        assert call(**bad) == F.ERR_SHAPE, bad
    need = L.fp8w_logprobs_workspace_bytes(4, 100000, 3)
    assert need > 0 and L.fp8w_logprobs_workspace_bytes(4096, 100000, 3) == 0
    assert call(v=100000, stride=100000, ws=None) == F.ERR_NULL
    assert call(v=100000, stride=100000, ws_n=need - 1) == F.ERR_SHAPE
    for bad in (dict(logits=A + 1), dict(logits=A + 2, dtype=1), dict(targets=B + 2), dict(lp=C + 1), dict(ent=D + 2),
                dict(ids=E + 1), dict(best=G + 2), dict(v=100000, stride=100000, ws=H + 4)):
        assert call(**bad) == F.ERR_ALIGN, bad
    for bad in (dict(lp=A + 700), dict(ent=C), dict(ids=G + 16), dict(lp=B)):
        assert call(**bad) == F.ERR_OVERLAP, bad
    assert call(t=0, logits=None, targets=None, lp=None, ids=None, best=None) == F.OK


def test_binding_refuses_before_the_library():
    import fp8_block_scaled_02_amd as F
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.fp8w_route_experts(x, 2)                                   # a CPU tensor
    with pytest.raises(ValueError):
        F.fp8w_logprobs(x)
    with pytest.raises(TypeError):
        F.fp8w_logprobs(np.zeros((2, 16)))
    assert ctypes.sizeof(ctypes.c_void_p) == 8
