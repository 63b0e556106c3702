"""Activations of the dense product where they are next to nothing, against
bounds of their own evaluation alone: each sum has one term, a product with 1,
and is exact.  And sums beyond fp32's range."""
import math

import numpy as np
import pytest
import torch

from oracle import dense as D
from gpu_util import dev, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
F32 = torch.float32
FAR = [-150, -103, -95, -90, -88, -86, -60, -40, -20, -13, -12, -10, -8, -6, -5, -4, -3, -2, -1, -0.5, -1e-3, -1e-30, 0,
       1e-30, 1e-3, 0.5, 1, 3, 6, 10, 90, 1e30]
ONE = 26   # of FAR, the values that gates multiply


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _bounds(act, v):
    """(act(v), error) in units of 2^-24 of the value, and 2^-119: below it
    results may be zero.

    v * sigmoid(t): an error of t moves it by (1 - sigmoid(t)) of that; silu's
    t is exact, gelu_tanh's has five roundings, 9 |t| with room.  The exponential
    and the reciprocal are good to an ulp each (2 units), and there are five more
    roundings: 16 with room.  v / 2 erfc(z): z has 1.3 units, which move erfc(z)
    by its condition |z erfc'(z) / erfc(z)| (1.5 with room), the function is good
    to 16 ulp and there are three more roundings: 36."""
    if act == "gelu":
        y, _ = D.activation("gelu", v)
        z = -v * math.sqrt(0.5)
        erfc = np.vectorize(math.erfc)(z)
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            cond = np.where(erfc > 0, np.abs(z) * 2 / math.sqrt(math.pi) * np.exp(-z * z) / erfc, 0)
        units = 1.5 * cond + 36
    else:
        y, _ = D.activation(act, v)
        if act == "relu":
            units = np.zeros_like(v)
        else:
            t = v if act in ("silu", "swiglu") else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
            with np.errstate(over="ignore"):
                units = 16 + (0 if act in ("silu", "swiglu") else 9 * np.abs(t) / (1 + np.exp(np.minimum(t, 700))))
    return y, units * 2.0 ** -24 * np.abs(y) + 2.0 ** -119


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"])
@pytest.mark.parametrize("fmt,m", [("block", 1), ("block", 40), ("block", 200), ("mx", 3)])
def test_activations_of_exact_sums(F, act, fmt, m):
    x = torch.tensor(FAR, dtype=torch.float64).to(torch.bfloat16)
    v = x.double().numpy()
    assert v[ONE] == 1
    codes = np.zeros((64, 32), np.uint8)
    codes[np.arange(32), np.arange(32)] = 0x38                        # gates: x's columns
    codes[np.arange(32, 64), ONE] = 0x38                              # values: 1
    scales = np.ones((1, 1), np.float32) if fmt == "block" else np.full((64, 1), 127, np.uint8)
    got = F.fp8w_linear(x[None].repeat(m, 1).to(dev()), to_dev(codes), to_dev(scales), fmt, act=act, out_dtype=F32)
    ref, err = _bounds(act, v)
    got = got.double().cpu().numpy()[:, :32]
    bad = ~(np.abs(got - ref) <= err)
    assert not bad.any(), [(v[j], got[i, j], ref[j], err[j]) for i, j in np.argwhere(bad)[:5]]


@pytest.mark.parametrize("fmt,m", [("block", 1), ("block", 40), ("block", 200), ("mx", 3)])
def test_sums_beyond_fp32(F, fmt, m):
    """+inf passes as the formula's limit; -inf is NaN but under relu, -inf * 0."""
    x = torch.zeros(m, 32, dtype=torch.bfloat16)
    x[:, 0], x[:, 1], x[:, 2] = 3e38, -3e38, 0.5
    codes = np.zeros((8, 32), np.uint8)
    codes[0, 0] = codes[1, 1] = codes[2, 2] = codes[3, 2] = 0x40      # 2.0: inf, -inf, 1, 1
    codes[4:, 2] = 0x40, 0x40, 0xC0, 0x40                             # values 1, 1, -1, 1
    scales = np.ones((1, 1), np.float32) if fmt == "block" else np.full((8, 1), 127, np.uint8)
    inf, nan = np.inf, np.nan

    def call(act):
        return F.fp8w_linear(x.to(dev()), to_dev(codes), to_dev(scales), fmt, act=act, out_dtype=F32).double().cpu().numpy()
    for act, want in (("none", [inf, -inf]), ("relu", [inf, 0]), ("silu", [inf, nan]), ("gelu", [inf, nan]), ("gelu_tanh", [inf, nan]),
                      ("swiglu", [inf, nan]), ("geglu", [inf, nan])):
        y = call(act)
        assert np.array_equal(y[:, :2], np.broadcast_to(want, (m, 2)), equal_nan=True), (act, y[0])
        assert np.isfinite(y[:, 2:4]).all()
