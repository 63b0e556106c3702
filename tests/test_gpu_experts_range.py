"""The products grouped by expert at the ends of fp32's range, on every kernel:
an infinity in any column of x shows where and as the definition says, and
gates near fp32's largest value and beyond it pass through silu."""
import numpy as np
import pytest
import torch

import oracle
from fp8_block_scaled_02_amd import workloads as W
from gpu_util import bf16_to_f64, dev, to_dev, to_dev_bf16
from test_gpu_experts import _experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


# streaming, 128 x 64 tiles, 256 x 128 tiles, these with last runs of half a tile
@pytest.mark.parametrize("slots", [3, 40, 300, 420])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("fmt,n,k", [("block", 64, 400), ("block", 6, 144), ("row", 64, 16), ("mx", 64, 48),
                                     ("mx", 96, 112), ("mx", 64, 208), ("block_bf16", 130, 272), ("tensor", 32, 240),
                                     ("row", 300, 384)])
def test_infinities_of_x(F, fmt, n, k, act, slots):
    """One infinite column in each row of x, every column among them: the
    products are infinite with the weight's sign, NaN where it is zero, and no
    column is met by anything else (k that is no multiple of 128 ends in
    places that read other columns)."""
    codes, scales, cd, sd = _experts(2, n, k, fmt)
    x = W.activation(90, slots, k)
    at = (np.arange(slots) * 5) % k                          # columns 0, 5, 10, ...
    x[np.arange(slots), at] = np.where(np.arange(slots) % 3 == 0, 0xFF80, 0x7F80)
    x[np.arange(slots) % 7 == 6] = W.activation(91, slots, k)[np.arange(slots) % 7 == 6]   # some rows are finite
    split = slots // 4
    off = torch.tensor([0, split, slots], dtype=torch.int32, device=dev())
    y = F.fp8w_gemm_experts(to_dev_bf16(x), cd, sd, off, fmt=fmt, act=act)
    torch.cuda.synchronize()
    got = bf16_to_f64(y)
    inf = np.flatnonzero(np.arange(slots) % 7 != 6)
    expert = (inf >= split).astype(int)
    with np.errstate(all="ignore"):
        w = oracle.e4m3_decode(codes[expert, :, at[inf]]).astype(np.float64)     # its weights, but for scales
        p = w * np.where(inf % 3 == 0, -np.inf, np.inf)[:, None]
        if act == "swiglu":
            h = n // 2
            g, u = p[:, :h], p[:, h:]
            p = np.where(g == -np.inf, np.nan, g) * u          # -inf * 0, as the formula has it
    assert np.array_equal(got[inf], p, equal_nan=True)
    x[inf] = 0
    clean = F.fp8w_gemm_experts(to_dev_bf16(x), cd, sd, off, fmt=fmt, act=act)
    rest = np.setdiff1d(np.arange(slots), inf)
    assert np.isfinite(got[rest]).all() and np.array_equal(got[rest], bf16_to_f64(clean)[rest])


@pytest.mark.parametrize("slots", [8, 40, 200, 130])         # of one expert: the kernels as above
@pytest.mark.parametrize("fmt,half,k", [("row", 64, 128), ("block", 128, 256), ("block", 3, 16), ("mx", 32, 128),
                                        ("mx", 32, 32), ("row", 5, 144)])
def test_gates_at_the_end_of_the_range(F, fmt, half, k, slots):
    """silu(g) is g where g is large, up to infinity: the gate 2^100 * 2^27 *
    f times an up product of one or of 2^-9."""
    n = 2 * half
    codes = np.zeros((1, n, k), np.uint8)
    codes[0, :half, 5] = 0x38                               # 1
    shape = (1, *oracle.scale_shape(fmt, n, k))
    if fmt == "mx":                                         # powers of two only
        scales, up = np.full(shape, 127 + 27, np.uint8), 1.0
        scales[0, half:] = 127 - 100
        codes[0, half:, 5] = 0x38
    elif fmt == "row":
        scales, up = np.full(shape, 2.0 ** 27, np.float32), 1.0
        scales[0, half:] = 2.0 ** -100
        codes[0, half:, 5] = 0x38
    elif half == 128:
        scales, up = np.full(shape, 2.0 ** 27, np.float32), 1.0
        scales[0, 1] = 2.0 ** -100
        codes[0, half:, 5] = 0x38
    else:                                                   # both halves in one scale block
        scales, up = np.full(shape, 2.0 ** 27, np.float32), None
        codes[0, half:, 5] = 0x01                           # 2^-9
    factor = torch.tensor([1.0, 1.5, 1.9375, -1.0, -1.9375, 2.0, 2.0 ** -20, float("inf")])[torch.arange(slots) % 8]
    x = torch.zeros(slots, k)
    x[:, 5] = factor * 2.0 ** 100
    off = torch.tensor([0, slots], dtype=torch.int32, device=dev())
    y = F.fp8w_gemm_experts(x.to(torch.bfloat16).to(dev()), to_dev(codes), to_dev(scales), off, fmt=fmt, act="swiglu")
    torch.cuda.synchronize()
    got = bf16_to_f64(y)
    f = factor.double().numpy()
    with np.errstate(all="ignore"):
        gate = f * 2.0 ** 127
        gate = np.where(np.abs(gate) > np.finfo(np.float32).max, np.sign(f) * np.inf, gate)
        want = np.where(gate > 0, gate, 0.0) * (f if up else gate * 2.0 ** -9)
    want = np.where(want > 2.0 ** 127 * (2 - 2.0 ** -8), np.inf, want)      # past bf16's largest value and half a step
    want = np.broadcast_to(want[:, None], got.shape)
    assert not np.isnan(got).any()
    with np.errstate(invalid="ignore"):
        near = np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 8 * 2.0 ** -23 * np.abs(want)
    assert ((got == want) | near).all(), (got[:8, 0], want[:8, 0])
