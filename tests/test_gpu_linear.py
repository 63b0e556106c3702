"""GPU parity of the product with bias, activation and residual against the
64-bit form: every scale format, activation and type, sizes around each
kernel's tiles, odd sizes, strides, results in place, infinities and far
values, streams and graphs."""
import numpy as np
import pytest
import torch

import oracle
from oracle import dense as D
from fp8_block_scaled_02_amd import workloads as W
from gpu_util import bf16_to_f64, dev, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
FORMATS = sorted(oracle.FORMATS)
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _weight(n, k, fmt, seed=0):
    """Codes and scales of a gaussian weight (the quantizer's own tests hold those)."""
    codes, scales = oracle.quantize_format(W.gaussian_weight(9, seed, n, k), fmt)
    return codes, scales, to_dev(codes), _scales(scales, fmt)


def _scales(scales, fmt):
    if fmt == "block_bf16":
        return to_dev_bf16(scales)
    s = to_dev(scales)
    return s.reshape(1) if fmt == "tensor" else s


def _near(got, ref, err):
    half = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    y = got.double().cpu().numpy()
    bad = ~(np.abs(y - ref) <= err + half * (np.abs(ref) + err) + 2.0 ** -134)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), y[bad][:3], ref[bad][:3], err[bad][:3])


def _check(F, m, n, k, fmt="block", act="none", bias=None, residual=False, out=BF16, x=None, pad=0, seed=0):
    codes, scales, cd, sd = _weight(n, k, fmt, seed)
    xb = W.activation(seed, m, k) if x is None else x
    g = torch.Generator(device="cuda").manual_seed(seed * 1009 + m * 31 + n)
    n_out = n // 2 if act in D.GATED else n
    xd = to_dev_bf16(xb)
    if pad:
        wide = torch.full((m, k + pad), float("nan"), dtype=BF16, device=dev())
        wide[:, :k] = xd
        xd = wide[:, :k]
    b = None if bias is None else torch.randn(n, generator=g, device=dev()).to(bias)
    r = torch.randn(m, n_out + pad, generator=g, device=dev()).to(BF16)[:, :n_out] if residual else None
    y = torch.full((m, n_out + pad), 7.0, dtype=out, device=dev())
    got = F.fp8w_linear(xd, cd, sd, fmt, b, act, r, y=y[:, :n_out])
    torch.cuda.synchronize()
    ref, err = D.linear(xb, codes, scales, fmt, None if b is None else b.double().cpu().numpy(), act,
                        None if r is None else bf16_to_f64(r))
    _near(got, ref, err)
    assert (y[:, n_out:] == 7).all(), "between the rows"
    return got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 2, 3, 5, 16, 17, 32, 33, 65, 130])
def test_rows(F, fmt, m):
    _check(F, m, 272, 640, fmt, bias=BF16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 33, 64, 127, 129, 257, 400])
@pytest.mark.parametrize("m", [1, 20, 70])
def test_weight_rows(F, fmt, n, m):
    _check(F, m, n, 272, fmt, bias=F32, residual=n % 2 == 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("k", [16, 32, 48, 96, 112, 128, 144, 256, 272, 384, 1040, 4112])
@pytest.mark.parametrize("m", [1, 9, 48])
def test_columns(F, fmt, k, m):
    _check(F, m, 96, k, fmt)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"])
@pytest.mark.parametrize("m", [1, 12, 40, 150])
@pytest.mark.parametrize("out", [BF16, F32])
def test_activations(F, act, m, out):
    _check(F, m, 192, 320, "block", act, BF16, True, out)
    _check(F, m, 192, 320, "mx", act, None, False, out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("half", [1, 3, 7, 16, 60, 64, 100, 130, 192, 201])
@pytest.mark.parametrize("m", [1, 40])
def test_gated_halves(F, fmt, half, m):
    """Halves that start anywhere in a scale block."""
    _check(F, m, 2 * half, 288, fmt, "swiglu", F32)


@pytest.mark.parametrize("fmt", ["block", "block_bf16", "mx"])
@pytest.mark.parametrize("m,half,k", [(20, 16500, 80), (20, 70, 1040), (100, 2001, 272), (100, 3001, 144), (30, 6801, 400), (30, 6816, 656), (270, 130, 2064),
                                      (270, 7001, 144), (600, 100, 400), (600, 1111, 272), (600, 1120, 272), (520, 64, 4112)])
def test_gated_halves_of_many_sizes(F, fmt, m, half, k):
    """Every tiling, with halves that start at the end of a scale block, of 32 or 16 rows, and anywhere."""
    _check(F, m, 2 * half, k, fmt, "geglu", BF16, True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(2, 300, 144), (1, 3000, 400), (3, 65600, 48), (12, 16400, 144), (16, 130, 8208), (20, 33000, 80),
                                   (100, 6100, 272), (25, 12400, 592), (33, 7000, 1552), (70, 500, 2064), (150, 400, 1296), (500, 8400, 144), (513, 300, 656), (700, 200, 3104)])
def test_sizes_of_every_kernel(F, fmt, m, n, k):
    _check(F, m, n, k, fmt, "silu", F32, True)


@pytest.mark.parametrize("m", [1, 6, 30, 100])
@pytest.mark.parametrize("pad", [8, 24, 128])
def test_strides(F, m, pad):
    _check(F, m, 136, 208, "block", "none", BF16, True, pad=pad)
    _check(F, m, 130, 208, "row", "geglu", None, True, F32, pad=pad)


@pytest.mark.parametrize("m", [1, 3, 31, 64, 200])
@pytest.mark.parametrize("shape", [(512, 2048), (256, 8192), (1000, 4096)])
def test_long_sums(F, m, shape):
    """Few rows and many columns, where the sums may be cut and joined."""
    _check(F, m, *shape, "block", "none", F32, True, F32)
    _check(F, m, *shape, "mx", "swiglu")


@pytest.mark.parametrize("m", [1, 17, 64, 200])
def test_in_place(F, m):
    codes, scales, cd, sd = _weight(144, 256, "block")
    xb = W.activation(1, m, 256)
    r = torch.randn(m, 144, device=dev()).to(BF16)
    ref, err = D.linear(xb, codes, scales, "block", residual=bf16_to_f64(r))
    y = F.fp8w_linear(to_dev_bf16(xb), cd, sd, residual=r, y=r)
    assert y is r
    _near(r, ref, err)


@pytest.mark.parametrize("m", [1, 10, 33, 150])
def test_infinities_reach_their_row_alone(F, m):
    """Also past the columns of a last block, which hold no infinity of another row."""
    codes, scales, cd, sd = _weight(160, 208, "block")
    codes[5] = 0x38                                                   # 1.0, so that the row is the sum of x
    cd = to_dev(codes)
    xb = W.activation(2, m, 208)
    xb[m // 2, 0], clean = 0x7F80, xb.copy()                          # +inf in the first column
    clean[m // 2] = 0
    want = F.fp8w_linear(to_dev_bf16(clean), cd, sd)
    got = F.fp8w_linear(to_dev_bf16(xb), cd, sd)
    rest = [i for i in range(m) if i != m // 2]
    assert torch.equal(got[rest], want[rest])
    assert got[m // 2, 5] == float("inf") and not torch.isfinite(got[m // 2]).any()
    xb[m // 2, 0] = 0x7FC0
    got = F.fp8w_linear(to_dev_bf16(xb), cd, sd)
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[m // 2]).all()


@pytest.mark.parametrize("k", [16, 208, 336, 400, 1040])
@pytest.mark.parametrize("m", [1, 20, 100, 300, 600])
@pytest.mark.parametrize("fmt", ["block", "mx"])
def test_infinities_in_any_column(F, fmt, m, k):
    """A column that is read in the place of one past the end may hold an infinity: it adds nothing twice."""
    codes, scales, _, sd = _weight(48, k, fmt)
    codes[:] = 0x38 | codes & 0x80                                    # 1.0 or -1.0
    cd = to_dev(codes)
    for col in (0, k - 16, k - 8, k - 1):
        xb = W.activation(2, m, k)
        xb[m // 2, col] = 0x7F80
        got = F.fp8w_linear(to_dev_bf16(xb), cd, sd, fmt).float().cpu().numpy()
        assert np.array_equal(got[m // 2], np.where(codes[:, col] < 0x80, np.inf, -np.inf)), col
        assert np.isfinite(np.delete(got, m // 2, 0)).all()


def test_rows_beyond_4_gib(F):
    """x, residual and y of rows far apart: the last begins past 2^32 bytes."""
    m, k, n, pitch = 18, 256, 96, (1 << 27) + 8
    codes, scales, cd, sd = _weight(n, k, "block")
    xb = W.activation(3, m, k)
    try:
        wide = torch.empty((m - 1) * pitch + k + n, dtype=BF16, device=dev())
    except torch.OutOfMemoryError:
        pytest.skip("needs 5 GiB")
    x, y = torch.as_strided(wide, (m, k), (pitch, 1)), torch.as_strided(wide, (m, n), (pitch, 1), k)
    r = torch.randn(m, n, generator=torch.Generator(device="cuda").manual_seed(1), device=dev()).to(BF16)
    x.copy_(to_dev_bf16(xb))
    y.copy_(r)
    want = F.fp8w_linear(x.contiguous(), cd, sd, residual=r)
    x2, y2 = x.contiguous(), torch.empty(m, n, dtype=BF16, device=dev())
    got = F.fp8w_linear(x, cd, sd, residual=r, y=y2)
    assert torch.equal(got, want)
    far = torch.as_strided(wide, (m, n), (pitch, 1), k)
    assert torch.equal(F.fp8w_linear(x2, cd, sd, residual=far, y=far), want)
    assert torch.equal(x, x2)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"])
@pytest.mark.parametrize("m", [1, 40])
def test_activations_far_out(F, act, m):
    """Products from -3e38 to 3e38, by columns of a weight of ones."""
    far = np.array([-3e38, -1e30, -200.0, -90.0, -20.0, -6.0, -1.0, -1e-30, 0.0, 1e-30, 1.0, 6.0, 20.0, 90.0, 200.0, 1e30])
    xb = np.zeros((m, 16), np.uint16)
    x = torch.from_numpy(far).to(BF16)
    xb[:] = np.diag(x.view(torch.int16).numpy().view(np.uint16)).sum(0)[None]
    codes = np.zeros((32, 16), np.uint8)
    codes[np.arange(16), np.arange(16)] = 0x38                         # gates: x's columns
    codes[np.arange(16, 32), 10] = 0x38                                # values: 1
    scales = np.ones((1, 1), np.float32)
    ref, err = D.linear(xb, codes, scales, "block", None, act)
    got = F.fp8w_linear(to_dev_bf16(xb), to_dev(codes), to_dev(scales), act=act, out_dtype=F32)
    _near(got, ref, err)


def test_no_rows(F):
    _, _, cd, sd = _weight(32, 64, "block")
    assert F.fp8w_linear(torch.empty(0, 64, dtype=BF16, device=dev()), cd, sd).shape == (0, 32)


def test_weight_method_and_refusals(F):
    w = F.Fp8Weight.quantize(to_dev_bf16(W.gaussian_weight(1, 0, 64, 128)), F.ROW)
    x = to_dev_bf16(W.activation(1, 5, 128))
    b = torch.ones(64, device=dev())
    assert torch.equal(w.linear(x, b, "gelu"), F.fp8w_linear(x, w.codes, w.scales, "row", b, "gelu"))
    for bad in (dict(bias=b[:60]), dict(act="tanh"), dict(residual=x), dict(y=x), dict(out_dtype=F32, y=torch.empty(5, 64, dtype=BF16, device=dev())),
                dict(x=x[:, ::2]), dict(x=x.float()), dict(bias=b.double()), dict(out_dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            w.linear(**{"x": x, **bad})
    room = torch.zeros(6 * 64, dtype=BF16, device=dev())
    with pytest.raises(F.Fp8wError):
        w.linear(x, residual=room[:320].view(5, 64), y=room[64:].view(5, 64))   # neither apart nor the same
    wide = torch.zeros(5, 132, dtype=BF16, device=dev())
    with pytest.raises(F.Fp8wError):
        w.linear(wide[:, :128])                                       # a stride that is no multiple of 8


@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (24, 512, 1024), (64, 256, 4096), (300, 384, 512)])
def test_repeatable_on_another_stream_and_in_a_graph(F, m, n, k):
    _, _, cd, sd = _weight(n, k, "block")
    x = to_dev_bf16(W.activation(1, m, k))
    b = torch.randn(n, device=dev())
    want = F.fp8w_linear(x, cd, sd, bias=b, act="silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.fp8w_linear(x, cd, sd, bias=b, act="silu", stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    need = F.lib().fp8w_linear_workspace_bytes(m, n, k, 0, 2)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev())
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp8w_linear(x, cd, sd, bias=b, act="silu", y=y, workspace=ws)
    for i in range(3):
        x.copy_(to_dev_bf16(W.activation(5 + i, m, k)))
        y.fill_(-1)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, F.fp8w_linear(x, cd, sd, bias=b, act="silu")), i
