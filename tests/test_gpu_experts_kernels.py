"""GPU parity of the products grouped by expert around the average group size
at which the kernel changes (8 / 9 and 112 / 113 slots an expert), for every
scale format and activation, halves that only the streaming kernel takes,
every e4m3 code, and drawn shapes; routing at the edges of its lane groups;
the weighted sum at every length of its row batches."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S
from fp8_block_scaled_02_amd import workloads as W
from gpu_util import bf16_to_f64, dev, to_dev, to_dev_bf16
from test_gpu_experts import _check as check_experts
from test_gpu_route import _check as check_route

pytestmark = pytest.mark.gpu
FORMATS = sorted(oracle.FORMATS)


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("sizes", [[17, 0, 7], [9, 1, 17], [200, 3, 181], [258, 0, 129]])
def test_formats_where_the_kernel_changes(F, sizes, act, fmt):
    check_experts(F, sizes, 320, 400, fmt, act)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("sizes", [[9, 8, 8], [9, 8, 10], [224, 112, 0], [226, 113, 0], [0, 0, 337]])
def test_sizes_next_to_the_changes(F, sizes, act, fmt):
    check_experts(F, sizes, 192, 272, fmt, act)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes", [[30, 9], [150, 170]])
def test_ragged_outputs_and_terms(F, sizes, fmt):
    check_experts(F, sizes, 258, 272, fmt)
    check_experts(F, sizes, 129, 48, fmt)
    check_experts(F, sizes, 130, 1040, fmt, "swiglu")      # halves of 65 rows
    check_experts(F, sizes, 8, 16, fmt, "swiglu")
    check_experts(F, sizes, 1, 4112, fmt, rows=None)


@pytest.mark.parametrize("fmt", ["block", "block_bf16"])
@pytest.mark.parametrize("half", [4, 12, 20, 36, 68, 140, 148])
def test_halves_off_the_scale_blocks_with_many_slots(F, half, fmt):
    check_experts(F, [40, 11, 90], 2 * half, 208, fmt, "swiglu")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("slots", [3, 60, 300])
def test_every_code(F, slots, fmt):
    """All 256 codes: finite ones exactly as decoded (NaN codes spoil their
    own row's outputs only)."""
    n, k = 96, 256
    codes = np.empty((2, n, k), np.uint8)
    codes[:, :, :] = np.random.default_rng(5).permutation(256).astype(np.uint8)
    codes[:, :-1][(codes[:, :-1] & 0x7F) == 0x7F] = 0        # NaN in the last row only
    shape = (2, *oracle.scale_shape(fmt, n, k))
    scales = np.full(shape, 127, np.uint8) if fmt == "mx" else np.ones(shape, np.float32)
    sd = torch.ones(shape, dtype=torch.bfloat16, device=dev()) if fmt == "block_bf16" else to_dev(scales)
    x = torch.zeros(slots, k, device=dev())
    pick = torch.arange(slots, device=dev()) * 7 % k
    x[torch.arange(slots, device=dev()), pick] = 1.0          # one code a slot: the product is the code
    off = torch.tensor([0, slots // 2, slots], dtype=torch.int32, device=dev())
    y = F.fp8w_gemm_experts(x.to(torch.bfloat16), to_dev(codes), sd, off, fmt=fmt)
    torch.cuda.synchronize()
    value = oracle.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64)
    want = value[codes[0][:, pick.cpu().numpy()]].T           # [slots, n]
    got = bf16_to_f64(y)
    assert np.array_equal(got[:, :-1], want[:, :-1])
    assert np.isnan(got[:, -1]).all()


@pytest.mark.parametrize("case", range(24))
def test_drawn_shapes(F, case):
    rng = np.random.default_rng(700 + case)
    e = int(rng.integers(1, 20))
    total = int(rng.choice([1, 5, 40, 300, 700]))
    sizes = rng.multinomial(total, rng.dirichlet(np.full(e, 0.5)))
    act = "swiglu" if case % 2 else "none"
    n = int(rng.integers(1, 150)) * 2
    k = int(rng.integers(1, 40)) * 16
    check_experts(F, list(sizes), n, k, FORMATS[case % len(FORMATS)], act, slots=total + int(rng.integers(0, 9)),
                  seed=case)


# ------------------------------------------------------------------ route --

@pytest.mark.parametrize("e,k", [(16, 16), (17, 17), (64, 16), (64, 17), (65, 16), (128, 16), (128, 17), (129, 16),
                                 (256, 16), (256, 17), (257, 16)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_lane_groups(F, e, k, biased):
    g = torch.Generator(device="cuda").manual_seed(e * 100 + k)
    bias = torch.randn(e, generator=g, device=dev()) if biased else None
    for t in (1, 3, 35):
        x = torch.randn(t, e, generator=g, device=dev())
        x[0, ::2] = -np.inf
        for score in ("softmax", "sigmoid"):
            check_route(F, x, k, score, bias=bias)
            check_route(F, x.to(torch.bfloat16), k, score, bias=bias, renorm=False)


def test_route_tokens_of_a_wave_differ_in_what_is_left(F):
    """Four tokens share a wave: none live, one, some, all; in every place."""
    g = torch.Generator(device="cuda").manual_seed(77)
    for shift in range(4):
        x = torch.randn(34, 50, generator=g, device=dev())
        for r in range(34):
            live = (0, 1, 3, 50)[(r + shift) % 4]
            x[r, torch.randperm(50, generator=g, device=dev())[live:]] = -np.inf
        check_route(F, x, 7)
        check_route(F, x, 7, "sigmoid", bias=torch.randn(50, generator=g, device=dev()))


# ---------------------------------------------------------------- combine --

@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 7, 8, 9, 11, 12, 13, 16, 17, 31, 63, 64])
@pytest.mark.parametrize("n", [8, 504, 520, 67])
def test_combine_row_batches(F, k, n):
    rng = np.random.default_rng(k * 1000 + n)
    t, m = 5, 40
    y = W.activation(68, m, n)
    slots = rng.integers(0, m, (t, k)).astype(np.int32)
    slots[rng.random((t, k)) < 0.2] = -1
    w = rng.standard_normal((t, k)).astype(np.float32)
    ref, bound = S.combine(oracle.bf16_to_f32(y).astype(np.float64).reshape(m, n), w, slots)
    out = F.fp8w_combine_experts(to_dev_bf16(y), to_dev(w), to_dev(slots))
    torch.cuda.synchronize()
    assert (np.abs(bf16_to_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * bound + 1e-38).all()


def test_combine_reads_nothing_for_no_slot(F):
    """A spoilt row 0 that no token names, and no rows at all."""
    y = torch.ones(4, 24, dtype=torch.bfloat16, device=dev())
    y[0] = float("nan")
    slots = torch.tensor([[-1, 1, -1], [-1, -1, -1], [2, 3, 4]], dtype=torch.int32, device=dev())
    w = torch.ones(3, 3, device=dev())
    out = F.fp8w_combine_experts(y, w, slots)
    assert out[:, 0].tolist() == [1.0, 0.0, 2.0] and (out == out[:, :1]).all()
    none = F.fp8w_combine_experts(y[:0], w, slots)
    assert none.shape == (3, 24) and (none == 0).all()


# --------------------------------------------------------------- refusals --

def test_refused_buffers_and_workspaces(F):
    """Nothing is launched with a buffer of another shape, type, place or
    layout, or with a workspace that the GPU cannot write."""
    x = torch.randn(40, 64, device=dev())
    i32 = dict(dtype=torch.int32, device=dev())
    for bad, error in ((torch.empty(40, 3, **i32), ValueError), (torch.empty(40, 4, device=dev()), TypeError),
                       (torch.empty(40, 4, dtype=torch.int32), ValueError), (torch.empty(4, 40, **i32).T, ValueError)):
        with pytest.raises(error, match="ids"):
            F.fp8w_route_experts(x, 4, ids=bad)
        with pytest.raises(error, match="top_ids"):
            F.fp8w_logprobs(x, top=4, top_ids=bad)
    for bad in (torch.empty(1 << 16, dtype=torch.uint8), torch.empty(1 << 9, 1 << 9, device=dev())[:, ::2]):
        with pytest.raises(ValueError, match="workspace"):
            F.fp8w_route_experts(x, 4, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            F.fp8w_logprobs(x, top=4, workspace=bad)
    with pytest.raises(F.Fp8wError):
        F.fp8w_route_experts(x, 4, workspace=torch.empty(3, dtype=torch.uint8, device=dev()))
