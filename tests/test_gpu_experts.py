"""GPU parity of the products grouped by expert and of the weighted sum of a
token's experts, against the 64-bit forms: every scale format, both outputs,
groups from none to several tiles, ragged n and k, indirect rows."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S
from fp8_block_scaled_02_amd import workloads as W
from gpu_util import bf16_to_f64, dev, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
FORMATS = sorted(oracle.FORMATS)


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


_weights = {}


def _experts(e, n, k, fmt):
    """(codes, scales) of e experts as numpy, and on the GPU."""
    key = (e, n, k, fmt)
    if key not in _weights:
        if len(_weights) > 40:
            _weights.clear()
        q = [oracle.quantize_format(W.gaussian_weight(60, i, n, k, outlier_rows=n >= 100), fmt) for i in range(e)]
        codes = np.stack([c for c, _ in q])
        scales = np.stack([np.asarray(s).reshape(oracle.scale_shape(fmt, n, k)) for _, s in q])
        sd = to_dev_bf16(scales) if fmt == "block_bf16" else to_dev(scales)
        _weights[key] = codes, scales, to_dev(codes), sd
    return _weights[key]


def _check(F, sizes, n, k, fmt, act="none", x_rows=None, rows="random", slots=None, seed=0):
    """One call with sizes[e] slots for expert e against the 64-bit form."""
    e, total = len(sizes), int(sum(sizes))
    slots = total if slots is None else slots
    rng = np.random.default_rng([seed, n, k, total])
    x_rows = max(slots, 1) if x_rows is None else x_rows
    x = W.activation(61 + seed, x_rows, k)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    at = rng.integers(0, x_rows, slots).astype(np.int32) if isinstance(rows, str) else rows
    codes, scales, cd, sd = _experts(e, n, k, fmt)
    n_out = n // 2 if act == "swiglu" else n
    y = torch.full((slots, n_out), 77.0, dtype=torch.bfloat16, device=dev())
    F.fp8w_gemm_experts(to_dev_bf16(x), cd, sd, to_dev(offsets), None if at is None else to_dev(at), fmt, act, y)
    torch.cuda.synchronize()
    got = bf16_to_f64(y)
    ref, bound = S.gemm_experts(x, codes, scales, offsets, np.arange(slots) if at is None else at, fmt)
    err = S.sum_error(k, bound)
    if act == "swiglu":
        ref, err = S.swiglu(ref, err)
    ref, err = ref[:total], err[:total]
    tol = err + 2.0 ** -8 * (np.abs(ref) + err) + 1e-38      # half a step of bf16
    bad = ~(np.abs(got[:total] - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), [tuple(map(int, i)) for i in np.argwhere(bad)[:4]], got[:total][bad][:4],
                           ref[bad][:4])
    assert (got[total:] == 77.0).all()                       # slots of no expert are not written
    return y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_formats(F, fmt, act):
    _check(F, [3, 0, 16, 1, 17], 260, 400, fmt, act)


@pytest.mark.parametrize("fmt", ["block", "mx", "row"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 64, 65, 127, 129, 200, 257])
def test_ragged_n(F, n, fmt):
    _check(F, [5, 1, 0, 18], n, 144, fmt)


@pytest.mark.parametrize("fmt", ["block", "mx", "row"])
@pytest.mark.parametrize("half", [1, 3, 16, 17, 63, 64, 100, 128, 190])
def test_swiglu_halves_that_split_a_scale_block(F, half, fmt):
    _check(F, [2, 9, 20], 2 * half, 272, fmt, "swiglu")


@pytest.mark.parametrize("fmt", ["block", "mx", "block_bf16"])
@pytest.mark.parametrize("k", [16, 32, 48, 112, 128, 144, 240, 256, 272, 496, 528, 1008, 1024, 1040, 2064, 4112])
def test_ragged_k(F, k, fmt):
    _check(F, [4, 0, 19], 72, k, fmt)


@pytest.mark.parametrize("sizes", [[0, 0, 0], [1], [0, 1, 0], [15, 16, 17], [31, 32, 33], [63, 64, 65],
                                   [127, 128, 129], [255, 0, 257], [0, 0, 300], [1] * 70, [3, 0] * 40])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_group_sizes(F, sizes, act):
    _check(F, sizes, 144, 288, "block", act, slots=max(sum(sizes), 1))


@pytest.mark.parametrize("avg", [1, 6, 12, 24, 48, 100, 200])
@pytest.mark.parametrize("fmt", ["block", "mx", "row"])
def test_uneven_groups_at_every_density(F, avg, fmt):
    rng = np.random.default_rng(avg)
    sizes = rng.multinomial(avg * 5, rng.dirichlet(np.ones(5)))
    _check(F, list(sizes), 320, 528, fmt, "swiglu" if avg % 8 else "none")
    _check(F, list(sizes), 514, 256, fmt, x_rows=7)


def test_one_expert_takes_all(F):
    _check(F, [0, 0, 0, 200, 0, 0, 0, 0], 272, 384, "block", "swiglu")
    _check(F, [64] + [0] * 63, 128, 128, "row")


def test_direct_rows_and_slots_of_no_expert(F):
    _check(F, [7, 0, 12], 96, 160, "block", rows=None, slots=30)
    _check(F, [40, 0, 90], 96, 160, "block", "swiglu", slots=150)


def test_rows_outside_x_are_zero(F):
    at = np.array([0, -1, 3, 4, 2**31 - 1, 1, -2**31, 2] * 5, np.int32)
    _check(F, [9, 31], 80, 192, "block", x_rows=4, rows=at)
    _check(F, [9, 31], 80, 192, "mx", "swiglu", x_rows=4, rows=at)


def test_offsets_outside_the_slots_are_cut(F):
    """Offsets that leave the slots or fall are cut to them: no write outside."""
    codes, scales, cd, sd = _experts(4, 48, 64, "row")
    x = to_dev_bf16(W.activation(62, 40, 64))
    room = torch.full((60, 48), 5.0, dtype=torch.bfloat16, device=dev())
    for off in ([-5, 3, 2, 50, 99], [0, 40, 40, 40, 2**31 - 1], [30, 20, 10, 0, -7]):
        F.fp8w_gemm_experts(x, cd, sd, torch.tensor(off, dtype=torch.int32, device=dev()), fmt="row", y=room[10:50])
        torch.cuda.synchronize()
        assert (room[:10] == 5).all() and (room[50:] == 5).all()


def test_infinite_inputs_stay_in_their_rows(F):
    """A row with an infinity or NaN spoils its own slots only."""
    k, n = 400, 96
    codes, scales, cd, sd = _experts(2, n, k, "block")
    x = W.activation(63, 30, k)
    off = torch.tensor([0, 20, 30], dtype=torch.int32, device=dev())
    clean = F.fp8w_gemm_experts(to_dev_bf16(x), cd, sd, off)
    x[4, 399], x[21, 3], x[29, 17] = 0x7F80, 0x7FC0, 0xFF80
    dirty = F.fp8w_gemm_experts(to_dev_bf16(x), cd, sd, off)
    torch.cuda.synchronize()
    keep = [i for i in range(30) if i not in (4, 21, 29)]
    assert torch.equal(clean[keep], dirty[keep]) and not torch.isfinite(dirty[[4, 21, 29]].float()).any(1).any()


def test_offsets_past_32_bits_of_weight_bytes(F):
    """Experts beyond 2^32 bytes of codes: the last one is read where it lies."""
    e, n, k = 70, 8192, 8192
    codes = torch.zeros(e, n, k, dtype=torch.uint8, device=dev())
    codes[-1, :, 5] = 0x38                                        # 1.0
    scales = torch.ones(e, n, device=dev())
    x = torch.randn(3, k, device=dev()).to(torch.bfloat16)
    off = torch.tensor([0] * e + [3], dtype=torch.int32, device=dev())
    y = F.fp8w_gemm_experts(x, codes, scales, off, fmt="row")
    assert torch.equal(y, x[:, 5:6].expand(3, n))


def test_repeatable_on_another_stream_and_in_a_graph(F):
    codes, scales, cd, sd = _experts(3, 260, 400, "block")
    x = to_dev_bf16(W.activation(64, 50, 400))
    off = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device=dev())
    rows = torch.arange(49, -1, -1, dtype=torch.int32, device=dev())
    want = F.fp8w_gemm_experts(x, cd, sd, off, rows, act="swiglu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.fp8w_gemm_experts(x, cd, sd, off, rows, act="swiglu", stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp8w_gemm_experts(x, cd, sd, off, rows, act="swiglu", y=y)
    for split in ([0, 20, 20, 50], [0, 0, 50, 50], [0, 1, 2, 50]):
        off.copy_(torch.tensor(split, dtype=torch.int32))
        y.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, F.fp8w_gemm_experts(x, cd, sd, off, rows, act="swiglu"))


def test_quantized_experts(F):
    w = to_dev_bf16(W.gaussian_weight(65, 0, 3 * 130, 272)).view(3, 130, 272)
    for fmt in FORMATS:
        q = F.Fp8Experts.quantize(w, fmt)
        for i in range(3):
            c, s = F.fp8w_quantize(w[i], fmt)
            assert torch.equal(q.codes[i], c) and torch.equal(q.scales[i], s)
        x = to_dev_bf16(W.activation(65, 4, 272))
        off = torch.tensor([0, 0, 4, 4], dtype=torch.int32, device=dev())
        y, one = q.matmul(x, off).float(), F.fp8w_gemv(x, q.codes[1], q.scales[1], fmt).float()
        assert (y - one).abs().max() <= 2.0 ** -7 * one.abs().max()   # two roundings of one product


# ---------------------------------------------------------------- combine --

@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (33, 6, 136), (100, 1, 1000), (257, 64, 24),
                                   (5, 3, 8192)])
def test_combine(F, t, k, n):
    rng = np.random.default_rng(t + n)
    m = t * k
    y = W.activation(66, m, n)
    slots = rng.permutation(m).reshape(t, k).astype(np.int32)
    slots[rng.random((t, k)) < 0.15] = -1
    w = rng.standard_normal((t, k)).astype(np.float32)
    if t > 2:
        slots[0], slots[1, 0] = -1, m                       # a token without experts; a slot past the end
        w[0], w[1, 0] = np.nan, np.inf                      # whose weights count for nothing
    out = F.fp8w_combine_experts(to_dev_bf16(y), to_dev(w), to_dev(slots))
    torch.cuda.synchronize()
    ref, bound = S.combine(oracle.bf16_to_f32(y).astype(np.float64).reshape(m, n), w, slots)
    assert (np.abs(bf16_to_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * bound + 1e-38).all()


def test_combine_unaligned_and_empty(F):
    y = to_dev_bf16(W.activation(67, 6, 16))
    slots = to_dev(np.array([[0, 5], [2, -1]], np.int32))
    w = to_dev(np.array([[0.5, 0.25], [2.0, 1.0]], np.float32))
    want = F.fp8w_combine_experts(y, w, slots)
    room = torch.zeros(2 * 16 + 3, dtype=torch.bfloat16, device=dev())
    got = F.fp8w_combine_experts(y, w, slots, out=room[3:].view(2, 16))     # 2-byte aligned
    assert torch.equal(got, want) and (room[:3] == 0).all()
    none = F.fp8w_combine_experts(y, w[:0].contiguous(), slots[:0].contiguous())
    assert none.shape == (0, 16)
