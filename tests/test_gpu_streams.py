"""Calls on a stream that is not the current one: what they made is not handed
out again while the stream is still busy, and their results are those of the
current stream's calls."""
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import fp8_block_scaled_02_amd as fp8w
    fp8w.lib()
    return fp8w


def _occupy(stream, a):
    """Some 20 ms of work that the calls behind it wait for."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(30):
            torch.mm(a, a)


@pytest.mark.parametrize("fmt", ["block", "mx", "block_bf16", "row", "tensor"])
@pytest.mark.parametrize("by", ["stream", "handle"])
def test_dropped_outputs_are_not_reused_early(F, fmt, by):
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device=dev())
    w = torch.randn(4, 512, 1024, device=dev()).to(torch.bfloat16)
    side = torch.cuda.Stream()
    torch.mm(a, a)
    want = F.Fp8Experts.quantize(w, fmt)
    torch.cuda.synchronize()
    _occupy(side, a)
    q = F.Fp8Experts.quantize(w, fmt, stream=side if by == "stream" else side.cuda_stream)
    at = q.codes.data_ptr()
    busy = not side.query()
    del q
    others = [torch.empty(4, 512, 1024, dtype=torch.uint8, device=dev()) for _ in range(3)]
    assert not busy or all(o.data_ptr() != at for o in others)
    side.synchronize()
    q = F.Fp8Experts.quantize(w, fmt, stream=side)
    side.synchronize()
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)


def test_default_stream_by_its_handle(F):
    """The handle 0 under another current stream is the default stream."""
    w = torch.randn(512, 1024, device=dev()).to(torch.bfloat16)
    want = F.fp8w_quantize(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = F.fp8w_quantize(w, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("by", ["stream", "handle", "current"])
def test_plans_dropped_behind_their_call(F, by):
    """A plan made and dropped around one call on a busy stream: its table,
    which names every buffer, is not reused before the call has run."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device=dev())
    ws = [torch.randn(256, 512, device=dev()).to(torch.bfloat16) for _ in range(5)]
    want = F.fp8w_quantize_grouped(F.fp8w_quant_plan_init(ws))
    x = torch.randn(2, 512, device=dev()).to(torch.bfloat16)
    ys = [y.clone() for y in F.fp8w_gemv_grouped(F.fp8w_grouped_plan_init([x] * 5, *want))]
    side = torch.cuda.Stream()
    torch.mm(a, a)
    torch.cuda.synchronize()
    plan, gemv = F.fp8w_quant_plan_init(ws), F.fp8w_grouped_plan_init([x] * 5, *want)
    table, other = plan.table.data_ptr(), gemv.table.data_ptr()
    _occupy(side, a)
    if by == "current":
        with torch.cuda.stream(side):
            got, out = F.fp8w_quantize_grouped(plan), F.fp8w_gemv_grouped(gemv)
    else:
        s = side if by == "stream" else side.cuda_stream
        got, out = F.fp8w_quantize_grouped(plan, s), F.fp8w_gemv_grouped(gemv, s)
    size = plan.table.numel(), gemv.table.numel()
    busy = not side.query()
    del plan, gemv
    fresh = [torch.empty(n, dtype=torch.uint8, device=dev()) for n in size for _ in range(4)]
    assert not busy or not {table, other} & {f.data_ptr() for f in fresh}
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got[0], *got[1]), (*want[0], *want[1])))
    assert all(torch.equal(p, q) for p, q in zip(out, ys))
