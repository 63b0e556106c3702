"""What a call makes for itself and uses on a stream that is not the current
one is recorded there, so that the allocator does not hand its memory out
while the kernels run.  On the CPU, with a library that does nothing: the
tensors that are made, and those that are recorded."""
import pytest
import torch

import fp8_block_scaled_02_amd as F

CURRENT, SIDE = 11, 22


class Library:
    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 64
        Current.order.append(name)
        return lambda *a: 0


class Raw:
    """A stream of another library: a handle and nothing else."""
    cuda_stream = SIDE


class Current:
    """The current stream; `order` is what happened to it and in the library."""
    order = []

    def synchronize(self):
        Current.order.append("synchronize")

    def __eq__(self, other):
        return isinstance(other, Current)


@pytest.fixture
def calls(monkeypatch):
    """(made, recorded): data pointers of the one, (data pointer, stream) of the other."""
    made, recorded = [], []
    empty = torch.empty

    def counted(*a, **k):
        t = empty(*a, **k)
        made.append(t)
        return t
    monkeypatch.setattr(F, "lib", Library)
    monkeypatch.setattr(F, "_current_handle", lambda: CURRENT)
    monkeypatch.setattr(F, "_require", lambda t, *a: t)
    monkeypatch.setattr(F, "_logits", lambda t, what: (1, t.shape[1]))
    monkeypatch.setattr(torch, "empty", counted)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t, s)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: ("stream", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "the default stream")
    monkeypatch.setattr(torch.cuda, "current_stream", Current)
    return made, recorded


n, k, m = 64, 128, 2
U8 = dict(dtype=torch.uint8)
w, x = torch.zeros(n, k, dtype=torch.bfloat16), torch.zeros(m, k, dtype=torch.bfloat16)
codes, block, mx = torch.zeros(n, k, **U8), torch.zeros(1, 1), torch.zeros(n, 4, **U8)
xc, xs = torch.zeros(m, k, **U8), torch.zeros(1)
offsets = torch.zeros(2, dtype=torch.int32)

CALLS = {
    "quantize": lambda s: F.fp8w_quantize(w, stream=s),
    "quantize_tensor": lambda s: F.fp8w_quantize(w, "tensor", stream=s),
    "quantize_block": lambda s: F.fp8w_quantize_block(w, stream=s),
    "quantize_mx": lambda s: F.fp8w_quantize_mx(w, stream=s),
    "quantize_act": lambda s: F.fp8w_quantize_act(x, stream=s),
    "dequantize": lambda s: F.fp8w_dequantize(codes, block, stream=s),
    "dequantize_block": lambda s: F.fp8w_dequantize_block(codes, block, stream=s),
    "dequantize_mx": lambda s: F.fp8w_dequantize_mx(codes, mx, stream=s),
    "gemv": lambda s: F.fp8w_gemv(x, codes, block, stream=s),
    "gemv_block": lambda s: F.fp8w_gemv_block(x, codes, block, stream=s),
    "gemv_mx": lambda s: F.fp8w_gemv_mx(x, codes, mx, stream=s),
    "gemm": lambda s: F.fp8w_gemm(x, codes, block, stream=s),
    "gemm_block": lambda s: F.fp8w_gemm_block(x, codes, block, stream=s),
    "gemm_mx": lambda s: F.fp8w_gemm_mx(x, codes, mx, stream=s),
    "gemv_w8a8": lambda s: F.fp8w_gemv_w8a8(xc, xs, codes, block, stream=s),
    "gemv_block_w8a8": lambda s: F.fp8w_gemv_block_w8a8(xc, xs, codes, block, stream=s),
    "gemv_mx_w8a8": lambda s: F.fp8w_gemv_mx_w8a8(xc, xs, codes, mx, stream=s),
    "route": lambda s: F.fp8w_route_experts(torch.zeros(40, 8), 2, stream=s),
    "gemm_experts": lambda s: F.fp8w_gemm_experts(x, codes[None], block[None], offsets, stream=s),
    "combine": lambda s: F.fp8w_combine_experts(x, torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.int32), stream=s),
    "logprobs": lambda s: F.fp8w_logprobs(torch.zeros(3, 50), torch.zeros(3, dtype=torch.int32), 4, stream=s),
    "experts": lambda s: F.Fp8Experts.quantize(torch.zeros(2, n, k, dtype=torch.bfloat16), stream=s),
    "experts_tensor": lambda s: F.Fp8Experts.quantize(torch.zeros(2, n, k, dtype=torch.bfloat16), "tensor", stream=s),
    "weight": lambda s: F.Fp8Weight.quantize(w, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream,recorded_as", [(Raw(), ("stream", SIDE)), (SIDE, ("stream", SIDE)),
                                                (0, "the default stream")])
def test_made_tensors_are_recorded(calls, name, stream, recorded_as):
    made, recorded = calls
    CALLS[name](stream)
    assert made and all(s == recorded_as for _, s in recorded)
    kept = {t.untyped_storage().data_ptr() for t, _ in recorded}
    assert {t.untyped_storage().data_ptr() for t in made if t.numel()} <= kept


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, CURRENT])
def test_nothing_is_recorded_on_the_current_stream(calls, name, stream):
    made, recorded = calls
    CALLS[name](stream)
    assert made and not recorded


PLANS = {
    "gemv": (lambda: F.fp8w_grouped_plan_init([x, x], [codes, codes], [block, block]), F.fp8w_gemv_grouped, 3),
    "quantize": (lambda: F.fp8w_quant_plan_init([w, w]), F.fp8w_quantize_grouped, 5),
}


@pytest.mark.parametrize("name", PLANS)
@pytest.mark.parametrize("stream,recorded_as", [(Raw(), ("stream", SIDE)), (SIDE, ("stream", SIDE)),
                                                (0, "the default stream"), (None, Current())])
def test_plans_are_recorded_once_a_stream(calls, name, stream, recorded_as):
    """Table and outputs, also on the current stream: the plan may have been
    made under another."""
    made, recorded = calls
    make, use, count = PLANS[name]
    plan = make()
    assert len(made) == count and not recorded
    use(plan, stream)
    assert {t.data_ptr() for t, _ in recorded} == {t.data_ptr() for t in made}
    assert all(s == recorded_as for _, s in recorded)
    use(plan, stream)
    assert len(recorded) == count
    use(plan, 33)
    assert len(recorded) == 2 * count and recorded[-1][1] == ("stream", 33)


@pytest.mark.parametrize("name", PLANS)
def test_tables_are_written_behind_the_current_stream(calls, name):
    """The set-up call writes the table at once; memory from the allocator may
    still be in use by what the current stream was given before."""
    Current.order.clear()
    PLANS[name][0]()
    assert Current.order == ["synchronize", {"gemv": "fp8w_grouped_plan_init", "quantize": "fp8w_quant_plan_init"}[name]]
