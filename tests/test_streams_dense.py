"""The dense product and drawn tokens on a stream that is not the current one:
what the calls make there is recorded, what they are given as well, and nothing
is on the current stream.  On the CPU, with a library that does nothing."""
import pytest
import torch

import fp8_block_scaled_02_amd as F

CURRENT, SIDE = 11, 22


class Library:
    def __getattr__(self, name):
        return lambda *a: 64 if name.endswith("_bytes") else 0


class Raw:
    """A stream of another library: a handle and nothing else."""
    cuda_stream = SIDE


@pytest.fixture
def calls(monkeypatch):
    made, recorded = [], []
    empty = torch.empty

    def counted(*a, **k):
        t = empty(*a, **k)
        made.append(t)
        return t
    monkeypatch.setattr(F, "lib", Library)
    monkeypatch.setattr(F, "_current_handle", lambda: CURRENT)
    monkeypatch.setattr(F, "_require", lambda t, *a: t)
    monkeypatch.setattr(F, "_rows_of", lambda t, dtypes, shape, what: t.shape[1])
    monkeypatch.setattr(F, "_on_current_device", lambda *a: None)
    monkeypatch.setattr(F, "_logits", lambda t, what: (1, t.shape[1]))
    monkeypatch.setattr(torch, "empty", counted)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t, s)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: ("stream", h))
    return made, recorded


X, CODES, SCALES = torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(1, 1)
CALLS = {
    "linear": (lambda s: F.fp8w_linear(X, CODES, SCALES, act="swiglu", bias=torch.zeros(64), stream=s), 2),
    "weight": (lambda s: F.Fp8Weight(CODES, SCALES, 64, 128, F.BLOCK128).linear(X, out_dtype=torch.float32, stream=s), 2),
    "sample": (lambda s: F.fp8w_sample(torch.zeros(3, 50), torch.zeros(3), stream=s), 4),
    "route": (lambda s: F.fp8w_route_experts(torch.zeros(40, 8), 2, groups=4, top_groups=2, stream=s), 6),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_made_on_another_stream(calls, name):
    made, recorded = calls
    call, count = CALLS[name]
    call(Raw())
    assert len(made) == count
    assert {t.data_ptr() for t, _ in recorded} == {t.data_ptr() for t in made}
    assert {s for _, s in recorded} == {("stream", SIDE)}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_made_on_the_current_stream(calls, name):
    made, recorded = calls
    call, count = CALLS[name]
    call(None)
    assert len(made) == count and recorded == []


def test_given_buffers(calls):
    made, recorded = calls
    y = torch.zeros(3, 64, dtype=torch.bfloat16)
    F.fp8w_linear(X, CODES, SCALES, y=y, stream=Raw())
    assert any(t is y for t, _ in recorded) and len(made) == 1 and any(t is made[0] for t, _ in recorded)
