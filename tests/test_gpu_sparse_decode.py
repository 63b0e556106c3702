"""The example that runs routing, the grouped products, the weighted sum, the
lm_head and log probabilities together: each stage against the 64-bit forms
on the stage's own inputs, and decoding from a captured graph against eager
steps."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S
from gpu_util import bf16_to_f64, dev

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_decode.py")


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    spec = importlib.util.spec_from_file_location("sparse_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m
    spec.loader.exec_module(m)
    return m


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("fmt", ["block", "mx", "row"])
@pytest.mark.parametrize("t", [1, 5, 90])
def test_layer_stages(ex, fmt, t):
    model = ex.SparseDecoder(vocab=500, d=160, f=64, experts=6, top_k=2, layers=1, fmt=fmt)
    layer, F = model.layers[0], ex.fp8w
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn(t, 160, generator=g, device=dev()).to(torch.bfloat16)
    logits = x.float() @ layer.router.float().T
    r = F.fp8w_route_experts(logits, 2)
    h = layer.gate_up.matmul(x, r.offsets, r.rows, act="swiglu")
    y = layer.down.matmul(h, r.offsets)
    out = layer(x)
    torch.cuda.synchronize()

    ids, w, slots, rows, offsets = S.route(logits.cpu().numpy(), 2)
    assert np.array_equal(r.ids.cpu().numpy(), ids) and np.array_equal(r.slots.cpu().numpy(), slots)
    for q, src, at, got, act in ((layer.gate_up, x, rows, h, True), (layer.down, h, np.arange(2 * t), y, False)):
        ref, bound = S.gemm_experts(_bits(src), q.codes.cpu().numpy(), q.scales.cpu().numpy(), offsets, at, fmt)
        err = S.sum_error(src.shape[1], bound)
        if act:
            ref, err = S.swiglu(ref, err)
        assert (np.abs(bf16_to_f64(got) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err) + 1e-38).all()
    ref, bound = S.combine(bf16_to_f64(y), r.weights.cpu().numpy(), slots)
    assert (np.abs(bf16_to_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * 2.0 ** -23 * bound + 1e-38).all()


def test_decoding_from_a_graph_equals_eager_steps(ex):
    model = ex.SparseDecoder(vocab=3000, d=256, f=128, experts=16, top_k=3)
    step = ex.GraphedStep(model, 5, 4)
    start = torch.arange(10, 15, dtype=torch.int32, device=dev())
    step.token.copy_(start)
    token = start
    for _ in range(6):
        got = step()
        want = ex.fp8w.fp8w_logprobs(model.logits(token), top=4)
        torch.cuda.synchronize()
        assert torch.equal(got.top_ids, want.top_ids) and torch.equal(got.top_logprobs, want.top_logprobs)
        assert torch.equal(got.entropy, want.entropy)
        token = want.top_ids[:, 0].contiguous()
        assert torch.equal(step.token, token)


def test_command(ex, capsys):
    text, total, scored = ex.main(["--sequences", "2", "--tokens", "3", "--fmt", "mx"])
    assert text.shape == (2, 4) and torch.isfinite(total).all() and torch.isfinite(scored).all()
    assert "ms a step" in capsys.readouterr().out
