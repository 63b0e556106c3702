"""The example with its shared expert, expert groups and drawn tokens: every new
stage against the 64-bit forms on the stage's own inputs, all of them together
eagerly, from a captured graph, and from two graphs on two streams at once."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from oracle import dense as D
from gpu_util import bf16_to_f64, dev

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_decode.py")


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    spec = importlib.util.spec_from_file_location("sparse_decode_drawn", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m
    spec.loader.exec_module(m)
    return m


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _settings(t):
    full = lambda v, d=torch.float32: torch.full((t,), v, dtype=d, device=dev())
    return dict(temperature=full(0.9), top_k=full(200, torch.int32), top_p=full(0.95), min_p=full(1e-3))


@pytest.mark.parametrize("fmt", ["block", "mx", "row"])
@pytest.mark.parametrize("t", [1, 5, 90])
def test_stages(ex, fmt, t):
    model = ex.SparseDecoder(vocab=700, d=160, f=64, experts=24, top_k=3, layers=1, fmt=fmt, shared=96, groups=6, top_groups=2)
    layer = model.layers[0]
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn(t, 160, generator=g, device=dev()).to(torch.bfloat16)
    n = ex.norm(x)
    router = n.float() @ layer.router.float().T
    r = ex.fp8w.fp8w_route_experts(router, 3, groups=6, top_groups=2)
    h = layer.shared_gate_up.linear(n, act="swiglu")
    y = layer.add_shared(n, x)
    logits = model.lm_head.linear(ex.norm(y), out_dtype=torch.float32)
    u = torch.rand(t, generator=g, device=dev())
    k = _settings(t)
    drawn = ex.fp8w.fp8w_sample(logits, u, **k)
    torch.cuda.synchronize()

    ids, _, slots, _, _ = D.route_grouped(router.cpu().numpy(), 3, 6, 2)
    assert np.array_equal(r.ids.cpu().numpy(), ids) and np.array_equal(r.slots.cpu().numpy(), slots)
    for q, src, act, add, got in ((layer.shared_gate_up, n, "swiglu", None, h), (layer.shared_down, h, "none", x, y),
                                  (model.lm_head, ex.norm(y), "none", None, logits)):
        ref, err = D.linear(_bits(src), q.codes.cpu().numpy(), _scales(q), q.format, None, act, None if add is None else bf16_to_f64(add))
        half = 2.0 ** -24 if got.dtype == torch.float32 else 2.0 ** -8
        got = got.double().cpu().numpy()
        assert (np.abs(got - ref) <= err + half * (np.abs(ref) + err)).all()
    tokens, logprob, kept = D.sample(logits.double().cpu().numpy(), u.cpu().numpy(), **{n: v.cpu().numpy() for n, v in k.items()})
    assert np.array_equal(drawn.tokens.cpu().numpy(), tokens) and np.array_equal(drawn.kept.cpu().numpy(), kept)
    assert (np.abs(drawn.logprob.double().cpu().numpy() - logprob) <= D.sample_tolerance(logprob, 700)).all()


def _scales(q):
    return q.scales.cpu().numpy()


def _eager(ex, model, token, u, k):
    return ex.fp8w.fp8w_sample(model.logits(token, torch.float32), u, **k)


@pytest.mark.parametrize("vocab", [3000, 60000])
@pytest.mark.parametrize("sequences", [1, 5, 40])
def test_drawing_from_a_graph_equals_eager_steps(ex, sequences, vocab):
    model = ex.SparseDecoder(vocab=vocab, d=256, f=128, experts=16, top_k=3, shared=192, groups=4, top_groups=2)
    k = _settings(sequences)
    step = ex.GraphedStep(model, sequences, 1, k)
    token = torch.arange(10, 10 + sequences, dtype=torch.int32, device=dev())
    step.token.copy_(token)
    random = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(5):
        step.uniforms.uniform_(generator=random)
        got = step()
        want = _eager(ex, model, token, step.uniforms, k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        token = want.tokens
        assert torch.equal(step.token, token) and (token >= 0).all()


def test_two_graphs_at_once(ex):
    """Each graph has workspaces of its own: replayed side by side they answer as they do alone."""
    model = ex.SparseDecoder(vocab=60000, d=256, f=128, experts=16, top_k=3, shared=192, groups=4, top_groups=2)
    k = _settings(3)
    steps = [ex.GraphedStep(model, 3, 1, k) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    tokens = [torch.arange(5, 8, dtype=torch.int32, device=dev()), torch.arange(20, 23, dtype=torch.int32, device=dev())]
    for i, s in enumerate(steps):
        s.token.copy_(tokens[i])
        s.uniforms.copy_(torch.rand(3, generator=torch.Generator(device="cuda").manual_seed(i), device=dev()))
    torch.cuda.synchronize()
    for _ in range(4):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s()
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            want = _eager(ex, model, tokens[i], s.uniforms, k)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(s.out, want)), i
            tokens[i] = want.tokens


def test_command(ex, capsys):
    text, total, scored = ex.main(["--sequences", "2", "--tokens", "3", "--shared", "128", "--groups", "4", "--top-groups", "2",
                                   "--temperature", "0.8", "--top-k", "50", "--top-p", "0.95"])
    assert text.shape == (2, 4) and torch.isfinite(total).all() and torch.isfinite(scored).all()
    assert "ms a step" in capsys.readouterr().out
