#!/usr/bin/env python3
"""Decoding through layers of fp8 experts, greedy or drawn, with log probabilities.

A step of every sequence: router logits -> fp8w_route_experts ->
fp8w_gemm_experts (gate and up, SwiGLU) -> fp8w_gemm_experts (down) ->
fp8w_combine_experts, added to the stream of each layer; then the fp8 lm_head
(Fp8Weight.matmul) and fp8w_logprobs, whose first alternative is the next
token.  One step is captured in a HIP graph and replayed; the same step runs
eagerly on a whole prompt to score it.  Weights are random: the text is noise.

With --shared a layer also has an expert that every token takes
(Fp8Weight.linear: gate and up with SwiGLU, then down, added to the stream in
the product's epilogue); with --groups the experts are chosen from each
token's best groups; with --temperature tokens are drawn (fp8w_sample) from
fp32 logits instead of taken.

    python examples/sparse_decode.py [--sequences 4] [--tokens 16] [--fmt block]
        [--shared 512] [--groups 8 --top-groups 4]
        [--temperature 0.8 --top-k 50 --top-p 0.95 --min-p 0]
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass
from typing import Optional

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_02_amd as fp8w  # noqa: E402

FORMATS = {"block": fp8w.BLOCK128, "mx": fp8w.MX32, "block_bf16": fp8w.BLOCK128_BF16, "row": fp8w.ROW, "tensor": fp8w.TENSOR}


@dataclass
class SparseLayer:
    """Router weight bf16 [E, d], and the experts' gate-and-up [E, 2f, d] and
    down [E, d, f] weights; of the expert that all tokens take, if there is
    one, [2s, d] and [d, s]."""
    router: torch.Tensor
    gate_up: fp8w.Fp8Experts
    down: fp8w.Fp8Experts
    top_k: int
    shared_gate_up: Optional[fp8w.Fp8Weight] = None
    shared_down: Optional[fp8w.Fp8Weight] = None
    groups: int = 1
    top_groups: Optional[int] = None

    def __call__(self, x):
        """What the chosen experts make of x."""
        logits = x.float() @ self.router.float().T
        r = fp8w.fp8w_route_experts(logits, self.top_k, groups=self.groups, top_groups=self.top_groups)
        h = self.gate_up.matmul(x, r.offsets, r.rows, act="swiglu")
        y = self.down.matmul(h, r.offsets)            # slots in, slots out
        return fp8w.fp8w_combine_experts(y, r.weights, r.slots)

    def add_shared(self, x, stream):
        """`stream` and what the shared expert makes of x."""
        if self.shared_gate_up is None:
            return stream
        return self.shared_down.linear(self.shared_gate_up.linear(x, act="swiglu"), residual=stream)


class SparseDecoder:
    def __init__(self, vocab=32000, d=1024, f=512, experts=32, top_k=4, layers=2, fmt="block", device="cuda:0", seed=0,
                 shared=0, groups=1, top_groups=None):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.embed = torch.randn(vocab, d, generator=g, device=device).to(torch.bfloat16)
        self.layers = [SparseLayer(weight(experts, d), fp8w.Fp8Experts.quantize(weight(experts, 2 * f, d), fmt),
                                   fp8w.Fp8Experts.quantize(weight(experts, d, f), fmt), top_k) for _ in range(layers)]
        self.lm_head = fp8w.Fp8Weight.quantize(weight(vocab, d))
        for layer in self.layers:
            layer.groups, layer.top_groups = groups, top_groups
            if shared:
                layer.shared_gate_up = fp8w.Fp8Weight.quantize(weight(2 * shared, d), FORMATS[fmt])
                layer.shared_down = fp8w.Fp8Weight.quantize(weight(d, shared), FORMATS[fmt])

    def logits(self, tokens, dtype=torch.bfloat16):
        """bf16 or fp32 [len(tokens), vocab]."""
        x = self.embed[tokens.long()]
        for layer in self.layers:
            n = norm(x)
            x = layer.add_shared(n, x) + layer(n)
        if dtype is torch.bfloat16:
            return self.lm_head.matmul(norm(x))
        return self.lm_head.linear(norm(x), out_dtype=dtype)

    def score(self, tokens, top=0):
        """Log probability of each token of a prompt after the first, given
        the one before it."""
        return fp8w.fp8w_logprobs(self.logits(tokens[:-1]), tokens[1:].contiguous(), top)


def norm(x):
    v = x.float()
    return (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class GraphedStep:
    """One decoding step captured once: `token` is read and replaced.  With
    `settings` (of fp8w_sample, a tensor each) tokens are drawn by `uniforms`,
    which the caller fills before each step."""

    def __init__(self, model: SparseDecoder, sequences: int, top: int, settings=None):
        self.token = torch.zeros(sequences, dtype=torch.int32, device=model.embed.device)
        self.uniforms = torch.zeros(sequences, device=model.embed.device)

        def step():
            if settings is not None:
                out = fp8w.fp8w_sample(model.logits(self.token, torch.float32), self.uniforms, **settings)
                self.token.copy_(out.tokens)
                return out
            out = fp8w.fp8w_logprobs(model.logits(self.token), top=top)
            self.token.copy_(out.top_ids[:, 0])
            return out

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = step()

    def __call__(self):
        self.graph.replay()
        return self.out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--fmt", default="block", choices=sorted(fp8w.FORMAT_IDS))
    ap.add_argument("--top", type=int, default=3)
    ap.add_argument("--shared", type=int, default=0, help="width of an expert that all tokens take")
    ap.add_argument("--groups", type=int, default=1)
    ap.add_argument("--top-groups", type=int, default=None)
    ap.add_argument("--temperature", type=float, default=0.0, help="0: the most likely token")
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args(argv)
    model = SparseDecoder(fmt=args.fmt, shared=args.shared, groups=args.groups, top_groups=args.top_groups)
    settings = None
    if args.temperature > 0:
        def rows(value, dtype=torch.float32):
            return torch.full((args.sequences,), value, dtype=dtype, device=model.embed.device)
        settings = dict(temperature=rows(args.temperature), top_k=rows(args.top_k, torch.int32), top_p=rows(args.top_p),
                        min_p=rows(args.min_p))
    step = GraphedStep(model, args.sequences, max(args.top, 1), settings)
    random = torch.Generator(device=model.embed.device).manual_seed(args.seed)
    step.token.copy_(torch.arange(1, args.sequences + 1, dtype=torch.int32))
    text, total = [step.token.clone()], torch.zeros(args.sequences, device=step.token.device)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.tokens):
        if settings is not None:
            step.uniforms.uniform_(generator=random)
        out = step()
        text.append(step.token.clone())
        total += out.top_logprobs[:, 0] if settings is None else out.logprob
    torch.cuda.synchronize()
    ms = (time.perf_counter() - start) / max(args.tokens, 1) * 1e3
    text = torch.stack(text, 1)
    scored = torch.stack([model.score(row.contiguous()).logprob.sum() for row in text])
    for i in range(args.sequences):
        print(f"sequence {i}: log p {total[i]:.3f} while decoding, {scored[i]:.3f} scored at once: {text[i].tolist()}")
    print(f"{ms:.3f} ms a step of {args.sequences} sequences")
    return text, total, scored


if __name__ == "__main__":
    main()
