#!/usr/bin/env python3
"""Greedy decoding through layers of fp8 experts, with log probabilities.

A step of every sequence: router logits -> fp8w_route_experts ->
fp8w_gemm_experts (gate and up, SwiGLU) -> fp8w_gemm_experts (down) ->
fp8w_combine_experts, added to the stream of each layer; then the fp8 lm_head
(Fp8Weight.matmul) and fp8w_logprobs, whose first alternative is the next
token.  One step is captured in a HIP graph and replayed; the same step runs
eagerly on a whole prompt to score it.  Weights are random: the text is noise.

    python examples/sparse_decode.py [--sequences 4] [--tokens 16] [--fmt block]
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_02_amd as fp8w  # noqa: E402


@dataclass
class SparseLayer:
    """Router weight bf16 [E, d], and the experts' gate-and-up [E, 2f, d] and
    down [E, d, f] weights."""
    router: torch.Tensor
    gate_up: fp8w.Fp8Experts
    down: fp8w.Fp8Experts
    top_k: int

    def __call__(self, x):
        logits = x.float() @ self.router.float().T
        r = fp8w.fp8w_route_experts(logits, self.top_k)
        h = self.gate_up.matmul(x, r.offsets, r.rows, act="swiglu")
        y = self.down.matmul(h, r.offsets)            # slots in, slots out
        return fp8w.fp8w_combine_experts(y, r.weights, r.slots)


class SparseDecoder:
    def __init__(self, vocab=32000, d=1024, f=512, experts=32, top_k=4, layers=2, fmt="block", device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.embed = torch.randn(vocab, d, generator=g, device=device).to(torch.bfloat16)
        self.layers = [SparseLayer(weight(experts, d), fp8w.Fp8Experts.quantize(weight(experts, 2 * f, d), fmt),
                                   fp8w.Fp8Experts.quantize(weight(experts, d, f), fmt), top_k) for _ in range(layers)]
        self.lm_head = fp8w.Fp8Weight.quantize(weight(vocab, d))

    def logits(self, tokens):
        """bf16 [len(tokens), vocab]."""
        x = self.embed[tokens.long()]
        for layer in self.layers:
            x = x + layer(norm(x))
        return self.lm_head.matmul(norm(x))

    def score(self, tokens, top=0):
        """Log probability of each token of a prompt after the first, given
        the one before it."""
        return fp8w.fp8w_logprobs(self.logits(tokens[:-1]), tokens[1:].contiguous(), top)


def norm(x):
    v = x.float()
    return (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class GraphedStep:
    """One decoding step captured once: `token` is read and replaced."""

    def __init__(self, model: SparseDecoder, sequences: int, top: int):
        self.token = torch.zeros(sequences, dtype=torch.int32, device=model.embed.device)

        def step():
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
    args = ap.parse_args(argv)
    model = SparseDecoder(fmt=args.fmt)
    step = GraphedStep(model, args.sequences, max(args.top, 1))
    step.token.copy_(torch.arange(1, args.sequences + 1, dtype=torch.int32))
    text, total = [step.token.clone()], torch.zeros(args.sequences, device=step.token.device)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.tokens):
        out = step()
        text.append(step.token.clone())
        total += out.top_logprobs[:, 0]
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
