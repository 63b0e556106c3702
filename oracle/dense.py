"""Plain forms of a dense layer's product with its epilogue, of sampling and of
expert routing in groups -- TEST INFRASTRUCTURE ONLY, in numpy, written from the
definitions in ``include/fp8w.h`` and sharing no code with the library.

Sums and exponentials are taken in at least 64 bits.  Where a result is inexact
the functions also return what its error is bounded by."""
from __future__ import annotations

import math

import numpy as np

from . import gemv_format_f64
from .serving import EPS32, sum_error

GATED = ("swiglu", "geglu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


def activation(act: str, v):
    """(act(v), what fp32 evaluation of it adds to the error, relative to its
    value).  With t the sigmoid's argument, its roundings (three of them, each
    2^-24 of a term no larger than 3 |t|) move sigmoid(t) by at most their sum
    relative to itself; the exponential, sum, reciprocal and products round by
    16 * 2^-24.  erfc(z) moves by 2 z^2 2^-24 relative where z is rounded, and
    is good to 16 units."""
    if act == "none":
        return v, np.zeros_like(v)
    if act == "relu":
        return np.where(v > 0, v, 0.0 * v), np.zeros_like(v)
    with np.errstate(invalid="ignore", over="ignore"):
        if act == "gelu":
            z = -v * math.sqrt(0.5)
            return 0.5 * v * _erfc(z), (2 * z * z + 32) * 2.0 ** -24
        t = v if act in ("silu", "swiglu") else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return v * _sigmoid(t), (9 * np.abs(t) + 16) * 2.0 ** -24


def linear(x_bits, codes, scales, fmt: str, bias=None, act: str = "none", residual=None):
    """(y, err) in fp64: the values before the last rounding, and what fp32 may
    have added to them by then.  The derivatives of the activations are at
    most 1.13."""
    v, bound = gemv_rows(x_bits, codes, scales, fmt)
    err = sum_error(x_bits.shape[1], bound)
    if bias is not None:
        v = v + bias
        err = err + 2.0 ** -24 * (np.abs(v) + err)
    h = v.shape[1] // 2
    if act in GATED:
        g, eg, u, eu = v[:, :h], err[:, :h], v[:, h:], err[:, h:]
        s, rel = activation(act, g)
        es = 1.13 * eg + rel * (np.abs(s) + 1.13 * eg)
        y = s * u
        err = es * (np.abs(u) + eu) + np.abs(s) * eu + 2.0 ** -23 * np.abs(y)
    else:
        y, rel = activation(act, v)
        if act != "none":
            err = 1.13 * err + rel * (np.abs(y) + 1.13 * err)
    if residual is not None:
        y = y + residual
        err = err + 2.0 ** -24 * (np.abs(y) + err)
    return y, err + 2.0 ** -125


def gemv_rows(x_bits, codes, scales, fmt: str):
    """The products and |x| . |deq W|^T, 32 rows of x at a time."""
    parts = [gemv_format_f64(x_bits[i:i + 32], codes, scales, fmt) for i in range(0, len(x_bits), 32)]
    return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])


def weight_bits(vocab: int) -> int:
    """Fraction bits of the library's weights."""
    return min(50, 62 - max(0, math.ceil(math.log2(vocab))))


def sample(logits, uniforms, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, logprob, kept) of float rows, one at a time."""
    t, vocab = logits.shape
    tokens, logprob, kept = np.full(t, -1, np.int64), np.full(t, -np.inf), np.zeros(t, np.int64)
    for r in range(t):
        x = np.asarray(logits[r], np.float64)
        x = np.where(np.isnan(x), -np.inf, x)
        order = np.argsort(-x, kind="stable")
        order = order[x[order] > -np.inf]
        if len(order) == 0:
            continue
        x = x[order]
        temp = 1.0 if temperature is None else float(temperature[r])
        if not temp > 0:
            tokens[r], logprob[r], kept[r] = order[0], 0.0, 1
            continue
        with np.errstate(invalid="ignore"):
            d = np.where(x == x[0], 0.0, x - x[0])
            scaled = np.where(np.isinf(d), d, d / temp)   # beside +inf nothing else has weight, at no temperature
        n = len(x)
        if top_k is not None and top_k[r] > 0:
            n = min(n, int(top_k[r]))
        w = np.exp(scaled.astype(np.longdouble))
        upto = w.cumsum()
        stop = n
        if top_p is not None and top_p[r] < 1:
            before = np.concatenate([[0], upto[:n - 1]])
            stop = min(stop, int((before < np.longdouble(top_p[r]) * upto[n - 1]).sum()))
        if min_p is not None and min_p[r] > 0:
            stop = min(stop, int((scaled >= math.log(float(min_p[r]))).sum()))
        stop = max(stop, 1)
        u = float(uniforms[r])
        goal = 0.0 if not u > 0 else np.longdouble(u) * upto[stop - 1]
        some = int((w[:stop] >= 2.0 ** -(weight_bits(vocab) + 1)).sum())   # of a weight that is not zero
        j = min(int((upto[:stop] <= goal).sum()), some - 1)
        tokens[r], kept[r] = order[j], stop
        logprob[r] = float(scaled[j] - np.log(upto[stop - 1]))
    return tokens, logprob, kept


def sample_tolerance(logprob, vocab: int):
    """A log probability is rounded once to fp32; the sum behind it is of at
    most `vocab` weights off by half a unit each, and at least 1.

    Where whole bins enter that sum, each weight is 1 + e times its bin's middle:
    e rounded to half of 2^-f (f = 31, two less for each doubling beyond 2^18
    tokens), with (0.021)^5 / 120 < 2^-34.7 left out of its series, 2^-41 of the
    middle's, and all of it at most e^0.021 of the weight: 1.03 (2^-(f+1) +
    2^-34.7 + 2^-41) < 2^-f of the sum, and as much of its logarithm."""
    f = 31 - 2 * max(0, math.ceil(math.log2(vocab)) - 18)
    return (2.0 ** -24 * np.abs(np.where(np.isfinite(logprob), logprob, 0)) + vocab * 2.0 ** -(weight_bits(vocab) + 1)
            + 2.0 ** -f + 2.0 ** -40)


def route_grouped(logits, top_k: int, groups: int, top_groups: int, by: str = "max", score: str = "softmax", bias=None,
                  renorm: bool = True, scale: float = 1.0):
    """(ids, weights, slots, rows, offsets) of a choice within each token's best
    groups, the weights in fp64."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    ids, w = np.full((t, top_k), -1, np.int64), np.zeros((t, top_k))
    for r in range(t):
        live = x[r] > -np.inf
        if not live.any():
            continue
        safe = np.where(live, x[r], 0.0)
        if score == "softmax":
            top = safe[live].max()
            with np.errstate(invalid="ignore"):
                p = np.where(live, np.exp(np.where(safe == top, 0.0, np.minimum(safe - top, 0.0))), 0.0)
            p = p / p.sum()
        else:
            p = np.where(live, _sigmoid(safe), 0.0)
        key = safe if bias is None else p + np.asarray(bias, np.float64)
        value = p if bias is None and by == "top2" else key
        live &= key > -np.inf
        parts = np.arange(e) // (e // groups)
        rating = []
        for g in range(groups):
            best = np.sort(value[live & (parts == g)])[::-1]
            rating.append(-np.inf if len(best) == 0 else best[0] if by == "max" else best[:2].sum())
        best = sorted(range(groups), key=lambda g: (-rating[g], g))[:top_groups]
        live &= np.isin(parts, best)
        order = sorted(np.flatnonzero(live), key=lambda i: (-key[i], i))[:top_k]
        ids[r, :len(order)] = order
        w[r, :len(order)] = p[order]
        if renorm and len(order):
            if score == "softmax":                 # of the chosen alone, however far below the best
                c = np.exp(x[r, order] - x[r, order].max())
                w[r, :len(order)] = c / c.sum()
            elif p[order].max() < 2.0 ** -150:     # zero in fp32: no ratio
                w[r] = 0.0
            else:
                w[r] /= p[order].sum()
    w *= np.float64(np.float32(scale))
    flat = ids.reshape(-1)
    order = [i for i in np.argsort(flat, kind="stable") if flat[i] >= 0]
    slots, rows = np.full(t * top_k, -1, np.int64), np.full(t * top_k, -1, np.int64)
    slots[order] = np.arange(len(order))
    rows[:len(order)] = np.array(order, np.int64) // top_k
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=e))])
    return ids, w, slots.reshape(t, top_k), rows, offsets
