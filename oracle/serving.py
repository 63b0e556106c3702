"""Plain 64-bit forms of the operators around the fp8 products: expert
routing, products grouped by expert, their weighted sum, and token log
probabilities -- TEST INFRASTRUCTURE ONLY, in numpy, written from the
definitions in ``include/fp8w.h`` and sharing no code with the library.

Where a result is inexact the functions also return the magnitude its error
is bounded by, as ``gemv_format_f64`` does."""
from __future__ import annotations

import numpy as np

from . import gemv_format_f64

EPS32 = 2.0 ** -23


def route(logits: np.ndarray, top_k: int, score: str = "softmax", bias=None, renorm: bool = True,
          scale: float = 1.0):
    """(ids, weights, slots, rows, offsets): ids, slots and the map as int
    arrays, the weights in fp64."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    ids = np.full((t, top_k), -1, np.int64)
    w = np.zeros((t, top_k))
    for r in range(t):
        live = x[r] > -np.inf                      # False for NaN too
        if not live.any():
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                p = np.where(live, np.exp(np.where(live, x[r] - x[r][live].max(), 0.0)), 0.0)
                p = p / p.sum()
            else:
                p = np.where(live, 1.0 / (1.0 + np.exp(np.where(live, -x[r], 0.0))), 0.0)
        key = x[r] if bias is None else p + np.asarray(bias, np.float64)
        order = sorted(np.flatnonzero(live & (key > -np.inf)), key=lambda i: (-key[i], i))[:top_k]
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
    pairs = sorted((ids[r, j], r, j) for r in range(t) for j in range(top_k) if ids[r, j] >= 0)
    slots = np.full((t, top_k), -1, np.int64)
    rows = np.full(t * top_k, -1, np.int64)
    offsets = np.zeros(e + 1, np.int64)
    for s, (i, r, j) in enumerate(pairs):
        slots[r, j], rows[s] = s, r
        offsets[i + 1] += 1
    return ids, w, slots, rows, np.cumsum(offsets)


def gemm_experts(x_bits, codes, scales, offsets, rows, fmt: str):
    """(y, bound) fp64 [slots, n]: the products and |x| . |deq W|^T; NaN for
    the slots that no expert has.  A row outside x is a row of zeros."""
    slots = len(rows)
    e, n, _ = codes.shape
    y, bound = np.full((slots, n), np.nan), np.full((slots, n), np.nan)
    for i in range(e):
        lo, hi = int(offsets[i]), int(offsets[i + 1])
        if hi <= lo:
            continue
        at = np.asarray(rows[lo:hi])
        there = (at >= 0) & (at < len(x_bits))
        xs = np.where(there[:, None], x_bits[np.where(there, at, 0)], 0).astype(np.uint16)
        y[lo:hi], bound[lo:hi] = gemv_format_f64(xs, codes[i], scales[i], fmt)
    return y, bound


def sum_error(k: int, bound):
    """What fp32 accumulation of k products (exact in fp32) and a few scale
    multiplications can add: a rounding of up to 2^-23 for each."""
    return (k + 8) * EPS32 * bound


def swiglu(y, err):
    """(silu(g) * u, its error) from the two halves of the products and
    theirs.  |silu'| < 1.1; the exponential, sum, quotient and product round
    by 16 * 2^-24 at most."""
    h = y.shape[1] // 2
    g, u = y[:, :h], y[:, h:]
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    eg, eu = 1.1 * err[:, :h], err[:, h:]
    return s * u, eg * np.abs(u) + np.abs(s) * eu + eg * eu + 8 * EPS32 * np.abs(s * u)


def combine(y, weights, slots):
    """(out, bound): the weighted sums and the sums of magnitudes."""
    t, k = slots.shape
    out, bound = np.zeros((t, y.shape[1])), np.zeros((t, y.shape[1]))
    for r in range(t):
        for j in range(k):
            if 0 <= slots[r, j] < len(y):
                v = np.float64(weights[r, j]) * y[slots[r, j]]
                out[r] += v
                bound[r] += np.abs(v)
    return out, bound


def logprobs(logits, targets, top: int):
    """(logprob, entropy, top_ids, top_logprobs), fp64 and int."""
    x = np.asarray(logits, np.float64)
    t, v = x.shape
    lp, ent = np.full(t, np.nan), np.full(t, np.nan)
    ids, best = np.zeros((t, top), np.int64), np.full((t, top), np.nan)
    for r in range(t):
        rank = np.where(np.isnan(x[r]), -np.inf, x[r])
        ids[r] = np.argsort(-rank, kind="stable")[:top]
        if np.isnan(x[r]).any() or np.isposinf(x[r]).any():
            continue
        if np.isneginf(x[r]).all():
            logp, ent[r] = np.full(v, -np.inf), 0.0
        else:
            m = x[r].max()
            logp = (x[r] - m) - np.log(np.exp(x[r] - m).sum())
            p = np.exp(logp)
            ent[r] = -(p * np.where(p > 0, logp, 0.0)).sum()
        if targets is not None and 0 <= targets[r] < v:
            lp[r] = logp[targets[r]]
        best[r] = logp[ids[r]]
    return lp, ent, ids, best


def logprobs_errors(logits):
    """What fp32 can add to each row's ln z (what its log probabilities share)
    and to its entropy; a log probability has one more rounding of itself.

    With d = max - x, a term is 2^(-d log2 e): the difference, the product and
    the constant are off by at most 2.5 * 2^-24 of d together, so a term by 2.5
    * 2^-24 * d of itself, however the running maximum got there and whatever
    the logits' own size.  Besides, the exponentials (one of its own, one for
    each new maximum) are good to a unit of 2^-23 each, and the sums round:
    16 values and two more operations a step of 8192 values, up to 19 joins.
    The entropy weighs its terms by d once more."""
    x = np.asarray(logits, np.float64)
    top = x.max(axis=1, keepdims=True)
    usable = np.isfinite(top)
    with np.errstate(invalid="ignore"):
        d = np.where(usable & (x > -np.inf), top - x, np.inf)
        p = np.exp(-d)
        z = p.sum(axis=1)
        z[z == 0] = 1.0
        far = np.where(p > 0, d, 0.0)
        mean, square = (p * far).sum(axis=1) / z, (p * far * far).sum(axis=1) / z
    n = 2.0 * -(-x.shape[1] // 8192) + 50
    err_z = EPS32 * (1.25 * mean + n)                      # relative
    err_ln = err_z + 2 * EPS32 * np.log(np.maximum(z, 1.0))
    return err_ln, err_ln + EPS32 * (1.25 * square + mean * (n + 2)) + mean * err_z


def logprobs_tolerance(logits, entropy):
    """The errors of a row's log probabilities and entropy, relative to 1 +
    their magnitude."""
    err_ln, err_h = logprobs_errors(logits)
    return np.maximum(err_ln + EPS32, err_h / (1 + np.nan_to_num(entropy)))
