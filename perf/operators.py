"""Cases of the operators around fp8 expert weights and the answer's scores.

Four operators are measured, each by the call a user's program makes:

* ``route``    router logits [T, E] -> the top experts of each token, their
               weights, and the map that sorts (token, choice) pairs by expert;
* ``experts``  the products grouped by expert, y[i] = x[rows[i]] . deq(W_e)^T
               for the slots i of expert e, fp8 weights in any scale format,
               plain or with the gated SiLU of two stacked halves;
* ``combine``  out[t] = sum_j weights[t, j] * y[slots[t, j]];
* ``logprobs`` lm_head logits [T, V] -> log probability of a given token,
               entropy, and the best alternatives of each row.

``run`` computes them in elementary torch operations where ``own`` is false
and by the library's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
FMAX = 448.0   # largest e4m3fn value


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decode step: the latency of choosing its experts
        dict(name="route_token", op="route", t=1, e=128, k=8, dtype="f32", score="softmax", bias=False, renorm=True),
        # a chunk of prefill, logits straight from a bf16 product
        dict(name="route_chunk", op="route", t=8192, e=128, k=8, dtype="bf16", score="softmax", bias=False, renorm=True),
        # a mixed batch on an odd number of experts, chosen with a load-balancing bias
        dict(name="route_biased", op="route", t=777, e=60, k=6, dtype="f32", score="sigmoid", bias=True, renorm=True),
        # one token: eight experts' gate and up weights, read once
        dict(name="experts_token", op="experts", t=1, e=64, k=8, n=2048, kk=2048, fmt="block", act="swiglu"),
        # a decode batch that reaches nearly every expert with a few rows each
        dict(name="experts_decode", op="experts", t=32, e=128, k=8, n=1536, kk=2048, fmt="block", act="swiglu"),
        # the down product of an odd batch, MX weights
        dict(name="experts_batch_mx", op="experts", t=301, e=64, k=8, n=2048, kk=1024, fmt="mx", act="none"),
        # prefill: gate and up products, hundreds of rows per expert
        dict(name="experts_prefill", op="experts", t=4096, e=64, k=8, n=2048, kk=2048, fmt="block", act="swiglu"),
        # the same chunk's down product, per-row scales
        dict(name="experts_prefill_row", op="experts", t=4096, e=64, k=8, n=2048, kk=1024, fmt="row", act="none"),
        # the experts' answers of a decode batch and of a prefill chunk added up
        dict(name="combine_decode", op="combine", t=32, k=8, n=2048, drop=0.0),
        dict(name="combine_chunk", op="combine", t=8192, k=8, n=2048, drop=0.02),
        # the sampled tokens of a small batch, with top alternatives
        dict(name="logprobs_step", op="logprobs", t=4, v=151936, pad=0, top=20, dtype="bf16", masked=0.0),
        # scoring a prompt: every position's next token
        dict(name="logprobs_prompt", op="logprobs", t=2048, v=151936, pad=0, top=5, dtype="bf16", masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "combine", "logprobs", "logprobs"])
    if op == "route":
        e = _log_int(rng, 8, 256)
        return dict(op=op, t=_log_int(rng, 1, 8192), e=e, k=rng.randint(1, min(8, e)), dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4, renorm=rng.random() < 0.7)
    if op == "combine":
        return dict(op=op, t=_log_int(rng, 1, 8192), k=rng.randint(1, 8), n=_log_int(rng, 256, 2048),
                    drop=rng.choice([0.0, 0.05]))
    if op == "logprobs":
        v = _log_int(rng, 1000, 151936)
        return dict(op=op, t=_log_int(rng, 1, 1024), v=v, pad=rng.choice([0, 0, 8, 61]), top=rng.randint(0, 20),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), masked=rng.choice([0.0, 0.0, 0.6]))
    while True:
        e = rng.choice([8, 16, 30, 64, 128])
        act = rng.choice(["none", "swiglu"])
        n = _log_int(rng, 64, 4096) // (2 if act == "swiglu" else 1) * (2 if act == "swiglu" else 1)
        c = dict(op=op, t=_log_int(rng, 1, 4096), e=e, k=rng.randint(1, 8), n=n, kk=16 * _log_int(rng, 8, 256),
                 fmt=rng.choice(["block", "block", "mx", "row", "block_bf16", "tensor"]), act=act)
        if 2 * c["t"] * c["k"] * c["n"] * c["kk"] <= 2.7e11 and e * c["n"] * c["kk"] <= 4e8:
            return c


def work(case):
    c = case
    if c["op"] == "route":
        t, e, k = c["t"], c["e"], c["k"]
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=t * e * size + t * k * 16 + (e + 1) * 4, flops=t * e * 4 + t * k * e)
    if c["op"] == "combine":
        t, k, n = c["t"], c["k"], c["n"]
        return dict(bytes=t * k * n * 2 * (1 - c["drop"]) + t * n * 2 + t * k * 8, flops=2 * t * k * n)
    if c["op"] == "logprobs":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["t"] * c["v"] * size + c["t"] * (12 + 8 * c["top"]), flops=c["t"] * c["v"] * 6)
    t, e, k, n, kk = c["t"], c["e"], c["k"], c["n"], c["kk"]
    hit = e * (1 - (1 - k / e) ** t)   # experts that some token chooses, were the choices even
    scales = {"block": 4 / 16384, "block_bf16": 2 / 16384, "mx": 1 / 32, "row": 4 / kk, "tensor": 0}[c["fmt"]]
    out = n // 2 if c["act"] == "swiglu" else n
    return dict(bytes=hit * n * kk * (1 + scales) + t * kk * 2 + t * k * (out * 2 + 4) + 4 * e,
                flops=2 * t * k * n * kk)


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _spread(v, n, k):
    """A [E, ceil(n/128), ceil(k/128)] grid widened to the [E, n, k] elements it covers."""
    return v.repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]


def _tiles_amax(w):
    e, n, k = w.shape
    p = torch.nn.functional.pad(w.abs(), (0, -k % 128, 0, -n % 128))
    return p.view(e, p.shape[1] // 128, 128, p.shape[2] // 128, 128).amax((2, 4))


def _quantized(w, fmt):
    """Codes and scales of bf16-valued weights [E, N, K], as load time leaves them."""
    e, n, k = w.shape
    if fmt in ("block", "block_bf16"):
        s = _tiles_amax(w) / FMAX
        s = torch.where(s > 0, s, torch.ones_like(s))
        if fmt == "block_bf16":
            s = s.to(torch.bfloat16)
        per = _spread(s.float(), n, k)
    elif fmt == "mx":
        p = torch.nn.functional.pad(w.abs(), (0, -k % 32)).view(e, n, -1, 32).amax(3)
        ex = torch.ceil(torch.log2(p.double() / FMAX)).clamp(-127, 127)
        s = (ex + 127).to(torch.uint8)
        per = torch.exp2(ex).float().repeat_interleave(32, 2)[:, :, :k]
    elif fmt == "row":
        s = w.abs().amax(2) / FMAX
        per = s[:, :, None]
    else:
        s = w.abs().amax((1, 2)) / FMAX
        per = s[:, None, None]
        s = s[:, None]
    codes = (w / per).clamp(-FMAX, FMAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), s.contiguous()


def _routed(g, t, e, k):
    """A router's answer: token of each slot (sorted by expert) and the experts' offsets."""
    logits = torch.randn(t, e, generator=g, device=DEV) + 0.5 * torch.randn(e, generator=g, device=DEV)
    ids = logits.topk(k, 1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    count = torch.zeros(e, dtype=torch.int64, device=DEV).index_add_(0, ids, torch.ones_like(ids))
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    return (order // k).int().contiguous(), offsets.int().contiguous(), order


def _room(*shape, dtype=torch.int32):
    """An output buffer, as a serving program keeps one from step to step."""
    return torch.empty(shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "route":
        logits = (torch.randn(c["t"], c["e"], generator=g, device=DEV) * 1.5).to(_dtype(c["dtype"]))
        bias = 0.1 * torch.randn(c["e"], generator=g, device=DEV) if c["bias"] else None
        t, k = c["t"], c["k"]
        kept = dict(ids=_room(t, k), weights=_room(t, k, dtype=torch.float32), slots=_room(t, k), rows=_room(t * k),
                    offsets=_room(c["e"] + 1))
        return dict(case=c, logits=logits, bias=bias, kept=kept)
    if c["op"] == "combine":
        t, k, n = c["t"], c["k"], c["n"]
        y = torch.randn(t * k, n, generator=g, device=DEV).to(torch.bfloat16)
        w = torch.rand(t, k, generator=g, device=DEV) + 0.05
        w = w / w.sum(1, keepdim=True)
        slots = torch.randperm(t * k, generator=g, device=DEV).int().view(t, k)
        if c["drop"]:
            slots = torch.where(torch.rand(t, k, generator=g, device=DEV) < c["drop"], -1, slots).int()
        out = _room(t, n, dtype=torch.bfloat16)
        return dict(case=c, y=y, weights=w, slots=slots.contiguous(), out=out)
    if c["op"] == "logprobs":
        t, v = c["t"], c["v"]
        full = torch.empty(t, v + c["pad"], dtype=_dtype(c["dtype"]), device=DEV)
        for r in range(0, t, 256):   # rows at a time: the fp32 samples of a long prompt stay small
            part = torch.randn(min(256, t - r), v + c["pad"], generator=g, device=DEV) * 2.5
            if c["masked"]:
                part[torch.rand(part.shape, generator=g, device=DEV) < c["masked"]] = -math.inf
            full[r:r + 256] = part.to(full.dtype)
        targets = torch.randint(0, v, (t,), generator=g, device=DEV).int()
        kept = dict(logprob=_room(t, dtype=torch.float32), entropy=_room(t, dtype=torch.float32),
                    top_ids=_room(t, c["top"]), top_logprobs=_room(t, c["top"], dtype=torch.float32))
        return dict(case=c, logits=full[:, :v], targets=targets, kept=kept)
    t, e, k, n, kk = c["t"], c["e"], c["k"], c["n"], c["kk"]
    x = torch.randn(t, kk, generator=g, device=DEV).to(torch.bfloat16)
    rows, offsets, _ = _routed(g, t, e, k)
    codes = torch.empty(e, n, kk, dtype=torch.uint8, device=DEV)
    scales = []
    for i in range(0, e, 16):   # 16 experts at a time
        w = (0.02 * torch.randn(min(16, e - i), n, kk, generator=g, device=DEV)).to(torch.bfloat16).float()
        q, s = _quantized(w, c["fmt"])
        codes[i:i + 16] = q
        scales.append(s)
    out = _room(t * k, n // 2 if c["act"] == "swiglu" else n, dtype=torch.bfloat16)
    return dict(case=c, x=x, rows=rows, offsets=offsets, codes=codes, scales=torch.cat(scales), out=out)


# ----------------------------------------------------------------- passes --

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _own_route(s):
    import fp8_block_scaled_02_amd as F
    c = s["case"]
    r = F.fp8w_route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], renorm=c["renorm"], **s["kept"])
    return dict(ids=r.ids, weights=r.weights, slots=r.slots, rows=r.rows, offsets=r.offsets)


def _own_experts(s):
    import fp8_block_scaled_02_amd as F
    c = s["case"]
    return dict(y=F.fp8w_gemm_experts(s["x"], s["codes"], s["scales"], s["offsets"], rows=s["rows"], fmt=c["fmt"],
                                      act=c["act"], y=s["out"]))


def _own_combine(s):
    import fp8_block_scaled_02_amd as F
    return dict(out=F.fp8w_combine_experts(s["y"], s["weights"], s["slots"], out=s["out"]))


def _own_logprobs(s):
    import fp8_block_scaled_02_amd as F
    r = F.fp8w_logprobs(s["logits"], s["targets"], top=s["case"]["top"], **s["kept"])
    return dict(logprob=r.logprob, entropy=r.entropy, top_ids=r.top_ids, top_logprobs=r.top_logprobs)


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    t, e, k = c["t"], c["e"], c["k"]
    key = x.double()   # the choice is made next to ties: in 64 bits
    if c["score"] == "softmax":
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
        if c["bias"]:
            key = torch.exp(key - key.amax(1, keepdim=True))
            key = key / key.sum(1, keepdim=True) + s["bias"].double()
    else:
        score = 1 / (1 + torch.exp(-x))
        if c["bias"]:
            key = 1 / (1 + torch.exp(-key)) + s["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    weights = score.gather(1, ids)
    if c["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(t * k, device=flat.device)
    count = torch.zeros(e, dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    return dict(ids=ids.int(), weights=weights, slots=slots.view(t, k).int(), rows=(order // k).int(),
                offsets=offsets.int())


def _weights_f32(codes, scales, fmt):
    e, n, k = codes.shape
    w = codes.view(torch.float8_e4m3fn).float()
    if fmt in ("block", "block_bf16"):
        return w * _spread(scales.float(), n, k)
    if fmt == "mx":
        return w * torch.exp2(scales.float() - 127).repeat_interleave(32, 2)[:, :, :k]
    return w * scales[:, :, None]   # one per row, or one per expert


def _plain_experts(s):
    c, offsets = s["case"], s["offsets"].long()
    slots = s["rows"].numel()
    at = torch.arange(slots, device=offsets.device)
    expert = torch.searchsorted(offsets[1:].contiguous(), at, right=True)
    place = at - offsets[expert]
    most = int((offsets[1:] - offsets[:-1]).max())
    xs = torch.zeros(c["e"], most, c["kk"], device=offsets.device)
    xs[expert, place] = s["x"][s["rows"].long()].float()
    y = torch.bmm(xs, _weights_f32(s["codes"], s["scales"], c["fmt"]).transpose(1, 2).contiguous())[expert, place]
    if c["act"] == "swiglu":
        gate, up = y.chunk(2, 1)
        y = gate / (1 + torch.exp(-gate)) * up
    return dict(y=y.to(torch.bfloat16))


def _plain_combine(s):
    slots = s["slots"].long()
    w = torch.where(slots >= 0, s["weights"], torch.zeros_like(s["weights"]))
    picked = s["y"][slots.clamp(min=0)].float()
    return dict(out=(picked * w[:, :, None]).sum(1).to(torch.bfloat16))


def _plain_logprobs(s):
    c, x = s["case"], s["logits"].float()
    v, top = c["v"], c["top"]
    m = x.amax(1, keepdim=True)
    ex = torch.exp(x - m)
    z = ex.sum(1, keepdim=True)
    logp = x - m - torch.log(z)
    entropy = -torch.where(ex > 0, ex / z * logp, torch.zeros_like(ex)).sum(1)
    logprob = logp.gather(1, s["targets"].long()[:, None])[:, 0]
    # unique keys, larger values first and lower places first among equals
    bits = x.view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    keys = bits * (1 << 24) + ((1 << 24) - 1 - torch.arange(v, device=x.device))
    ids = keys.topk(top, 1).indices
    return dict(logprob=logprob, entropy=entropy, top_ids=ids.int(), top_logprobs=logp.gather(1, ids))


_run_own = dict(route=_own_route, experts=_own_experts, combine=_own_combine, logprobs=_own_logprobs)
_run_plain = dict(route=_plain_route, experts=_plain_experts, combine=_plain_combine, logprobs=_plain_logprobs)


# ------------------------------------------------------- the definition, 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, experts=_exact_experts, combine=_exact_combine, logprobs=_exact_logprobs)[case["op"]](s)


def _exact_route(s):
    c, x = s["case"], s["logits"].double()
    p = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    want = p + s["bias"].double() if c["bias"] else x
    w = torch.zeros(c["t"], c["k"], dtype=torch.float64, device=x.device)
    left = want.clone()
    for j in range(c["k"]):
        i = left.argmax(1, keepdim=True)
        w[:, j] = p.gather(1, i)[:, 0]
        left.scatter_(1, i, -math.inf)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(ids=None, weights=w, slots=None, rows=None, offsets=None)


def _code_values():
    """e4m3fn: sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinities."""
    v = []
    for b in range(256):
        ex, man = (b >> 3) & 15, b & 7
        a = man / 8 * 2.0 ** -6 if ex == 0 else (1 + man / 8) * 2.0 ** (ex - 7)
        v.append(-a if b & 128 else a)
    return v


def _exact_experts(s):
    c = s["case"]
    table = torch.tensor(_code_values(), dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    y = torch.zeros(ends[-1], c["n"], dtype=torch.float64, device=DEV)
    kcol, nrow = torch.arange(c["kk"], device=DEV), torch.arange(c["n"], device=DEV)
    for e in range(c["e"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        w, sc = table[s["codes"][e].long()], s["scales"][e].double()
        if c["fmt"] in ("block", "block_bf16"):
            w = w * sc[nrow // 128][:, kcol // 128]
        elif c["fmt"] == "mx":
            w = w * (2.0 ** (sc - 127))[:, kcol // 32]
        else:
            w = w * sc.view(-1, 1)
        y[lo:hi] = s["x"][s["rows"][lo:hi].long()].double() @ w.T
    if c["act"] == "swiglu":
        h = c["n"] // 2
        y = y[:, :h] * torch.sigmoid(y[:, :h]) * y[:, h:]
    return dict(y=y)


def _exact_combine(s):
    c = s["case"]
    out = torch.zeros(c["t"], c["n"], dtype=torch.float64, device=DEV)
    for j in range(c["k"]):
        i = s["slots"][:, j].long()
        live = i >= 0
        out[live] += s["weights"][live, j, None].double() * s["y"][i[live]].double()
    return dict(out=out)


def _exact_logprobs(s):
    c = s["case"]
    lp, en, best = [], [], []
    for r in range(0, c["t"], 128):
        x = s["logits"][r:r + 128].double()
        logp = torch.log_softmax(x, 1)
        p = logp.exp()
        en.append(-(p * logp.masked_fill(p == 0, 0.0)).sum(1))
        lp.append(logp.gather(1, s["targets"][r:r + 128, None].long())[:, 0])
        best.append(logp.topk(c["top"], 1).values)
    return dict(logprob=torch.cat(lp), entropy=torch.cat(en), top_ids=None, top_logprobs=torch.cat(best))
