"""Cases of the operators of a dense fp8 layer and of the token it answers with.

Three operators are measured, each by the call a user's program makes:

* ``linear``  y = act(x . deq(W)^T + bias) + residual, fp8 weights in any scale
              format, any number of rows, bf16 or f32 results;
* ``sample``  logits [T, V] and one random number a row -> a token drawn under
              the row's temperature, top-k, top-p and min-p, its log
              probability, and how many tokens it was drawn from;
* ``route``   router logits [T, E] -> each token's experts, chosen within its
              best groups of experts.

``run`` computes them in elementary torch operations where ``own`` is false
and by the library's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
FMAX = 448.0   # largest e4m3fn value
GATED = ("swiglu", "geglu")


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's query, key and value projections, with their bias
        dict(name="linear_token", op="linear", m=1, n=6144, k=4096, fmt="block", act="none", bias="bf16", residual=False, out="bf16", pad=0),
        # a decode batch's down projection, added to the stream
        dict(name="linear_decode_down", op="linear", m=16, n=4096, k=12288, fmt="block", act="none", bias="none", residual=True, out="bf16", pad=0),
        # a full decode batch's gate and up projections
        dict(name="linear_decode_gate", op="linear", m=32, n=24576, k=4096, fmt="block", act="swiglu", bias="none", residual=False, out="bf16", pad=0),
        # the head of a small batch: logits in fp32 for the sampler
        dict(name="linear_head", op="linear", m=8, n=151936, k=2048, fmt="block", act="none", bias="none", residual=False, out="f32", pad=0),
        # an odd batch of short prompts, MX weights, x a part of wider rows
        dict(name="linear_batch_mx", op="linear", m=203, n=6144, k=4096, fmt="mx", act="gelu_tanh", bias="f32", residual=False, out="bf16", pad=64),
        # prefill: gate and up projections
        dict(name="linear_prefill", op="linear", m=2048, n=24576, k=4096, fmt="block", act="swiglu", bias="none", residual=False, out="bf16", pad=0),
        # an odd chunk's down projection, per-row scales, added to the stream
        dict(name="linear_prefill_row", op="linear", m=1777, n=4096, k=12288, fmt="row", act="none", bias="none", residual=True, out="bf16", pad=0),
        # a few sequences' next tokens, usual filters
        dict(name="sample_step", op="sample", t=4, v=151936, pad=0, dtype="bf16", filters="topk_topp"),
        # a serving batch, every row with settings of its own, greedy ones among them
        dict(name="sample_mixed", op="sample", t=64, v=151936, pad=0, dtype="f32", filters="mixed"),
        # many rollouts drawn from the whole distribution's nucleus
        dict(name="sample_nucleus", op="sample", t=512, v=32000, pad=0, dtype="bf16", filters="topp"),
        # one token on experts in groups, sigmoid scores and a balancing bias
        dict(name="route_groups_token", op="route", t=1, e=256, k=8, groups=8, top_groups=4, dtype="f32", score="sigmoid", bias=True, by="top2"),
        # a chunk of prefill, groups by their best expert
        dict(name="route_groups_chunk", op="route", t=4096, e=160, k=6, groups=8, top_groups=3, dtype="bf16", score="softmax", bias=False, by="max"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "linear", "sample", "sample", "sample", "route"])
    if op == "route":
        groups = rng.choice([2, 3, 4, 8, 16])
        e = groups * _log_int(rng, 2, 256 // groups)
        top_groups = rng.randint(1, groups)
        return dict(op=op, t=_log_int(rng, 1, 4096), e=e, k=rng.randint(1, min(8, e // groups * top_groups)), groups=groups,
                    top_groups=top_groups, dtype=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, by=rng.choice(["max", "top2"]))
    if op == "sample":
        while True:
            c = dict(op=op, t=_log_int(rng, 1, 512), v=_log_int(rng, 1000, 151936), pad=rng.choice([0, 0, 8, 61]),
                     dtype=rng.choice(["bf16", "f32"]), filters=rng.choice(["none", "topk", "topp", "minp", "topk_topp", "mixed"]))
            if c["t"] * c["v"] <= 1.6e7:
                return c
    while True:
        act = rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"])
        gated = act in GATED
        n = _log_int(rng, 64, 24576) // (2 if gated else 1) * (2 if gated else 1)
        c = dict(op=op, m=_log_int(rng, 1, 2048), n=n, k=16 * _log_int(rng, 8, 768),
                 fmt=rng.choice(["block", "block", "mx", "row", "block_bf16", "tensor"]), act=act,
                 bias=rng.choice(["none", "bf16", "f32"]), residual=rng.random() < 0.4, out=rng.choice(["bf16", "bf16", "f32"]),
                 pad=rng.choice([0, 0, 8, 128]))
        if 2 * c["m"] * c["n"] * c["k"] <= 4e11 and c["n"] * c["k"] <= 1.5e8:
            return c


def work(case):
    c = case
    if c["op"] == "route":
        t, e, k = c["t"], c["e"], c["k"]
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=t * e * size + t * k * 16 + (e + 1) * 4 + (4 * e if c["bias"] else 0), flops=t * e * 6 + t * k * e)
    if c["op"] == "sample":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["t"] * c["v"] * size + c["t"] * 32, flops=c["t"] * c["v"] * 8)
    m, n, k = c["m"], c["n"], c["k"]
    n_out = n // 2 if c["act"] in GATED else n
    scales = {"block": 4 / 16384, "block_bf16": 2 / 16384, "mx": 1 / 32, "row": 4 / k, "tensor": 0}[c["fmt"]]
    bias = {"none": 0, "bf16": 2, "f32": 4}[c["bias"]]
    out = (4 if c["out"] == "f32" else 2) + (2 if c["residual"] else 0)
    return dict(bytes=n * k * (1 + scales) + m * k * 2 + n * bias + m * n_out * out, flops=2 * m * n * k)


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _spread(v, n, k):
    """A [ceil(n/128), ceil(k/128)] grid widened to the [n, k] elements it covers."""
    return v.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def _quantized(w, fmt):
    """Codes and scales of bf16-valued weights [n, k], as load time leaves them."""
    n, k = w.shape
    if fmt in ("block", "block_bf16"):
        p = torch.nn.functional.pad(w.abs(), (0, -k % 128, 0, -n % 128))
        s = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128).amax((1, 3)) / FMAX
        s = torch.where(s > 0, s, torch.ones_like(s))
        if fmt == "block_bf16":
            s = s.to(torch.bfloat16)
        per = _spread(s.float(), n, k)
    elif fmt == "mx":
        p = torch.nn.functional.pad(w.abs(), (0, -k % 32)).view(n, -1, 32).amax(2)
        ex = torch.ceil(torch.log2(p.double() / FMAX)).clamp(-127, 127)
        s = (ex + 127).to(torch.uint8)
        per = torch.exp2(ex).float().repeat_interleave(32, 1)[:, :k]
    elif fmt == "row":
        s = w.abs().amax(1) / FMAX
        per = s[:, None]
    else:
        s = (w.abs().amax() / FMAX).view(1)
        per = s
    codes = (w / per).clamp(-FMAX, FMAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), s.contiguous()


def _room(*shape, dtype=torch.int32):
    """An output buffer, as a serving program keeps one from step to step."""
    return torch.empty(shape, dtype=dtype, device=DEV)


def _settings(c, g):
    """Each row's temperature, top-k, top-p and min-p, None where unused."""
    t, f = c["t"], c["filters"]

    def among(values, dtype=torch.float32):
        v = torch.tensor(values, dtype=dtype, device=DEV)
        return v[torch.randint(0, len(values), (t,), generator=g, device=DEV)].contiguous()
    if f == "mixed":
        return dict(temperature=among([0.0, 0.6, 0.8, 1.0, 1.5]), top_k=among([0, 1, 20, 50, 400], torch.int32),
                    top_p=among([1.0, 0.95, 0.8, 0.5]), min_p=among([0.0, 0.0, 0.02, 0.1]))
    return dict(temperature=among([0.7, 1.0]), top_k=among([40, 50], torch.int32) if "topk" in f else None,
                top_p=among([0.9, 0.95]) if "topp" in f else None, min_p=among([0.01, 0.05]) if f == "minp" else None)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "route":
        t, e, k = c["t"], c["e"], c["k"]
        logits = (torch.randn(t, e, generator=g, device=DEV) * 1.5).to(_dtype(c["dtype"]))
        bias = 0.1 * torch.randn(e, generator=g, device=DEV) if c["bias"] else None
        kept = dict(ids=_room(t, k), weights=_room(t, k, dtype=torch.float32), slots=_room(t, k), rows=_room(t * k),
                    offsets=_room(e + 1))
        return dict(case=c, logits=logits, bias=bias, kept=kept)
    if c["op"] == "sample":
        t, v = c["t"], c["v"]
        full = torch.empty(t, v + c["pad"], dtype=_dtype(c["dtype"]), device=DEV)
        for r in range(0, t, 128):   # rows at a time: the fp32 samples stay small
            n = min(128, t - r)
            part = torch.randn(n, v + c["pad"], generator=g, device=DEV) * 2.0
            # most rows have some likely tokens, from a clear favourite to dozens; the rest are flat
            likely = torch.randint(0, v, (n, 48), generator=g, device=DEV)
            lift = 4 - 4 * torch.log(torch.rand(n, 48, generator=g, device=DEV) + 1e-6)
            lift = lift * (torch.rand(n, 1, generator=g, device=DEV) < 0.8)
            part.scatter_add_(1, likely, lift.clamp(max=22.0))
            full[r:r + n] = part.to(full.dtype)
        uniforms = torch.rand(t, generator=g, device=DEV)
        kept = dict(tokens=_room(t), logprob=_room(t, dtype=torch.float32), kept=_room(t))
        return dict(case=c, logits=full[:, :v], uniforms=uniforms, settings=_settings(c, g), kept=kept)
    m, n, k = c["m"], c["n"], c["k"]
    x = torch.randn(m, k + c["pad"], generator=g, device=DEV).to(torch.bfloat16)[:, :k]
    if c["fmt"] in ("row", "mx"):   # formats that need no more than a row at a time
        codes, scales = torch.empty(n, k, dtype=torch.uint8, device=DEV), []
        for i in range(0, n, 8192):
            w = (0.02 * torch.randn(min(8192, n - i), k, generator=g, device=DEV)).to(torch.bfloat16).float()
            codes[i:i + 8192], s = _quantized(w, c["fmt"])
            scales.append(s)
        scales = torch.cat(scales)
    else:
        codes, scales = _quantized((0.02 * torch.randn(n, k, generator=g, device=DEV)).to(torch.bfloat16).float(), c["fmt"])
    n_out = n // 2 if c["act"] in GATED else n
    bias = None if c["bias"] == "none" else (0.2 * torch.randn(n, generator=g, device=DEV)).to(_dtype(c["bias"]))
    residual = torch.randn(m, n_out, generator=g, device=DEV).to(torch.bfloat16) if c["residual"] else None
    return dict(case=c, x=x, codes=codes, scales=scales, bias=bias, residual=residual, out=_room(m, n_out, dtype=_dtype(c["out"])))


# ----------------------------------------------------------------- passes --

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _own_linear(s):
    import fp8_block_scaled_02_amd as F
    c = s["case"]
    return dict(y=F.fp8w_linear(s["x"], s["codes"], s["scales"], fmt=c["fmt"], bias=s["bias"], act=c["act"],
                                residual=s["residual"], y=s["out"]))


def _own_sample(s):
    import fp8_block_scaled_02_amd as F
    r = F.fp8w_sample(s["logits"], s["uniforms"], **s["settings"], **s["kept"])
    return dict(tokens=r.tokens, logprob=r.logprob, kept=r.kept)


def _own_route(s):
    import fp8_block_scaled_02_amd as F
    c = s["case"]
    r = F.fp8w_route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                             top_groups=c["top_groups"], group_score=c["by"], **s["kept"])
    return dict(ids=r.ids, weights=r.weights, slots=r.slots, rows=r.rows, offsets=r.offsets)


def _weights_f32(codes, scales, fmt):
    n, k = codes.shape
    w = codes.view(torch.float8_e4m3fn).float()
    if fmt in ("block", "block_bf16"):
        return w * _spread(scales.float(), n, k)
    if fmt == "mx":
        return w * torch.exp2(scales.float() - 127).repeat_interleave(32, 1)[:, :k]
    return w * (scales[:, None] if fmt == "row" else scales)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _gelu_tanh(v):
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _plain_linear(s):
    c = s["case"]
    v = torch.matmul(s["x"].float(), _weights_f32(s["codes"], s["scales"], c["fmt"]).t())
    if s["bias"] is not None:
        v = v + s["bias"].float()
    if c["act"] in GATED:
        gate, up = v.chunk(2, 1)
        v = (_silu(gate) if c["act"] == "swiglu" else _gelu_tanh(gate)) * up
    elif c["act"] == "silu":
        v = _silu(v)
    elif c["act"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        v = _gelu_tanh(v)
    elif c["act"] == "relu":
        v = v.clamp(min=0)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return dict(y=v.to(_dtype(c["out"])))


def _plain_sample(s):
    c, k = s["case"], s["settings"]
    t, v = c["t"], c["v"]
    x, ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    x = x.double()   # what is left is decided at borders of long sums: in 64 bits
    temp = k["temperature"].double()[:, None]
    greedy = temp <= 0
    scaled = (x - x[:, :1]) / torch.where(greedy, torch.ones_like(temp), temp)
    rank = torch.arange(v, device=x.device)
    stay = torch.ones(t, v, dtype=torch.bool, device=x.device)
    if k["top_k"] is not None:
        stay = (k["top_k"][:, None] <= 0) | (rank < k["top_k"][:, None])
    w = torch.exp(scaled) * stay
    if k["top_p"] is not None:
        p = k["top_p"].double()[:, None]
        total = w.cumsum(1)
        stay = stay & ((p >= 1) | (total - w < p * total[:, -1:]))
    if k["min_p"] is not None:
        low = k["min_p"].double()[:, None]
        stay = stay & ((low <= 0) | (scaled >= torch.log(low)))
    stay = torch.where(greedy, rank < 1, stay | (rank < 1))
    w = w * stay
    total = w.cumsum(1)
    count = stay.sum(1)
    place = (total <= s["uniforms"].double()[:, None] * total[:, -1:]).sum(1).minimum(count - 1)[:, None]
    logprob = torch.log(w.gather(1, place) / total[:, -1:])
    return dict(tokens=ids.gather(1, place)[:, 0].int(), logprob=logprob[:, 0].float(), kept=count.int())


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    t, e, k, groups = c["t"], c["e"], c["k"], c["groups"]
    d = x.double()   # the choices are made next to ties: in 64 bits
    if c["score"] == "softmax":
        score = torch.exp(d - d.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-d))
    key = score + s["bias"].double() if c["bias"] else score
    best = torch.sort(key.view(t, groups, e // groups), dim=2, descending=True).values
    rating = best[:, :, 0] if c["by"] == "max" or e == groups else best[:, :, 0] + best[:, :, 1]
    if c["by"] == "max" and not c["bias"]:   # scores rise with the logits, which are exact
        key = d
        rating = d.view(t, groups, e // groups).amax(2)
    order = torch.sort(rating, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
    open_ = torch.zeros(t, groups, dtype=torch.bool, device=x.device).scatter_(1, order, True)
    if not c["bias"]:
        key = d
    key = torch.where(open_.repeat_interleave(e // groups, 1), key, torch.full_like(key, -math.inf))
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    weights = score.gather(1, ids)
    weights = (weights / weights.sum(1, keepdim=True)).float()
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(t * k, device=flat.device)
    count = torch.zeros(e, dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    return dict(ids=ids.int(), weights=weights, slots=slots.view(t, k).int(), rows=(order // k).int(), offsets=offsets.int())


_run_own = dict(linear=_own_linear, sample=_own_sample, route=_own_route)
_run_plain = dict(linear=_plain_linear, sample=_plain_sample, route=_plain_route)


# ------------------------------------------------------- the definition, 64 bits --

def exact(case, seed):
    return dict(linear=_exact_linear, sample=_exact_sample, route=_exact_route)[case["op"]](prepare(case, seed))


def _code_values():
    """e4m3fn: sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinities."""
    v = []
    for b in range(256):
        ex, man = (b >> 3) & 15, b & 7
        a = man / 8 * 2.0 ** -6 if ex == 0 else (1 + man / 8) * 2.0 ** (ex - 7)
        v.append(-a if b & 128 else a)
    return v


def _exact_linear(s):
    c = s["case"]
    m, n, k = c["m"], c["n"], c["k"]
    table = torch.tensor(_code_values(), dtype=torch.float64, device=DEV)
    col = torch.arange(k, device=DEV)
    x = s["x"].double()
    v = torch.empty(m, n, dtype=torch.float64, device=DEV)
    for lo in range(0, n, 4096):
        row = torch.arange(lo, min(lo + 4096, n), device=DEV)
        w = table[s["codes"][lo:lo + 4096].long()]
        if c["fmt"] in ("block", "block_bf16"):
            w *= s["scales"].double()[row // 128][:, col // 128]
        elif c["fmt"] == "mx":
            w *= (2.0 ** (s["scales"][lo:lo + 4096].double() - 127))[:, col // 32]
        elif c["fmt"] == "row":
            w *= s["scales"].double()[row][:, None]
        else:
            w *= s["scales"].double()
        v[:, lo:lo + 4096] = x @ w.T
    if s["bias"] is not None:
        v += s["bias"].double()
    f = torch.nn.functional
    h = n // 2
    v = {"none": lambda: v, "silu": lambda: f.silu(v), "gelu": lambda: f.gelu(v), "gelu_tanh": lambda: f.gelu(v, approximate="tanh"),
         "relu": lambda: f.relu(v), "swiglu": lambda: f.silu(v[:, :h]) * v[:, h:],
         "geglu": lambda: f.gelu(v[:, :h], approximate="tanh") * v[:, h:]}[c["act"]]()
    return dict(y=v if s["residual"] is None else v + s["residual"].double())


def _exact_sample(s):
    """Row by row: the tokens in order, cut three times, and the place that the random number falls to."""
    c, k = s["case"], s["settings"]
    out = torch.empty(c["t"], dtype=torch.float64, device=DEV)
    for r in range(c["t"]):
        temp = float(k["temperature"][r])
        x = torch.sort(s["logits"][r].double(), descending=True).values
        if temp <= 0:
            out[r] = 0.0
            continue
        if k["top_k"] is not None and int(k["top_k"][r]) > 0:
            x = x[:int(k["top_k"][r])]
        logp = torch.log_softmax(x / temp, 0)
        n = len(x)
        if k["top_p"] is not None and float(k["top_p"][r]) < 1:
            n = 1 + int((logp.exp().cumsum(0)[:-1] < float(k["top_p"][r])).sum())
        if k["min_p"] is not None and float(k["min_p"][r]) > 0:
            n = min(n, int((logp >= logp[0] + math.log(float(k["min_p"][r]))).sum()))
        logp = torch.log_softmax(logp[:max(n, 1)], 0)
        j = int((logp.exp().cumsum(0) <= float(s["uniforms"][r])).sum())
        out[r] = logp[min(j, len(logp) - 1)]
    return dict(tokens=None, logprob=out, kept=None)


def _exact_route(s):
    c, x = s["case"], s["logits"].double()
    t, e, groups = c["t"], c["e"], c["groups"]
    p = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    want = p + s["bias"].double() if c["bias"] else p
    g = want.view(t, groups, e // groups)
    rating = g.amax(2) if c["by"] == "max" else g.topk(min(2, e // groups), 2).values.sum(2)
    left = want.clone().view(t, groups, -1)
    for _ in range(groups - c["top_groups"]):   # the worst group goes, the last of equals first
        worst = groups - 1 - rating.flip(1).argmin(1)
        left[torch.arange(t, device=DEV), worst] = -math.inf
        rating[torch.arange(t, device=DEV), worst] = math.inf
    left = left.view(t, e)
    w = torch.empty(t, c["k"], dtype=torch.float64, device=DEV)
    for j in range(c["k"]):
        i = left.argmax(1, keepdim=True)
        w[:, j] = p.gather(1, i)[:, 0]
        left.scatter_(1, i, -math.inf)
    return dict(ids=None, weights=w / w.sum(1, keepdim=True), slots=None, rows=None, offsets=None)
