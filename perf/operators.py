"""The operators of a transformer block around the quantized layers, as they are measured: attention over packed
sequences, the 16-bit linear layer with its epilogue, and the norms around a block with its gate and residual.

`run` computes an operator in its plain form, or calls the framework's where `own` is true; `exact` computes its
definition in 64 bits.
"""
import random

import torch

own = False

BF16, F16, F32 = "bfloat16", "float16", "float32"


def _lengths(text):
    return [int(n) for n in text.split(",")]


def _text(lengths):
    return ",".join(str(n) for n in lengths)


def _spread(rng, low, high):
    """A length whose logarithm is spread evenly over [low, high]."""
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def listed():
    some = random.Random(20)
    return [
        # the joint attention of a FLUX-shaped block: 4096 image and 512 text tokens, every token sees every other
        {"name": "attention joint", "op": "attention", "dtype": BF16, "heads": 24, "kv_heads": 24, "dim": 128,
         "causal": False, "q_lengths": "4608", "k_lengths": "4608"},
        # prompts of very different lengths, packed without padding, grouped heads
        {"name": "attention prompts", "op": "attention", "dtype": BF16, "heads": 32, "kv_heads": 8, "dim": 128,
         "causal": True, "q_lengths": "8192,4096,2049,1,1500,546", "k_lengths": "8192,4096,2049,1,1500,546"},
        # a piece of a prompt against the keys of what came before it, for two requests of odd lengths, narrow heads
        {"name": "attention piece", "op": "attention", "dtype": F16, "heads": 16, "kv_heads": 2, "dim": 64,
         "causal": True, "q_lengths": "511,130", "k_lengths": "7103,1301"},
        # one new token of each request of a batch: every key is read once
        {"name": "attention step", "op": "attention", "dtype": BF16, "heads": 32, "kv_heads": 8, "dim": 128,
         "causal": True, "q_lengths": _text([1] * 64), "k_lengths": _text([_spread(some, 200, 16000) for _ in range(64)])},
        # one new token of a lone request: latency
        {"name": "attention step alone", "op": "attention", "dtype": F16, "heads": 16, "kv_heads": 4, "dim": 128,
         "causal": True, "q_lengths": "1", "k_lengths": "777"},
        # the modulation vector of a FLUX-shaped block from its conditioning vector: one row, all of the weight read
        {"name": "linear modulation", "op": "linear", "dtype": BF16, "rows": 1, "inner": 3072, "outer": 18432,
         "activation": "none", "bias": True, "residual": False},
        # a small batch through an odd-sized layer
        {"name": "linear small batch", "op": "linear", "dtype": F16, "rows": 37, "inner": 2056, "outer": 1000,
         "activation": "silu", "bias": True, "residual": True},
        # the two layers of a FLUX-shaped MLP kept in 16 bits: GELU after the first, the residual stream added by the second
        {"name": "linear up", "op": "linear", "dtype": BF16, "rows": 4608, "inner": 3072, "outer": 12288,
         "activation": "gelu", "bias": True, "residual": False},
        {"name": "linear down", "op": "linear", "dtype": BF16, "rows": 4608, "inner": 12288, "outer": 3072,
         "activation": "none", "bias": True, "residual": True},
        # between the blocks of a FLUX-shaped model: gated residual, then layer norm with modulation
        {"name": "norm modulated", "op": "norm", "dtype": BF16, "stream": BF16, "dim": 3072, "rows": "4608",
         "norm": "layer", "post_norm": "none", "modulated": True, "weights": False, "residual_scale": 1.0},
        # between the blocks of a language model with norms on both sides and a 32-bit residual stream, packed prompts
        {"name": "norm both sides", "op": "norm", "dtype": BF16, "stream": F32, "dim": 4096, "rows": "8192,4096,2049,1,1500,546",
         "norm": "rms", "post_norm": "rms", "modulated": True, "weights": True, "residual_scale": 0.22},
        # the same for one token of each of seven requests, an odd width
        {"name": "norm step", "op": "norm", "dtype": F16, "stream": F16, "dim": 2050, "rows": "1,1,1,1,1,1,1",
         "norm": "rms", "post_norm": "rms", "modulated": False, "weights": True, "residual_scale": 1.0},
    ]


def _draw_attention(rng):
    dim = rng.choice([64, 64, 72, 96, 128, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 8])
    dtype = rng.choice([BF16, BF16, F16])
    kind = rng.choice(["prompts", "joint", "piece", "step"])
    if kind == "step":
        batch = _spread(rng, 1, 96)
        q, k = [1] * batch, [_spread(rng, 30, 12000) for _ in range(batch)]
    elif kind == "piece":
        batch = rng.randint(1, 3)
        q = [_spread(rng, 2, 700) for _ in range(batch)]
        k = [n + _spread(rng, 1, 6000) for n in q]
    else:
        batch = _spread(rng, 1, 6) if kind == "prompts" else rng.randint(1, 2)
        q = [_spread(rng, 16, 4200) for _ in range(batch)]
        k = q if kind == "prompts" else [n + rng.choice([0, 77]) for n in q]
    return {"op": "attention", "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": kind != "joint", "q_lengths": _text(q), "k_lengths": _text(k)}


def _draw_linear(rng):
    return {"op": "linear", "dtype": rng.choice([BF16, BF16, F16]),
            "rows": _spread(rng, 1, 4608) if rng.random() < 0.7 else _spread(rng, 1, 64),
            "inner": 8 * _spread(rng, 32, 1500), "outer": 8 * _spread(rng, 16, 1500),
            "activation": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
            "bias": rng.random() < 0.7, "residual": rng.random() < 0.6}


def _draw_norm(rng):
    dtype = rng.choice([BF16, BF16, F16])
    batch = _spread(rng, 1, 12)
    longest = 1 if rng.random() < 0.25 else _spread(rng, 8, 1300)
    return {"op": "norm", "dtype": dtype, "stream": rng.choice([dtype, F32]),
            "dim": rng.choice([8 * _spread(rng, 16, 1024), 8 * _spread(rng, 16, 1024), _spread(rng, 128, 6000)]),
            "rows": _text([rng.randint(1, longest) for _ in range(batch)]), "norm": rng.choice(["layer", "rms"]),
            "post_norm": rng.choice(["none", "layer", "rms"]), "modulated": rng.random() < 0.6,
            "weights": rng.random() < 0.6, "residual_scale": rng.choice([1.0, 0.5])}


def draw(rng):
    return rng.choice([_draw_attention, _draw_linear, _draw_norm])(rng)


class _Maker:
    """Random tensors on the GPU, from the seed alone."""

    def __init__(self, seed):
        self.generator = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, scale=1.0, offset=0.0, dtype=F32):
        t = torch.randn(*shape, generator=self.generator, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(offset).to(getattr(torch, dtype))


def _offsets(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    make, dtype = _Maker(seed), case["dtype"]
    state = {"case": case}
    if case["op"] == "attention":
        q, k = _lengths(case["q_lengths"]), _lengths(case["k_lengths"])
        state["q"] = make.normal(sum(q), case["heads"], case["dim"], scale=1.5, dtype=dtype)
        state["k"] = make.normal(sum(k), case["kv_heads"], case["dim"], dtype=dtype)
        state["v"] = make.normal(sum(k), case["kv_heads"], case["dim"], offset=0.1, dtype=dtype)
        state["lengths"] = q, k
        state["offsets"] = _offsets(q), _offsets(k)
        return state
    if case["op"] == "linear":
        rows, inner, outer = case["rows"], case["inner"], case["outer"]
        gain = torch.ones(inner, device="cuda")
        gain[torch.randperm(inner, generator=make.generator, device="cuda")[: max(1, inner // 100)]] = 8.0
        state["X"] = (make.normal(rows, inner) * gain).to(getattr(torch, dtype))  # a few channels are outliers
        state["W"] = make.normal(inner, outer, scale=0.02, dtype=dtype)
        state["bias"] = make.normal(outer, scale=0.1, dtype=dtype) if case["bias"] else None
        state["residual"] = make.normal(rows, outer, dtype=dtype) if case["residual"] else None
        return state
    rows, dim = _lengths(case["rows"]), case["dim"]
    state["x"] = make.normal(sum(rows), dim, scale=2.0, offset=0.3, dtype=case["stream"])
    state["y"] = make.normal(sum(rows), dim, dtype=dtype)
    state["offsets"] = _offsets(rows)
    state["sequence"] = torch.repeat_interleave(torch.tensor(rows, device="cuda"))
    state["vectors"] = {}
    if case["modulated"]:
        for name in ("gate", "scale", "shift"):
            state["vectors"][name] = make.normal(len(rows), dim, scale=0.4, dtype=dtype)
    if case["weights"]:
        state["vectors"]["weight"] = make.normal(dim, scale=0.1, offset=1.0, dtype=dtype)
        if case["post_norm"] != "none":
            state["vectors"]["post_weight"] = make.normal(dim, scale=0.1, offset=1.0, dtype=dtype)
        if case["norm"] == "layer":
            state["vectors"]["bias"] = make.normal(dim, scale=0.1, dtype=dtype)
    return state


def _softmax_product(scores, hidden, v):
    """softmax over the last axis of scores, hidden places left out, times v; 0 for rows with nothing visible. Overwrites scores."""
    if hidden is not None:
        scores.masked_fill_(hidden, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    return (scores @ v) / torch.where(total == 0, 1.0, total)


def _attention_step(state):
    """One query a sequence: the keys of all sequences side by side, as long as the longest."""
    case, (_, lengths) = state["case"], state["lengths"]
    q, k, v, start = state["q"], state["k"], state["v"], state["offsets"][1]
    batch, groups, dim = q.shape[0], case["kv_heads"], case["dim"]
    place = torch.arange(max(lengths), device="cuda")
    at = (start[:-1, None] + place).clamp_(max=k.shape[0] - 1)
    hidden = (place >= (start[1:] - start[:-1])[:, None])[:, None, None, :]
    scores = q.float().view(batch, groups, -1, dim) @ k[at].float().permute(0, 2, 3, 1)
    o = _softmax_product(scores.mul_(dim ** -0.5), hidden, v[at].float().transpose(1, 2))
    return o.view(q.shape).to(q.dtype)


def _attention(state):
    case, (q_lengths, k_lengths) = state["case"], state["lengths"]
    if max(q_lengths) == 1:
        return _attention_step(state)
    groups, dim, out, pieces = case["kv_heads"], case["dim"], [], zip(
        state["q"].split(q_lengths), state["k"].split(k_lengths), state["v"].split(k_lengths))
    for q, k, v in pieces:
        n, m = q.shape[0], k.shape[0]
        rows = q.float().view(n, groups, -1, dim).permute(1, 2, 0, 3)
        scores = (rows @ k.float().permute(1, 2, 0)[:, None]).mul_(dim ** -0.5)
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")
        o = _softmax_product(scores, j > i + (m - n) if case["causal"] else None, v.float().transpose(0, 1)[:, None])
        out.append(o.permute(2, 0, 1, 3).reshape(q.shape).to(q.dtype))
    return torch.cat(out)


def _activated(t, name):
    if name == "relu":
        return t.clamp_min(0)
    if name == "silu":
        return t / (1 + torch.exp(-t))
    if name == "gelu":
        return 0.5 * t * (1 + torch.erf(t * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * t * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (t + 0.044715 * t * t * t)))
    return t


def _linear(state):
    t = state["X"].float() @ state["W"].float()
    if state["bias"] is not None:
        t += state["bias"].float()
    t = _activated(t, state["case"]["activation"])
    if state["residual"] is not None:
        t += state["residual"].float()
    return t.to(state["X"].dtype)


def _normed(t, kind, eps=1e-6):
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    return t if kind == "none" else t * torch.rsqrt((t * t).mean(-1, keepdim=True) + eps)


def _norm(state):
    case, sequence = state["case"], state["sequence"]
    vector = {name: t.float() for name, t in state["vectors"].items()}
    y = _normed(state["y"].float(), case["post_norm"])
    if "post_weight" in vector:
        y = y * vector["post_weight"]
    if "gate" in vector:
        y = y * vector["gate"][sequence]
    x = case["residual_scale"] * state["x"].float() + y
    h = _normed(x, case["norm"])
    if "weight" in vector:
        h = h * vector["weight"]
    if "bias" in vector:
        h = h + vector["bias"]
    if "scale" in vector:
        h = h * (1 + vector["scale"][sequence]) + vector["shift"][sequence]
    return x.to(state["x"].dtype), h.to(state["y"].dtype)


def run(state):
    case = state["case"]
    if own:
        import rank_gemm_quantize_b200 as rq

        if case["op"] == "attention":
            return rq.attention(state["q"], state["k"], state["v"], *state["offsets"], causal=case["causal"])
        if case["op"] == "linear":
            return rq.linear(state["X"], state["W"], state["bias"], activation=None if case["activation"] == "none" else case["activation"],
                             residual=state["residual"])
        return rq.residual_norm(state["x"], state["y"], offsets=state["offsets"], residual_scale=case["residual_scale"],
                                post_norm=None if case["post_norm"] == "none" else case["post_norm"], norm=case["norm"],
                                **state["vectors"])
    return {"attention": _attention, "linear": _linear, "norm": _norm}[case["op"]](state)


def work(case):
    if case["op"] == "attention":
        q, k = _lengths(case["q_lengths"]), _lengths(case["k_lengths"])
        # query i of n sees the first i + m - n + 1 of m keys, or all of them
        pairs = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(q, k))
        values = 2 * sum(q) * case["heads"] + 2 * sum(k) * case["kv_heads"]
        return {"bytes": 2 * case["dim"] * values, "flops": 4 * case["dim"] * case["heads"] * pairs}
    if case["op"] == "linear":
        rows, inner, outer = case["rows"], case["inner"], case["outer"]
        values = rows * inner + inner * outer + rows * outer * (2 if case["residual"] else 1) + (outer if case["bias"] else 0)
        return {"bytes": 2 * values, "flops": 2 * rows * inner * outer}
    rows = _lengths(case["rows"])
    vectors = (3 * len(rows) if case["modulated"] else 0) + (2 if case["weights"] else 0)
    wide = 4 if case["stream"] == F32 else 2
    return {"bytes": case["dim"] * (sum(rows) * (2 * wide + 4) + 2 * vectors), "flops": 20 * sum(rows) * case["dim"]}


def _exact_attention(case, state):
    group, out = case["heads"] // case["kv_heads"], torch.empty(state["q"].shape, dtype=torch.float64, device="cuda")
    first_q = first_k = 0
    for n, m in zip(*state["lengths"]):
        for head in range(case["heads"]):
            q = state["q"][first_q:first_q + n, head].double()
            k = state["k"][first_k:first_k + m, head // group].double()
            v = state["v"][first_k:first_k + m, head // group].double()
            s = q.mm(k.t()) / case["dim"] ** 0.5
            if case["causal"]:
                s = s + torch.full_like(s, -torch.inf).triu_(m - n + 1)
            out[first_q:first_q + n, head] = torch.softmax(s, dim=1).mm(v)
        first_q, first_k = first_q + n, first_k + m
    return out


def _exact_linear(case, state):
    t = torch.mm(state["X"].double(), state["W"].double())
    if case["bias"]:
        t = t + state["bias"].double()
    name = case["activation"]
    if name in ("gelu", "gelu_tanh"):
        t = torch.nn.functional.gelu(t, approximate="tanh" if name == "gelu_tanh" else "none")
    elif name == "silu":
        t = torch.nn.functional.silu(t)
    elif name == "relu":
        t = torch.nn.functional.relu(t)
    return t + state["residual"].double() if case["residual"] else t


def _exact_norm(case, state):
    def norm(t, kind, weight, bias):
        if kind == "layer":
            t = (t - t.mean(1, keepdim=True)) / (t.var(1, keepdim=True, unbiased=False) + 1e-6).sqrt()
        elif kind == "rms":
            t = t / (t.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()
        t = t if weight is None else t * weight.double()
        return t if bias is None else t + bias.double()

    vector, times = state["vectors"].get, torch.tensor(_lengths(case["rows"]), device="cuda")
    y = norm(state["y"].double(), case["post_norm"], vector("post_weight"), None)
    if case["modulated"]:
        y = y * vector("gate").double().repeat_interleave(times, 0)
    x = state["x"].double() * case["residual_scale"] + y
    h = norm(x, case["norm"], vector("weight"), vector("bias"))
    if case["modulated"]:
        h = h * (vector("scale").double() + 1).repeat_interleave(times, 0) + vector("shift").double().repeat_interleave(times, 0)
    return x, h


def exact(case, seed):
    return {"attention": _exact_attention, "linear": _exact_linear, "norm": _exact_norm}[case["op"]](case, prepare(case, seed))
