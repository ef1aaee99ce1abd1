"""Operators measured on one MI355X beside those of perf/operators.py: what each case is, its inputs, its plain form,
and its result in 64 bits.

Three operators around a row-scaled linear layer and a gated feed-forward block:

- "int8": the linear layer in 8-bit integers with a scale per token and per output channel, from a bf16 activation
  (quantized by token within the call) or from one already quantized ("codes");
- "route": a mixture-of-experts router: logits, the best experts of every token and their weights;
- "moe": the whole mixture of gated feed-forward blocks for a few tokens, from the router's choice, with experts in
  bf16, 8-bit integers with a scale per channel, or 4-bit floats with group scales.

`run` computes the plain form with elementary torch operations, or (`own`) calls the package.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST = 8 * 4096 * 14336  # values of the experts' largest projection


def listed():
    return [
        # single-token decode, attention output projection: latency
        {"name": "int8_m1", "kind": "int8", "m": 1, "n": 4096, "k": 4096, "bias": True, "codes": False},
        # a decode batch, down projection
        {"name": "int8_m16", "kind": "int8", "m": 16, "n": 4096, "k": 14336, "bias": False, "codes": False},
        # a short prompt through odd sizes, its activation quantized before (shared by several projections)
        {"name": "int8_m100", "kind": "int8", "m": 100, "n": 5648, "k": 2080, "bias": True, "codes": True},
        # a ragged prompt
        {"name": "int8_m517", "kind": "int8", "m": 517, "n": 14336, "k": 4096, "bias": False, "codes": False},
        # prefill
        {"name": "int8_m8192", "kind": "int8", "m": 8192, "n": 14336, "k": 4096, "bias": False, "codes": False},
        # single-token decode, many small experts: latency
        {"name": "route_m1", "kind": "route", "m": 1, "k": 2048, "experts": 64, "top": 8, "score": "softmax"},
        # the prompts that join a running batch, an odd number of experts
        {"name": "route_m1000", "kind": "route", "m": 1000, "k": 4096, "experts": 161, "top": 6, "score": "sigmoid"},
        # single-token decode of few large experts
        {"name": "moe_bf16_m1", "kind": "moe", "m": 1, "k": 4096, "f": 14336, "experts": 8, "top": 2, "weight": "bf16",
         "act": "silu", "empty": False},
        # single-token decode of many small experts with 8-bit weights
        {"name": "moe_int8_m1", "kind": "moe", "m": 1, "k": 2048, "f": 1408, "experts": 64, "top": 6, "weight": "int8",
         "act": "silu", "empty": False},
        # a few sequences, or one with drafted tokens, on 4-bit weights
        {"name": "moe_fp4_m5", "kind": "moe", "m": 5, "k": 4096, "f": 14336, "experts": 8, "top": 2, "weight": "fp4",
         "act": "gelu", "empty": False},
        # a decode batch on many small experts, padded rows and experts of another device among the slots
        {"name": "moe_bf16_m16", "kind": "moe", "m": 16, "k": 2048, "f": 1408, "experts": 64, "top": 8,
         "weight": "bf16", "act": "silu", "empty": True},
        # the largest batch that still counts as a few tokens
        {"name": "moe_int8_m64", "kind": "moe", "m": 64, "k": 4096, "f": 14336, "experts": 8, "top": 2,
         "weight": "int8", "act": "silu", "empty": False},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    kind = rng.choice(["int8", "int8", "route", "moe", "moe"])
    if kind == "int8":
        n, k = 16 * _spread(rng, 16, 896), 16 * _spread(rng, 16, 896)
        return {"kind": kind, "m": _spread(rng, 1, min(8192, 8192 * 14336 * 4096 // (n * k))), "n": n, "k": k,
                "bias": rng.random() < 0.5, "codes": rng.random() < 0.3}
    if kind == "route":
        experts = _spread(rng, 4, 256)
        return {"kind": kind, "m": _spread(rng, 1, 1024), "k": 32 * _spread(rng, 8, 128), "experts": experts,
                "top": rng.randint(1, min(8, experts)), "score": rng.choice(["softmax", "sigmoid"])}
    k, f = 32 * _spread(rng, 8, 128), 32 * _spread(rng, 8, 448)
    experts = _spread(rng, 4, min(128, LARGEST // (k * f)))
    return {"kind": kind, "m": _spread(rng, 1, 64), "k": k, "f": f, "experts": experts,
            "top": rng.randint(1, min(8, experts)), "weight": rng.choice(["bf16", "int8", "fp4"]),
            "act": rng.choice(["silu", "gelu", "relu"]), "empty": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs


def _activation(gen, m, k):
    """Normal values, a few loud channels, -0.0 entries, and now and then a row of zeros, as of padding."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    x *= 1 + 9 * (torch.rand(k, generator=gen, device="cuda") < 0.01)
    x = torch.where(torch.rand(m, k, generator=gen, device="cuda") < 0.001, -0.0, x)
    x[7::64] = 0
    return x.bfloat16()


def _int8(x):
    """Codes and scales of rows: the nearest whole number to 127 x / amax, ties to even."""
    amax = x.abs().amax(1, keepdim=True)
    codes = torch.round(127 * x / torch.where(amax > 0, amax, 1))
    return codes.to(torch.int8), (amax / 127)[:, 0]


def _fp4(w):
    """A weight held in 4 bits: codes [r, c / 2], even column in the low half, and biased scale exponents per 32."""
    b = w.reshape(w.shape[0], -1, 32)
    e = torch.ceil(torch.log2(b.abs().amax(2).clamp(min=2.0 ** -60) / 6))
    t = b * torch.exp2(-e)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    codes = torch.bucketize(t.abs(), edges, out_int32=True).to(torch.uint8) + 8 * torch.signbit(t).to(torch.uint8)
    codes = codes.reshape(w.shape)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _weight(gen, rows, k, form):
    w = 0.02 * torch.randn(rows, k, generator=gen, device="cuda")
    return (w.bfloat16(), None) if form == "bf16" else _int8(w.bfloat16().float()) if form == "int8" else _fp4(w)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    m, k = case["m"], case["k"]
    x = _activation(gen, m, k)
    if case["kind"] == "int8":
        s["w"], s["ws"] = _weight(gen, case["n"], k, "int8")
        if case["bias"]:
            s["bias_values"] = (0.01 * torch.randn(case["n"], generator=gen, device="cuda")).bfloat16()
        if case["codes"]:
            s["x"], s["xs"] = _int8(x.float())
        else:
            s["x"] = x
        return s
    s["x"] = x
    experts, top = case["experts"], case["top"]
    if case["kind"] == "route":
        s["w"] = (0.02 * torch.randn(experts, k, generator=gen, device="cuda")).bfloat16()
        s["bias_values"] = 0.1 * torch.randn(experts, generator=gen, device="cuda")
        return s
    logits = torch.randn(m, experts, generator=gen, device="cuda") + torch.randn(experts, generator=gen, device="cuda")
    values, ids = torch.topk(logits, top)
    s["ids"], s["weights"] = ids.int(), torch.softmax(values, 1)
    if case["empty"]:  # slots that this device does not serve, and rows that are padding
        off = torch.rand(m, top, generator=gen, device="cuda") < 0.1
        off[5::8] = True
        s["ids"] = torch.where(off, -1, s["ids"]).int()
    s["gu"], s["gu_scale"] = _weight(gen, experts * 2 * case["f"], k, case["weight"])
    s["down"], s["down_scale"] = _weight(gen, experts * k, case["f"], case["weight"])
    return s


# ------------------------------------------------------------------ the operators


ACT = {"silu": "silu", "gelu": "gelu_tanh", "relu": "relu"}


def _own(s):
    import sparse_fp8_row_amd as sfr
    if s["kind"] == "int8":
        x = sfr.Int8Tensor(s["x"], s["xs"]) if s["codes"] else s["x"]
        return {"out": sfr.int8_linear(x, sfr.Int8Tensor(s["w"], s["ws"]), s.get("bias_values"))}
    if s["kind"] == "route":
        r = sfr.moe_route(s["x"], s["w"], s["top"], bias=s["bias_values"], score=s["score"])
        return {"ids": r.ids, "weights": r.weights, "logits": r.logits}
    k, f = s["k"], s["f"]
    if s["weight"] == "bf16":
        gu, down = s["gu"].view(-1, 2 * f, k), s["down"].view(-1, k, f)
    elif s["weight"] == "int8":
        gu, down = sfr.Int8Tensor(s["gu"], s["gu_scale"]), sfr.Int8Tensor(s["down"], s["down_scale"])
    else:
        gu, down = (sfr.MxTensor(q.view(torch.float4_e2m1fn_x2), e.view(torch.float8_e8m0fnu))
                    for q, e in ((s["gu"], s["gu_scale"]), (s["down"], s["down_scale"])))
    return {"out": sfr.moe_layer(s["x"], sfr.MoeRoute(s["ids"], s["weights"]), gu, down, ACT[s["act"]])}


def _values(w, scale, form):
    """The binary32 values of a weight."""
    if form == "bf16":
        return w.float()
    if form == "int8":
        return w.float() * scale[:, None]
    c = torch.stack((w & 15, w >> 4), 2).reshape(w.shape[0], -1).int()
    v = torch.tensor(E2M1, device=w.device)[c & 7] * (1 - 2 * (c >> 3))
    return (v.reshape(w.shape[0], -1, 32) * torch.exp2(scale.float() - 127)[:, :, None]).reshape(v.shape)


def _act(g, act):
    if act == "relu":
        return g.clamp(min=0)
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def run(state):
    if own:
        return _own(state)
    s = state
    if s["kind"] == "int8":
        x, xs = (s["x"], s["xs"]) if s["codes"] else _int8(s["x"].float())
        y = (x.float() @ s["w"].float().t()) * (xs[:, None] * s["ws"])
        return {"out": (y + s["bias_values"].float() if s["bias"] else y).bfloat16()}
    if s["kind"] == "route":
        # 64 bits: the choice between two nearly equal experts; the logits are rounded once to 32
        logits = (s["x"].double() @ s["w"].double().t() + s["bias_values"].double()).float()
        best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
        best, ids = best[:, : s["top"]], ids[:, : s["top"]].int()
        p = torch.exp(best - best[:, :1]) if s["score"] == "softmax" else 1 / (1 + torch.exp(-best))
        return {"ids": ids, "weights": p / p.sum(1, keepdim=True), "logits": logits}
    m, k, f, experts, top, form = s["m"], s["k"], s["f"], s["experts"], s["top"], s["weight"]
    if m * top < experts:  # the chosen experts' weights, one set for every choice
        ids = s["ids"].reshape(-1)

        def chosen(name, n):  # a slot without an expert: expert 0, weighted by zero below
            e, scale = ids.clamp(min=0).long(), s[name + "_scale"]
            w = s[name].view(experts, n, -1)[e].view(m * top * n, -1)
            scale = None if scale is None else scale.view(experts, n, -1)[e].view(m * top * n, -1).squeeze(1)
            return _values(w, scale, form).view(m * top, n, -1)

        x = s["x"].float().repeat_interleave(top, 0)
        gu = (chosen("gu", 2 * f) @ x[:, :, None]).view(m * top, 2, f)
        h = _act(gu[:, 0], s["act"]) * gu[:, 1] * torch.where(ids < 0, 0.0, s["weights"].reshape(-1))[:, None]
        return {"out": (chosen("down", k) @ h[:, :, None]).view(m, top, k).sum(1).bfloat16()}
    # every expert on every token, weighted by zero where the token did not choose it
    gu = (s["x"].float() @ _values(s["gu"], s["gu_scale"], form).t()).view(m, experts, 2, f)
    h = _act(gu[:, :, 0], s["act"]) * gu[:, :, 1]
    chosen = s["ids"][:, :, None] == torch.arange(experts, device="cuda")
    h = h * (chosen * s["weights"][:, :, None]).sum(1)[:, :, None]
    down = _values(s["down"], s["down_scale"], form).view(experts, k, f).transpose(1, 2).reshape(-1, k)
    return {"out": (h.view(m, -1) @ down).bfloat16()}


def work(case):
    kind, m, k = case["kind"], case["m"], case["k"]
    if kind == "int8":
        n = case["n"]
        x = m * k + 4 * m if case["codes"] else 2 * m * k
        return {"bytes": x + n * k + 4 * n + 2 * n * case["bias"] + 2 * m * n, "flops": 2 * m * n * k}
    experts, top = case["experts"], case["top"]
    if kind == "route":
        return {"bytes": 2 * m * k + 2 * experts * k + 4 * experts + 4 * m * experts + 8 * m * top,
                "flops": 2 * m * experts * k}
    f = case["f"]
    # experts that at least one token chose: all that can be different, or what so many choices leave in the mean
    used = min(experts, m * top) if m == 1 else experts * (1 - (1 - top / experts) ** m)
    each = {"bf16": 2, "int8": 1, "fp4": 17 / 32}[case["weight"]]
    scales = 4 * (2 * f + k) if case["weight"] == "int8" else 0
    return {"bytes": used * (each * (3 * k * f) + scales) + 4 * m * k + 8 * m * top, "flops": 6 * m * top * k * f}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _exact_rows(w, scale, form):
    """Values of stored rows in binary64, element by element from their bit fields."""
    if form == "bf16":
        return w.double()
    if form == "int8":
        return w.double() * scale.double()[:, None]
    c = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.int64, device=w.device)
    c[:, 0::2], c[:, 1::2] = w % 16, w // 16
    exp, man = (c // 2) % 4, (c % 2).double() / 2
    v = torch.where(exp > 0, (1 + man) * torch.exp2(exp.double() - 1), man) * (1 - 2 * (c // 8))
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)


def _exact_act(g, act):
    if act == "relu":
        return torch.where(g > 0, g, 0.0)
    return g * torch.sigmoid(g if act == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3))


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["kind"] == "int8":
        if case["codes"]:
            scale = s["xs"].double()
        else:
            scale = x.abs().amax(1) / 127
            x = torch.round(127 * x / torch.where(scale > 0, 127 * scale, 1.0)[:, None])
        y = torch.matmul(x, s["w"].double().t())
        y = y * scale[:, None] * s["ws"].double()[None, :]
        return {"out": y + s["bias_values"].double()[None, :] if case["bias"] else y}
    top = case["top"]
    if case["kind"] == "route":
        logits = torch.matmul(x, s["w"].double().t()) + s["bias_values"].double()[None, :]
        rounded = logits.float().double()
        ids = torch.argsort(rounded, dim=1, descending=True, stable=True)[:, :top]
        best = torch.gather(rounded, 1, ids)
        p = torch.softmax(best, 1) if case["score"] == "softmax" else torch.sigmoid(best)
        return {"ids": ids.int(), "weights": p / p.sum(1, keepdim=True), "logits": logits}
    k, f = case["k"], case["f"]
    out = torch.zeros(case["m"], k, dtype=torch.float64, device="cuda")
    ids = s["ids"].cpu()
    for e in range(case["experts"]):
        rows, slots = torch.nonzero(ids == e, as_tuple=True)
        if rows.numel():
            def part(name, n):
                scale = s[name + "_scale"]
                return _exact_rows(s[name][e * n:(e + 1) * n], None if scale is None else scale[e * n:(e + 1) * n],
                                   case["weight"])
            rows, slots = rows.cuda(), slots.cuda()
            gu = torch.matmul(x[rows], part("gu", 2 * f).t())
            h = _exact_act(gu[:, :f], case["act"]) * gu[:, f:]
            out[rows] += torch.matmul(h, part("down", k).t()) * s["weights"][rows, slots].double()[:, None]
    return {"out": out}
