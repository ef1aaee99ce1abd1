"""Operators measured on one MI355X: what each case is, its inputs, its plain form, and its result in 64 bits.

Three groups that a gated feed-forward block needs beside the row-scaled FP8 linear layer:

- "checkpoint": an activation saved in 8 bits for the backward pass and restored (MX format: blocks of 32 values along
  a row share one power-of-two scale; elements are FP8);
- "gated" / "backward" / "train": h = act(x Wg^T) * (x Wu^T) for a bf16 weight w = [Wg; Wu] of [2f, k], its gradients
  from saved 8-bit (or bf16) activations, and a training step of both;
- "mxfp4" / "mxfp4_gated": the linear layer, and the gated block, for a weight of 4-bit floats with group scales.

`run` computes the plain form in binary32 with elementary torch operations, or (`own`) calls the package.
"""
import math

import torch

own = False

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# Largest element of each format is FRACTION * 2^TOP with FRACTION in [1/2, 1).
FRACTION = {"e4m3": 0.875, "e5m2": 0.875, "e2m1": 0.75}
TOP = {"e4m3": 9, "e5m2": 16, "e2m1": 3}
LOWEST = -110  # smallest scale exponent
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one micro-batch's odd rest of rows: launch latency of a save and a restore
        {"name": "checkpoint_37x2080", "kind": "checkpoint", "rows": 37, "cols": 2080, "fmt": "e4m3"},
        # the gated product of a prefill-sized step, saved for the backward pass
        {"name": "checkpoint_8192x14336", "kind": "checkpoint", "rows": 8192, "cols": 14336, "fmt": "e4m3"},
        # single-token decode of the block with its bf16 weight (bound by reading the weight)
        {"name": "gated_m1", "kind": "gated", "m": 1, "k": 4096, "f": 14336, "act": "silu"},
        # a ragged prompt
        {"name": "gated_m517", "kind": "gated", "m": 517, "k": 4096, "f": 14336, "act": "gelu"},
        # prefill, and the forward half of a large training step
        {"name": "gated_m8192", "kind": "gated", "m": 8192, "k": 4096, "f": 14336, "act": "silu"},
        # a small block's backward pass with activations kept in bf16, odd rows
        {"name": "backward_m1000", "kind": "backward", "m": 1000, "k": 2048, "f": 5632, "act": "relu", "fmt": "bf16"},
        # a large step's backward pass from 8-bit activations
        {"name": "backward_m8192", "kind": "backward", "m": 8192, "k": 4096, "f": 14336, "act": "silu", "fmt": "e4m3"},
        # one training step of a micro-batch: forward, 8-bit save, backward
        {"name": "train_m2048", "kind": "train", "m": 2048, "k": 4096, "f": 14336, "act": "silu", "fmt": "e4m3"},
        # single-token decode, attention output projection
        {"name": "mxfp4_m1", "kind": "mxfp4", "m": 1, "n": 4096, "k": 4096, "bias": True},
        # a decode batch, down projection
        {"name": "mxfp4_m16", "kind": "mxfp4", "m": 16, "n": 4096, "k": 14336, "bias": False},
        # single-token decode of the gated block with a 4-bit weight
        {"name": "mxfp4_gated_m1", "kind": "mxfp4_gated", "m": 1, "k": 4096, "f": 14336, "act": "silu"},
        # a short ragged prompt with a 4-bit weight
        {"name": "mxfp4_gated_m300", "kind": "mxfp4_gated", "m": 300, "k": 4096, "f": 14336, "act": "silu"},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    kind = rng.choice(["checkpoint", "gated", "gated", "backward", "train", "mxfp4", "mxfp4_gated"])
    act = rng.choice(["silu", "gelu", "relu"])
    k, f = 32 * _spread(rng, 8, 128), 32 * _spread(rng, 16, 448)
    if kind == "checkpoint":
        return {"kind": kind, "rows": _spread(rng, 1, 8192), "cols": 32 * _spread(rng, 1, 448),
                "fmt": rng.choice(["e4m3", "e5m2"])}
    if kind == "gated":
        return {"kind": kind, "m": _spread(rng, 1, 8192), "k": k, "f": f, "act": act}
    if kind in ("backward", "train"):
        return {"kind": kind, "m": _spread(rng, 1, 4096), "k": k, "f": f, "act": act,
                "fmt": rng.choice(["bf16", "e4m3", "e4m3", "e5m2"])}
    if kind == "mxfp4":
        return {"kind": kind, "m": _spread(rng, 1, 1024), "n": 16 * _spread(rng, 16, 896),
                "k": 32 * _spread(rng, 8, 448), "bias": rng.random() < 0.5}
    return {"kind": kind, "m": _spread(rng, 1, 1024), "k": k, "f": f, "act": act}


# ------------------------------------------------------------------ plain form of the block format


def _exp2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x):
    return x.reshape(x.shape[0], x.shape[1] // 32, 32)


def _mx_encode(x, fmt):
    """binary32 [r, c] -> (codes uint8 [r, c] (4-bit: [r, c/2], even column in the low half), scales uint8 [r, c/32])."""
    b = _blocks(x)
    amax = b.abs().amax(2)
    part, e = torch.frexp(amax)
    e = (e - TOP[fmt] + (part > FRACTION[fmt])).clamp(min=LOWEST)
    e = torch.where(amax == 0, LOWEST, e)
    t = b * _exp2(-e)[:, :, None]
    if fmt == "e2m1":
        a = t.abs()
        code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
                + 8 * torch.signbit(t)).to(torch.uint8).reshape(x.shape)
        codes = code[:, 0::2] | (code[:, 1::2] << 4)
    else:
        codes = t.to(FP8[fmt]).view(torch.uint8).reshape(x.shape)
    return codes, (e + 127).to(torch.uint8)


def _mx_decode(codes, scale, fmt):
    """The binary32 values that the codes stand for."""
    if fmt == "e2m1":
        c = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1).int()
        v = torch.tensor(E2M1, device=codes.device)[c & 7] * (1 - 2 * (c >> 3))
    else:
        v = codes.view(FP8[fmt]).float()
    return (_blocks(v) * _exp2(scale.int() - 127)[:, :, None]).reshape(v.shape)


def _act(g, act):
    """act(g) and its derivative."""
    if act == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _gradients(dh, x, g, u, w, act):
    a, d = _act(g, act)
    dgu = torch.cat((dh * u * d, dh * a), 1)
    return dgu @ w, dgu.t() @ x


# ------------------------------------------------------------------ inputs


def _activation(gen, m, k, dev):
    """Normal values, a few loud channels, some blocks all zero, as after a ReLU or a mask, and -0.0 entries."""
    x = torch.randn(m, k, generator=gen, device=dev)
    x *= 1 + 9 * (torch.rand(k, generator=gen, device=dev) < 0.01)
    zero = torch.rand(m, k // 32, 1, generator=gen, device=dev) < 0.01
    x = torch.where(zero, torch.zeros((), device=dev), _blocks(x)).reshape(m, k)
    return torch.where(torch.rand(m, k, generator=gen, device=dev) < 0.001, -0.0, x).bfloat16()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind == "checkpoint":
        s["x"] = _activation(gen, case["rows"], case["cols"], dev)
        return s
    m, k = case["m"], case["k"]
    rows = case["n"] if kind == "mxfp4" else 2 * case["f"]
    w = (0.02 * torch.randn(rows, k, generator=gen, device=dev)).bfloat16()
    if kind != "backward" or case["fmt"] == "bf16":
        s["x"] = _activation(gen, m, k, dev)
    if kind in ("gated", "backward", "train"):
        s["w"] = w
    else:
        s["wq"], s["ws"] = _mx_encode(w.float(), "e2m1")
    if case.get("bias"):
        s["bias_values"] = (0.01 * torch.randn(rows, generator=gen, device=dev)).bfloat16()
    if kind in ("backward", "train"):
        s["dh"] = (0.05 * torch.randn(m, case["f"], generator=gen, device=dev)).bfloat16()
    if kind == "backward":
        gu = 0.02 * math.sqrt(k) * torch.randn(m, rows, generator=gen, device=dev)
        if case["fmt"] == "bf16":
            s["gu"] = gu.bfloat16()
        else:
            s["gu"], s["gu_scale"] = _mx_encode(gu, case["fmt"])
            s["x"], s["x_scale"] = _mx_encode(_activation(gen, m, k, dev).float(), case["fmt"])
    return s


# ------------------------------------------------------------------ the operators


ACT = {"silu": "silu", "gelu": "gelu_tanh", "relu": "relu"}


def _own(s):
    import sparse_fp8_row_amd as sfr
    kind = s["kind"]
    if kind == "checkpoint":
        return {"restored": sfr.dequantize_mx(sfr.quantize_mx(s["x"], FP8[s["fmt"]]))}
    if kind == "gated":
        return {"h": sfr.gated_linear(s["x"], s["w"], ACT[s["act"]])}
    if kind == "train":
        fmt = FP8.get(s["fmt"], torch.bfloat16)
        h, saved = sfr.gated_linear_checkpointed(s["x"], s["w"], ACT[s["act"]], checkpoint=fmt)
        dx, dw = sfr.gated_linear_backward(s["dh"], s["w"], saved)
        return {"h": h, "dx": dx, "dw": dw}
    if kind == "backward":
        if s["fmt"] == "bf16":
            saved = sfr.GatedCheckpoint(s["x"], s["gu"], ACT[s["act"]])
        else:
            def mx(q, e):
                return sfr.MxTensor(q.view(FP8[s["fmt"]]), e.view(torch.float8_e8m0fnu))
            saved = sfr.GatedCheckpoint(mx(s["x"], s["x_scale"]), mx(s["gu"], s["gu_scale"]), ACT[s["act"]])
        dx, dw = sfr.gated_linear_backward(s["dh"], s["w"], saved)
        return {"dx": dx, "dw": dw}
    w = sfr.MxTensor(s["wq"].view(torch.float4_e2m1fn_x2), s["ws"].view(torch.float8_e8m0fnu))
    if kind == "mxfp4":
        return {"out": sfr.mxfp4_linear(s["x"], w, s.get("bias_values"))}
    return {"h": sfr.mxfp4_gated_linear(s["x"], w, ACT[s["act"]])}


def run(state):
    if own:
        return _own(state)
    s, kind = state, state["kind"]
    if kind == "checkpoint":
        return {"restored": _mx_decode(*_mx_encode(s["x"].float(), s["fmt"]), s["fmt"]).bfloat16()}
    if kind == "mxfp4":
        y = s["x"].float() @ _mx_decode(s["wq"], s["ws"], "e2m1").t()
        return {"out": (y + s["bias_values"].float() if s.get("bias") else y).bfloat16()}
    if kind == "backward":
        saved = s["fmt"] == "bf16"
        x = s["x"].float() if saved else _mx_decode(s["x"], s["x_scale"], s["fmt"])
        gu = s["gu"].float() if saved else _mx_decode(s["gu"], s["gu_scale"], s["fmt"])
        dx, dw = _gradients(s["dh"].float(), x, *gu.chunk(2, 1), s["w"].float(), s["act"])
        return {"dx": dx.bfloat16(), "dw": dw.bfloat16()}
    x = s["x"].float()
    w = s["w"].float() if "w" in s else _mx_decode(s["wq"], s["ws"], "e2m1")
    gu = x @ w.t()
    g, u = gu.chunk(2, 1)
    h = (_act(g, s["act"])[0] * u).bfloat16()
    if kind != "train":
        return {"h": h}
    if s["fmt"] == "bf16":
        gu = gu.bfloat16().float()
    else:
        gu, x = (_mx_decode(*_mx_encode(v, s["fmt"]), s["fmt"]) for v in (gu, x))
    dx, dw = _gradients(s["dh"].float(), x, *gu.chunk(2, 1), w, s["act"])
    return {"h": h, "dx": dx.bfloat16(), "dw": dw.bfloat16()}


def work(case):
    kind = case["kind"]
    if kind == "checkpoint":  # read, save the codes, read them back, write
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n + 2 * n * 33 / 32, "flops": 4 * n}
    m, k = case["m"], case["k"]
    if kind == "mxfp4":
        n = case["n"]
        return {"bytes": 2 * m * k + n * k * 17 / 32 + 2 * m * n + 2 * n * case["bias"], "flops": 2 * m * n * k}
    f = case["f"]
    product = 4 * m * k * f  # of x with both halves of the weight
    if kind == "mxfp4_gated":
        return {"bytes": 2 * m * k + 2 * f * k * 17 / 32 + 2 * m * f, "flops": product}
    if kind == "gated":
        return {"bytes": 2 * m * k + 4 * f * k + 2 * m * f, "flops": product}
    each = 2 if case["fmt"] == "bf16" else 33 / 32
    back = 2 * m * f + each * (2 * m * f + m * k) + 4 * f * k + 2 * m * k + 4 * f * k
    if kind == "backward":
        return {"bytes": back, "flops": 2 * product}
    save = (2 * m * f if case["fmt"] == "bf16" else each * (2 * m * f + m * k)) if kind == "train" else 0
    return {"bytes": 2 * m * k + 4 * f * k + 2 * m * f + save + back, "flops": 3 * product}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _exact_power(e):
    """2^e for whole e, in binary64."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_grid(x, fmt):
    """Values of binary64 x [r, c] after the 8-bit block format: each block's scale is the smallest power of two s
    with |x| <= largest * s (not below 2^LOWEST); elements go to the nearest multiple of their binade's step."""
    largest, bits, low = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}[fmt]
    b = _blocks(x)
    amax = b.abs().amax(2, keepdim=True)
    one = torch.ones((), dtype=torch.float64, device=x.device)
    power = _exact_power
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, one) / largest))
    e = e + (amax > largest * power(e)).double()
    e = e + (amax > largest * power(e)).double()
    e = torch.where(amax > 0, e, LOWEST * one).clamp(min=LOWEST)
    s = power(e)
    t = b / s
    binade = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** low))).clamp(min=low)
    binade = binade - (power(binade) > t.abs().clamp(min=2.0 ** low)).double()
    step = power(binade - bits)
    return (torch.round(t / step) * step * s).reshape(x.shape)


def _exact_value(codes, scale, fmt):
    """Values of stored codes in binary64, element by element from their bit fields."""
    if fmt == "e2m1":
        c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.int64, device=codes.device)
        c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
        sign, exp, man, bits, bias = c // 8, (c // 2) % 4, c % 2, 1, 1
    else:
        bits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
        c = codes.long()
        sign, exp, man = c // 128, (c % 128) // 2 ** bits, c % 2 ** bits
    man = man.double() / 2 ** bits
    v = torch.where(exp > 0, (1 + man) * _exact_power(exp - bias), man * 2.0 ** (1 - bias))
    return (1 - 2 * sign) * v * _exact_power(scale.long() - 127).repeat_interleave(32, 1)


def _exact_act(g, act):
    if act == "relu":
        return torch.where(g > 0, g, 0.0), torch.where(g > 0, 1.0, 0.0).double()
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)  # 0.5 (1 + tanh(z / 2)) = sigmoid(z)
    s = torch.sigmoid(z)
    return g * s, s + g * s * (1 - s) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "checkpoint":
        return {"restored": _exact_grid(s["x"].double(), s["fmt"])}
    if kind == "backward":
        if s["fmt"] == "bf16":
            x, gu = s["x"].double(), s["gu"].double()
        else:
            x, gu = _exact_value(s["x"], s["x_scale"], s["fmt"]), _exact_value(s["gu"], s["gu_scale"], s["fmt"])
        w = s["w"].double()
    else:
        x = s["x"].double()
        w = s["w"].double() if "w" in s else _exact_value(s["wq"], s["ws"], "e2m1")
        gu = torch.matmul(x, w.t())
        if kind == "mxfp4":
            return {"out": gu + s["bias_values"].double()[None, :] if s.get("bias") else gu}
    f = case["f"]
    if kind != "backward":
        h = _exact_act(gu[:, :f], s["act"])[0] * gu[:, f:]
        if kind != "train":
            return {"h": h}
        if s["fmt"] == "bf16":
            gu = gu.bfloat16().double()
        else:
            gu, x = _exact_grid(gu, s["fmt"]), _exact_grid(x, s["fmt"])
    a, d = _exact_act(gu[:, :f], s["act"])
    dh = s["dh"].double()
    dg, du = dh * gu[:, f:] * d, dh * a
    dx = torch.matmul(dg, w[:f]) + torch.matmul(du, w[f:])
    dw = torch.cat((torch.matmul(dg.t(), x), torch.matmul(du.t(), x)))
    return {"dx": dx, "dw": dw} if kind == "backward" else {"h": h, "dx": dx, "dw": dw}
