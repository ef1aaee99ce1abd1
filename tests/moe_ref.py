"""64-bit forms of the expert router and the mixture-of-experts layer, with the
error bounds that their tests use (the parts of block_ref).

Layer, per output: every h is off by block_ref.gated64's bound (the two binary32
sums, the activation and the rounding to bf16), which the second product carries
linearly with the weight's size; that product is a binary32-grade sum over at most
top * f terms and the wavefronts' joins, each addition losing at most 2^-23 of S =
sum |weight h wd|; a scale and a weight are one rounding (2^-24) each, and a scale
of the first product moves g and u by as much; the result is rounded to bf16."""
import math

import torch

from block_ref import HALF_BF16, U, gated64, mx_values

FP4 = torch.float4_e2m1fn_x2


def experts64(w, n):
    """binary64 [experts, n, c] of an experts' weight in any of its forms."""
    if isinstance(w, torch.Tensor):
        return w.double()
    if w.codes.dtype == torch.int8:
        v = w.codes.double() * w.scale.double()[:, None]
    else:
        v = mx_values(w)
    return v.view(-1, n, v.shape[1])


def layer64(x, ids, weights, w_gate_up, w_down, act):
    """(out, bound) for bf16 x [m, k]; ids outside the experts are no choice."""
    m, k = x.shape
    down = experts64(w_down, k)
    experts, _, f = down.shape
    gu = experts64(w_gate_up, 2 * f)
    x = x.double()
    out = torch.zeros(m, k, dtype=torch.float64, device=x.device)
    bound, size = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(experts):
        wt = (weights.double() * (ids == e)).sum(1)
        rows = torch.nonzero((ids == e).any(1))[:, 0]
        if not rows.numel():
            continue
        h, eh, _ = gated64(x[rows], gu[e], act)
        eh = eh + 3 * U * h.abs()  # scales of g and u: half a step each, twice over in the activation's slope
        wt, d = wt[rows, None], down[e]
        out[rows] += wt * (h @ d.t())
        bound[rows] += wt.abs() * (eh @ d.abs().t())
        size[rows] += wt.abs() * ((h.abs() + eh) @ d.abs().t())
    bound = bound + (ids.shape[1] * f + 32) * U * size
    return out, (1 + HALF_BF16) * bound + HALF_BF16 * out.abs() + 2.0 ** -133


def weights64(logits, ids, score, renormalize):
    """(weights, relative bound) from the router's own logits and ids.

    exp(l - best): the difference is rounded (|l - best| 2^-24), expf is good to two
    steps; s(l) by differences of log s, each a few roundings of |log s| <= |l| + 1;
    sums and the quotient: a rounding per six joins and two more."""
    l = logits.double()
    best = torch.gather(l, 1, ids.clamp(min=0).long())
    best = torch.where(ids < 0, -math.inf, best)
    if score == "softmax":
        top = l.amax(1, keepdim=True)
        p = torch.exp(best - top)
        total = p.sum(1, keepdim=True) if renormalize else torch.exp(l - top).sum(1, keepdim=True)
        args = torch.where(ids < 0, 0.0, top - best)
    else:
        log_s = torch.nn.functional.logsigmoid(best)
        top = log_s.amax(1, keepdim=True)
        p = torch.exp(log_s - top) if renormalize else torch.sigmoid(best)
        total = p.sum(1, keepdim=True) if renormalize else torch.ones_like(top)
        args = 2 * (torch.where(ids < 0, 0.0, best.abs()).amax(1, keepdim=True) + 1)
    w = p / total
    return torch.where(ids < 0, 0.0, w), (args + 12) * U


def stacked(gen_seed, m, k, f, experts, top, form, sfr, scale=0.1):
    """x, ids, weights and the experts' weights in `form` on the GPU."""
    g = torch.Generator("cuda").manual_seed(gen_seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = r(m, k).bfloat16()
    ids = torch.argsort(r(m, experts), 1)[:, :top].int().contiguous()
    weights = torch.softmax(r(m, ids.shape[1]), 1)
    gu = (scale * r(experts, 2 * f, k)).bfloat16()
    down = (scale * r(experts, k, f)).bfloat16()
    return (x, ids, weights, *as_form(sfr, gu, down, form))


def as_form(sfr, gu, down, form):
    if form == "bf16":
        return gu, down
    flat = [w.reshape(-1, w.shape[2]) for w in (gu, down)]
    if form == "int8":
        return tuple(sfr.quantize_rowwise_int8(w) for w in flat)
    return tuple(sfr.quantize_mx(w, FP4) for w in flat)
