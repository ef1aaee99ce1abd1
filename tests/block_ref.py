"""Plain 64-bit forms of the gated feed-forward block and the MX formats, and
the error bounds their tests use.

Everything here is computed on the CPU or the tensors' device in binary64 from
the definitions.  Bounds count, per output:
  * one rounding to bf16: half a step, 2^-8 of the value (and 2^-133, half the
    smallest subnormal step);
  * the matrix cores' binary32-grade sums: every addition loses at most 2^-23 of
    the running magnitude, which never exceeds S = sum |a b| of the sum's
    terms, so a sum of n terms is off by at most n 2^-23 S;
  * act(g): the exponential's argument z is rounded, which moves exp(z) by
    |z| 2^-23 relative, and the few roundings after it by 2^-21 together: a
    relative (|z| + 4) 2^-22, z = g (SiLU) or the GELU polynomial's argument.
"""
import math

import torch

HALF_BF16 = 2.0 ** -8
U = 2.0 ** -23
MX = {  # largest element, mantissa bits, smallest normal exponent
    torch.float8_e4m3fn: (448.0, 3, -6),
    torch.float8_e5m2: (57344.0, 2, -14),
    torch.float4_e2m1fn_x2: (6.0, 1, 0),
}


def pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def floor_log2(a):
    """Exponent of positive binary64 values."""
    return ((a.view(torch.int64) >> 52) & 0x7FF) - 1023


def mx_round(x, dtype):
    """(values after the block format, scale bytes) of binary64 x [r, c], from the definition."""
    top, bits, low = MX[dtype]
    r, c = x.shape
    b = x.reshape(r, c // 32, 32)
    finite = torch.isfinite(b).all(2)
    b = torch.where(finite[:, :, None], b, 0.0)
    amax = b.abs().amax(2)
    e = torch.full_like(amax, -110.0)
    pos = amax > 0
    # smallest e with amax <= top 2^e: the exponent of amax / top, one up unless it is a whole power of two
    q = torch.where(pos, amax, 1.0)
    guess = floor_log2(q) - floor_log2(torch.tensor(top, dtype=torch.float64)).item()
    guess = guess + (q > top * pow2(guess)).long()
    e = torch.where(pos, guess.double(), e).clamp(min=-110)
    t = b / pow2(e)[:, :, None]
    step = pow2(floor_log2(t.abs().clamp(min=2.0 ** low)) - bits)
    v = torch.round(t / step) * step * pow2(e)[:, :, None]  # torch.round: halves to even
    # an element that would stand for 2^128 (past bf16 and binary32) is the one below: 2^128 less half its step there
    v = torch.where(v.abs() >= 2.0 ** 128, torch.copysign(torch.tensor(2.0 ** 128 - 2.0 ** (127 - bits), dtype=torch.float64), v), v)
    v = torch.where(finite[:, :, None], torch.copysign(v, b), math.nan)
    return v.reshape(r, c), torch.where(finite, e + 127, 255.0).to(torch.uint8)


def mx_values(t):
    """binary64 values of an MxTensor, from its bit fields."""
    codes, scale = t.codes.view(torch.uint8), t.scale.view(torch.uint8).long()
    if t.codes.dtype == torch.float4_e2m1fn_x2:
        c = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1).long()
        sign, exp, man, bits, bias = c >> 3, (c >> 1) & 3, c & 1, 1, 1
    elif t.codes.dtype == torch.float8_e4m3fn:
        c = codes.long()
        sign, exp, man, bits, bias = c >> 7, (c >> 3) & 15, c & 7, 3, 7
    else:
        c = codes.long()
        sign, exp, man, bits, bias = c >> 7, (c >> 2) & 31, c & 3, 2, 15
    frac = man.double() / 2 ** bits
    v = torch.where(exp > 0, (1 + frac) * pow2(exp - bias), frac * 2.0 ** (1 - bias)) * (1.0 - 2.0 * sign)
    s = torch.where(scale == 255, math.nan, pow2(scale - 127))
    return v * s.repeat_interleave(32, 1)


def act64(g, name):
    """act(g), its derivative and the magnitude of the exponential's argument, binary64."""
    if name == "relu":
        return torch.where(g < 0, 0.0, g), (g > 0).double(), torch.zeros_like(g)
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g), g.abs()
    # 0.5 (1 + tanh z) = sigmoid(2 z), which does not cancel for negative z
    c = math.sqrt(8 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    s, r = torch.sigmoid(z), torch.sigmoid(-z)
    return g * s, s + g * s * r * c * (1 + 3 * 0.044715 * g * g), z.abs().clamp(max=200)


def products64(x, w):
    """x @ w.T and the bound of a binary32-grade sum's error, for binary64 operands."""
    return x @ w.t(), x.shape[1] * U * (x.abs() @ w.abs().t())


def gated64(x, w, act):
    """(h, bound) of the gated block and (g, u, their bounds)."""
    f = w.shape[0] // 2
    p, e = products64(x, w)
    g, u, eg, eu = p[:, :f], p[:, f:], e[:, :f], e[:, f:]
    a, _, z = act64(g, act)
    ea = 1.13 * eg + (z + 4) * 2.0 ** -22 * a.abs()  # |act'| <= 1.13
    before = ea * (u.abs() + eu) + a.abs() * eu + U * (a * u).abs()
    h = a * u
    return h, (1 + HALF_BF16) * before + HALF_BF16 * h.abs() + 2.0 ** -133, (g, u, eg, eu)


def gated_grad64(dh, x, g, u, w, act):
    """(dx, bound, dw, bound) for binary64 operands taken as given.

    dg, du are rounded to bf16 (half a step each, and the activation's error),
    which the products then carry linearly; act' = s + g s (1 - s) ... has terms
    of magnitude up to 1 + |z|, so its error is that times (|z| + 4) 2^-22."""
    f = g.shape[1]
    a, d, z = act64(g, act)
    dg, du = dh * u * d, dh * a
    rel = (z + 4) * 2.0 ** -22
    eg = HALF_BF16 * dg.abs() + 2 * rel * (1 + z) * (dh * u).abs() + 2.0 ** -133
    eu = HALF_BF16 * du.abs() + 2 * rel * du.abs() + 2.0 ** -133
    dgu, e = torch.cat((dg, du), 1), torch.cat((eg, eu), 1)
    dx, dw = dgu @ w, dgu.t() @ x
    ex = e @ w.abs() + 2 * f * U * ((dgu.abs() + e) @ w.abs())
    ew = e.t() @ x.abs() + x.shape[0] * U * ((dgu.abs() + e).t() @ x.abs())
    return (dx, (1 + HALF_BF16) * ex + HALF_BF16 * dx.abs() + 2.0 ** -133,
            dw, (1 + HALF_BF16) * ew + HALF_BF16 * dw.abs() + 2.0 ** -133)


def check(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= bound)
    n = int(bad.sum())
    if n:
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {n} of {got.numel()} off; first at {i}: got {got[i].item()}, "
                             f"exact {ref[i].item()}, bound {bound[i].item()}")


def inputs(seed, m, k, rows, device="cuda", scale=0.05):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g).bfloat16()
    w = (scale * torch.randn(rows, k, generator=g)).bfloat16()
    return x.to(device), w.to(device)


def shapes_of(test):
    """The sizes that a test is parametrized over."""
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0].startswith("m,k,"):
            return list(mark.args[1])
    raise AssertionError(f"{test.__name__} has no sizes")
