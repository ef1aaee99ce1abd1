"""64-bit forms of the 8-bit integer layer.

Codes are whole numbers decided by an exact quotient, sums are whole numbers
under 2^31: both are exact in binary64, and tests ask for equality.  A binary32
output is the sum rounded to binary32, times the binary32 product of the scales,
plus the bias, rounded once: the last rounding is half a step, 2^-24 of the value
(2^-150 below the normal numbers), beside what binary64 itself loses (2^-50)."""
import torch


def codes64(x):
    """(codes, scale) of bf16 x, from the definition.  127 x has 15 bits, so the
    binary64 quotient is off by 2^-53 of itself at most and a quotient that is no
    half-integer is 2^-16 of itself away from one: rounding it rounds the exact one."""
    x = x.double().cpu()
    amax = x.abs().amax(1, keepdim=True)
    finite = torch.isfinite(x).all(1, keepdim=True)
    live = finite & (amax > 0)
    q = torch.where(live, torch.round(127 * torch.where(live, x, 0.0) / torch.where(live, amax, 1.0)), 0.0)
    scale = amax[:, 0].float() / 127  # one IEEE division
    return q.to(torch.int8), torch.where(finite[:, 0], scale, torch.nan)


def linear64(xq, xs, wq, ws, bias=None):
    """(out, bound) of a binary32 output, for int8 codes and float32 scales."""
    total = (xq.double() @ wq.double().t()).float().double()  # exact, then rounded as the kernels do
    s = (xs[:, None] * ws[None, :]).double()                  # a binary32 product
    y = total * s
    if bias is not None:
        y = y + bias.double()
    return y, 2.0 ** -24 * (1 + 2.0 ** -20) * y.abs() + 2.0 ** -149
