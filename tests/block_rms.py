"""Root-mean-square bounds of the gated block's and the 4-bit linear layer's
outputs, beside the per-output bounds of block_ref.

A per-output bound of a sum allows every rounding its worst sign, so for a long
sum it is wider than a block of missing terms.  Over many outputs of random
operands the roundings' signs do not agree, and the root mean square is known:

  * one rounding to bf16 is off by at most 2^-8 of the lower end of the value's
    binade, evenly spread, so by 2^-8 / sqrt(3) of the value at most in root
    mean square (ROUND);
  * a gradient's terms are products with dg or du, each rounded once: random
    operands of mean zero carry the same ratio to the sum, and the sum is
    rounded once more: 2 ROUND;
  * an addition of a binary32-grade sum loses at most 2^-23 of the running
    sum, whose root mean square over the outputs is sqrt(i / n) of the final
    one after i of n terms: (2 / 3) n 2^-23 together, whatever the signs;
  * the activation: below 2^-14 of its value and slope for the arguments here.

A sum of n terms that lacks 32 of them is off by sqrt(32 / n) of its value: 4%
at n = 20544, where the bounds allow 0.6%.  The ratio needs many outputs: with
1024 the mean square of an even spread is within 10% of its mean (three standard
deviations), and ROUND itself is a third above what values spread evenly over a
binade give.
"""
import math

import torch

from block_ref import U, act64

ROUND = 2.0 ** -8 / math.sqrt(3)
ENOUGH = 1024


def rms(t):
    return t.double().square().mean().sqrt().item()


def sums(n):
    return 2 / 3 * n * U


def check_rms(got, ref, allowed, what):
    """got's error is at most `allowed` of ref, both in root mean square."""
    off, size = rms(got.double() - ref), rms(ref)
    assert off <= allowed * size, f"{what}: off by {off / size:.3g} of its value, {allowed:.3g} allowed"


def gated_rms(g, u, act, k):
    """What h of a sum over k may be off by, from the exact projections."""
    a = act64(g, act)[0]
    moved = sums(k) * (1.13 * rms(g) + rms(a)) * rms(u) / rms(a * u)  # |act'| <= 1.13
    return ROUND + 2.0 ** -14 + (1 + ROUND) * moved


def linear_rms(k, bf16):
    return sums(k) + U + (ROUND if bf16 else 0)


def grad_rms(n):
    """dx (n = 2 f) or dw (n = m)."""
    return 2 * ROUND + 2.0 ** -14 + (1 + 2 * ROUND) * sums(n)


def gradients64(dh, x, g, u, w, act):
    """dx, dw and [dg du] in binary64."""
    a, d, _ = act64(g, act)
    dgu = torch.cat((dh * u * d, dh * a), 1)
    return dgu @ w, dgu.t() @ x, dgu
