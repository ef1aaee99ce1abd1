"""The root mean square bounds of the block's GPU tests, on the CPU: a result that
lacks 32 terms of a sum, or whose partial sums were rounded to bf16, fails them
at every shape those tests use, and a right one passes."""
import pytest
import torch

import block_rms
import test_gpu_block_rms as rms_tests
from block_ref import HALF_BF16, U, act64, inputs
from block_rms import check_rms, gated_rms, grad_rms, gradients64, linear_rms


def told(got, wrong, ref, allowed, what):
    check_rms(got, ref, allowed, what)
    with pytest.raises(AssertionError):
        check_rms(wrong, ref, allowed, what)


def without(t, n, dim):
    """t with up to 32 (half at most) of its n terms zero, at the end of the sum."""
    count = min(32, max(1, n // 2))
    t = t.clone()
    t.narrow(dim, n - count, count).zero_()
    return t


def part(t, dim, n=64):
    """64 rows or columns at most: the mistake is planted in a block of the oracle's outputs."""
    return t.narrow(dim, 0, min(n, t.shape[dim]))


@pytest.mark.parametrize("m,k,f", sorted(set(rms_tests.FORWARD)))
def test_forward_bound_tells_lost_terms(m, k, f):
    x, w = inputs(m, min(m, 256), k, 2 * min(f, 96), "cpu")
    x, w = x.double(), w.double()
    n = w.shape[0] // 2

    def h(x):
        p = x @ w.t()
        return act64(p[:, :n], "silu")[0] * p[:, n:], p[:, :n], p[:, n:]
    ref, g, u = h(x)
    told(ref.bfloat16(), h(without(x, k, 1))[0].bfloat16(), ref, gated_rms(g, u, "silu", k), "h")


@pytest.mark.parametrize("m,k,n", sorted(set(rms_tests.LINEAR)))
def test_linear_bound_tells_lost_terms_and_partial_roundings(m, k, n):
    x, w = inputs(m, min(m, 256), k, min(n, 256), "cpu")
    x, w = x.double(), w.double()
    ref = x @ w.t()
    lost = without(x, k, 1) @ w.t()
    told(ref.bfloat16(), lost.bfloat16(), ref, linear_rms(k, True), "bf16")
    told(ref.float(), lost.float(), ref, linear_rms(k, False), "binary32")
    # two halves of the sum, each rounded to bf16 before they are added
    half = k // 2
    halves = (x[:, :half] @ w[:, :half].t()).bfloat16().double() + (x[:, half:] @ w[:, half:].t()).bfloat16().double()
    told(ref.float(), halves.float(), ref, linear_rms(k, False), "binary32, partial sums in bf16")


@pytest.mark.parametrize("m,k,f", sorted(set(rms_tests.BACKWARD)))
def test_gradient_bounds_tell_lost_terms(m, k, f):
    g = torch.Generator().manual_seed(m + k)
    x, w = inputs(m, m, min(k, 64), 2 * f, "cpu")
    dh, gu = (torch.randn(m, c, generator=g).bfloat16().double() for c in (f, 2 * f))
    x, w = x.double(), w.double()
    dgu = gradients64(dh, x, gu[:, :f], gu[:, f:], w, "silu")[2]
    rounded = dgu.bfloat16().double()
    rows, wide = part(rounded, 0), part(rounded, 1)
    rx, rw = part(dgu, 0) @ w, part(dgu, 1).t() @ x
    told((rows @ w).bfloat16(), (without(rows, 2 * f, 1) @ w).bfloat16(), rx, grad_rms(2 * f), "dx")
    told((wide.t() @ x).bfloat16(), (without(wide, m, 0).t() @ x).bfloat16(), rw, grad_rms(m), "dw")


def test_worst_case_bound_does_not():
    """What the root mean square is for: at 20544 terms the per-output bound lets the lost terms pass."""
    g = torch.Generator().manual_seed(0)
    dgu, w = torch.randn(8, 20544, generator=g).double(), 0.05 * torch.randn(20544, 64, generator=g).double()
    ref = dgu @ w
    off = (without(dgu, 20544, 1) @ w - ref).abs()
    bound = (HALF_BF16 + 20544 * U) * (dgu.abs() @ w.abs())
    assert float((off <= bound).double().mean()) > 0.99
    assert block_rms.rms(off) > 5 * grad_rms(20544) * block_rms.rms(ref)
