"""GPU: the gated block, its gradients and its 4-bit forms against 64-bit
results in root mean square (bounds: block_rms), on the shapes that reach every
kernel."""
import pytest
import torch

import test_gpu_block_kernels
import test_gpu_gated
import test_gpu_gated_more
from block_ref import gated64, inputs, mx_values, products64, shapes_of
from block_rms import ENOUGH, check_rms, gated_rms, grad_rms, gradients64, linear_rms

pytestmark = pytest.mark.gpu
FP4 = torch.float4_e2m1fn_x2
FORWARD = [s for s in test_gpu_gated.SHAPES + shapes_of(test_gpu_gated_more.test_forward_tiles)
           + shapes_of(test_gpu_block_kernels.test_forward_few_rows) if s[0] * s[2] >= ENOUGH]
LINEAR = [s for s in shapes_of(test_gpu_gated.test_mxfp4_linear) + shapes_of(test_gpu_gated_more.test_mxfp4_linear_tiles)
          + shapes_of(test_gpu_gated_more.test_mxfp4_streamed) if s[0] * s[2] >= ENOUGH]
BACKWARD = [s for s in test_gpu_gated.SHAPES + shapes_of(test_gpu_gated_more.test_backward_tiles)
            + shapes_of(test_gpu_block_kernels.test_backward_sliced) if s[0] * min(s[1], s[2]) >= ENOUGH]


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("m,k,f", FORWARD)
def test_forward_rms(sfr, m, k, f):
    x, w = inputs(m + f, m, k, 2 * f)
    h, _, (g, u, _, _) = gated64(x.double(), w.double(), "silu")
    allowed = gated_rms(g, u, "silu", k)
    check_rms(sfr.gated_linear(x, w), h, allowed, "h")
    got, saved = sfr.gated_linear_checkpointed(x, w, checkpoint=torch.bfloat16)
    check_rms(got, h, allowed, "h, saving")
    check_rms(saved.gu, torch.cat((g, u), 1), linear_rms(k, True), "gu")
    q = sfr.quantize_mx(w, FP4)
    h, _, (g, u, _, _) = gated64(x.double(), mx_values(q), "silu")
    check_rms(sfr.mxfp4_gated_linear(x, q), h, gated_rms(g, u, "silu", k), "h, 4-bit weight")


@pytest.mark.parametrize("m,k,n", LINEAR)
def test_mxfp4_linear_rms(sfr, m, k, n):
    x, w = inputs(m + n, m, k, n)
    q = sfr.quantize_mx(w, FP4)
    ref, _ = products64(x.double(), mx_values(q))
    check_rms(sfr.mxfp4_linear(x, q, out_dtype=torch.float32), ref, linear_rms(k, False), "binary32")
    check_rms(sfr.mxfp4_linear(x, q), ref, linear_rms(k, True), "bf16")
    bias = randn(n, n)
    check_rms(sfr.mxfp4_linear(x, q, bias), ref + bias.double(), linear_rms(k, True), "bf16, with a bias")


@pytest.mark.parametrize("m,k,f", BACKWARD)
def test_backward_rms(sfr, m, k, f):
    x, w = inputs(m + f, m, k, 2 * f)
    dh, gu = randn(m, m, f), randn(m + 1, m, 2 * f)
    for act in ("silu", "relu"):
        dx, dw = sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(x, gu, act))
        rx, rw, _ = gradients64(dh.double(), x.double(), gu[:, :f].double(), gu[:, f:].double(), w.double(), act)
        check_rms(dx, rx, grad_rms(2 * f), f"dx, {act}")
        check_rms(dw, rw, grad_rms(m), f"dw, {act}")


def test_gradient_error_is_two_roundings(sfr):
    """The gradients' error at a size of a model: dg and du are rounded to bf16
    before the products and the result once after, so between one rounding's
    spread and two's."""
    m, k, f = 700, 1184, 1056
    x, w = inputs(m, m, k, 2 * f)
    dh, gu = randn(m, m, f), randn(m + 1, m, 2 * f)
    dx, dw = sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(x, gu, "silu"))
    rx, rw, dgu = gradients64(dh.double(), x.double(), gu[:, :f].double(), gu[:, f:].double(), w.double(), "silu")
    rounded = dgu.bfloat16().double()
    # Against the products of the rounded dg and du the last rounding is left, and
    # the dg and du whose binary32 value lies on the other side of a rounding
    # border: off by 2^-16 at most (the activation, for |g| < 8), that is one in
    # 256 of the steps of 2^-8, and then by a step: sqrt(2^-8) 2^-8, a quarter of ROUND's 2^-8 / sqrt(3) at most.
    check_rms(dx, rounded @ w.double(), 1.25 * linear_rms(2 * f, True), "dx")
    check_rms(dw, rounded.t() @ x.double(), 1.25 * linear_rms(m, True), "dw")
