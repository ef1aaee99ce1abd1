"""GPU: what the gated block's documentation says of the edges: no autograd
graph, ReLU's slope at NaN and zero, the factor that act loses far below zero."""
import math

import pytest
import torch

from block_ref import check, gated64, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def test_no_graph(sfr):
    """Results of leaves that require grad have no graph; the same numbers as without."""
    x, w = inputs(1, 20, 96, 128)
    q = sfr.quantize_mx(w, torch.float4_e2m1fn_x2)
    lx, lw = x.clone().requires_grad_(), torch.nn.Parameter(w.clone())
    for checkpoint in (torch.bfloat16, torch.float8_e4m3fn):
        h, saved = sfr.gated_linear_checkpointed(lx, lw, checkpoint=checkpoint)
        dx, dw = sfr.gated_linear_backward(h, lw, saved)
        hp, sp = sfr.gated_linear_checkpointed(x, w, checkpoint=checkpoint)
        px, pw = sfr.gated_linear_backward(hp, w, sp)
        for a, b in ((h, hp), (dx, px), (dw, pw)):
            assert not a.requires_grad and torch.equal(a, b)
    for a, b in ((sfr.gated_linear(lx, lw), sfr.gated_linear(x, w)), (sfr.mxfp4_linear(lx, q), sfr.mxfp4_linear(x, q)),
                 (sfr.mxfp4_gated_linear(lx, q), sfr.mxfp4_gated_linear(x, q))):
        assert not a.requires_grad and torch.equal(a, b)
    assert lx.grad is None and lw.grad is None


def test_relu_slope_at_nan_and_zero(sfr):
    """relu' is 1 above zero and 0 elsewhere, at NaN too: a NaN g reaches dx and the up rows of dw through act(g)."""
    m, k, f = 5, 96, 64
    x, w = inputs(2, m, k, 2 * f)
    gu = torch.ones(m, 2 * f, dtype=torch.bfloat16, device="cuda")
    gu[:, 3], gu[:, 4], gu[1, 5] = 0.0, -0.0, math.nan
    dh = torch.ones(m, f, dtype=torch.bfloat16, device="cuda")
    dx, dw = sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(x, gu, "relu"))
    rows = torch.arange(m, device="cuda") != 1
    assert bool(torch.isnan(dx[1]).all()) and bool(torch.isfinite(dx[rows]).all())
    assert bool(torch.isnan(dw[f + 5]).all())
    assert bool((dw[3] == 0).all()) and bool((dw[4] == 0).all())
    rest = torch.arange(2 * f, device="cuda") != f + 5
    assert bool(torch.isfinite(dw[rest]).all())
    # dw[5] is the sum over the other rows; each g = u = 1, so dg = dh
    ref = x[rows].double().sum(0)
    assert bool(((dw[5].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + m * 2.0 ** -23 * x.double().abs().sum(0)).all())


@pytest.mark.parametrize("m", [1, 8, 40])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_far_below_zero(sfr, m, act):
    """The logistic factor may be 0 where it is below 2^-126 (SiLU: g < -87.3): h is
    off by |g u| 2^-126 at most, and right above."""
    k, f = 32, 512
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 2.0 ** 100
    w = torch.zeros(2 * f, k, device="cuda")
    w[:f, 0] = torch.linspace(-110, -1, f)
    w[f:, 1] = 1.0
    w = w.bfloat16()
    h, bound, (g, u, _, _) = gated64(x.double(), w.double(), act)
    assert bool((h.abs() > 1e-6).any())
    check(sfr.gated_linear(x, w, act), h, bound + (g * u).abs() * 2.0 ** -126, "h")
