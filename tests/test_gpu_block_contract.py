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


def calls(sfr, x, w, q, dh, **kw):
    """One call of each operator, with `kw`, and of those with `out` into one."""
    m, f = dh.shape
    h, saved = sfr.gated_linear_checkpointed(x, w, **kw)
    dx, dw = sfr.gated_linear_backward(dh, w, saved, **kw)
    outs = [torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for n in (f, f, 2 * f, x.shape[1])]
    return [h, dx, dw, sfr.gated_linear(x, w, out=outs[0], **kw), sfr.mxfp4_gated_linear(x, q, out=outs[1], **kw),
            sfr.mxfp4_linear(x, q, out=outs[2], **kw), sfr.dequantize_mx(saved.x, out=outs[3], **kw), *outs]


@pytest.mark.parametrize("m,k,f", [(3, 4128, 1056), (130, 4128, 2080)])
def test_explicit_stream_in_a_graph(sfr, m, k, f):
    """Calls with an explicit stream captured into a graph: the capturing stream
    named, and a side stream that the capture forks into and joins again.
    Replayed with new inputs and eager work between, and after the inputs'
    neighbours in memory were freed."""
    x, w = inputs(3, m, k, 2 * f)
    q, dh = sfr.quantize_mx(w, torch.float4_e2m1fn_x2), inputs(4, m, f, 16)[0]
    calls(sfr, x, w, q, dh)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        first = calls(sfr, x, w, q, dh, stream=here)
        side.wait_stream(here)
        second = calls(sfr, x, w, q, dh, stream=side)
        here.wait_stream(side)
    for i in range(3):
        nx, nw = inputs(10 + i, m, k, 2 * f)
        nq = sfr.quantize_mx(nw, torch.float4_e2m1fn_x2)
        x.copy_(nx)
        w.copy_(nw)
        dh.copy_(inputs(20 + i, m, f, 16)[0])
        q.codes.view(torch.uint8).copy_(nq.codes.view(torch.uint8))
        q.scale.view(torch.uint8).copy_(nq.scale.view(torch.uint8))
        del nx, nw, nq
        graph.replay()
        want = calls(sfr, x, w, q, dh)
        torch.cuda.synchronize()
        for a, b, c in zip(first, second, want):
            assert torch.equal(a, c) and torch.equal(b, c), i


def test_inputs_that_are_one_tensor(sfr):
    """The same tensor as activation and weight, and h as its own gradient."""
    w = inputs(5, 16, 96, 128)[1]
    copy = w.clone()
    h, saved = sfr.gated_linear_checkpointed(w, w, checkpoint=torch.bfloat16)
    hp, sp = sfr.gated_linear_checkpointed(copy, w, checkpoint=torch.bfloat16)
    assert torch.equal(h, hp) and torch.equal(w, copy)
    for a, b in zip(sfr.gated_linear_backward(h, w, saved), sfr.gated_linear_backward(hp.clone(), copy, sp)):
        assert torch.equal(a, b)
