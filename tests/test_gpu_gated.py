"""GPU: the gated feed-forward block, its gradients and its 4-bit form against
plain 64-bit forms; bounds are derived in block_ref."""
import pytest
import torch

from block_ref import (act64, check, gated64, gated_grad64, inputs, mx_round, mx_values, products64, HALF_BF16)

pytestmark = pytest.mark.gpu
ACTS = ["silu", "gelu_tanh", "relu"]
FP4 = torch.float4_e2m1fn_x2
CHECKPOINTS = [torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2]
# m, k, f: one row to several tiles, odd rows, k and f at the ends of tiles and inside them
SHAPES = [(1, 32, 32), (1, 4096, 160), (2, 96, 64), (15, 160, 96), (16, 128, 32), (17, 224, 128), (32, 288, 288),
          (33, 512, 64), (63, 64, 96), (64, 320, 160), (65, 96, 192), (127, 416, 96), (128, 128, 128),
          (129, 1056, 224), (255, 192, 160), (257, 64, 352), (300, 608, 544), (513, 256, 288), (700, 1184, 1056)]


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k,f", SHAPES)
def test_forward(sfr, m, k, f, act):
    x, w = inputs(m + k, m, k, 2 * f)
    h, bound, _ = gated64(x.double(), w.double(), act)
    check(sfr.gated_linear(x, w, act), h, bound, "h")


@pytest.mark.parametrize("checkpoint", CHECKPOINTS, ids=str)
@pytest.mark.parametrize("m,k,f", SHAPES)
def test_checkpoint(sfr, m, k, f, checkpoint):
    """h, and the saved x and projections: a projection's saved value lies
    between the format's values of the ends of its binary32 error interval."""
    x, w = inputs(m + k, m, k, 2 * f)
    h, bound, (g, u, eg, eu) = gated64(x.double(), w.double(), "silu")
    got, saved = sfr.gated_linear_checkpointed(x, w, "silu", checkpoint=checkpoint)
    check(got, h, bound, "h")
    gu, e = torch.cat((g, u), 1), torch.cat((eg, eu), 1)
    if checkpoint == torch.bfloat16:
        assert saved.x is x
        check(saved.gu, gu, e + HALF_BF16 * (gu.abs() + e) + 2.0 ** -133, "gu")
        return
    assert torch.equal(mx_values(saved.x), mx_round(x.double().cpu(), checkpoint)[0].cuda())
    # The scale is one of the two that the block maximum's interval allows; a
    # step of the format under the larger one is at most 2^-3 (e4m3) or 2^-2
    # (e5m2) of the value, or 2^-9 / 2^-16 of the scale below its normals: half
    # of that is the rounding.
    bits, low = (3, 2.0 ** -9) if checkpoint == torch.float8_e4m3fn else (2, 2.0 ** -16)
    v = mx_values(saved.gu)
    block = (gu.abs() + e).reshape(m, -1, 32).amax(2)
    top = 448.0 if checkpoint == torch.float8_e4m3fn else 57344.0
    s = saved.gu.scale.view(torch.uint8).double()
    scale = torch.exp2(s - 127)
    lower = (gu.abs() - e).clamp(min=0).reshape(m, -1, 32).amax(2)
    assert bool((lower <= top * scale).all()) and bool(((block > top * scale / 2) | (s == 17)).all())
    half = torch.maximum(2.0 ** -(bits + 1) * (gu.abs() + e), (low / 2 * scale).repeat_interleave(32, 1))
    check(v, gu, e + half, "gu")


def dequantized(sfr, t):
    return mx_values(t) if isinstance(t, sfr.MxTensor) else t.double()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("checkpoint", CHECKPOINTS, ids=str)
@pytest.mark.parametrize("m,k,f", SHAPES)
def test_backward(sfr, m, k, f, checkpoint, act):
    x, w = inputs(m + k, m, k, 2 * f)
    dh = torch.randn(m, f, generator=torch.Generator().manual_seed(m)).bfloat16().cuda()
    _, saved = sfr.gated_linear_checkpointed(x, w, act, checkpoint=checkpoint)
    dx, dw = sfr.gated_linear_backward(dh, w, saved)
    gu = dequantized(sfr, saved.gu)
    rx, bx, rw, bw = gated_grad64(dh.double(), dequantized(sfr, saved.x), gu[:, :f], gu[:, f:], w.double(), act)
    check(dx, rx, bx, "dx")
    check(dw, rw, bw, "dw")
    only_dx, none = sfr.gated_linear_backward(dh, w, saved, need_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = sfr.gated_linear_backward(dh, w, saved, need_dx=False)
    assert none is None and torch.equal(only_dw, dw)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradient_against_differences(sfr, act):
    """The gradients against central differences of the plain form in 64 bits
    along random directions.  The step's own error is h^2 / 6 of a third
    derivative: with h = 1e-4 far below the gradients' rounding (2^-7 of the
    terms' root sum of squares, ten times which is allowed for the direction's sum)."""
    m, k, f = 24, 64, 96
    x, w = inputs(5, m, k, 2 * f)
    dh = torch.randn(m, f, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    _, saved = sfr.gated_linear_checkpointed(x, w, act, checkpoint=torch.bfloat16)
    # the saved projections are rounded to bf16 too: half a step in g and u
    dx, dw = sfr.gated_linear_backward(dh, w, saved)

    def loss(xx, ww):
        p = xx @ ww.t()
        return (act64(p[:, :f], act)[0] * p[:, f:] * dh.double()).sum()
    g = torch.Generator().manual_seed(7)
    for i in range(4):
        vx = torch.randn(m, k, generator=g, dtype=torch.float64).cuda()
        vw = torch.randn(2 * f, k, generator=g, dtype=torch.float64).cuda()
        t = 1e-4
        nx = (loss(x.double() + t * vx, w.double()) - loss(x.double() - t * vx, w.double())) / (2 * t)
        nw = (loss(x.double(), w.double() + t * vw) - loss(x.double(), w.double() - t * vw)) / (2 * t)
        ax, aw = (dx.double() * vx).sum(), (dw.double() * vw).sum()
        assert abs(nx - ax) <= 10 * 2.0 ** -7 * (dx.double() * vx).norm(), (i, nx, ax)
        assert abs(nw - aw) <= 10 * 2.0 ** -7 * (dw.double() * vw).norm(), (i, nw, aw)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,k,n", [(1, 32, 16), (1, 4096, 48), (2, 96, 64), (5, 14336, 80), (16, 160, 16),
                                   (17, 224, 144), (32, 128, 32), (33, 288, 96), (64, 1056, 272), (65, 96, 16),
                                   (128, 512, 128), (130, 416, 400), (300, 608, 1040)])
def test_mxfp4_linear(sfr, m, k, n, bias, out_dtype):
    x, w = inputs(m + k, m, k, n)
    q = sfr.quantize_mx(w, FP4)
    b = torch.randn(n, generator=torch.Generator().manual_seed(n)).bfloat16().cuda() if bias else None
    ref, e = products64(x.double(), mx_values(q))
    if bias:
        ref = ref + b.double()
        e = e + 2.0 ** -24 * (ref.abs() + e)  # the addition's own rounding
    bound = e if out_dtype == torch.float32 else e + HALF_BF16 * (ref.abs() + e) + 2.0 ** -133
    check(sfr.mxfp4_linear(x, q, b, out_dtype=out_dtype), ref, bound, "out")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k,f", SHAPES)
def test_mxfp4_gated(sfr, m, k, f, act):
    x, w = inputs(m + k, m, k, 2 * f)
    q = sfr.quantize_mx(w, FP4)
    h, bound, _ = gated64(x.double(), mx_values(q), act)
    check(sfr.mxfp4_gated_linear(x, q, act), h, bound, "h")


def test_no_rows(sfr):
    k, f = 96, 64
    x, w = inputs(1, 0, k, 2 * f)
    assert sfr.gated_linear(x, w).shape == (0, f)
    for c in CHECKPOINTS:
        h, saved = sfr.gated_linear_checkpointed(x, w, checkpoint=c)
        dx, dw = sfr.gated_linear_backward(h, w, saved)
        assert h.shape == (0, f) and dx.shape == (0, k)
        assert dw.shape == (2 * f, k) and int((dw != 0).sum()) == 0
    q = sfr.quantize_mx(w, FP4)
    assert sfr.mxfp4_linear(x, q).shape == (0, 2 * f)
    assert sfr.mxfp4_gated_linear(x, q).shape == (0, f)
