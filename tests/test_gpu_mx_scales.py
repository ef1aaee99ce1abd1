"""GPU: MX blocks that quantize_mx did not write: every element code, the ones
that are no numbers among them, under every scale byte, decoded and in the
products.  Such a block stands for code * 2^(scale - 127), rounded to bf16."""
import pytest
import torch

from block_ref import MX, check, gated64, gated_grad64, inputs, mx_values, products64, HALF_BF16

pytestmark = pytest.mark.gpu
FP4 = torch.float4_e2m1fn_x2
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def decoded(t):
    """binary64 values of an MxTensor in bf16.  A value has four significant bits
    at most and is a whole multiple of 2^-149, so binary32 holds it exactly (or
    as an infinity) and it is rounded once."""
    v = mx_values(t)
    if t.codes.dtype != FP4:  # codes that are no numbers
        e = t.codes.float().double()
        nan = torch.isnan(v)
        v = torch.where(torch.isfinite(e) | nan, v, e)
    return v.float().bfloat16().double()


@pytest.mark.parametrize("dtype", list(MX), ids=str)
def test_decode(sfr, dtype):
    per = 16 if dtype == FP4 else 256
    codes = torch.arange(per, dtype=torch.uint8)
    if dtype == FP4:
        codes = codes.repeat(2)
        codes = codes[0::2] | (codes[1::2] << 4)
    scales = torch.arange(256, dtype=torch.uint8)
    q = sfr.MxTensor(codes[None].repeat(256, 1).view(dtype).contiguous(),
                     scales[:, None].repeat(1, max(per, 32) // 32).view(torch.float8_e8m0fnu).contiguous())
    want = decoded(q)
    got = sfr.dequantize_mx(sfr.MxTensor(q.codes.cuda(), q.scale.cuda())).cpu().double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan]) and torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))
    assert bool(nan[255].all()) and not bool(nan[:255, :16].any())
    if dtype == FP4:  # every value is a bf16 number up to scale 252
        assert torch.equal(want[:253], mx_values(q)[:253])


def weight(sfr, n, k, first, last, seed):
    """A 4-bit weight of random codes whose blocks have the scale bytes first .. last."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8)
    scale = torch.randint(first, last + 1, (n, 1), generator=g).to(torch.uint8).repeat(1, k // 32)
    return sfr.MxTensor(codes.view(FP4).cuda(), scale.view(torch.float8_e8m0fnu).cuda())


# The streamed forms and tiles.  x keeps every product and sum among binary32's normal numbers.
@pytest.mark.parametrize("first,last,power", [(0, 16, 100), (17, 60, 60), (200, 252, -110)])
@pytest.mark.parametrize("m", [1, 5, 16, 40, 130, 300])
def test_products(sfr, m, first, last, power):
    k, n = 288, 320
    q = weight(sfr, n, k, first, last, m)
    x = inputs(m, m, k, 16)[0] * 2.0 ** power
    ref, e = products64(x.double(), decoded(q))
    check(sfr.mxfp4_linear(x, q, out_dtype=torch.float32), ref, e, "binary32")
    check(sfr.mxfp4_linear(x, q), ref, e + HALF_BF16 * (ref.abs() + e) + 2.0 ** -133, "bf16")
    if power > 0:  # h = act(g) u stays finite
        for act in ("silu", "relu"):
            h, bound, _ = gated64(x.double(), decoded(q), act)
            check(sfr.mxfp4_gated_linear(x, q, act), h, bound, "h")


@pytest.mark.parametrize("dtype", [E4M3, E5M2], ids=str)
@pytest.mark.parametrize("m,k,f", [(5, 96, 64), (300, 288, 160)])
def test_gradients(sfr, dtype, m, k, f):
    """Saved activations of the smallest scales, with a gradient that makes up for them."""
    g = torch.Generator().manual_seed(m)

    def saved(cols):
        codes = torch.randn(m, cols, generator=g).to(dtype).cuda()
        scale = torch.randint(0, 17, (m, cols // 32), generator=g).to(torch.uint8).view(torch.float8_e8m0fnu).cuda()
        return sfr.MxTensor(codes, scale)
    sx, sgu = saved(k), saved(2 * f)
    w = inputs(m, m, k, 2 * f)[1]
    dh = (torch.randn(m, f, generator=g) * 2.0 ** 110).bfloat16().cuda()
    gu = decoded(sgu)
    rx, bx, rw, bw = gated_grad64(dh.double(), decoded(sx), gu[:, :f], gu[:, f:], w.double(), "silu")
    dx, dw = sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(sx, sgu, "silu"))
    assert bool((rx.abs() > 2.0 ** -60).any())
    check(dx, rx, bx, "dx")
    # dw's terms dg * x lie below 2^-100: the products' own steps are 2^-149
    check(dw, rw, bw + m * 2.0 ** -149, "dw")


def test_past_the_largest_number(sfr):
    """Elements that stand for 2^128 or more are infinities, as in bf16, in the products too."""
    codes = torch.zeros(16, 16, dtype=torch.uint8)
    codes[:, 0] = torch.arange(16, dtype=torch.uint8)  # column 0: every code; the others zero
    scale = torch.full((16, 1), 254, dtype=torch.uint8)
    q = sfr.MxTensor(codes.view(FP4).cuda(), scale.view(torch.float8_e8m0fnu).cuda())
    want = decoded(q)[:, 0]
    assert int(torch.isinf(want).sum()) == 8 and float(want[2]) == 2.0 ** 127  # 2, 3, 4, 6 and their negatives; 1
    x = torch.zeros(5, 32, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    got = sfr.mxfp4_linear(x, q, out_dtype=torch.float32)
    assert torch.equal(got.double(), want[None].repeat(5, 1))
