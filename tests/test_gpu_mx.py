"""GPU: MX block formats against their definition in 64 bits, bit for bit."""
import math

import pytest
import torch

from block_ref import MX, mx_round, mx_values

pytestmark = pytest.mark.gpu
DTYPES = list(MX)


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def same_values(got, want):
    """Equal, zeros by sign and NaN as NaN."""
    got, want = got.double().cpu(), want.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])
    assert torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))


def data(kind, rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if kind == "wide":      # magnitudes over the whole range of bf16
        x = x * torch.exp2(torch.randint(-126, 120, (rows, cols // 32), generator=g).float()).repeat_interleave(32, 1)
    elif kind == "zeros":   # zero blocks of both signs, single values
        x = x * (torch.rand(rows, cols, generator=g) < 0.03)
        x = torch.where(torch.rand(rows, cols, generator=g) < 0.5, -x, x)
    elif kind == "bits":    # every finite bf16 pattern may appear
        b = torch.randint(0, 65536, (rows, cols), generator=g)
        b = torch.where((b & 0x7F80) == 0x7F80, b & 0xBFFF, b)
        return b.to(torch.int32).to(torch.int16).view(torch.bfloat16)
    elif kind == "halves":  # values halfway between two elements, and block maxima at the largest element
        x = torch.randint(-64, 65, (rows, cols), generator=g).float() / 16
        x[:, ::32] = torch.tensor([448.0, 6.0, 57344.0, 449.0])[torch.randint(0, 4, x[:, ::32].shape, generator=g)]
    return x.bfloat16()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("kind", ["normal", "wide", "zeros", "bits", "halves"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (37, 2080), (129, 4096)])
def test_round_trip(sfr, dtype, kind, rows, cols):
    x = data(kind, rows, cols, rows + cols)
    v, s = mx_round(x.double(), dtype)
    q = sfr.quantize_mx(x.cuda(), dtype)
    assert torch.equal(q.scale.view(torch.uint8).cpu(), s)
    cpu = sfr.MxTensor(q.codes.cpu(), q.scale.cpu())
    same_values(mx_values(cpu), v)
    same_values(sfr.dequantize_mx(q), v)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_not_finite(sfr, dtype):
    x = data("normal", 4, 128, 1)
    x[0, 5], x[1, 40], x[2, 64] = math.nan, math.inf, -math.inf
    x[3, 96:] = math.nan
    v, s = mx_round(x.double(), dtype)
    assert int((s == 255).sum()) == 4
    q = sfr.quantize_mx(x.cuda(), dtype)
    assert torch.equal(q.scale.view(torch.uint8).cpu(), s)
    same_values(sfr.dequantize_mx(q), v)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_decode_every_code(sfr, dtype):
    """Every element code under every scale byte that quantize_mx writes."""
    per = 16 if dtype == torch.float4_e2m1fn_x2 else 256
    codes = torch.arange(per, dtype=torch.uint8)
    if per == 16:
        codes = codes.repeat(2)
        codes = codes[0::2] | (codes[1::2] << 4)
    else:  # a NaN or infinity code is never written in a finite block
        codes = torch.where(torch.isfinite(codes.view(dtype).float()), codes, 0)
    top = {torch.float8_e4m3fn: 246, torch.float8_e5m2: 239, torch.float4_e2m1fn_x2: 252}[dtype]
    scales = torch.tensor(list(range(17, top + 1)) + [255], dtype=torch.uint8)
    cols = max(per, 32)
    q = sfr.MxTensor(codes[None].repeat(len(scales), 1).view(dtype).contiguous(),
                     scales[:, None].repeat(1, cols // 32).view(torch.float8_e8m0fnu).contiguous())
    want = mx_values(q)
    got = sfr.dequantize_mx(sfr.MxTensor(q.codes.cuda(), q.scale.cuda()))
    same_values(got, want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_rows_behind_are_left(sfr, dtype):
    """Outputs end at the last row: what lies behind it is untouched."""
    lib, h = sfr.load(), int(torch.cuda.current_stream().cuda_stream)
    rows, cols, per = 5, 96, (48 if dtype == torch.float4_e2m1fn_x2 else 96)
    x = data("normal", rows, cols, 3).cuda()
    q = torch.full((rows + 2, per), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((rows * 3 + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    o = torch.full((rows + 2, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    kind = sfr._MX[dtype]
    assert lib.quantize_mx(x.data_ptr(), rows, cols, kind, q.data_ptr(), s.data_ptr(), h) == 0
    assert lib.dequantize_mx(q.data_ptr(), s.data_ptr(), rows, cols, kind, o.data_ptr(), h) == 0
    assert int((q[rows:] != 0xA5).sum()) == 0 and int((s[rows * 3:] != 0xA5).sum()) == 0
    assert int((o[rows:] != 7.0).sum()) == 0
    v, _ = mx_round(x.double().cpu(), dtype)
    same_values(o[:rows], v)


def test_empty(sfr):
    q = sfr.quantize_mx(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 64) and q.scale.shape == (0, 2)
    assert sfr.dequantize_mx(q).shape == (0, 64)
