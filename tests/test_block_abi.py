"""The gated block's and the MX formats' entry points on the CPU: invalid
arguments are refused with the documented status before anything is launched
(so these calls need no GPU), and the 64-bit references agree with themselves."""
import math
import os

import pytest
import torch

from block_ref import MX, mx_round, mx_values

OK, NULL, SHAPE, ALIGN, DTYPE = 0, 1, 2, 3, 4
A, U = 0x10000, 0x10001  # 16-byte aligned and misaligned stand-in addresses, never dereferenced
BIG = 1 << 20


@pytest.fixture(scope="module")
def sfr():
    import sparse_fp8_row_amd as sfr
    if not os.path.exists(sfr.LIB_PATH):
        from sparse_fp8_row_amd import build
        build.build()
    sfr.load()
    return sfr


def caller(fn, order, good):
    def call(**kw):
        a = dict(good, **kw)
        return fn(*[a[k] for k in order.split()], None)
    return call


@pytest.mark.parametrize("name", ["quantize_mx", "dequantize_mx"])
def test_mx_validation(sfr, name):
    if name == "quantize_mx":
        call = caller(sfr.load().quantize_mx, "x rows cols dt q s", dict(x=A, rows=4, cols=64, dt=0, q=A, s=A))
    else:
        call = caller(sfr.load().dequantize_mx, "q s rows cols dt x", dict(x=A, rows=4, cols=64, dt=0, q=A, s=A))
    assert call(dt=3) == DTYPE and call(dt=-1) == DTYPE
    for bad in (dict(cols=48), dict(cols=0), dict(cols=-32), dict(rows=-1), dict(rows=(1 << 30) + 1),
                dict(cols=(1 << 30) + 32), dict(rows=1 << 30, cols=1 << 20)):
        assert call(**bad) == SHAPE, bad
    assert call(rows=0, x=None, q=None, s=None) == OK
    for t in ("x", "q", "s"):
        assert call(**{t: None}) == NULL and call(**{t: U}) == ALIGN


def test_gated_validation(sfr):
    call = caller(sfr.load().gated_linear_bf16, "x m k w f act h save gu gs",
                  dict(x=A, m=4, k=64, w=A, f=96, act=0, h=A, save=2, gu=A, gs=A))
    assert call(act=3) == DTYPE and call(act=-1) == DTYPE and call(save=4) == DTYPE and call(save=-1) == DTYPE
    for bad in (dict(m=-1), dict(m=(1 << 30) + 1), dict(k=48), dict(k=0), dict(k=BIG + 32), dict(f=48), dict(f=0),
                dict(f=-32), dict(f=BIG // 2 + 32), dict(m=1 << 30, f=BIG // 2), dict(f=32 - (1 << 63))):
        assert call(**bad) == SHAPE, bad
    assert call(m=0, x=None, h=None, gu=None, gs=None) == OK
    for t in ("x", "w", "h", "gu", "gs"):
        assert call(**{t: None}) == NULL and call(**{t: U}) == ALIGN
    # without the 8-bit form its arguments are not looked at (checked by what is refused next)
    assert call(save=0, gu=None, gs=None, x=None) == NULL
    assert call(save=1, gs=U, x=U) == ALIGN
    assert call(save=1, gu=None) == NULL


def test_gated_backward_validation(sfr):
    lib = sfr.load()
    need = lib.sfr_gated_backward_workspace_bytes
    assert need(4, 64, 96, 1) == 4 * 192 * 2 and need(4, 64, 96, 2) == 4 * 192 * 2 + 4 * 64 * 2
    assert need(4, 64, 1 << 14, 1) > 4 * (1 << 15) * 2  # a long sum over f: slices
    assert need(0, 64, 96, 2) == 0 and need(4, 48, 96, 2) == 0 and need(4, 64, 96, 0) == 0 and need(-1, 64, 96, 1) == 0
    call = caller(lib.gated_linear_bf16_backward, "dh m k f act gu gs gsave x xs xsave w dx dw work bytes",
                  dict(dh=A, m=4, k=64, f=96, act=1, gu=A, gs=A, gsave=2, x=A, xs=A, xsave=3, w=A, dx=A, dw=A, work=A,
                       bytes=1 << 20))
    assert call(act=7) == DTYPE
    for s in (0, 4, -1):
        assert call(gsave=s) == DTYPE and call(xsave=s) == DTYPE
    for bad in (dict(m=-1), dict(k=40), dict(k=0), dict(f=16), dict(f=0), dict(k=BIG + 32), dict(f=32 - (1 << 63)),
                dict(bytes=need(4, 64, 96, 3) - 1), dict(bytes=-1)):
        assert call(**bad) == SHAPE, bad
    assert call(dx=None, dw=None) == OK
    for t in ("dh", "gu", "gs", "x", "xs", "w", "work"):
        assert call(**{t: None}) == NULL, t
        assert call(**{t: U}) == ALIGN, t
    assert call(dx=U) == ALIGN and call(dw=U) == ALIGN
    assert call(dw=None, x=None, xs=None, dh=None) == NULL  # x is not needed, dh is
    assert call(dx=None, w=None, dh=U) == ALIGN             # nor w


@pytest.mark.parametrize("gated", [False, True])
def test_mxfp4_validation(sfr, gated):
    lib = sfr.load()
    need = lib.sfr_mxfp4_workspace_bytes
    assert need(0, 64, 64) == 0 and need(4, 64, 48) == 0 and need(4, 40, 64) == 0
    assert need(1, 64, 64) == 0
    if gated:
        call = caller(lib.mxfp4_gated_linear, "x m k wq ws f act out",
                      dict(x=A, m=4, k=64, wq=A, ws=A, f=64, act=0, out=A))
        assert call(act=5) == DTYPE
        bads = (dict(f=0), dict(f=48), dict(f=BIG // 2 + 32), dict(f=32 - (1 << 63)))
    else:
        call = caller(lib.mxfp4_linear, "x m k wq ws n bias out od work bytes",
                      dict(x=A, m=4, k=64, wq=A, ws=A, n=64, bias=None, out=A, od=0, work=A, bytes=1 << 40))
        assert call(od=2) == DTYPE
        assert call(bias=U) == ALIGN
        assert call(n=0, wq=None, ws=None, out=None) == OK
        bads = (dict(n=40), dict(n=-16), dict(n=BIG + 16))
    for bad in bads + (dict(m=-1), dict(m=(1 << 30) + 1), dict(k=48), dict(k=0), dict(k=BIG + 32)):
        assert call(**bad) == SHAPE, bad
    assert call(m=0, x=None, out=None) == OK
    for t in ("x", "wq", "ws", "out"):
        assert call(**{t: None}) == NULL and call(**{t: U}) == ALIGN
    if not gated:  # few outputs and a long sum: slices of the sum in the workspace
        m, k = 200, 1 << 15
        assert need(m, 64, k) > 0 and need(m, 64, k) % (m * 64 * 4) in range(256)
        assert call(m=m, k=k, bytes=need(m, 64, k) - 1) == SHAPE
        assert call(m=m, k=k, work=None) == NULL and call(m=m, k=k, work=U) == ALIGN


def test_binding_refuses(sfr):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((128, 64), dtype=torch.bfloat16)
    q = sfr.MxTensor(torch.zeros((128, 32), dtype=torch.uint8).view(torch.float4_e2m1fn_x2),
                     torch.zeros((128, 2), dtype=torch.uint8).view(torch.float8_e8m0fnu))
    for call in (lambda: sfr.quantize_mx(x), lambda: sfr.dequantize_mx(q), lambda: sfr.gated_linear(x, w),
                 lambda: sfr.gated_linear_checkpointed(x, w), lambda: sfr.mxfp4_linear(x, q),
                 lambda: sfr.mxfp4_gated_linear(x, q),
                 lambda: sfr.gated_linear_backward(x, w, sfr.GatedCheckpoint(x, w, "silu"))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("dtype", list(MX), ids=str)
def test_reference_round_trip(dtype):
    """The reference's rounding gives values that its own decoder returns for
    every code, and no value between two neighbouring codes is nearer to a third."""
    top, bits, low = MX[dtype]
    per = 16 if bits == 1 else 256
    codes = torch.arange(per, dtype=torch.uint8)
    if bits == 1:
        t = codes.repeat(2)
        raw = (t[0::2] | (t[1::2] << 4))[None].view(dtype)
    else:
        raw = torch.where(torch.isfinite(codes.view(dtype).float()), codes, 0)[None].view(dtype)

    class T:
        pass
    q = T()
    q.codes, q.scale = raw, torch.full((1, max(per, 32) // 32), 127, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    v = mx_values(q)[0].unique()
    assert v.max() == top and v.abs()[v.abs() > 0].min() == 2.0 ** (low - bits)
    x = (v[:-1] + v[1:]) / 2  # halfway points, and just beside them
    for y, near in ((v, v), (x - x.abs() * 2.0 ** -30, v[:-1]), (x + x.abs() * 2.0 ** -30, v[1:])):
        rows = torch.cat((y[:, None], torch.full((len(y), 1), top, dtype=torch.float64),
                          torch.zeros(len(y), 30, dtype=torch.float64)), 1)
        r, s = mx_round(rows, dtype)
        keep = torch.ones(len(y), dtype=torch.bool) if y is v else x != 0
        assert torch.equal(r[keep, 0], near[keep]) and bool((s == 127).all())


def test_reference_not_finite():
    x = torch.zeros(1, 64, dtype=torch.float64)
    x[0, 3] = math.inf
    v, s = mx_round(x, torch.float8_e4m3fn)
    assert s.tolist() == [[255, 17]] and bool(torch.isnan(v[0, :32]).all()) and bool((v[0, 32:] == 0).all())
