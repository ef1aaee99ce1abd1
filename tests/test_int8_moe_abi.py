"""The 8-bit integer layer's, the router's and the mixture-of-experts layer's
entry points on the CPU: invalid arguments are refused with the documented
status before anything is launched (so these calls need no GPU), the sizes of
the GPU tests reach every kernel, and the 64-bit references agree with plain
forms and see planted mistakes."""
import itertools
import math
import os

import pytest
import torch

import test_gpu_int8 as int8_tests
from block_ref import U, act64
from block_rms import ROUND, rms, sums
from int8_ref import codes64, linear64
from moe_ref import layer64, weights64
from test_block_abi import caller

OK, NULL, SHAPE, ALIGN, DTYPE = 0, 1, 2, 3, 4
A, U1 = 0x10000, 0x10001  # 16-byte aligned and misaligned stand-in addresses, never dereferenced
BIG = 1 << 20


@pytest.fixture(scope="module")
def sfr():
    import sparse_fp8_row_amd as sfr
    if not os.path.exists(sfr.LIB_PATH):
        from sparse_fp8_row_amd import build
        build.build()
    sfr.load()
    return sfr


def test_quantize_validation(sfr):
    call = caller(sfr.load().quantize_rowwise_int8, "x rows cols q s", dict(x=A, rows=4, cols=64, q=A, s=A))
    for bad in (dict(cols=12), dict(cols=0), dict(cols=-8), dict(rows=-1), dict(rows=(1 << 30) + 1),
                dict(cols=(1 << 30) + 8), dict(rows=1 << 30, cols=1 << 20)):
        assert call(**bad) == SHAPE, bad
    assert call(rows=0, x=None, q=None, s=None) == OK
    for t in ("x", "q", "s"):
        assert call(**{t: None}) == NULL and call(**{t: U1}) == ALIGN


@pytest.mark.parametrize("dynamic", [False, True])
def test_int8_validation(sfr, dynamic):
    lib = sfr.load()
    need = lambda m, n, k: lib.sfr_int8_workspace_bytes(m, n, k, dynamic)  # noqa: E731
    if dynamic:
        call = caller(lib.int8_linear_dynamic, "x m k wq ws n bias out od work bytes",
                      dict(x=A, m=4, k=64, wq=A, ws=A, n=64, bias=None, out=A, od=0, work=A, bytes=1 << 40))
        tensors = ("x", "wq", "ws", "out")
        assert need(300, 64, 64) >= 300 * 64 + 300 * 4 and need(1, 64, 64) == 0
    else:
        call = caller(lib.int8_scaled_linear, "x xs m k wq ws n bias out od work bytes",
                      dict(x=A, xs=A, m=4, k=64, wq=A, ws=A, n=64, bias=None, out=A, od=0, work=A, bytes=1 << 40))
        tensors = ("x", "xs", "wq", "ws", "out")
        assert need(1, 64, 64) == 0
    assert call(od=2) == DTYPE and call(od=-1) == DTYPE
    for bad in (dict(m=-1), dict(m=(1 << 30) + 1), dict(k=40), dict(k=0), dict(k=-16), dict(k=131072), dict(n=40),
                dict(n=-16), dict(n=BIG + 16), dict(m=1 << 30, n=BIG), dict(n=16 - (1 << 63))):
        assert call(**bad) == SHAPE, bad
        if "n" in bad or "k" in bad:
            assert need(bad.get("m", 4), bad.get("n", 64), bad.get("k", 64)) == 0
    assert call(m=0, x=None, out=None, work=None) == OK and call(n=0, wq=None, ws=None, out=None, work=None) == OK
    for t in tensors:
        assert call(**{t: None}) == NULL and call(**{t: U1}) == ALIGN
    assert call(bias=U1) == ALIGN
    if dynamic:
        call = caller(lib.int8_linear_dynamic, "x m k wq ws n bias out od work bytes",
                      dict(x=A, m=40, k=64, wq=A, ws=A, n=64, bias=None, out=A, od=0, work=A, bytes=1 << 40))
        assert call(work=None) == NULL and call(work=U1) == ALIGN and call(bytes=0) == SHAPE
    m, k = 200, 1 << 15  # few outputs and a long sum: slices of the sum in the workspace
    assert need(m, 64, k) >= 2 * m * 64 * 4
    assert call(m=m, k=k, bytes=need(m, 64, k) - 1) == SHAPE and call(m=m, k=k, bytes=-1) == SHAPE
    assert call(m=m, k=k, work=None) == NULL and call(m=m, k=k, work=U1) == ALIGN


def test_route_validation(sfr):
    call = caller(sfr.load().moe_route, "x m k w experts bias top score renorm logits ids weights",
                  dict(x=A, m=4, k=64, w=A, experts=20, bias=None, top=3, score=0, renorm=1, logits=A, ids=A, weights=A))
    assert call(score=2) == DTYPE and call(score=-1) == DTYPE
    for bad in (dict(m=-1), dict(m=(1 << 30) + 1), dict(k=48), dict(k=0), dict(k=BIG + 32), dict(experts=0),
                dict(experts=-1), dict(experts=1025), dict(top=0), dict(top=-1), dict(top=21), dict(top=17, experts=40)):
        assert call(**bad) == SHAPE, bad
    assert call(m=0, x=None, logits=None) == OK
    for t in ("x", "w", "logits", "ids", "weights"):
        assert call(**{t: None}) == NULL and call(**{t: U1}) == ALIGN
    assert call(bias=U1) == ALIGN


@pytest.mark.parametrize("form", [0, 1, 2])
def test_layer_validation(sfr, form):
    lib = sfr.load()
    need = lambda m, f, top, k=64: lib.sfr_moe_workspace_bytes(m, k, f, top)  # noqa: E731
    up = lambda b: (b + 255) // 256 * 256  # noqa: E731
    # h of a pass in bf16; with more tokens the experts' parts in binary32 too
    assert need(3, 96, 2) == up(3 * 2 * 96 * 2)
    assert need(64, 96, 2) == need(1000, 96, 2) == up(64 * 2 * 96 * 2) + 64 * 2 * 64 * 4
    assert need(0, 96, 2) == 0 and need(4, 48, 2) == 0 and need(4, 96, 0) == 0 and need(4, 96, 17) == 0 and need(-1, 96, 2) == 0
    assert need(4, 96, 2, 48) == 0 and need(4, 96, 2, 0) == 0
    call = caller(lib.moe_layer, "x m k ids weights top experts f form gu gus down downs act out work bytes",
                  dict(x=A, m=4, k=64, ids=A, weights=A, top=2, experts=5, f=96, form=form, gu=A, gus=A, down=A, downs=A,
                       act=0, out=A, work=A, bytes=1 << 20))
    assert call(act=3) == DTYPE and call(act=-1) == DTYPE and call(form=3) == DTYPE and call(form=-1) == DTYPE
    for bad in (dict(m=-1), dict(m=(1 << 30) + 1), dict(k=48), dict(k=0), dict(k=BIG + 32), dict(f=48), dict(f=0),
                dict(f=BIG // 2 + 32), dict(f=32 - (1 << 63)), dict(experts=0), dict(experts=1025), dict(top=0),
                dict(top=17), dict(bytes=need(4, 96, 2) - 1), dict(bytes=-1)):
        assert call(**bad) == SHAPE, bad
    assert call(m=0, x=None, out=None, work=None, bytes=0) == OK
    for t in ("x", "ids", "weights", "gu", "down", "out", "work") + (("gus", "downs") if form else ()):
        assert call(**{t: None}) == NULL, t
        assert call(**{t: U1}) == ALIGN, t
    assert call(ids=A + 4, weights=A + 4, out=U1) == ALIGN and call(ids=A + 2) == ALIGN
    if not form:  # the scales are not looked at (checked by what is refused next)
        assert call(gus=None, downs=U1, x=None) == NULL


def test_binding_refuses(sfr):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q = sfr.Int8Tensor(torch.zeros((32, 64), dtype=torch.int8), torch.zeros(32))
    route = sfr.MoeRoute(torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)))
    gu, down = torch.zeros((3, 64, 64), dtype=torch.bfloat16), torch.zeros((3, 64, 32), dtype=torch.bfloat16)
    for call in (lambda: sfr.quantize_rowwise_int8(x), lambda: sfr.int8_linear(x, q),
                 lambda: sfr.int8_linear(sfr.Int8Tensor(q.codes, q.scale), q), lambda: sfr.moe_route(x, x, 2),
                 lambda: sfr.moe_layer(x, route, gu, down)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("dynamic", [False, True])
def test_every_int8_kernel_is_compared(sfr, dynamic):
    def kernel(m, n, k):
        name, slices = sfr.int8_kernel(m, n, k, dynamic)
        return name, slices > 1
    reached = {kernel(*s) for s in int8_tests.SHAPES}
    missing = {}
    rows = (1, 2, 3, 4, 5, 8, 9, 16, 17, 24, 33, 48, 64, 65, 77, 100, 128, 129, 160, 200, 256, 257, 300, 420, 513, 600,
            769, 1025, 1300, 1800, 2049, 2500, 4097, 8192)
    sizes = (16, 32, 48, 112, 160, 272, 528, 784, 1040, 1552, 2080, 3600, 4096, 5648, 8192, 14336, 28672)
    for s in itertools.product(rows, sizes, sizes):
        if kernel(*s) not in reached:
            missing.setdefault(kernel(*s), s)
    assert not missing, missing


def test_kernel_query(sfr):
    for bad in ((0, 64, 64), (-1, 64, 64), (4, 40, 64), (4, 64, 40), (4, 0, 64), (4, 64, 0), (4, 64, 131072)):
        assert sfr.int8_kernel(*bad) is None and sfr.int8_kernel(*bad, dynamic=False) is None, bad
    assert sfr.load().sfr_int8_kernel(4, 64, 64, 0, None)
    lib = sfr.load()
    up = lambda b: (b + 255) // 256 * 256  # noqa: E731
    for m, n, k in itertools.product((1, 20, 68, 300, 1000, 4097), (32, 416, 3616), (32, 2080, 32768)):
        _, slices = sfr.int8_kernel(m, n, k, False)
        assert lib.sfr_int8_workspace_bytes(m, n, k, 0) == (up(slices * m * n * 4) if slices > 1 else 0)


# ------------------------------------------------------------------ references


def test_reference_codes():
    """Against whole-number arithmetic: |127 a - q b| is least, ties to the even q."""
    for b in (128, 129, 200, 254, 255):
        a = torch.arange(-b, b + 1, dtype=torch.float64)
        x = torch.cat((torch.tensor([float(b)], dtype=torch.float64), a))[None].bfloat16()
        codes, scale = codes64(x)
        assert scale.item() == torch.tensor(b / 127).item()
        for v, q in zip(a.tolist(), codes[0, 1:].tolist()):
            best = min(range(-127, 128), key=lambda c: (abs(254 * int(v) - 2 * c * b), c % 2))
            assert q == best, (b, v)


def test_reference_linear():
    g = torch.Generator().manual_seed(1)
    xq = torch.randint(-128, 128, (5, 48), generator=g).to(torch.int8)
    wq = torch.randint(-128, 128, (7, 48), generator=g).to(torch.int8)
    xs, ws = torch.rand(5, generator=g), torch.rand(7, generator=g)
    y, bound = linear64(xq, xs, wq, ws)
    plain = (xq.long() @ wq.long().t()).double() * xs.double()[:, None] * ws.double()
    assert bool(((y - plain).abs() <= bound + 2.0 ** -24 * y.abs()).all())


def plain_layer(x, ids, weights, gu, down, act):
    """Slot by slot."""
    f = down.shape[2]
    out = torch.zeros(x.shape, dtype=torch.float64)
    for t, s in itertools.product(range(x.shape[0]), range(ids.shape[1])):
        e = int(ids[t, s])
        if 0 <= e < gu.shape[0]:
            v = gu[e].double() @ x[t].double()
            out[t] += weights[t, s].double() * (down[e].double() @ (act64(v[:f], act)[0] * v[f:]))
    return out


def cpu_case(m, k, f, experts, top, seed=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ids = torch.randint(-1, experts + 1, (m, top), generator=g).int()  # repeats and none among them
    return r(m, k).bfloat16(), ids, torch.rand(m, top, generator=g), (0.1 * r(experts, 2 * f, k)).bfloat16(), \
        (0.1 * r(experts, k, f)).bfloat16()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_reference_layer(act):
    case = cpu_case(6, 32, 64, 4, 3)
    ref = layer64(*case, act)[0]
    assert torch.allclose(ref, plain_layer(*case, act), rtol=1e-12, atol=1e-12)


def test_root_mean_square_sees_a_missing_unit():
    """The bound of the GPU test against 32 of an output's f * top terms, and against a
    slot's weight off by a hundredth."""
    m, k, f, top = 16, 256, 1440, 2
    x, _, weights, gu, down = cpu_case(m, k, f, 3, top)
    ids = torch.tensor([[0, 2]] * m, dtype=torch.int32)
    ref = layer64(x, ids, weights, gu, down, "silu")[0]
    limit = (1.1 * math.sqrt(2) * ROUND + sums(k) + sums(f * top)) * rms(ref)
    short = down.clone()
    short[2, :, -32:] = 0
    assert rms(layer64(x, ids, weights, gu, short, "silu")[0] - ref) > limit
    other = weights.clone()
    other[:, 1] *= 1.01
    assert rms(layer64(x, ids, other, gu, down, "silu")[0] - ref) > limit
    assert U < limit


def test_reference_weights():
    l = torch.tensor([[0.5, -1.0, 2.0, 0.0]])
    ids = torch.tensor([[2, 0, -1]])
    w = weights64(l, ids, "softmax", True)[0]
    e = [math.exp(2.0), math.exp(0.5)]
    assert torch.allclose(w, torch.tensor([[e[0], e[1], 0.0]], dtype=torch.float64) / sum(e))
    total = sum(map(math.exp, l[0].tolist()))
    assert torch.allclose(weights64(l, ids, "softmax", False)[0], torch.tensor([[e[0], e[1], 0.0]], dtype=torch.float64) / total)
    s = [1 / (1 + math.exp(-2.0)), 1 / (1 + math.exp(-0.5))]
    assert torch.allclose(weights64(l, ids, "sigmoid", True)[0], torch.tensor([[s[0], s[1], 0.0]], dtype=torch.float64) / sum(s))
    assert torch.allclose(weights64(l, ids, "sigmoid", False)[0], torch.tensor([[s[0], s[1], 0.0]], dtype=torch.float64))
