"""GPU: the row quantizer to 8-bit integers and the integer linear layer, against
exact results (int8_ref)."""
import itertools
import math
import threading

import pytest
import torch

from int8_ref import codes64, linear64

pytestmark = pytest.mark.gpu
# m, n, k: every row count around the forms' limits, sizes inside and at the ends of tiles
SHAPES = [(1, 16, 16), (1, 4096, 4096), (2, 48, 144), (3, 272, 400), (5, 16, 8192), (8, 1040, 272), (9, 4112, 528),
          (16, 64, 1040), (17, 48, 32), (31, 5008, 656), (33, 112, 2064), (64, 144, 160), (65, 16, 112),
          (100, 5648, 2080), (128, 128, 128), (129, 272, 16), (200, 64, 32768), (257, 1552, 784), (300, 4096, 1024),
          (517, 784, 4112), (700, 3600, 272), (1025, 528, 3088), (2100, 4368, 528),
          # one for every other kernel, with and without slices of the sum
          (1, 16, 28672), (1, 5648, 28672), (1, 5648, 16), (3, 5648, 16), (5, 5648, 16), (17, 3600, 28672), (17, 4096, 14336), (17, 5648, 8192), (17, 28672, 2080),
          (65, 5648, 5648), (65, 5648, 28672), (129, 5648, 14336), (200, 14336, 16), (257, 14336, 16),
          (769, 14336, 528), (1025, 14336, 528), (4097, 272, 28672), (4097, 528, 14336), (4097, 784, 272),
          (17, 28672, 8192), (65, 28672, 5648), (129, 2080, 28672), (129, 8192, 14336), (200, 5648, 28672)]


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def operands(seed, m, n, k, low=-127):
    g = torch.Generator("cuda").manual_seed(seed)
    draw = lambda *s: torch.randint(low, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)  # noqa: E731
    scale = lambda r: torch.rand(r, generator=g, device="cuda") * 0.01 + 1e-4  # noqa: E731
    bias = torch.randn(n, generator=g, device="cuda").bfloat16()
    return draw(m, k), scale(m), draw(n, k), scale(n), bias


def check(out, ref, bound):
    assert out.shape == ref.shape
    assert bool(((out.double() - ref).abs() <= bound).all()), float(((out.double() - ref).abs() - bound).max())


# ------------------------------------------------------------------ quantizer


@pytest.mark.parametrize("exponent", [-133, -126, -100, 0, 100, 126])
def test_codes_of_every_pair(sfr, exponent):
    """Every significand of amax against every element of its nine lower binades
    (below them every code is 0), both signs: ties and the quotients next to them."""
    b = torch.arange(128, 256, dtype=torch.float64)
    a = torch.cat([torch.arange(128, 256, dtype=torch.float64) * 2.0 ** -j for j in range(10)])
    x = torch.cat((b[:, None], a.repeat(128, 1), -a.repeat(128, 1)), 1) * 2.0 ** exponent * 2.0 ** -7
    x = torch.where(x.abs() > b[:, None] * 2.0 ** (exponent - 7), 0.0, x).bfloat16()
    x = torch.cat((x, x.new_zeros(128, -x.shape[1] % 8)), 1).cuda()
    q = sfr.quantize_rowwise_int8(x)
    codes, scale = codes64(x)
    assert torch.equal(q.codes.cpu(), codes)
    assert torch.equal(q.scale.cpu(), scale)


# a row held in registers, one read twice, in both forms (rows of a wavefront, of a workgroup)
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 2080), (7, 4104), (5, 8200), (2, 16384), (3, 16400), (1023, 24),
                                       (1024, 2048), (1025, 2056), (1031, 4096), (1026, 4104), (1027, 8208)])
def test_codes(sfr, rows, cols):
    g = torch.Generator("cuda").manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())).bfloat16()
    x[rows // 2] = 0
    x[-1, -1] = -1e30  # the maximum in the last column, negative
    q = sfr.quantize_rowwise_int8(x)
    codes, scale = codes64(x)
    assert torch.equal(q.codes.cpu(), codes) and torch.equal(q.scale.cpu(), scale)


@pytest.mark.parametrize("rows", [5, 1100])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite_rows(sfr, rows, bad):
    x = torch.randn(rows, 272, device="cuda").bfloat16()
    x[2, 100] = bad
    q = sfr.quantize_rowwise_int8(x)
    codes, scale = codes64(x)
    assert math.isnan(q.scale[2].item()) and bool((q.codes[2] == 0).all())
    keep = torch.arange(rows) != 2
    assert torch.equal(q.codes.cpu()[keep], codes[keep]) and torch.equal(q.scale.cpu()[keep], scale[keep])
    out = sfr.int8_linear(x, sfr.quantize_rowwise_int8(torch.randn(32, 272, device="cuda").bfloat16()))
    assert bool(torch.isnan(out[2]).all()) and bool(torch.isfinite(out.cpu()[keep]).all())


# ------------------------------------------------------------------ linear layer


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(sfr, m, n, k):
    """Both output types, with and without a bias, codes down to -128; the bf16
    output is the binary32 one rounded."""
    xq, xs, wq, ws, bias = operands(m + n + k, m, n, k, low=-128)
    x, w = sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws)
    for b in (None, bias):
        ref, bound = linear64(xq, xs, wq, ws, b)
        out = sfr.int8_linear(x, w, b, out_dtype=torch.float32)
        check(out, ref, bound)
        assert torch.equal(sfr.int8_linear(x, w, b), out.bfloat16())


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_dynamic(sfr, m, n, k):
    """From bf16: the same bits as quantizing first."""
    g = torch.Generator("cuda").manual_seed(k)
    x = (torch.randn(m, k, generator=g, device="cuda") * (1 + 9 * (torch.rand(k, generator=g, device="cuda") < 0.02)))
    x = x.bfloat16()
    x[m // 2, : k // 2] = 0
    w = sfr.quantize_rowwise_int8((0.02 * torch.randn(n, k, generator=g, device="cuda")).bfloat16())
    bias = torch.randn(n, generator=g, device="cuda").bfloat16()
    q = sfr.quantize_rowwise_int8(x)
    rows = torch.unique(torch.tensor([0, m // 2, m - 1]))
    codes, scale = codes64(x[rows])
    assert torch.equal(q.codes[rows].cpu(), codes) and torch.equal(q.scale[rows].cpu(), scale)
    for dtype, b in itertools.product((torch.float32, torch.bfloat16), (None, bias)):
        out = sfr.int8_linear(x, w, b, out_dtype=dtype)
        assert torch.equal(out, sfr.int8_linear(q, w, b, out_dtype=dtype))
        if dtype == torch.float32:
            check(out, *linear64(q.codes, q.scale, w.codes, w.scale, b))


@pytest.mark.parametrize("m", [1, 4, 20, 200])
def test_largest_sums(sfr, m):
    """The largest k with every code -128: the sum just below 2^31."""
    k, n = 131056, 32
    xq = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    one = lambda r: torch.ones(r, device="cuda")  # noqa: E731
    out = sfr.int8_linear(sfr.Int8Tensor(xq, one(m)), sfr.Int8Tensor(wq, one(n)), out_dtype=torch.float32)
    ref = torch.full((m, n), float(16384 * k), device="cuda")
    ref[:, 1] = float(-16256 * k)
    assert torch.equal(out, ref)


def test_rows_do_not_depend_on_the_batch(sfr):
    """Every kernel gives a row the same bits."""
    n, k = 1040, 4096
    xq, xs, wq, ws, bias = operands(3, 2500, n, k)
    w = sfr.Int8Tensor(wq, ws)
    want = sfr.int8_linear(sfr.Int8Tensor(xq, xs), w, bias, out_dtype=torch.float32)
    for m in (1, 2, 3, 8, 9, 16, 17, 40, 64, 100, 129, 300, 600, 1500):
        got = sfr.int8_linear(sfr.Int8Tensor(xq[:m].clone(), xs[:m].clone()), w, bias, out_dtype=torch.float32)
        assert torch.equal(got, want[:m]), m


@pytest.mark.parametrize("m,n,k", [(1, 64, 4096), (3, 64, 272), (40, 272, 272), (300, 272, 272), (200, 64, 32768)])
def test_scales(sfr, m, n, k):
    """Zero and NaN scales: zeros (the bias) and NaN in their own row or column only."""
    xq, xs, wq, ws, bias = operands(9, m, n, k)
    xs[0], ws[5], ws[n - 1] = 0.0, 0.0, math.nan
    out = sfr.int8_linear(sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws), bias, out_dtype=torch.float32)
    fine = torch.arange(n, device="cuda") != n - 1
    assert bool(torch.isnan(out[:, n - 1]).all()) and bool(torch.isfinite(out[:, fine]).all())
    assert torch.equal(out[0, fine], bias.float()[fine]) and torch.equal(out[:, 5], bias.float()[5].expand(m))


@pytest.mark.parametrize("m,n,k", [(1, 48, 144), (5, 272, 400), (17, 48, 32), (129, 272, 16), (200, 64, 32768)])
def test_padding_is_not_read_or_written(sfr, m, n, k):
    """Operands in larger buffers of NaN scales and of -128 codes; nothing around the output changes."""
    def within(t, fill):
        flat = torch.full((t.numel() + 2048,), fill, dtype=t.dtype, device="cuda")
        flat[1024:1024 + t.numel()] = t.reshape(-1)
        return flat[1024:1024 + t.numel()].view(t.shape), flat
    xq, xs, wq, ws, bias = operands(4, m, n, k)
    x = torch.randn(m, k, device="cuda").bfloat16()
    want = sfr.int8_linear(sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws), bias)
    dyn = sfr.int8_linear(x, sfr.Int8Tensor(wq, ws), bias)
    xq, xs, wq, ws, bias, x = (within(t, f)[0] for t, f in ((xq, -128), (xs, math.nan), (wq, -128), (ws, math.nan),
                                                         (bias, math.nan), (x, math.nan)))
    out, flat = within(torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), 7.0)
    sfr.int8_linear(sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws), bias, out=out)
    assert torch.equal(out, want)
    assert bool((flat[:1024] == 7).all()) and bool((flat[1024 + m * n:] == 7).all())
    assert torch.equal(sfr.int8_linear(x, sfr.Int8Tensor(wq, ws), bias, out=out), dyn)
    assert bool((flat[:1024] == 7).all()) and bool((flat[1024 + m * n:] == 7).all())


def test_past_32_bit_offsets(sfr):
    """Outputs, and a weight, past 2^32 bytes."""
    m, n, k = 66000, 33008, 16
    xq, xs, wq, ws, _ = operands(5, m, n, k)
    out = sfr.int8_linear(sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws))
    rows = torch.tensor([0, 1, 32768, 65000, m - 1], device="cuda")
    ref, bound = linear64(xq[rows], xs[rows], wq, ws)
    check(out[rows], ref, bound + 2.0 ** -8 * ref.abs() + 2.0 ** -133)
    del out
    n, k = 32784, 131056
    wq = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    wq[-3:, -16:] = 5
    ws = torch.ones(n, device="cuda")
    for m in (1, 20, 70):
        xq = torch.ones(m, k, dtype=torch.int8, device="cuda")
        out = sfr.int8_linear(sfr.Int8Tensor(xq, torch.ones(m, device="cuda")), sfr.Int8Tensor(wq, ws))
        assert bool((out[:, -3:] == 80).all()) and bool((out[:, :-3] == 0).all())


@pytest.mark.parametrize("m,n,k", [(1, 64, 4096), (12, 4096, 1024), (200, 64, 32768), (600, 1552, 784)])
def test_graph_replay(sfr, m, n, k):
    """Captured from bf16 and replayed with new inputs, eager calls and synchronizations between."""
    x = torch.randn(m, k, device="cuda").bfloat16()
    w = sfr.quantize_rowwise_int8(torch.randn(n, k, device="cuda").bfloat16())
    sfr.int8_linear(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sfr.int8_linear(x, w)
    for i in range(4):
        x.copy_(torch.randn(m, k, device="cuda") * 10.0 ** i)
        graph.replay()
        torch.cuda.synchronize()
        want = sfr.int8_linear(x.clone(), w)
        assert torch.equal(out, want)


def test_streams_and_threads(sfr):
    """An explicit stream, the current one, and several host threads at once."""
    w = sfr.quantize_rowwise_int8(torch.randn(1040, 2080, device="cuda").bfloat16())
    xs = [torch.randn(m, 2080, device="cuda").bfloat16() for m in (1, 7, 40, 300)]
    want = [sfr.int8_linear(x, w) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [sfr.int8_linear(x, w, stream=side) for x in xs]
    q = sfr.quantize_rowwise_int8(xs[2], stream=side)
    again = sfr.int8_linear(q, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(again, want[2])
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                if not torch.equal(sfr.int8_linear(xs[i], w), want[i]):
                    bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_refusals(sfr):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = sfr.quantize_rowwise_int8(torch.zeros(32, 64, device="cuda", dtype=torch.bfloat16))
    q = sfr.quantize_rowwise_int8(x)
    ok = sfr.int8_linear(x, w)
    for bad in (lambda: sfr.int8_linear(x.float(), w), lambda: sfr.int8_linear(x[:, :32].contiguous(), w),
                lambda: sfr.int8_linear(x[0], w), lambda: sfr.int8_linear(x.t(), w), lambda: sfr.int8_linear(x, x),
                lambda: sfr.int8_linear(x, sfr.Int8Tensor(w.codes, w.scale[:31])),
                lambda: sfr.int8_linear(x, sfr.Int8Tensor(w.codes, w.scale.double())),
                lambda: sfr.int8_linear(x, sfr.Int8Tensor(w.codes.float(), w.scale)),
                lambda: sfr.int8_linear(x, sfr.Int8Tensor(w.codes.cpu(), w.scale)),
                lambda: sfr.int8_linear(x, sfr.Int8Tensor(w.codes.t(), w.scale)),
                lambda: sfr.int8_linear(sfr.Int8Tensor(q.codes, q.scale.cpu()), w),
                lambda: sfr.int8_linear(x.cpu(), w), lambda: sfr.int8_linear(x, w, torch.zeros(32, device="cuda")),
                lambda: sfr.int8_linear(x, w, torch.zeros(16, device="cuda", dtype=torch.bfloat16)),
                lambda: sfr.int8_linear(x, w, out_dtype=torch.float16),
                lambda: sfr.int8_linear(x, w, out=ok.float()), lambda: sfr.int8_linear(x, w, out=ok[:3]),
                lambda: sfr.int8_linear(x, w, out=x.view(-1)[:128].view(4, 32)),
                lambda: sfr.quantize_rowwise_int8(x.float()), lambda: sfr.quantize_rowwise_int8(x.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sfr.quantize_rowwise_int8(x[:, :12].contiguous()),
                lambda: sfr.int8_linear(x.view(-1)[1:193].view(3, 64), w),  # 2 bytes past an aligned address
                lambda: sfr.int8_linear(x, sfr.quantize_rowwise_int8(torch.zeros(24, 64, device="cuda").bfloat16()))):
        with pytest.raises(sfr.SfrError):
            bad()
    empty = sfr.int8_linear(x[:0], w)
    assert empty.shape == (0, 32) and sfr.quantize_rowwise_int8(x[:0]).shape == (0, 64)
    assert not sfr.int8_linear(x.clone().requires_grad_(), w).requires_grad


def test_same_every_time(sfr):
    xq, xs, wq, ws, bias = operands(8, 150, 512, 4096)
    first = sfr.int8_linear(sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws), bias)
    for _ in range(20):
        assert torch.equal(sfr.int8_linear(sfr.Int8Tensor(xq, xs), sfr.Int8Tensor(wq, ws), bias), first)
