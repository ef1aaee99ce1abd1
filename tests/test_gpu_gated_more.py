"""GPU: the gated block, its gradients and its 4-bit form on the shapes that
reach every kernel (tiles of every size, sliced sums), in padded buffers, with
values that are not finite, past 32-bit offsets, captured into graphs, on other
streams and together as a model uses them."""
import math

import pytest
import torch

from block_ref import check, gated64, gated_grad64, inputs, mx_round, mx_values, products64, HALF_BF16

pytestmark = pytest.mark.gpu
FP4 = torch.float4_e2m1fn_x2
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def randn(seed, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).bfloat16().cuda()


# Per product shapes (m, k, f) at which the choice takes each tile size, the
# smallest with half a stage of k (k = 32), others with more and odd stages.
@pytest.mark.parametrize("m,k,f", [(3000, 32, 2080), (2049, 32, 2080), (2049, 32, 4128), (1001, 32, 2080),
                                   (513, 32, 3104), (3000, 288, 2080), (300, 544, 14336), (517, 288, 14336),
                                   (1001, 416, 2080), (200, 1056, 14336), (130, 32, 32), (513, 288, 3104),
                                   (385, 1056, 2080), (130, 96, 160), (77, 1120, 96), (1300, 288, 3104),
                                   (257, 288, 16416), (16, 1056, 8224), (27, 2080, 8224), (50, 1120, 1056)])
def test_forward_tiles(sfr, m, k, f):
    x, w = inputs(m + f, m, k, 2 * f)
    h, bound, (g, u, eg, eu) = gated64(x.double(), w.double(), "silu")
    check(sfr.gated_linear(x, w), h, bound, "h")
    got, saved = sfr.gated_linear_checkpointed(x, w, checkpoint=torch.bfloat16)
    check(got, h, bound, "h, saving")
    gu, e = torch.cat((g, u), 1), torch.cat((eg, eu), 1)
    check(saved.gu, gu, e + HALF_BF16 * (gu.abs() + e) + 2.0 ** -133, "gu")
    got, saved = sfr.gated_linear_checkpointed(x, w, checkpoint=E4M3)
    check(got, h, bound, "h, saving in 8 bits")
    # half a step of e4m3 is 2^-4 of the value or, below 2^-6 of the block's largest-element scale, 2^-10 of that
    scale = torch.exp2(saved.gu.scale.view(torch.uint8).double() - 127).repeat_interleave(32, 1)
    check(mx_values(saved.gu), gu, e + torch.maximum(2.0 ** -4 * (gu.abs() + e), 2.0 ** -10 * scale), "gu in 8 bits")
    q = sfr.quantize_mx(w, FP4)
    h, bound, _ = gated64(x.double(), mx_values(q), "silu")
    check(sfr.mxfp4_gated_linear(x, q), h, bound, "h, 4-bit weight")


@pytest.mark.parametrize("m,k,n", [(3000, 32, 4128), (385, 8224, 6176), (2049, 32, 4128), (130, 4128, 8224),
                                   (4097, 32, 4128), (300, 8224, 16416), (2049, 32, 2080), (65, 4128, 8224),
                                   (3000, 32, 1056), (65, 2080, 8224), (130, 2080, 48), (4097, 96, 4128),
                                   (130, 4128, 4128), (130, 32, 32), (65, 4128, 4128), (1001, 288, 3104),
                                   (65, 4128, 6176), (385, 1056, 4128), (65, 8224, 2080), (130, 96, 48),
                                   (3000, 288, 4128), (2049, 288, 4128), (4097, 288, 4128), (130, 8224, 6176),
                                   (385, 4128, 1056), (4097, 8224, 32)])
def test_mxfp4_linear_tiles(sfr, m, k, n):
    x, w = inputs(m + n, m, k, n)
    q = sfr.quantize_mx(w, FP4)
    bias = randn(n, n)
    ref, e = products64(x.double(), mx_values(q))
    ref = ref + bias.double()
    e = e + 2.0 ** -24 * (ref.abs() + e)
    check(sfr.mxfp4_linear(x, q, bias, out_dtype=torch.float32), ref, e, "binary32")
    check(sfr.mxfp4_linear(x, q, bias), ref, e + HALF_BF16 * (ref.abs() + e) + 2.0 ** -133, "bf16")


@pytest.mark.parametrize("m,k,f", [(1, 2080, 2080), (1, 1056, 2080), (1, 4128, 416), (3000, 4128, 32), (385, 2080, 10272),
                                   (2049, 4128, 32), (130, 4128, 6176), (4097, 4128, 32), (257, 8224, 6176),
                                   (2049, 2080, 32), (65, 4128, 4128), (3000, 1056, 32), (1, 4128, 4128),
                                   (1, 32, 1056), (1000, 2048, 5632), (130, 8224, 2080), (4097, 288, 8224),
                                   (1, 32, 32), (1, 32, 96), (1, 4128, 3104), (3000, 1056, 416), (1, 2080, 8224),
                                   (3000, 4128, 416), (2049, 4128, 416), (4097, 4128, 416), (257, 2080, 2080)])
def test_backward_tiles(sfr, m, k, f):
    x, w = inputs(m + f, m, k, 2 * f)
    dh = randn(m, m, f)
    gu = randn(m + 1, m, 2 * f)
    for saved in (sfr.GatedCheckpoint(x, gu, "silu"),
                  sfr.GatedCheckpoint(sfr.quantize_mx(x, E4M3), sfr.quantize_mx(gu, torch.float8_e5m2), "silu")):
        mx = isinstance(saved.x, sfr.MxTensor)
        xd, gd = (mx_values(saved.x), mx_values(saved.gu)) if mx else (x.double(), gu.double())
        dx, dw = sfr.gated_linear_backward(dh, w, saved)
        rx, bx, rw, bw = gated_grad64(dh.double(), xd, gd[:, :f], gd[:, f:], w.double(), "silu")
        check(dx, rx, bx, "dx")
        check(dw, rw, bw, "dw")


# The streamed 4-bit forms: up to 2, 8, 16 rows and more passes, each with few
# and many tiles of 16 weight rows (n / 16 an odd number of them, too).
@pytest.mark.parametrize("m,k,n", [(1, 96, 4112), (2, 1056, 8224), (5, 96, 4112), (8, 544, 16), (16, 1056, 4112),
                                   (9, 1056, 8208), (16, 1056, 16400), (27, 2080, 4112), (48, 4128, 8208), (100, 32, 32)])
def test_mxfp4_streamed(sfr, m, k, n):
    x, w = inputs(m + n, m, k, n)
    q = sfr.quantize_mx(w, FP4)
    ref, e = products64(x.double(), mx_values(q))
    check(sfr.mxfp4_linear(x, q, out_dtype=torch.float32), ref, e, "out")
    f = (n + 31) // 32 * 32
    x, w = inputs(m + f, m, k, 2 * f)
    q = sfr.quantize_mx(w, FP4)
    h, bound, _ = gated64(x.double(), mx_values(q), "relu")
    check(sfr.mxfp4_gated_linear(x, q, "relu"), h, bound, "h")


def padded(rows, cols, dtype, fill, before=3, after=5):
    """A [rows, cols] view inside a buffer of `fill`, and the buffer's rows outside it."""
    b = torch.full((before + rows + after, cols), fill, dtype=dtype, device="cuda")
    return b[before:before + rows], (b[:before], b[before + rows:])


def untouched(outside, fill):
    for t in outside:
        assert bool((t == fill).all())


@pytest.mark.parametrize("m,k,f", [(1, 4096, 96), (5, 160, 64), (17, 96, 160), (100, 288, 224), (300, 544, 1056),
                                   (2049, 32, 2080), (517, 96, 14336)])
def test_padding_is_not_read_or_written(sfr, m, k, f):
    """Inputs lie among NaNs, outputs among marks: no call reads or writes past its rows."""
    x, w = inputs(m + k, m, k, 2 * f)
    want = sfr.gated_linear(x, w)
    px, _ = padded(m, k, torch.bfloat16, math.nan)
    pw, _ = padded(2 * f, k, torch.bfloat16, math.nan)
    px.copy_(x)
    pw.copy_(w)
    o, out = padded(m, f, torch.bfloat16, 7.0)
    assert torch.equal(sfr.gated_linear(px, pw, out=o), want)
    untouched(out, 7.0)
    q = sfr.quantize_mx(w, FP4)
    assert bool((mx_values(sfr.quantize_mx(pw, FP4)) == mx_values(q)).all())
    pc, _ = padded(2 * f, k // 2, torch.uint8, 0xFF)
    ps = torch.full((2 * f * k // 32 + 4096,), 255, dtype=torch.uint8, device="cuda")
    scale = ps[2048:2048 + 2 * f * k // 32].view(2 * f, k // 32)
    pc.copy_(q.codes.view(torch.uint8))
    scale.copy_(q.scale.view(torch.uint8))
    pq = sfr.MxTensor(pc.view(FP4), scale.view(torch.float8_e8m0fnu))
    o, out = padded(m, f, torch.bfloat16, 7.0)
    assert torch.equal(sfr.mxfp4_gated_linear(px, pq, out=o), sfr.mxfp4_gated_linear(x, q))
    untouched(out, 7.0)
    for dt in (torch.bfloat16, torch.float32):
        o, out = padded(m, 2 * f, dt, 7.0)
        assert torch.equal(sfr.mxfp4_linear(px, pq, out_dtype=dt, out=o), sfr.mxfp4_linear(x, q, out_dtype=dt))
        untouched(out, 7.0)
    # the checkpoint and the gradients through the C ABI, into marked buffers
    lib, h = sfr.load(), int(torch.cuda.current_stream().cuda_stream)
    for save, ty in ((1, torch.bfloat16), (2, torch.uint8), (3, torch.uint8)):
        fill = 7.0 if save == 1 else 0xA5
        o, out = padded(m, f, torch.bfloat16, 7.0)
        gu, gout = padded(m, 2 * f, ty, fill, 4, 4)
        gs = torch.full((m * 2 * f // 32 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        assert lib.gated_linear_bf16(px.data_ptr(), m, k, pw.data_ptr(), f, 0, o.data_ptr(), save, gu.data_ptr(),
                                     gs.data_ptr(), h) == 0
        # (saving takes the tiled kernels at every m: its own order of the sums)
        kind = {1: torch.bfloat16, 2: E4M3, 3: torch.float8_e5m2}[save]
        assert torch.equal(o, sfr.gated_linear_checkpointed(x, w, checkpoint=kind)[0])
        untouched(out, 7.0)
        untouched(gout, fill)
        assert bool((gs[m * 2 * f // 32:] == 0xA5).all())
        dh, _ = padded(m, f, torch.bfloat16, math.nan)
        dh.copy_(randn(m, m, f))
        dx, xout = padded(m, k, torch.bfloat16, 7.0)
        dw, wout = padded(2 * f, k, torch.bfloat16, 7.0)
        need = lib.sfr_gated_backward_workspace_bytes(m, k, f, 1)
        work = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        assert lib.gated_linear_bf16_backward(dh.data_ptr(), m, k, f, 0, gu.data_ptr(), gs.data_ptr(), save,
                                              px.data_ptr(), None, 1, pw.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                                              work.data_ptr(), need, h) == 0
        untouched(xout, 7.0)
        untouched(wout, 7.0)
        assert bool((work[need:] == 0xFF).all())
        saved = sfr.GatedCheckpoint(x, gu.clone() if save == 1 else sfr.MxTensor(
            gu.clone().view(E4M3 if save == 2 else torch.float8_e5m2),
            gs[:m * 2 * f // 32].clone().view(m, -1).view(torch.float8_e8m0fnu)), "silu")
        ex, ew = sfr.gated_linear_backward(dh.clone(), w, saved)
        assert torch.equal(dx, ex) and torch.equal(dw, ew)


@pytest.mark.parametrize("m,k,f", [(3, 160, 96), (40, 96, 64), (300, 544, 1056)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(sfr, m, k, f, bad):
    """A NaN or infinity in one row of x stays in that row: it reaches every one
    of the row's outputs (as NaN or, for an infinity, as plain arithmetic has
    it), and no other row's bits change."""
    x, w = inputs(m + k, m, k, 2 * f)
    y = x.clone()
    r = m // 2
    y[r, 7] = bad
    others = [i for i in range(m) if i != r]
    q = sfr.quantize_mx(w, FP4)
    for call in (lambda t: sfr.gated_linear(t, w), lambda t: sfr.mxfp4_gated_linear(t, q),
                 lambda t: sfr.mxfp4_linear(t, q)):
        clean, got = call(x), call(y)
        assert torch.equal(got[others], clean[others])
        if math.isnan(bad):
            assert bool(torch.isnan(got[r]).all())
        else:
            assert not bool(torch.isfinite(got[r]).any())
    _, sc = sfr.gated_linear_checkpointed(x, w)
    _, sy = sfr.gated_linear_checkpointed(y, w)
    vc, vy = mx_values(sc.gu), mx_values(sy.gu)
    assert torch.equal(vc[others], vy[others]) and bool(torch.isnan(vy[r]).all())
    dh = randn(3, m, f)
    cx, _ = sfr.gated_linear_backward(dh, w, sc)
    gx, gw = sfr.gated_linear_backward(dh, w, sy)
    assert torch.equal(cx[others], gx[others]) and bool(torch.isnan(gx[r]).all()) and bool(torch.isnan(gw).all())


def test_extreme_values(sfr):
    """Activations of very large and very small arguments: 64-bit values, and no NaN."""
    m, k, f = 16, 32, 32
    x = torch.zeros(m, k)
    x[:, 0] = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1.0, -1.0, 10.0, -10.0, 90.0, -90.0, 200.0, -200.0, 1e4, -1e4,
                            1e18, -1e18])
    w = torch.zeros(2 * f, k)
    w[:f, 0] = 1.0
    w[f:, 0] = 0.5
    x, w = x.bfloat16().cuda(), w.bfloat16().cuda()
    for act in ("silu", "gelu_tanh", "relu"):
        h, bound, _ = gated64(x.double(), w.double(), act)
        tiny = 2.0 ** -126  # below: the exponential's result may be flushed
        got = sfr.gated_linear(x, w, act)
        check(got, h, bound + tiny, act)
        dh = torch.ones(m, f, dtype=torch.bfloat16, device="cuda")
        _, saved = sfr.gated_linear_checkpointed(x, w, act, checkpoint=torch.bfloat16)
        dx, dw = sfr.gated_linear_backward(dh, w, saved)
        assert bool(torch.isfinite(dx).all()) and not bool(torch.isnan(dw).any())


def test_past_32_bit_offsets(sfr):
    """More than 2^31 saved values: the last rows are as right as the first."""
    m, k, f = 75000, 32, 14336
    x, w = inputs(9, m, k, 2 * f)
    h, saved = sfr.gated_linear_checkpointed(x, w)
    assert saved.gu.codes.numel() > 2 ** 31
    pick = torch.tensor([0, 1, 37449, 37450, 74898, m - 2, m - 1], device="cuda")
    ref, bound, (g, u, eg, eu) = gated64(x[pick].double(), w.double(), "silu")
    check(h[pick], ref, bound, "h")
    part = sfr.MxTensor(saved.gu.codes.view(torch.uint8)[pick].view(E4M3), saved.gu.scale.view(torch.uint8)[pick].view(
        torch.float8_e8m0fnu))
    gu, e = torch.cat((g, u), 1), torch.cat((eg, eu), 1)
    scale = torch.exp2(part.scale.view(torch.uint8).double() - 127).repeat_interleave(32, 1)
    check(mx_values(part), gu, e + torch.maximum(2.0 ** -4 * (gu.abs() + e), 2.0 ** -10 * scale), "gu")
    dh = torch.zeros(m, f, dtype=torch.bfloat16, device="cuda")
    dh[pick] = randn(4, len(pick), f)
    dx, dw = sfr.gated_linear_backward(dh, w, saved)
    v = mx_values(part)
    xq = mx_values(sfr.quantize_mx(x[pick], E4M3))
    # rows of zero gradient add exact zeros to dw, so its sum has 7 terms
    rx, bx, rw, bw = gated_grad64(dh[pick].double(), xq, v[:, :f], v[:, f:], w.double(), "silu")
    check(dx[pick], rx, bx, "dx")
    check(dw, rw, bw, "dw")
    rest = torch.ones(m, dtype=torch.bool, device="cuda")
    rest[pick] = False
    assert int((dx[rest] != 0).sum()) == 0
    back = sfr.dequantize_mx(saved.gu)
    assert torch.equal(back[pick].double(), v)
    again = sfr.quantize_mx(back, E4M3)  # values of the format survive it
    assert torch.equal(sfr.dequantize_mx(again)[-3:], back[-3:])


def everything(sfr, x, w, q, dh, bias, checkpoint):
    """One call of each operator on given inputs."""
    h, saved = sfr.gated_linear_checkpointed(x, w, checkpoint=checkpoint)
    dx, dw = sfr.gated_linear_backward(dh, w, saved)
    t = sfr.quantize_mx(x, checkpoint if checkpoint != torch.bfloat16 else E4M3)
    return [h, dx, dw, sfr.gated_linear(x, w, "gelu_tanh"), sfr.mxfp4_gated_linear(x, q, "relu"),
            sfr.mxfp4_linear(x, q, bias), sfr.mxfp4_linear(x, q, out_dtype=torch.float32), sfr.dequantize_mx(t)]


@pytest.mark.parametrize("m,k,f", [(1, 4096, 4128), (20, 288, 96), (130, 4128, 2080), (300, 544, 1056)])
@pytest.mark.parametrize("checkpoint", [torch.bfloat16, E4M3], ids=str)
def test_graph_replay(sfr, m, k, f, checkpoint):
    """Captured calls replayed with new inputs, eager work between the replays; sliced sums among them."""
    x, w = inputs(1, m, k, 2 * f)
    q, dh, bias = sfr.quantize_mx(w, FP4), randn(2, m, f), randn(3, 2 * f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        everything(sfr, x, w, q, dh, bias, checkpoint)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything(sfr, x, w, q, dh, bias, checkpoint)
    for i in range(4):
        nx, nw = inputs(10 + i, m, k, 2 * f)
        nq = sfr.quantize_mx(nw, FP4)
        x.copy_(nx)
        w.copy_(nw)
        dh.copy_(randn(20 + i, m, f))
        q.codes.view(torch.uint8).copy_(nq.codes.view(torch.uint8))
        q.scale.view(torch.uint8).copy_(nq.scale.view(torch.uint8))
        graph.replay()
        want = everything(sfr, x, w, q, dh, bias, checkpoint)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_two_graphs_and_streams(sfr):
    """Two captured graphs replayed at once on two streams, and eager calls with an explicit stream: each has its own
    workspace, so all give what they give alone."""
    shapes = [(300, 544, 1056), (130, 4128, 2080)]
    sets, graphs, outs, wants = [], [], [], []
    for i, (m, k, f) in enumerate(shapes):
        x, w = inputs(30 + i, m, k, 2 * f)
        a = (x, w, sfr.quantize_mx(w, FP4), randn(40 + i, m, f), randn(50 + i, 2 * f), E4M3)
        wants.append([t.clone() for t in everything(sfr, *a)])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(sfr, *a))
        sets.append(a)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    # explicit streams: results are allocated on them, inputs are kept for them
    for (x, w, q, dh, bias, _), s, want in zip(sets, streams, wants):
        s.wait_stream(torch.cuda.current_stream())
        tmp = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        h, saved = sfr.gated_linear_checkpointed(tmp, w, stream=s)
        del tmp
        torch.full_like(x, math.nan)  # would take the freed memory if the call had not kept it
        dx, dw = sfr.gated_linear_backward(dh, w, saved, stream=s)
        y = sfr.mxfp4_linear(x, q, bias, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip((h, dx, dw, y), (want[0], want[1], want[2], want[5])):
            assert torch.equal(a, b)


def test_host_threads(sfr):
    """Calls from several host threads at once, each on a stream of its own: no state is shared."""
    import threading
    sets = []
    for i, (m, k, f) in enumerate([(300, 544, 1056), (130, 4128, 2080), (5, 160, 64)]):
        x, w = inputs(60 + i, m, k, 2 * f)
        sets.append((x, w, sfr.quantize_mx(w, FP4), randn(70 + i, m, f), randn(80 + i, 2 * f), E4M3))
    wants = [[t.clone() for t in everything(sfr, *a)] for a in sets]
    torch.cuda.synchronize()
    same = [False] * len(sets)

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [everything(sfr, *sets[i]) for _ in range(5)]
        s.synchronize()
        same[i] = all(torch.equal(a, b) for g in got for a, b in zip(g, wants[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same)


def test_refusals(sfr):
    x, w = inputs(1, 8, 64, 128)
    q, dh = sfr.quantize_mx(w, FP4), randn(2, 8, 64)
    _, saved = sfr.gated_linear_checkpointed(x, w)
    bad = [
        lambda: sfr.gated_linear(x.t().contiguous().t(), w),                       # not contiguous
        lambda: sfr.gated_linear(x, w[:, ::2]),
        lambda: sfr.gated_linear(x.float(), w),
        lambda: sfr.gated_linear(x[0], w),
        lambda: sfr.gated_linear(x, w[:127]),                                      # odd rows
        lambda: sfr.gated_linear(x, w, "tanh"),
        lambda: sfr.gated_linear(x, w.cpu()),
        lambda: sfr.gated_linear(x, w, out=torch.empty(8, 65, dtype=torch.bfloat16, device="cuda")),
        lambda: sfr.gated_linear(x, w, out=torch.empty(8, 64, device="cuda")),
        lambda: sfr.gated_linear(x, w, out=x),                                     # [8, 64] like h, but an input
        lambda: sfr.gated_linear(x, w, out=w[3:11]),
        lambda: sfr.mxfp4_gated_linear(x, q, out=x),
        lambda: sfr.gated_linear_checkpointed(x, w, checkpoint=torch.float16),
        lambda: sfr.gated_linear_checkpointed(x, w, checkpoint=None),
        lambda: sfr.gated_linear_backward(dh[:4], w, saved),
        lambda: sfr.gated_linear_backward(dh, w[:64], saved),
        lambda: sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(q, saved.gu, "silu")),
        lambda: sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(saved.x, saved.gu, "none")),
        lambda: sfr.gated_linear_backward(dh, w, sfr.GatedCheckpoint(saved.gu, saved.x, "silu")),
        lambda: sfr.mxfp4_linear(x, saved.x),                                      # an 8-bit tensor
        lambda: sfr.mxfp4_linear(x, w),
        lambda: sfr.mxfp4_linear(x[:, :32].contiguous(), q),
        lambda: sfr.mxfp4_linear(x, q, randn(3, 64)),
        lambda: sfr.mxfp4_linear(x, q, out_dtype=torch.float16),
        lambda: sfr.mxfp4_linear(x, sfr.MxTensor(q.codes, q.scale[:, :1].contiguous())),
        lambda: sfr.mxfp4_linear(x, sfr.MxTensor(q.codes, q.scale.view(torch.uint8))),
        lambda: sfr.quantize_mx(x, torch.float16),
        lambda: sfr.dequantize_mx(x),
        lambda: sfr.dequantize_mx(q, out=torch.empty(128, 32, dtype=torch.bfloat16, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    for call in (lambda: sfr.gated_linear(x[:, :48].contiguous(), w[:, :48].contiguous()),   # k % 32
                 lambda: sfr.gated_linear(x, w[:96].contiguous()),                           # f % 32
                 lambda: sfr.quantize_mx(x[:, :48].contiguous()),
                 lambda: sfr.mxfp4_linear(x, sfr.MxTensor(q.codes.view(torch.uint8)[:24].view(FP4),
                                                          q.scale.view(torch.uint8)[:24].view(torch.float8_e8m0fnu)))):
        with pytest.raises(sfr.SfrError):
            call()
    with pytest.raises(sfr.SfrError):  # misaligned: the second row of a tensor whose rows are 8 bytes past 16
        flat = torch.zeros(8 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        sfr.gated_linear(flat[4:].view(8, 64), w)


@pytest.mark.skipif(not torch.cuda.is_available() or torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_other_device(sfr):
    x, w = inputs(1, 40, 96, 128)
    q, dh = sfr.quantize_mx(w, FP4), randn(2, 40, 64)
    want = everything(sfr, x, w, q, dh, randn(3, 128), E4M3)
    to = lambda t: t.to("cuda:1")  # noqa: E731
    q1 = sfr.MxTensor(to(q.codes.view(torch.uint8)).view(FP4), to(q.scale.view(torch.uint8)).view(torch.float8_e8m0fnu))
    got = everything(sfr, to(x), to(w), q1, to(dh), to(randn(3, 128)), E4M3)
    for a, b in zip(got, want):
        assert a.device.index == 1 and torch.equal(a.cpu(), b.cpu())
    with pytest.raises(ValueError):
        sfr.gated_linear(x, to(w))


def test_same_every_time(sfr):
    """Repeated calls give the same bits (fixed order of every sum)."""
    for m, k, f in ((4, 4096, 1056), (130, 4128, 2080), (600, 1056, 2080)):
        x, w = inputs(m, m, k, 2 * f)
        a = (x, w, sfr.quantize_mx(w, FP4), randn(2, m, f), randn(3, 2 * f), E4M3)
        first = everything(sfr, *a)
        for _ in range(3):
            for p, r in zip(first, everything(sfr, *a)):
                assert torch.equal(p, r)


def test_feed_forward_block(sfr):
    """The operators as a model uses them: a training step of the whole block
    (gated projections, then the down projection) from 8-bit checkpoints, and
    the trained weights served in 4 bits, for a prompt and token by token.

    dy -> dh is a plain product here.  Bounds: those of each operator, with the
    operands that it was given."""
    m, k, f = 96, 256, 416
    x, w = inputs(70, m, k, 2 * f)
    wd = randn(71, k, f, scale=0.05)
    h, saved = sfr.gated_linear_checkpointed(x, w)
    ref, bound, _ = gated64(x.double(), w.double(), "silu")
    check(h, ref, bound, "h")
    dy = randn(72, m, k)
    dh = (dy.float() @ wd.float()).bfloat16()
    dx, dw = sfr.gated_linear_backward(dh, w, saved)
    g = mx_values(saved.gu)
    rx, bx, rw, bw = gated_grad64(dh.double(), mx_values(saved.x), g[:, :f], g[:, f:], w.double(), "silu")
    check(dx, rx, bx, "dx")
    check(dw, rw, bw, "dw")
    w = (w.float() - 0.1 * dw.float()).bfloat16()
    q, qd = sfr.quantize_mx(w, FP4), sfr.quantize_mx(wd, FP4)
    hp = sfr.mxfp4_gated_linear(x, q)
    y = sfr.mxfp4_linear(hp, qd)
    ref, bound, _ = gated64(x.double(), mx_values(q), "silu")
    check(hp, ref, bound, "served h")
    ry, ey = products64(hp.double(), mx_values(qd))
    check(y, ry, ey + HALF_BF16 * (ry.abs() + ey) + 2.0 ** -133, "served y")
    for i in (0, 17, m - 1):  # one token at a time: the same sums in another order
        hi = sfr.mxfp4_gated_linear(x[i:i + 1], q)
        check(hi, ref[i:i + 1], bound[i:i + 1], "token h")
        ri, ei = products64(hi.double(), mx_values(qd))
        check(sfr.mxfp4_linear(hi, qd), ri, ei + HALF_BF16 * (ri.abs() + ei) + 2.0 ** -133, "token y")
