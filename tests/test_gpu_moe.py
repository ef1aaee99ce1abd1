"""GPU: the expert router and the mixture-of-experts layer against 64-bit forms
(moe_ref), at the sizes, choices and values where they can go wrong."""
import math
import threading

import pytest
import torch

from block_rms import ROUND, rms, sums
from moe_ref import FP4, as_form, experts64, layer64, stacked, weights64

pytestmark = pytest.mark.gpu
FORMS = ["bf16", "int8", "fp4"]
# m, k, f, experts, top: token counts around the forms' limits and past one pass, sizes
# inside units and tiles, one expert, more slots than experts' worth of tokens
LAYERS = [(1, 32, 32, 1, 1), (1, 4096, 64, 4, 2), (1, 96, 1408, 8, 8), (2, 288, 160, 5, 3), (3, 64, 4128, 3, 2),
          (5, 544, 96, 33, 6), (8, 160, 288, 64, 8), (9, 256, 416, 4, 2), (15, 32, 96, 130, 16), (16, 320, 224, 16, 4),
          (17, 96, 352, 8, 2), (31, 416, 160, 3, 1), (32, 128, 128, 12, 4), (33, 224, 64, 6, 3), (47, 64, 544, 64, 8),
          (64, 352, 288, 8, 2), (65, 128, 96, 9, 2), (130, 96, 160, 1000, 5), (200, 64, 32, 2, 2),
          # the tiles of many and of large experts
          (10, 1536, 512, 48, 4), (40, 2048, 768, 36, 3), (9, 2112, 1440, 40, 2), (33, 1024, 2080, 32, 2), (46, 544, 768, 64, 3), (16, 1056, 288, 60, 3),
          # more groups of tiles than workgroups, of one expert and of several
          (20, 64, 16416, 5, 2), (20, 8224, 64, 5, 2), (12, 2080, 1056, 40, 3), (2, 64, 8224, 16, 16), (8, 8224, 96, 6, 4)]


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def check(got, ref, bound, what=""):
    assert got.shape == ref.shape
    far = (got.double() - ref).abs() - bound
    assert bool((far <= 0).all()), (what, far.max().item())


def compare(sfr, x, ids, weights, gu, down, act="silu", **kw):
    out = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down, act, **kw)
    check(out, *layer64(x, ids, weights, gu, down, act), "out")
    return out


# ------------------------------------------------------------------ layer


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("m,k,f,experts,top", LAYERS)
def test_layer(sfr, m, k, f, experts, top, form):
    compare(sfr, *stacked(m + k + f, m, k, f, experts, top, form, sfr), ["silu", "gelu_tanh", "relu"][(m + f // 32) % 3])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("form", FORMS)
def test_activations(sfr, form, act):
    compare(sfr, *stacked(11, 6, 128, 96, 4, 2, form, sfr), act)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("m,k,f,experts,top", [(1, 4096, 1408, 16, 4), (7, 2048, 1440, 12, 3), (16, 1056, 2080, 8, 2),
                                               (40, 1024, 1024, 8, 2), (64, 2048, 544, 16, 4)])
def test_root_mean_square(sfr, m, k, f, experts, top, form):
    """Two independent roundings (h, and out) and the two sums: a wider error is
    a missing or doubled term (32 of the f * top terms that an output sums are 7% of it)."""
    x, ids, weights, gu, down = stacked(5, m, k, f, experts, top, form, sfr, 0.05)
    out = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down, "silu")
    ref = layer64(x, ids, weights, gu, down, "silu")[0]
    assert rms(out.double() - ref) <= (1.1 * math.sqrt(2) * ROUND + sums(k) + sums(f * top)) * rms(ref)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("m", [1, 2, 7, 16, 20, 32, 33, 48, 49, 64, 70])
def test_every_token_to_one_expert(sfr, m, form):
    """The longest list an expert can have, in the last place."""
    x, ids, weights, gu, down = stacked(m, m, 160, 96, 6, 2, form, sfr)
    ids[:, 0], ids[:, 1] = 5, -1
    compare(sfr, x, ids, weights, gu, down)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("m", [1, 4, 16, 33, 64])
def test_slots_without_an_expert(sfr, m, form):
    """ids outside the experts, tokens with none at all, an expert named twice (and three times)."""
    x, ids, weights, gu, down = stacked(m, m, 96, 128, 7, 6, form, sfr)
    outside = torch.tensor([-1, 7, 8, -2 ** 31, 2 ** 31 - 1, 1 << 16], dtype=torch.int32, device="cuda")
    drop = torch.rand(m, 6, device="cuda") < 0.4
    ids = torch.where(drop, outside.expand(m, 6), ids)
    ids[:, 3] = ids[:, 0]
    if m > 2:
        ids[m // 2] = outside
        ids[0, :3] = 4
    ids = ids.contiguous()
    out = compare(sfr, x, ids, weights, gu, down)
    if m > 2:
        assert bool((out[m // 2] == 0).all())
    # nobody chose anything
    none = sfr.moe_layer(x, sfr.MoeRoute(torch.full_like(ids, -1), weights), gu, down)
    assert bool((none == 0).all())


@pytest.mark.parametrize("form", FORMS)
def test_shares_of_two_devices(sfr, form):
    """Experts split between two calls with shifted ids: each call's ids outside its
    own are no choice, and the shares add up."""
    x, ids, weights, gu, down = stacked(3, 12, 64, 96, 10, 4, "bf16", sfr)
    whole, bound = layer64(x, ids, weights, *as_form(sfr, gu, down, form), "silu")
    total = torch.zeros_like(whole)
    for a, b in ((0, 4), (4, 10)):
        part = as_form(sfr, gu[a:b].contiguous(), down[a:b].contiguous(), form)
        share = compare(sfr, x, ids - a, weights, *part)
        total += share.double()
    assert bool(((total - whole).abs() <= 3 * bound + 2.0 ** -7 * whole.abs().max()).all())


@pytest.mark.parametrize("m", [1, 5, 16, 20, 64])
@pytest.mark.parametrize("form", FORMS)
def test_not_finite_stays_with_its_tokens(sfr, m, form):
    """NaN and infinities in an expert's weights and in tokens' rows."""
    x, ids, weights, gu, down = stacked(7, m, 128, 96, 4, 2, "bf16", sfr)
    ids[:, 0], ids[:, 1] = 0, 1
    ids[m // 2:, 1] = 3  # the broken expert belongs to the upper half
    gu[3, 5, 7], down[3, 2, 3] = math.inf, math.nan
    if m > 4:
        x[1] = math.nan
        x[2, 3], ids[2] = math.inf, -1
        ids[m - 1, 0] = -1
        ids[m - 1, 1] = 2
    parts = as_form(sfr, gu, down, form)
    out = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), *parts)
    # tokens of the sound experts, by themselves
    good = torch.arange(m, device="cuda") < m // 2
    if m > 4:
        good[1] = False
        good[m - 1] = True
        assert bool(torch.isnan(out[1]).all()) and bool((out[2] == 0).all())
    xs = torch.where(torch.isfinite(x), x, 0.0)
    gu[3], down[3] = 0, 0
    sound = as_form(sfr, gu, down, form)
    ref, bound = layer64(xs, ids, weights, *sound, "silu")
    check(out[good], ref[good], bound[good])
    broken = ~good
    if m > 4:
        broken[1] = broken[2] = False
    assert bool(torch.isnan(out[broken]).any(1).all())


@pytest.mark.parametrize("m", [2, 16, 33])
def test_weights_that_are_not_finite(sfr, m):
    x, ids, weights, gu, down = stacked(8, m, 64, 64, 4, 2, "bf16", sfr)
    weights[0, 1] = math.nan
    weights[1, 0] = 0.0
    ids[1, 1] = -1
    weights[1, 1] = math.nan  # of no choice: not read into the sum
    out = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down)
    assert bool(torch.isnan(out[0]).all()) and bool((out[1] == 0).all()) and bool(torch.isfinite(out[2:]).all())


def within(t, fill):
    flat = torch.full((t.numel() + 4096,), fill, device="cuda").to(t.dtype)
    flat[2048:2048 + t.numel()] = t.reshape(-1)
    return flat[2048:2048 + t.numel()].view(t.shape), flat


@pytest.mark.parametrize("form", ["bf16", "int8"])
@pytest.mark.parametrize("m", [1, 7, 16, 30, 64])
def test_padding_is_not_read_or_written(sfr, m, form):
    """Operands inside larger buffers of NaN (codes: -128), the output inside one of sevens."""
    x, ids, weights, gu, down = stacked(m, m, 96, 160, 5, 2, form, sfr)
    want = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down)
    if form == "bf16":
        gu, down = within(gu, math.nan)[0], within(down, math.nan)[0]
    else:
        gu, down = (sfr.Int8Tensor(within(w.codes, -128)[0], within(w.scale, math.nan)[0]) for w in (gu, down))
    x, ids, weights = within(x, math.nan)[0], within(ids, 0)[0], within(weights, math.nan)[0]
    out, flat = within(torch.zeros_like(x), 7.0)
    sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down, out=out)
    assert torch.equal(out, want)
    assert bool((flat[:2048] == 7).all()) and bool((flat[2048 + out.numel():] == 7).all())


@pytest.mark.parametrize("form", FORMS)
def test_past_32_bit_offsets(sfr, form):
    """Experts past 2^32 values: the last of them is the one that counts."""
    k, f, experts = 2080, 8192, 130
    last = stacked(1, 3, k, f, 1, 1, "bf16", sfr, 0.02)
    x, weights = last[0], last[2]
    parts = as_form(sfr, *last[3:], form)
    ids = torch.full((3, 1), experts - 1, dtype=torch.int32, device="cuda")

    def at_the_end(t, axis=0):
        n = t.shape[0]
        big = torch.zeros((experts * n, *t.shape[1:]), dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
        big[(experts - 1) * n:] = t.view(big.dtype)
        return big.view(t.dtype)
    if form == "bf16":
        gu, down = (at_the_end(w) for w in parts)
    else:
        gu, down = (type(w)(at_the_end(w.codes), at_the_end(w.scale)) for w in parts)
    out = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down)
    check(out, *layer64(x, torch.zeros_like(ids), weights, *parts, "silu"))


@pytest.mark.parametrize("m", [1, 16, 70])
@pytest.mark.parametrize("form", FORMS)
def test_graph_replay(sfr, m, form):
    """Router and layer captured together, replayed with new tokens (and so new experts),
    eager calls and synchronizations between."""
    k, f, experts, top = 256, 160, 20, 4
    x, _, _, gu, down = stacked(2, m, k, f, experts, top, form, sfr)
    w = torch.randn(experts, k, device="cuda").bfloat16()
    sfr.moe_layer(x, sfr.moe_route(x, w, top), gu, down)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        route = sfr.moe_route(x, w, top)
        out = sfr.moe_layer(x, route, gu, down)
    for i in range(4):
        x.copy_(torch.randn(m, k, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        r = sfr.moe_route(x, w, top)
        assert torch.equal(r.ids, route.ids) and torch.equal(r.weights, route.weights)
        assert torch.equal(sfr.moe_layer(x, r, gu, down), out)
        check(out, *layer64(x, r.ids, r.weights, gu, down, "silu"))


def test_streams_graphs_and_threads(sfr):
    """An explicit stream, two captured graphs run at once, several host threads."""
    k, f, experts, top = 512, 416, 8, 2
    data = [stacked(i, m, k, f, experts, top, form, sfr) for i, (m, form) in
            enumerate([(1, "bf16"), (9, "int8"), (30, "fp4"), (100, "bf16")])]
    want = [sfr.moe_layer(x, sfr.MoeRoute(i, w), *p) for x, i, w, *p in data]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [sfr.moe_layer(x, sfr.MoeRoute(i, w), *p, stream=side) for x, i, w, *p in data]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for x, i, w, *p in data[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sfr.moe_layer(x, sfr.MoeRoute(i, w), *p)
        graphs.append((g, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, out, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, w) for (_, out, _), w in zip(graphs, want))
    bad = []

    def work(n):
        x, i, w, *p = data[n]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                if not torch.equal(sfr.moe_layer(x, sfr.MoeRoute(i, w), *p), want[n]):
                    bad.append(n)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(data))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


@pytest.mark.parametrize("form", FORMS)
def test_tokens_do_not_depend_on_the_batch(sfr, form):
    """From nine tokens on a token's bits are its own, whoever else is in the pass."""
    x, ids, weights, gu, down = stacked(9, 64, 288, 416, 6, 2, form, sfr)
    ids[::2, 0] = 5  # 32 tokens and more to one expert
    whole = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down)
    for rows in (slice(0, 9), slice(3, 20), slice(20, 57), slice(0, 64, 2), slice(0, 64, 5)):
        part = [t[rows].contiguous() for t in (x, ids, weights)]
        assert torch.equal(sfr.moe_layer(part[0], sfr.MoeRoute(*part[1:]), gu, down), whole[rows]), rows
    # one more than a pass: the last token in a pass of its own
    twice = [torch.cat((t, t[:1])) for t in (x, ids, weights)]
    again = sfr.moe_layer(twice[0], sfr.MoeRoute(*twice[1:]), gu, down)
    assert torch.equal(again[:64], whole) and torch.equal(again[64:], whole[:1])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("k,f", [(1024, 1024), (2080, 544), (288, 4128)])
def test_tokens_do_not_depend_on_the_kernels(sfr, form, k, f):
    """Nine tokens on few experts and 64 on many take tiles of different sizes."""
    x, ids, weights, gu, down = stacked(k, 64, k, f, 64, 1, form, sfr, 0.05)
    ids[:9] = 7
    whole = compare(sfr, x, ids, weights, gu, down)
    for rows in (slice(0, 9), slice(5, 16), slice(10, 35), slice(0, 64, 3)):
        part = [t[rows].contiguous() for t in (x, ids, weights)]
        assert torch.equal(sfr.moe_layer(part[0], sfr.MoeRoute(*part[1:]), gu, down), whole[rows]), rows


def test_layer_refusals(sfr):
    x, ids, weights, gu, down = stacked(1, 4, 64, 96, 5, 2, "bf16", sfr)
    r = sfr.MoeRoute(ids, weights)
    q, qd = as_form(sfr, gu, down, "int8")
    p, pd = as_form(sfr, gu, down, "fp4")
    ok = sfr.moe_layer(x, r, gu, down)
    M = sfr.MoeRoute
    for bad in (lambda: sfr.moe_layer(x.float(), r, gu, down), lambda: sfr.moe_layer(x[:, :32].contiguous(), r, gu, down),
                lambda: sfr.moe_layer(x[:3], r, gu, down), lambda: sfr.moe_layer(x, M(ids.long(), weights), gu, down),
                lambda: sfr.moe_layer(x, M(ids, weights.double()), gu, down),
                lambda: sfr.moe_layer(x, M(ids, weights[:, :1]), gu, down),
                lambda: sfr.moe_layer(x, M(ids.cpu(), weights), gu, down),
                lambda: sfr.moe_layer(x, M(ids.t().contiguous().t(), weights), gu, down),
                lambda: sfr.moe_layer(x, r, gu, qd), lambda: sfr.moe_layer(x, r, q, pd),
                lambda: sfr.moe_layer(x, r, gu[:4], down), lambda: sfr.moe_layer(x, r, gu, down[:4]),
                lambda: sfr.moe_layer(x, r, gu.view(10, 96, 64), down), lambda: sfr.moe_layer(x, r, gu.view(-1, 64), down),
                lambda: sfr.moe_layer(x, r, gu.float(), down), lambda: sfr.moe_layer(x, r, down, gu),
                lambda: sfr.moe_layer(x, r, gu.transpose(1, 2), down),
                lambda: sfr.moe_layer(x, r, sfr.Int8Tensor(q.codes[:-1], q.scale[:-1]), qd),
                lambda: sfr.moe_layer(x, r, sfr.quantize_mx(gu.view(-1, 64)), sfr.quantize_mx(down.view(-1, 96))),
                lambda: sfr.moe_layer(x, r, gu, down, "tanh"), lambda: sfr.moe_layer(x, r, gu, down, out=ok[:3]),
                lambda: sfr.moe_layer(x, r, gu, down, out=x), lambda: sfr.moe_layer(x, r, gu, down, out=down.view(-1)[:256].view(4, 64)),
                lambda: sfr.moe_layer(x.cpu(), r, gu, down)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sfr.moe_layer(x, M(ids.repeat(1, 9), weights.repeat(1, 9)), gu, down),
                lambda: sfr.moe_layer(x, M(ids[:, :0], weights[:, :0]), gu, down),
                lambda: sfr.moe_layer(x.view(-1)[1:193].view(3, 64), M(ids[:3], weights[:3]), gu, down)):
        with pytest.raises(sfr.SfrError):
            bad()
    # rows of a larger batch: ids and weights at addresses of 8 bytes
    compare(sfr, x[1:], ids[1:], weights[1:], gu, down)
    assert sfr.moe_layer(x[:0], M(ids[:0], weights[:0]), gu, down).shape == (0, 64)
    assert not sfr.moe_layer(x.clone().requires_grad_(), r, gu, down).requires_grad


@pytest.mark.parametrize("form", FORMS)
def test_same_every_time(sfr, form):
    x, ids, weights, gu, down = stacked(4, 40, 512, 416, 16, 4, form, sfr)
    first = sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down)
    for _ in range(20):
        assert torch.equal(sfr.moe_layer(x, sfr.MoeRoute(ids, weights), gu, down), first)


# ------------------------------------------------------------------ router


def check_route(r, logits64, top, score, renormalize):
    """Logits against the exact ones; ids by the order of the logits; weights from both."""
    l = r.logits
    fin = torch.isfinite(logits64)
    assert bool(((l.double() - logits64).abs()[fin] <= 2.0 ** -24 * (1 + 2.0 ** -20) * logits64.abs()[fin] + 2.0 ** -149).all())
    order = torch.argsort(torch.where(l == 0, 0.0, l).double().cpu(), dim=1, descending=True, stable=True)[:, :top]
    dead = torch.gather(l.cpu(), 1, order) == -math.inf
    assert torch.equal(r.ids.cpu().long(), torch.where(dead, -1, order))
    w, rel = weights64(l, r.ids, score, renormalize)
    assert bool(((r.weights.double() - w).abs() <= rel * w + 2.0 ** -125).all())


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("m,k,experts,top", [(1, 32, 1, 1), (1, 2048, 64, 8), (2, 96, 5, 5), (3, 4096, 130, 6),
                                             (5, 7200, 256, 16), (16, 160, 63, 4), (17, 544, 65, 2), (33, 1056, 129, 8),
                                             (64, 256, 1024, 16), (300, 416, 257, 7), (1000, 4096, 161, 6), (1100, 96, 250, 3), (70000, 32, 3, 2),
                                             (6000, 32, 2, 1)])
def test_route(sfr, m, k, experts, top, score, renormalize):
    g = torch.Generator("cuda").manual_seed(m + k)
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    w = (2 / math.sqrt(k) * torch.randn(experts, k, generator=g, device="cuda")).bfloat16()
    bias = torch.randn(experts, generator=g, device="cuda") if m % 2 else None
    r = sfr.moe_route(x, w, top, bias, score, renormalize)
    ref = x.double() @ w.double().t()
    check_route(r, ref if bias is None else ref + bias.double(), top, score, renormalize)


def test_route_ties(sfr):
    """Equal logits in every pattern: the lowest expert first; -0 is 0."""
    x = torch.zeros(40, 64, device="cuda", dtype=torch.bfloat16)
    x[torch.arange(40), torch.arange(40)] = 1
    w = torch.randint(-1, 2, (200, 64), device="cuda").bfloat16()
    w = torch.where(w == 0, torch.where(torch.rand(200, 64, device="cuda") < 0.5, -0.0, 0.0).bfloat16(), w)
    for bias in (None, torch.where(torch.rand(200, device="cuda") < 0.5, -0.0, 0.0)):
        r = sfr.moe_route(x, w, 12, bias)
        check_route(r, x.double() @ w.double().t(), 12, "softmax", True)


def test_route_nearly_equal(sfr):
    """Two experts that differ by the last bit of one product among 4096: the choice
    follows the exact logits, alone and in every batch."""
    k = 4096
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(70, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(40, k, generator=g, device="cuda").bfloat16()
    w[20:] = w[:20]
    at = torch.randint(0, k, (20,), generator=g, device="cuda")
    w.view(torch.int16)[20 + torch.arange(20, device="cuda"), at] ^= 1
    whole = sfr.moe_route(x, w, 8)
    check_route(whole, x.double() @ w.double().t(), 8, "softmax", True)
    for rows in (slice(0, 1), slice(3, 7), slice(10, 30), slice(5, 70)):
        part = sfr.moe_route(x[rows].clone(), w, 8)
        assert torch.equal(part.ids, whole.ids[rows]) and torch.equal(part.logits, whole.logits[rows])
        assert torch.equal(part.weights, whole.weights[rows])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_masked_and_far(sfr, score, renormalize):
    """Experts shut off by a bias of -inf, all of them too; logits far from zero."""
    x = torch.randn(9, 64, device="cuda").bfloat16()
    w = torch.randn(70, 64, device="cuda").bfloat16()
    ref = x.double() @ w.double().t()
    bias = torch.full((70,), -math.inf, device="cuda")
    r = sfr.moe_route(x, w, 5, bias, score, renormalize)
    assert bool((r.ids == -1).all()) and bool((r.weights == 0).all())
    bias[3] = bias[66] = bias[69] = 0.5
    check_route(sfr.moe_route(x, w, 5, bias, score, renormalize), ref + bias.double(), 5, score, renormalize)
    for shift in (-3e4, -150.0, 150.0, 3e4):
        bias = torch.full((70,), shift, device="cuda")
        check_route(sfr.moe_route(x, w, 5, bias, score, renormalize), ref + shift, 5, score, renormalize)


@pytest.mark.parametrize("m,experts", [(4, 20), (200, 100), (1100, 300)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_not_finite(sfr, score, m, experts):
    x = torch.randn(m, 64, device="cuda").bfloat16()
    x[1, 5] = math.nan
    w = torch.randn(experts, 64, device="cuda").bfloat16()
    bias = torch.zeros(experts, device="cuda")
    bias[7] = math.nan
    r = sfr.moe_route(x, w, 3, None, score)
    assert torch.equal(r.ids[1].cpu(), torch.arange(3, dtype=torch.int32)) and bool(torch.isnan(r.weights[1]).all())
    keep = torch.arange(m, device="cuda") != 1
    assert bool(torch.isfinite(r.weights[keep]).all())
    r = sfr.moe_route(x[keep], w, 3, bias, score)
    assert bool((r.ids[:, 0] == 7).all()) and bool(torch.isnan(r.weights[:, 0]).all())


def test_route_refusals(sfr):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(10, 64, device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: sfr.moe_route(x.float(), w, 2), lambda: sfr.moe_route(x, w[:, :32].contiguous(), 2),
                lambda: sfr.moe_route(x, w, 0), lambda: sfr.moe_route(x, w, 11), lambda: sfr.moe_route(x, w, 2, score="top"),
                lambda: sfr.moe_route(x, w, 2, torch.zeros(9, device="cuda")),
                lambda: sfr.moe_route(x, w, 2, torch.zeros(10, device="cuda", dtype=torch.bfloat16)),
                lambda: sfr.moe_route(x, w, 2, torch.zeros(10)), lambda: sfr.moe_route(x.cpu(), w, 2),
                lambda: sfr.moe_route(x, w.cpu(), 2)):
        with pytest.raises(ValueError):
            bad()
    many = torch.zeros(1056, 64, device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: sfr.moe_route(x, many, 2), lambda: sfr.moe_route(x, many[:64], 17),
                lambda: sfr.moe_route(x[:, :40].contiguous(), w[:, :40].contiguous(), 2)):
        with pytest.raises(sfr.SfrError):
            bad()
    r = sfr.moe_route(x[:0], w, 2)
    assert r.ids.shape == (0, 2) and r.logits.shape == (0, 10)


def test_block_of_all(sfr):
    """A feed-forward half of a layer as a model runs it: an 8-bit projection, the
    router, the experts in each form, and an 8-bit projection of the result, for one
    token and for a batch."""
    k, f, experts, top = 512, 288, 12, 3
    g = torch.Generator("cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    wi, wo = (sfr.quantize_rowwise_int8((r(k, k) / math.sqrt(k)).bfloat16()) for _ in range(2))
    wr = (r(experts, k) / math.sqrt(k)).bfloat16()
    gu, down = (r(experts, 2 * f, k) / math.sqrt(k)).bfloat16(), (r(experts, k, f) / math.sqrt(f)).bfloat16()
    for m in (1, 24, 90):
        x = r(m, k).bfloat16()
        for form in FORMS:
            parts = as_form(sfr, gu, down, form)
            a = sfr.int8_linear(x, wi)
            route = sfr.moe_route(a, wr, top)
            check_route(route, a.double() @ wr.double().t(), top, "softmax", True)
            y = compare(sfr, a, route.ids, route.weights, *parts)
            z = sfr.int8_linear(sfr.quantize_rowwise_int8(y), wo)
            assert torch.equal(z, sfr.int8_linear(y, wo))
            # against the whole in 64 bits: what 8- and 4-bit weights and 8-bit tokens leave, far under the values
            h = x.double() @ experts64(wi, k)[0].t()
            full = layer64(h.bfloat16(), route.ids, route.weights, *parts, "silu")[0] @ experts64(wo, k)[0].t()
            assert rms(z.double() - full) <= 0.05 * rms(full)
