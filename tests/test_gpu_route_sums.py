"""GPU: the router's logits where products of two bf16 values leave binary32, in each
of the kernels that form them (by the size of the call)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
# tokens of a call of ten experts: each of the kernels
CALLS = [1, 7, 40, 2000, 5000, 17000]


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def tokens(kinds, m):
    """m tokens, the kinds of row in turn."""
    return kinds[torch.arange(m) % kinds.shape[0]].bfloat16().cuda()


def same(a, b):
    """Equal values, NaN equal to NaN."""
    return torch.equal(torch.nan_to_num(a, 0.0), torch.nan_to_num(b, 0.0)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("m", CALLS)
def test_products_outside_binary32(sfr, m):
    """Products past 2^128 that cancel, under 2^-149, and among the subnormal numbers.
    Every sum is exact in binary64, in any order, so the logit is the exact one rounded."""
    k = 1024
    x, w = torch.zeros(4, k, dtype=torch.float64), torch.zeros(10, k, dtype=torch.float64)
    x[0, :3] = torch.tensor([2.0 ** 70, 2.0 ** 70, 1.5 * 2.0 ** 40])
    w[0, :2] = torch.tensor([2.0 ** 70, -2.0 ** 70])                  # 2^140 - 2^140
    w[1, :3] = torch.tensor([2.0 ** 70, -2.0 ** 70, 2.0 ** 80])       # and 1.5 2^120
    w[2, :2] = torch.tensor([-2.0 ** 70, 2.0 ** 70 * (1 - 2.0 ** -7)])  # -2^133: out of range after rounding
    w[3, :2] = torch.tensor([2.0 ** 127, 2.0 ** 127])
    x[1] = 2.0 ** -75
    w[4] = 2.0 ** -80                                                 # 1024 of 2^-155: 2^-145
    w[5] = 1.5 * 2.0 ** -74                                           # 1024 of 1.5 2^-149
    w[6], w[6, ::2] = 2.0 ** -76, -2.0 ** -76 * (1 - 2.0 ** -7)       # 512 of 2^-158: 2^-149
    x[2, 5], w[7, 5] = 2.0 ** -133, 2.0 ** 127                        # of a subnormal value
    x[3, 6:8] = torch.tensor([3.0 * 2.0 ** -100, 2.0 ** -133])
    w[8, 6:8] = torch.tensor([2.0 ** -49, -2.0 ** -16])               # 3 2^-149 - 2^-149
    assert torch.equal(x.bfloat16().double(), x) and torch.equal(w.bfloat16().double(), w)
    want = (x @ w.t())[torch.arange(m) % 4].float()
    r = sfr.moe_route(tokens(x, m), w.bfloat16().cuda(), 3)
    assert torch.equal(r.logits.cpu(), want)
    order = torch.argsort(want.double(), dim=1, descending=True, stable=True)[:, :3]
    dead = torch.gather(want, 1, order) == -math.inf
    assert torch.equal(r.ids.cpu().long(), torch.where(dead, -1, order))


@pytest.mark.parametrize("m", CALLS)
def test_infinities(sfr, m):
    """Infinities in x and in w, against zeros, ordinary values and each other."""
    k = 64
    x, w = torch.ones(4, k, dtype=torch.float64), torch.ones(10, k, dtype=torch.float64)
    x[0, 3], x[1, 4], x[2, 3], x[2, 40] = math.inf, -math.inf, math.inf, math.inf
    w[1, 3], w[2, 40], w[3, 3] = 0.0, -1.0, -2.0
    w[4, 50], w[5, 50] = math.inf, -math.inf
    r = sfr.moe_route(tokens(x, m), w.bfloat16().cuda(), 2)
    want = (x[:, None] * w[None]).sum(2)[torch.arange(m) % 4].float()
    assert same(r.logits.cpu(), want)


@pytest.mark.parametrize("k", [32, 64, 288, 1024, 1056, 2080, 4096, 7200])
def test_sums_do_not_depend_on_the_call(sfr, k):
    """Sums that cancel until only what binary64 lost is left, so that another order of
    their terms is another logit: the same bits for a token alone, in small and in large
    calls, and for an expert among others."""
    g = torch.Generator().manual_seed(k)
    m, experts = 17000, 10

    def wide(rows):  # values over 2^80, every one of them once more
        v = torch.randn(rows, k // 2, generator=g) * torch.exp2(torch.randint(-40, 40, (rows, k // 2), generator=g).float())
        return torch.cat((v, v), 1).bfloat16()
    x, w = wide(40)[torch.arange(m) % 40].cuda(), wide(experts).cuda()
    w[:, k // 2:] *= -1
    order = torch.randperm(k, generator=g).cuda()
    x, w = x[:, order].contiguous(), w[:, order].contiguous()
    whole = sfr.moe_route(x, w, 3)
    # sums that lost nothing would be 0
    assert bool((whole.logits[:40] != 0).any()) or k < 64
    for rows in (slice(0, 1), slice(1, 6), slice(3, 40), slice(7, 1300), slice(100, 6000), slice(10, 16900)):
        part = sfr.moe_route(x[rows].clone(), w, 3)
        assert torch.equal(part.logits, whole.logits[rows]) and torch.equal(part.ids, whole.ids[rows]), rows
        assert torch.equal(part.weights, whole.weights[rows]), rows
    among = torch.randperm(300, generator=g)[:experts].cuda()
    many = wide(300).cuda()
    many[among] = w
    for rows in (slice(0, 1), slice(0, 30), slice(0, 100), slice(0, 1000)):
        part = sfr.moe_route(x[rows].clone(), many, 3)
        assert torch.equal(part.logits[:, among], whole.logits[rows]), rows


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m", [1, 40, 6000])
def test_weights_of_logits_that_are_not_finite(sfr, score, renormalize, m):
    x, w = torch.zeros(m, 32, device="cuda").bfloat16(), torch.zeros(10, 32, device="cuda").bfloat16()
    bias = torch.tensor([0.5, -1.0, 2.0, 0.0, 1.0, -math.inf, 3.0, -2.0, 0.25, -0.5], device="cuda")
    for value in (math.nan, math.inf):
        bias[4] = value
        r = sfr.moe_route(x, w, 3, bias, score, renormalize)
        assert bool((r.ids.cpu() == torch.tensor([4, 6, 2])).all())
        l = torch.tensor([value, 3.0, 2.0], dtype=torch.float64)
        if score == "softmax":
            want = torch.full((3,), math.nan, dtype=torch.float64)
        else:
            want = torch.sigmoid(l)
            want = want / want.sum() if renormalize else want
        got = r.weights.double().cpu()
        assert torch.equal(got.isnan(), want.isnan().expand(m, 3))
        # exponentials and logarithms good to two steps, a quotient, sums of three: under 16 roundings
        assert bool(((got - want).abs()[~got.isnan()] <= 16 * 2.0 ** -24).all())
