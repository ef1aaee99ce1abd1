"""GPU: more rows than the wavefronts of one grid (2^26)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
P, REPS = 1025, 65537  # 67175425 rows, the same 1025 again and again


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def rows(cols, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(P, cols, generator=g, device="cuda").bfloat16()


def repeats(whole, part):
    return torch.equal(whole.view(REPS, *part.shape), part.expand(REPS, *part.shape))


def test_router(sfr):
    x = rows(32, 1)
    w = rows(32, 2)[:3].contiguous()
    part = sfr.moe_route(x, w, 2)
    whole = sfr.moe_route(x.repeat(REPS, 1), w, 2)
    assert whole.ids.shape[0] > 1 << 26
    assert repeats(whole.logits, part.logits) and repeats(whole.ids, part.ids) and repeats(whole.weights, part.weights)


def test_int8(sfr):
    """The quantizer, by itself and within the layer."""
    x = rows(16, 3)
    w = sfr.quantize_rowwise_int8(rows(16, 4)[:16].contiguous())
    part, y = sfr.quantize_rowwise_int8(x), sfr.int8_linear(x, w)
    x = x.repeat(REPS, 1)
    whole = sfr.quantize_rowwise_int8(x)
    assert repeats(whole.codes, part.codes) and repeats(whole.scale, part.scale)
    del whole
    assert repeats(sfr.int8_linear(x, w), y)


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_fp8(sfr, fmt):
    x = rows(8, 5)
    codes, scale = sfr.quantize_rowwise_fp8(x, fmt)
    many, scales = sfr.quantize_rowwise_fp8(x.repeat(REPS, 1), fmt)
    assert repeats(many.view(torch.uint8), codes.view(torch.uint8)) and repeats(scales, scale)
