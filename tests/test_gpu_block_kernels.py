"""GPU: the gated block and its gradients against 64-bit results on shapes whose
kernels the other tests' shapes do not reach."""
import pytest
import torch

from block_ref import check, gated64, gated_grad64, inputs, mx_values

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


# 3 .. 8 rows of a bf16 weight: few and many units of k per wavefront, k at the
# ends of a unit (128) and inside it, one pair of row tiles to many
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m,k,f", [(3, 32, 32), (3, 416, 96), (4, 128, 64), (5, 4128, 1056), (7, 1056, 224),
                                   (8, 96, 4128), (8, 4128, 96), (8, 4096, 2048)])
def test_forward_few_rows(sfr, m, k, f, act):
    x, w = inputs(m + k, m, k, 2 * f)
    h, bound, _ = gated64(x.double(), w.double(), act)
    check(sfr.gated_linear(x, w, act), h, bound, "h")


# dx of few rows and a long sum, in sliced 128 x 128 tiles
@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("m,k,f", [(68, 3616, 8608), (65, 8224, 2048), (77, 8224, 2080)])
def test_backward_sliced(sfr, m, k, f, eight_bits):
    x, w = inputs(m + f, m, k, 2 * f)
    dh, gu = randn(m, m, f), randn(m + 1, m, 2 * f)
    if eight_bits:
        saved = sfr.GatedCheckpoint(sfr.quantize_mx(x, torch.float8_e5m2), sfr.quantize_mx(gu, E4M3), "silu")
        x, gu = mx_values(saved.x), mx_values(saved.gu)
    else:
        saved = sfr.GatedCheckpoint(x, gu, "silu")
        x, gu = x.double(), gu.double()
    dx, dw = sfr.gated_linear_backward(dh, w, saved)
    rx, bx, rw, bw = gated_grad64(dh.double(), x, gu[:, :f], gu[:, f:], w.double(), "silu")
    check(dx, rx, bx, "dx")
    check(dw, rw, bw, "dw")
