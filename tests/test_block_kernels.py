"""The gated block's and the 4-bit layer's kernels on the CPU: the shapes of the
reference-checked GPU tests reach every kernel that any size takes."""
import itertools
import os

import pytest

import test_gpu_block_kernels as kernel_tests
import test_gpu_gated as gated_tests
import test_gpu_gated_more as more_tests
from block_ref import shapes_of

PRODUCTS = ("gated", "gated_saving", "dx", "dw", "mxfp4", "mxfp4_gated")
ROWS = (1, 2, 3, 5, 8, 9, 16, 17, 24, 33, 48, 63, 64, 65, 68, 77, 90, 100, 128, 129, 140, 160, 200, 256, 257, 300, 385,
        420, 513, 600, 769, 900, 1025, 1300, 1800, 2049, 2500, 3500, 4097, 6000, 8192)
SIZES = (32, 64, 96, 160, 224, 416, 512, 704, 1056, 1408, 2048, 2560, 3616, 4096, 5632, 7168, 8224, 10272, 14336, 28672)


@pytest.fixture(scope="module")
def sfr():
    import sparse_fp8_row_amd as sfr
    if not os.path.exists(sfr.LIB_PATH):
        from sparse_fp8_row_amd import build
        build.build()
    sfr.load()
    return sfr


def compared():
    """The sizes at which each product is compared with a 64-bit result."""
    forward = gated_tests.SHAPES + shapes_of(more_tests.test_forward_tiles)
    back = gated_tests.SHAPES + shapes_of(more_tests.test_backward_tiles) + shapes_of(kernel_tests.test_backward_sliced)
    streamed = shapes_of(more_tests.test_mxfp4_streamed)
    return {"gated": forward + shapes_of(kernel_tests.test_forward_few_rows), "gated_saving": forward, "dx": back, "dw": back,
            "mxfp4": shapes_of(gated_tests.test_mxfp4_linear) + shapes_of(more_tests.test_mxfp4_linear_tiles) + streamed,
            "mxfp4_gated": forward + [(m, k, (n + 31) // 32 * 32) for m, k, n in streamed]}


@pytest.mark.parametrize("product", PRODUCTS)
def test_every_kernel_is_compared(sfr, product):
    def kernel(m, k, f):
        name, slices = sfr.block_kernel(product, m, k, f)
        return name, slices > 1
    reached = {kernel(*s) for s in compared()[product]}
    missing = {}
    for s in itertools.product(ROWS, SIZES, SIZES):
        if kernel(*s) not in reached:
            missing.setdefault(kernel(*s), s)
    assert not missing, missing


def test_kernel_query(sfr):
    for product in PRODUCTS:
        name, slices = sfr.block_kernel(product, 1000, 2048, 5632)
        assert name and slices >= 1
        for bad in ((0, 64, 64), (-1, 64, 64), ((1 << 30) + 1, 64, 64), (4, 48, 64), (4, 64, 40), (4, 0, 64), (4, 64, 0),
                    (4, (1 << 20) + 32, 64), (4, 64, (1 << 20) + 32), (4, 64, 32 - (1 << 63)), (1 << 30, 64, 1 << 19)):
            assert sfr.block_kernel(product, *bad) is None, (product, bad)
    assert sfr.block_kernel("mxfp4", 4, 64, 16) and sfr.block_kernel("gated", 4, 64, 16) is None
    with pytest.raises(ValueError):
        sfr.block_kernel("linear", 4, 64, 64)
    assert sfr.load().sfr_block_kernel(6, 4, 64, 64, None) is None
    assert sfr.load().sfr_block_kernel(0, 4, 64, 64, None)  # without asking for the slices
    # a workspace for partial sums exactly where the sum has slices
    lib = sfr.load()
    for m, k, f in itertools.product((1, 20, 68, 300, 1000, 4097), (32, 416, 3616), (32, 2080, 8608)):
        _, slices = sfr.block_kernel("dx", m, k, f)
        up = lambda b: (b + 255) // 256 * 256  # noqa: E731
        assert lib.sfr_gated_backward_workspace_bytes(m, k, f, 1) == up(m * 4 * f) + (up(slices * m * k * 4) if slices > 1 else 0)
        _, slices = sfr.block_kernel("mxfp4", m, k, f)
        assert lib.sfr_mxfp4_workspace_bytes(m, f, k) == (up(slices * m * f * 4) if slices > 1 else 0)
