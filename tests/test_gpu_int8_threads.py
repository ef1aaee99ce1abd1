"""GPU: calls of the one-launch 8-bit layer from several host threads at once, each of
another size, so of another size of workgroup memory."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
SIZES = [(1, 256), (1, 16384), (4, 4096), (2, 8192), (3, 1040), (1, 32)]


@pytest.fixture(scope="module")
def sfr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_fp8_row_amd as sfr
    sfr.load()
    return sfr


def test_threads_with_different_sizes(sfr):
    data = []
    for m, k in SIZES:
        assert sfr.int8_kernel(m, 64, k)[0] == "fused_int8"
        x = torch.randn(m, k, device="cuda").bfloat16()
        w = sfr.quantize_rowwise_int8(torch.randn(64, k, device="cuda").bfloat16())
        data.append((x, w, sfr.int8_linear(sfr.quantize_rowwise_int8(x), w)))
    torch.cuda.synchronize()
    start, bad = threading.Barrier(len(data)), []

    def work(x, w, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(200):
                try:
                    ok = torch.equal(sfr.int8_linear(x, w), want)
                except sfr.SfrError as e:
                    ok = e
                if ok is not True:
                    bad.append((tuple(x.shape), ok))
    threads = [threading.Thread(target=work, args=d) for d in data]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad, bad[:4]
