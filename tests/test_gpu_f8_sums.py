"""Sums of the 8-bit floating-point products on the GPU: how they are held within a block, and the range of the scales."""

import pytest

from grouping import even, spans

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402
from test_gpu_grouped import blocks, close, f8, f8_reference, gen, offsets_of  # noqa: E402

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.set_device(0)
    g.gemm_init(0)
    yield


def finite(seed, *shape):
    """All finite codes, alike often."""
    x = torch.randint(0, 254, shape, generator=gen(seed), device="cuda")
    return (x + (x >= 127)).to(torch.uint8).view(F8)        # without 0x7F and 0xFF


# plain products and groups of few rows, in all sizes of row and weight tiles, whole and in pieces of K
@pytest.mark.parametrize("M,E,N,K", [(1, 0, 120, 128), (1, 0, 5504, 300), (16, 0, 120, 4096), (16, 0, 9000, 128), (17, 0, 120, 128), (33, 0, 120, 1000),
                                     (33, 0, 4096, 4096), (64, 0, 5504, 4096), (64, 8, 120, 128), (100, 50, 1376, 300), (300, 20, 120, 128)])
def test_few_rows_sum_in_float32(M, E, N, K):
    """2^16 at one k, -2^16 at another and a product down to 2^-17 of them at a third, in one block: the third is the
    output, bit for bit, as float32 holds 2^16 + 2^-1. And random codes within the bound of float32 sums."""
    off = offsets_of(even(M, E)) if E else None
    at = spans(even(M, max(E, 1)), M)
    run = lambda A, Sa, W, Sw: g.f8_grouped_matmul(A, Sa, W, Sw, off) if E else g.f8_matmul(A, Sa, W[0], Sw[0])  # noqa: E731
    A, W, want = torch.zeros(M, K), torch.zeros(max(E, 1), N, K), torch.zeros(N)
    A[:] = 256.0
    for n in range(N):
        gap = n % 18
        a, b, c = [(0, 1, 2), (0, 64, 127), (1, 2, 32), (7, 40, 90), (0, 16, 1)][n // 18 % 5]
        block = 128 * (n % blocks(K) if (n % blocks(K) + 1) * 128 <= K else 0)
        W[:, n, block + a], W[:, n, block + b], W[:, n, block + c] = 256.0, -256.0, 2.0 ** (8 - gap)
        want[n] = 2.0 ** (16 - gap)
    Sa, Sw = torch.ones(blocks(K), M, device="cuda"), torch.ones(max(E, 1), blocks(N), blocks(K), device="cuda")
    C = run(f8(A.cuda(), -K % 16), Sa, f8(W.cuda(), -K % 16), Sw)
    assert g.gemm_last_plan()["kernel"] == "f8_decode"
    assert (C.float().cpu() == want).all(), (C.float().cpu() != want).nonzero()[:3].tolist()
    if M == 1 and not E:                                    # quantised in the product's kernel: codes 448, scale 256 / 448
        C = g.f8_linear(A.bfloat16().cuda(), f8(W.cuda(), -K % 16)[0], Sw[0])
        assert (C.float().cpu() == want).all()
    A, W = (f8(finite(i, *s).float(), -K % 16) for i, s in enumerate(((M, K), (max(E, 1), N, K))))
    Sa, Sw = torch.rand(blocks(K), M, generator=gen(3), device="cuda") + 0.5, torch.rand(Sw.shape, generator=gen(4), device="cuda") + 0.5
    ref, sabs = f8_reference(A.float(), Sa, W.float(), Sw, at, M)
    close(run(A, Sa, W, Sw), ref, sabs, K, "random codes")
