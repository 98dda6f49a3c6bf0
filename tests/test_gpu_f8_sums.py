"""Sums of the 8-bit floating-point products on the GPU: how they are held within a block, and the range of the scales."""

import pytest

from grouping import even, spans

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402
from test_gpu_grouped import CUT, blocks, close, f8, f8_reference, gen, offsets_of  # noqa: E402

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
                                     (33, 0, 4096, 4096), (64, 0, 5504, 4096), (32, 8, 120, 128), (100, 50, 1376, 300), (80, 20, 120, 128)])
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


def factors(seed, low, high, *shape):
    """1.25 times powers of two between 2^low and 2^high."""
    e = torch.randint(low, high + 1, shape, generator=gen(seed), device="cuda")
    return torch.exp2(e.double()).mul(1.25).float()


def codes_of(values, seed, *shape):
    return torch.tensor(values, device="cuda")[torch.randint(0, len(values), shape, generator=gen(seed), device="cuda")]


LARGE, SMALL = [256.0, 288.0, 320.0, 384.0, 448.0], [m * 2.0**-8 for m in (-3, -2, -1, 0, 1, 2, 3)]


# each kernel: one row, few rows, tiles of 64, 128 and 256, the general one; plain and grouped
@pytest.mark.parametrize("M,E,N,bm", [(1, 0, 300, 0), (40, 0, 300, 0), (70, 0, 300, 64), (1024, 0, 4096, 128), (8192, 0, 2048, 256),
                                      (16, 4, 300, 0), (300, 3, 264, 64), (7000, 2, 2000, 256)])
@pytest.mark.parametrize("values,sa,sw", [(LARGE, (-126, -125), (-23, -21)),   # products of scales below 2^-126
                                          (LARGE, (-147, -140), (0, 3)),       # subnormal scales
                                          (SMALL, (105, 110), (20, 21)),       # above 2^128
                                          (SMALL, (20, 21), (105, 110)), (LARGE, (127, 127), (-126, -120)), (LARGE, (-126, -126), (100, 127))])
def test_scales_of_any_size(M, E, N, bm, values, sa, sw):
    """Codes whose sums of products, and those times (5/4)^2, float32 holds exactly, and scales whose product it does not hold:
    the outputs are in its normal range, and the exact ones rounded once. (LARGE: products are 1024 times whole numbers
    below 2^8, so 200 of them have 16 bits, and 25/16 five more; SMALL: 2^-16 times whole numbers up to 9. The matrix
    instruction keeps all of their bits.)"""
    K, off, at = 200, offsets_of(even(M, E)) if E else None, spans(even(M, max(E, 1)), M)
    A, W = codes_of(values, M, M, K), codes_of(values, N, max(E, 1), N, K)
    # (one exponent for both blocks of a row and of a weight's columns: their sum is exact)
    Sa, Sw = factors(1, *sa, 1, M).repeat(2, 1), factors(2, *sw, max(E, 1), blocks(N), 1).repeat(1, 1, 2)
    ref, _ = f8_reference(A, Sa, W, Sw, at, M)
    assert ref.abs().max() < 2.0**127 and ref[ref != 0].abs().min() >= 2.0**-126
    want = ref.float().bfloat16()
    for room, offset in ((8, 0), (3, 1)):                   # rows of 208 bytes, and the general kernel
        if room == 3 and M * N > 1 << 20:
            continue
        a, w = f8(A, room, offset), f8(W, room, offset)
        C = g.f8_grouped_matmul(a, Sa, w, Sw, off) if E else g.f8_matmul(a, Sa, w[0], Sw[0])
        plan = g.gemm_last_plan()
        assert room == 3 or plan["kernel"] == ("tile" if bm else "f8_decode") and (not bm or plan["bm"] == bm)
        bad = (C != want).nonzero()
        assert not len(bad), f"{len(bad)} differ, first {bad[0].tolist()}: {float(C[tuple(bad[0])])} for {float(ref[tuple(bad[0])])}"


@pytest.mark.parametrize("M", [1, 20, 100, 1024])
def test_activations_of_the_smallest_scale(M):
    """Activations about 2^-117, whose scales are about 2^-125, and weights about 2^-12, with 2^-20: outputs are about 2^-121."""
    K, N = 300, 520
    A = (2.0**-117 * (1 + torch.rand(M, K, generator=gen(1), device="cuda"))).bfloat16()
    Wq, Sw = g.f8_quantize_weight((2.0**-12 * (1 + torch.rand(N, K, generator=gen(2), device="cuda"))).bfloat16())
    Aq, Sa = g.f8_quantize(A)
    assert Sa.max() * Sw.max() < 2.0**-140
    ref, sabs = f8_reference(Aq.float(), Sa, Wq.float()[None], Sw[None], [(0, 0, M)], M)
    close(g.f8_linear(A, Wq, Sw), ref, sabs, K, "linear", CUT)


def test_zeros_beside_scales_of_any_size():
    """A block of zero codes adds nothing, whatever the scales, and one of a zero scale neither."""
    for M in (1, 40, 300):
        A, W = torch.ones(M, 256, device="cuda"), torch.ones(136, 256, device="cuda")
        A[:, 128:] = 0
        Sa, Sw = torch.ones(2, M, device="cuda"), torch.ones(2, 2, device="cuda")
        Sa[1], Sw[:, 1] = 2.0**100, 2.0**100
        assert (g.f8_matmul(f8(A), Sa, f8(W), Sw) == 128).all()
        A[:, 128:], Sa[1], Sw[:, 1] = 448.0, 0.0, 2.0**127
        assert (g.f8_matmul(f8(A), Sa, f8(W), Sw) == 128).all()


# tiles whose K is in pieces: of 64 and 128 rows, of 256 past whole rounds, of a group's few rows
@pytest.mark.parametrize("M,E,N,K,bm", [(200, 0, 130, 8300, 64), (1024, 0, 4096, 4130, 128), (4096, 0, 4352, 4130, 256), (300, 3, 264, 4130, 64),
                                        (3900, 1, 4352, 4130, 256), (40, 0, 300, 4130, 0), (16, 4, 300, 4130, 0)])
@pytest.mark.parametrize("values,sa,sw", [([256.0, 384.0], (-126, -125), (-23, -21)), ([2.0**-9, 2.0**-8], (108, 109), (21, 21))])
def test_scales_of_any_size_in_pieces(M, E, N, K, bm, values, sa, sw):
    """As above, every third row with scales about 1, and every seventh of zeros with a zero scale. (Products are 2^14 or 2^-18
    times whole numbers up to 9, their sums have 17 bits, and 25/16 five more.)"""
    off, at = offsets_of(even(M, E)) if E else None, spans(even(M, max(E, 1)), M)
    A, W = codes_of(values, M, M, K), codes_of(values, N, max(E, 1), N, K)
    Sa, Sw = factors(1, *sa, 1, M).repeat(blocks(K), 1), factors(2, *sw, max(E, 1), blocks(N), 1).repeat(1, 1, blocks(K))
    Sa[:, ::3] = 1.25
    A[::7], Sa[:, ::7] = 0.0, 0.0
    ref, _ = f8_reference(A, Sa, W, Sw, at, M)
    assert ref.abs().max() < 2.0**127 and ref[ref != 0].abs().min() >= 2.0**-126 and not ref[::7].any()
    a, w = f8(A, -K % 16), f8(W, -K % 16)
    run = lambda: g.f8_grouped_matmul(a, Sa, w, Sw, off) if E else g.f8_matmul(a, Sa, w[0], Sw[0])  # noqa: E731
    C = run()
    plan = g.gemm_last_plan()
    assert (plan["kernel"], plan["bm"]) == ("tile", bm) if bm else plan["kernel"] == "f8_decode"
    assert plan["splits"] > 1 or plan["grid"] > plan["tiles"]
    bad = (C != ref.float().bfloat16()).nonzero()
    assert not len(bad), f"{len(bad)} differ, first {bad[0].tolist()}: {float(C[tuple(bad[0])])} for {float(ref[tuple(bad[0])])}"
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other = run()
    again = run()
    torch.cuda.synchronize()
    assert torch.equal(other, C) and torch.equal(again, C)


@pytest.mark.parametrize("M,E,kernel", [(32, 8, "f8_decode"), (33, 8, "tile"), (64, 64, "f8_decode"), (512, 32, "tile")])
@pytest.mark.parametrize("hit", [1, 3])
def test_routers_of_few_groups(M, E, kernel, hit):
    """All rows in one group or three of many."""
    N, K, cuts = 264, 300, sorted([M // 5, M // 3][: hit - 1])
    offsets = [0] * (E - hit) + [0, *cuts, M]
    A, W = codes_of([-2.0, -1.0, 0.0, 1.0, 2.0], M, M, K), codes_of([-2.0, -1.0, 0.0, 1.0, 2.0], N, E, N, K)
    Sa, Sw = torch.ones(blocks(K), M, device="cuda"), torch.ones(E, blocks(N), blocks(K), device="cuda")
    ref, _ = f8_reference(A, Sa, W, Sw, spans(offsets, M), M)
    C = g.f8_grouped_matmul(f8(A, -K % 16), Sa, f8(W, -K % 16), Sw, offsets_of(offsets))
    assert g.gemm_last_plan()["kernel"] == kernel and torch.equal(C, ref.float().bfloat16())


def test_scales_of_any_size_in_a_graph():
    """A captured product replayed with scales that ask for a second run of every tile, of some and of none, and with rows of
    zeros and NaN, between eager calls: the bits of those."""
    cases = []
    for M, N, K in ((40, 300, 1000), (200, 130, 8300), (1024, 4096, 520), (4096, 4352, 4130)):
        A, W = (f8(codes_of([-2.0, -1.0, 1.0, 1.5], i, *s), -K % 16) for i, s in enumerate(((M, K), (N, K))))
        cases.append((A, torch.ones(blocks(K), M, device="cuda"), W, torch.ones(blocks(N), blocks(K), device="cuda")))

    def fill(turn):
        for A, Sa, W, Sw in cases:
            Sa.copy_(torch.rand(Sa.shape, generator=gen(turn), device="cuda") + 0.5)
            Sw.copy_(torch.rand(Sw.shape, generator=gen(10 + turn), device="cuda") + 0.5)
            if turn % 4 == 1:                               # sums of magnitudes from 2^-118 on, whose bound is 2^-128 at least,
                Sa.mul_(2.0**-126)                          # beside outputs' roundings of 2^-134 at most below 2^-126
                Sw.mul_(0.25)
            if turn % 4 == 2:
                Sa[:, 3::50] *= 2.0**-126
                Sw[-1] *= 0.25
                Sa[:, 5::70] = 0.0
            if turn % 4 == 3:
                Sa[-1, 7] = float("nan")
                Sa[:, ::9] = 0.0

    fill(0)
    run = lambda: [g.f8_matmul(*c) for c in cases]  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for turn in range(8):
        fill(turn)
        fresh = run()
        graph.replay()
        torch.cuda.synchronize()
        for h, f, (A, Sa, W, Sw) in zip(held, fresh, cases):
            assert torch.equal(h.view(torch.int16), f.view(torch.int16)), turn
            ref, sabs = f8_reference(A.float(), Sa, W.float()[None], Sw[None], [(0, 0, A.shape[0])], A.shape[0])
            fine = ~torch.isnan(ref).any(1)
            assert torch.isnan(f[~fine]).all() and int((~fine).sum()) == (1 if turn % 4 == 3 and A.shape[0] > 7 else 0)
            close(f[fine], ref[fine], sabs[fine], A.shape[1], f"turn {turn}", CUT)
