"""Products grouped by expert on the GPU, bf16 and e4m3, against float64 products of each group's rows.

Two kinds of inputs. Small whole numbers (with scales that are powers of two), whose products and sums float32
holds exactly: the output has to be the exact sum rounded once to bf16, bit for bit, from every kernel, split and
order. Normal ones: the output is off by its own rounding, 2^-8 |ref|, and by float32 sums of K products, each
addition within 2^-23 (a rounding in either direction) of the partial sum, which sum |a b| bounds; the scales add
three roundings a block: |c - ref| <= 2^-8 |ref| + (K + 8) 2^-23 sum |a b|, and the errors' norm over that of ref is
below 2^-8, the largest that a rounding alone makes of it (the sums add 2^-24 sqrt(K) in the mean).

The 8-bit matrix instruction does not sum in float32 throughout: it takes products by eights, aligned to the one of
the largest exponent sum E, and cuts what lies below 2^(E - 13) (test_what_the_matrix_instruction_keeps). The largest of eight
products is 2^E at least, so each of the seven others loses less than 2^-13 of it, and the eight together less than
7 2^-13 of their sum |a b|: close() adds 7 2^-13 sum |a b| for codes. The bound on the norm stays.
"""

import numpy as np
import pytest

from grouping import even, ragged, spans

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.set_device(0)
    g.gemm_init(0)
    yield


F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(seed, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").float()


def strided(x, pad, offset, poison):
    """x with `pad` columns between its rows and `offset` elements before, all of them `poison` bits."""
    *lead, rows, cols = x.shape
    ld, n = cols + pad, int(np.prod(lead, dtype=np.int64)) * rows * (cols + pad)
    kind = torch.uint8 if x.element_size() == 1 else torch.int16
    mem = torch.full((offset + n,), poison, dtype=kind, device="cuda").view(x.dtype)
    view = mem[offset:].view(*lead, rows, ld)[..., :cols]
    view.copy_(x)
    return view


def bf(x, pad=0, offset=0):
    return strided(x.bfloat16(), pad, offset, 0x7FC0)


def f8(x, pad=0, offset=0):
    return strided(x.to(F8), pad, offset, 0x7F)


def offsets_of(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def same(got, want, what):
    """bf16 `got` is float64 `want` rounded once (want's values fit float32)."""
    want = want.float().bfloat16()
    bad = got.contiguous().view(torch.int16) != want.view(torch.int16)
    bad &= ~((got == 0) & (want == 0))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


CUT = 7 * 2.0**-13  # of sum |a b|: what the 8-bit matrix instruction cuts


def close(got, ref, sabs, K, what, cut=0.0):
    err = (got.double() - ref).abs()
    bound = 2.0**-8 * ref.abs() + ((K + 8) * 2.0**-23 + cut) * sabs
    assert (err <= bound).all(), f"{what}: {float((err / bound).nan_to_num().max()):.3f} of the bound"
    norm = float(ref.norm())
    assert float(err.norm()) <= 2.0**-8 * norm, f"{what}: {float(err.norm()) / norm:.5f}"


def product(A, B, at, M, N):
    """float64 C of a grouped product: A (M x K) times B[e] (K x N) for the rows of each group, else zeros."""
    C = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for e, a, b in at:
        if b > a:
            torch.mm(A[a:b].double(), B[e].double(), out=C[a:b])
    return C


# M, N, K, offsets
CASES = [
    (1, 8, 8, [0, 1]), (1, 8, 8, [0, 0, 1]), (3, 16, 40, [0, 1, 1, 2, 3]), (5, 24, 64, [0, 0, 0]), (7, 520, 328, [2, 4, 5]),
    (16, 1376, 512, ragged(16, 8, 1)), (64, 264, 1000, even(64, 64)), (65, 136, 72, [0, 64, 65]),
    (130, 256, 128, [0, 65, 66, 130]), (300, 520, 328, ragged(300, 8, 2, 5, 280)), (600, 520, 328, ragged(600, 5, 3)),
    (257, 64, 2056, [0, 129, 257]), (513, 256, 96, [0, 256, 513]), (1018, 1376, 512, ragged(1018, 8, 4, 0, 981)),
    (2000, 1000, 264, ragged(2000, 70, 5)), (4096, 512, 264, ragged(4096, 300, 6, 9, 4000, empty=0.6)),
    (2048, 2056, 520, [0, 700, 2048]), (3000, 768, 1032, ragged(3000, 4, 7)), (1500, 4096, 264, [0, 1500]),
    (6000, 2048, 136, ragged(6000, 8, 8, 0, 5999)), (5000, 2304, 520, even(5000, 3)),
    # offsets that are no such thing
    (100, 136, 72, [-5, 40, 20, 300]), (100, 136, 72, [50, 10, 60]), (100, 136, 72, [100, 100, 0]),
    (100, 136, 72, [-(2**31), 2**31 - 1]), (700, 264, 72, [0, 700, 0, 700, 0, 700]),
]
# widths and leading dimensions that the matrix kernels do not take: pad, offset
LOOSE = [(3, 0), (0, 1), (5, 1)]


@pytest.mark.parametrize("M,N,K,offsets", CASES)
def test_forward(M, N, K, offsets):
    E, at = len(offsets) - 1, spans(offsets, M)
    A, B = ints(M, M, K), ints(N, E, K, N)
    off = offsets_of(offsets)
    ref = product(A, B, at, M, N)
    same(g.grouped_matmul(bf(A), bf(B), off), ref, "whole numbers")
    out = bf(torch.zeros(M, N), 8, 8)
    assert g.grouped_matmul(bf(A, 8, 8), bf(B, 16, 8), off, out=out) is out
    same(out, ref, "padded rows")
    assert (out.as_strided((M, 8), (N + 8, 1), out.storage_offset() - 8).contiguous().view(torch.int16) == 0x7FC0).all()
    a, b = torch.randn(M, K, generator=gen(1), device="cuda").bfloat16(), torch.randn(E, K, N, generator=gen(2), device="cuda").bfloat16()
    close(g.grouped_matmul(a, b, off), product(a, b, at, M, N), product(a.abs(), b.abs(), at, M, N), K, "normal")


@pytest.mark.parametrize("M,N,K,offsets", CASES)
def test_backward(M, N, K, offsets):
    E, at = len(offsets) - 1, spans(offsets, M)
    A, B, D = ints(M, M, K), ints(N, E, K, N), ints(K, M, N)
    covered = torch.zeros(M, dtype=torch.bool, device="cuda")
    for _, a, b in at:
        covered[a:b] = True
    refA = product(D, B.transpose(1, 2), at, M, K)
    refB = torch.zeros(E, K, N, dtype=torch.float64, device="cuda")
    for e, a, b in at:
        if b > a:
            refB[e] = torch.mm(A[a:b].double().t(), D[a:b].double())
    # what no group's row holds is not read
    A[~covered] = float("nan")
    D[~covered] = float("inf")
    off = offsets_of(offsets)
    for pad, offset in ((0, 0), (8, 8)):
        a, b, d = bf(A, pad, offset), bf(B, pad, offset), bf(D, pad, offset)
        dA, dB = g.grouped_matmul_backward(d, a, b, off)
        same(dA, refA, "dA")
        same(dB, refB, "dB")
        oneA, none = g.grouped_matmul_backward(d, a, b, off, need_dB=False)
        assert none is None and torch.equal(oneA, dA)
        none, oneB = g.grouped_matmul_backward(d, a, b, off, need_dA=False)
        assert none is None and torch.equal(oneB, dB)


# few tiles of 256 x 256 past whole rounds of the CUs: those are in pieces of K, the last of them short
@pytest.mark.parametrize("M,N,K,offsets", [(3840, 4400, 1100, even(3840, 3)), (4200, 4100, 4700, [0, 4096]), (4300, 4104, 3600, [7, 4100]),
                                           (4096, 4352, 2184, even(4096, 4)), (4100, 4352, 16456, [0, 4100]), (4096, 4096, 4800, [0, 4100]),
                                           (3840, 4400, 1104, even(3840, 3)), (4200, 4104, 4712, [0, 4096])])
def test_last_round_in_pieces(M, N, K, offsets):
    E, at = len(offsets) - 1, spans(offsets, M)
    A, B = ints(M, M, K), ints(N, E, K, N)
    a, b, off = bf(A, -K % 8), bf(B, -N % 8), offsets_of(offsets)
    ref = product(A, B, at, M, N)
    first = g.grouped_matmul(a, b, off)
    assert g.gemm_last_plan()["bm"] == (256 if K % 8 == N % 8 == 0 else 0)
    same(first, ref, "C")
    # the gradient of a product with K outputs is as long
    bt = bf(B.transpose(1, 2).contiguous(), -K % 8)
    dA, _ = g.grouped_matmul_backward(a, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), bt, off, need_dB=False)
    same(dA, ref, "dA")
    # the order of the pieces changes no bit
    x, w = torch.randn(M, K, generator=gen(1), device="cuda").bfloat16(), torch.randn(E, K, N, generator=gen(2), device="cuda").bfloat16()
    once = g.grouped_matmul(x, w, off)
    for _ in range(3):
        assert torch.equal(g.grouped_matmul(x, w, off), once)
    close(once, product(x, w, at, M, N), product(x.abs(), w.abs(), at, M, N), K, "normal")


# groups about the numbers that one pass over the offsets takes, with rows of no group before and behind
@pytest.mark.parametrize("E", [61, 62, 63, 64, 125, 126, 127, 128, 253, 254, 255, 256, 257, 511, 1500])
def test_many_groups(E):
    for M, first, last, empty in ((E + 40, 3, E + 17, 0.2), (777, 0, 777, 0.0), (70, 0, 69, 0.9)):
        N, K = 72, 40
        offsets = ragged(M, E, E + M, first, last, empty)
        A, B, D, at = ints(M, M, K), ints(N, E, K, N), ints(K, M, N), spans(offsets, M)
        a, b, d, off = bf(A), bf(B), bf(D), offsets_of(offsets)
        same(g.grouped_matmul(a, b, off), product(A, B, at, M, N), "C")
        dA, dB = g.grouped_matmul_backward(d, a, b, off)
        same(dA, product(D, B.transpose(1, 2), at, M, K), "dA")
        refB = torch.zeros(E, K, N, dtype=torch.float64, device="cuda")
        for e, r0, r1 in at:
            if r1 > r0:
                refB[e] = torch.mm(A[r0:r1].double().t(), D[r0:r1].double())
        same(dB, refB, "dB")
        W, Sa, Sw = ints(N, E, N, K), powers(1, blocks(K), M), powers(2, E, blocks(N), blocks(K))
        ref, _ = f8_reference(A, Sa, W, Sw, at, M)
        same(g.f8_grouped_matmul(f8(A, -K % 16), Sa, f8(W, -K % 16), Sw, off), ref, "codes")


@pytest.mark.parametrize("pad,offset", LOOSE)
@pytest.mark.parametrize("M,N,K,offsets", [(5, 3, 7, [0, 2, 5]), (130, 100, 90, ragged(130, 5, 1, 3, 120)),
                                           (300, 131, 70, ragged(300, 70, 2))])
def test_any_alignment(M, N, K, offsets, pad, offset):
    E, at = len(offsets) - 1, spans(offsets, M)
    A, B, D = ints(M, M, K), ints(N, E, K, N), ints(K, M, N)
    off = offsets_of(offsets)
    a, b, d = bf(A, pad, offset), bf(B, pad, offset), bf(D, pad, offset)
    out = bf(torch.zeros(M, N), pad, offset)
    same(g.grouped_matmul(a, b, off, out=out), product(A, B, at, M, N), "C")
    assert g.gemm_last_plan()["op"] == "grouped"
    dA, dB = g.grouped_matmul_backward(d, a, b, off)
    same(dA, product(D, B.transpose(1, 2), at, M, K), "dA")
    for e, r0, r1 in at:
        same(dB[e], torch.mm(A[r0:r1].double().t(), D[r0:r1].double()), f"dB {e}")


def blocks(n):
    return -(-n // 128)


def spread(S, rows, cols):
    return S.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def powers(seed, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=gen(seed), device="cuda").float())


def f8_reference(A, Sa, W, Sw, at, M):
    """float64 C, and the sum of magnitudes, of the grouped 8-bit product of values (not codes)."""
    N, K = W.shape[1:]
    C, S = (torch.zeros(M, N, dtype=torch.float64, device="cuda") for _ in range(2))
    a = A.double() * Sa.double().t().repeat_interleave(128, 1)[:, :K]
    for e, r0, r1 in at:
        if r1 > r0:
            w = W[e].double() * spread(Sw[e].double(), N, K)
            C[r0:r1] = a[r0:r1] @ w.t()
            S[r0:r1] = a[r0:r1].abs() @ w.abs().t()
    return C, S


# widths of any residue
F8_CASES = [(1, 1, 1, [0, 1]), (2, 17, 130, [0, 1, 2]), (16, 131, 257, ragged(16, 5, 1)), (33, 500, 16, [0, 33]),
            (64, 1376, 4096, ragged(64, 64, 2)), (100, 264, 129, [3, 60, 90]), (257, 129, 1003, [0, 128, 257]),
            (600, 520, 328, ragged(600, 70, 3, 2, 590)), (1018, 1375, 509, ragged(1018, 8, 4)),
            (2048, 2051, 390, [0, 900, 2048]), (6000, 2048, 136, ragged(6000, 8, 5, 0, 5999)),
            (5000, 2304, 520, even(5000, 3)), (3000, 1500, 1100, ragged(3000, 4, 6)),
            (100, 136, 72, [-5, 40, 20, 300]), (300, 136, 200, [0, 300, 0, 300])]


@pytest.mark.parametrize("M,N,K,offsets", F8_CASES)
def test_f8_grouped(M, N, K, offsets):
    E, at = len(offsets) - 1, spans(offsets, M)
    A, W = ints(M, M, K), ints(N, E, N, K)
    Sa, Sw = powers(1, blocks(K), M), powers(2, E, blocks(N), blocks(K))
    off = offsets_of(offsets)
    ref, _ = f8_reference(A, Sa, W, Sw, at, M)
    room = -K % 16
    codes = f8(A, room), f8(W, room)                       # NaN codes behind each row
    same(g.f8_grouped_matmul(codes[0], Sa, codes[1], Sw, off), ref, "whole numbers")
    sa, sw = strided4(Sa, 3), strided4(Sw, 2)
    out = bf(torch.zeros(M, N), 3, 1)
    g.f8_grouped_matmul(f8(A, room + 16, 16), sa, f8(W, room + 32, 32), sw, off, out=out)
    same(out, ref, "padded rows")
    assert (out.as_strided((M, 3), (N + 3, 1), out.storage_offset() + N)[:-1].contiguous().view(torch.int16) == 0x7FC0).all()
    same(g.f8_grouped_matmul(f8(A, 3, 1), Sa, f8(W, 5, 3), Sw, off), ref, "any alignment")
    # from bf16, with codes and scales of every size
    a = torch.randn(M, K, generator=gen(3), device="cuda").mul_(torch.exp2(torch.randn(M, 1, generator=gen(4), device="cuda"))).bfloat16()
    Wq, Sw = g.f8_quantize_weight(torch.randn(E, N, K, generator=gen(5), device="cuda").mul_(0.05).bfloat16())
    Aq, Sa = g.f8_quantize(a)
    ref, sabs = f8_reference(Aq.float(), Sa, Wq.float(), Sw, at, M)
    C = g.f8_grouped_linear(a, Wq, Sw, off)
    close(C, ref, sabs, K, "normal", CUT)
    assert torch.equal(C, g.f8_grouped_matmul(Aq, Sa, Wq, Sw, off))


def strided4(x, pad):
    mem = torch.full((*x.shape[:-1], x.shape[-1] + pad), float("nan"), device="cuda")
    mem[..., : x.shape[-1]] = x
    return mem[..., : x.shape[-1]]


def test_a_shared_weight():
    """Groups whose weights are one: the outputs are those of copies, and its gradient is the sum of theirs."""
    M, N, K, offsets = 300, 264, 136, [0, 100, 170, 300]
    off = offsets_of(offsets)
    A, B, D = ints(1, M, K), ints(2, K, N), ints(3, M, N)
    a, b, d = A.bfloat16(), B.bfloat16(), D.bfloat16()
    shared = b.expand(3, K, N)
    same(g.grouped_matmul(a, shared, off), A.double() @ B.double(), "C")
    dA, dB = g.grouped_matmul_backward(d, a, shared, off)
    same(dA, D.double() @ B.double().t(), "dA")
    assert dB.abs().max() <= 256                            # whole numbers that bf16 holds
    assert torch.equal(dB.double().sum(0), A.double().t() @ D.double())
    Wq, Sw = g.f8_quantize_weight(b.t().contiguous())
    Aq, Sa = g.f8_quantize(a)
    one = g.f8_matmul(Aq, Sa, Wq, Sw)
    assert torch.equal(g.f8_grouped_matmul(Aq, Sa, Wq.expand(3, N, K), Sw.expand(3, *Sw.shape), off), one)


def test_sub_weights_of_a_larger_tensor():
    """Weights that are slices in every dimension, and a stack in reverse order of memory's neighbours."""
    E, M, N, K = 4, 200, 72, 64
    off = offsets_of(ragged(M, E, 3, empty=0))
    big = ints(1, 2 * E, K + 8, N + 16).bfloat16()
    B = big[::2, 8:, 8 : N + 8]
    A = ints(2, M, K).bfloat16()
    same(g.grouped_matmul(A, B, off), product(A, B, spans(off.tolist(), M), M, N), "C")
    D = ints(3, M, N).bfloat16()
    dA, dB = g.grouped_matmul_backward(D, A, B, off)
    same(dA, product(D, B.transpose(1, 2), spans(off.tolist(), M), M, K), "dA")


@pytest.mark.parametrize("M,N,K", [(5, 16, 0), (0, 16, 8), (5, 0, 8)])
def test_empty_sizes(M, N, K):
    E = 3
    off = offsets_of([0, M // 2, M, M])
    A, B, D = (torch.ones(*s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (E, K, N), (M, N)))
    C = g.grouped_matmul(A, B, off)
    assert C.shape == (M, N) and not C.any()
    dA, dB = g.grouped_matmul_backward(D, A, B, off)
    assert dA.shape == (M, K) and dB.shape == (E, K, N) and not dA.any() and not dB.any()
    Wq, Sw = g.f8_quantize_weight(torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda"))
    assert not g.f8_grouped_linear(A, Wq, Sw, off).any()
    none = torch.zeros(0, 8, 16, dtype=torch.bfloat16, device="cuda")
    assert not g.grouped_matmul(torch.ones(4, 8, dtype=torch.bfloat16, device="cuda"), none, offsets_of([2])).any()


def test_infinities_stay_in_their_rows():
    M, N, K = 130, 136, 200
    off = offsets_of([0, 60, 130])
    A, B = ints(1, M, K), ints(2, 2, K, N, top=1) + 0.5     # no zero weight
    A[7, 3], A[100, 5] = float("inf"), float("nan")
    C = g.grouped_matmul(A.bfloat16(), B.bfloat16(), off)
    finite = torch.isfinite(C).all(1)
    assert not finite[7] and not finite[100] and int((~finite).sum()) == 2
    Wq, Sw = g.f8_quantize_weight(B.transpose(1, 2).contiguous().bfloat16())
    C = g.f8_grouped_linear(A.bfloat16(), Wq, Sw, off)
    bad = torch.isnan(C).all(1)
    assert bad[7] and bad[100] and torch.isfinite(C[~bad]).all() and int(bad.sum()) == 2


def test_gradients_against_differences():
    """The directional derivative of sum(D * C) in float64 from central differences of grouped products."""
    M, N, K, offsets = 40, 24, 16, [1, 12, 12, 39]
    at = spans(offsets, M)
    off = offsets_of(offsets)
    A, B, D = (torch.randn(*s, generator=gen(i), device="cuda").bfloat16() for i, s in enumerate(((M, K), (3, K, N), (M, N))))
    dA, dB = g.grouped_matmul_backward(D, A, B, off)
    for seed in range(4):
        vA, vB = torch.randn(M, K, generator=gen(10 + seed), device="cuda").double(), torch.randn(3, K, N, generator=gen(20 + seed), device="cuda").double()
        h = 1e-4

        def f(t):
            C = torch.zeros(M, N, dtype=torch.float64, device="cuda")
            for e, a, b in at:
                C[a:b] = (A.double() + t * vA)[a:b] @ (B.double() + t * vB)[e]
            return float((C * D.double()).sum())

        slope = (f(h) - f(-h)) / (2 * h)
        got = float((dA.double() * vA).sum() + (dB.double() * vB).sum())
        # each gradient element is rounded by at most 2^-8 of itself; the difference's own error is of order h^2 = 0 (f is quadratic)
        bound = 2.0**-8 * float((dA.double().abs() * vA.abs()).sum() + (dB.double().abs() * vB.abs()).sum()) + 1e-6
        assert abs(got - slope) <= bound


def bits(t):
    return t.contiguous().view(torch.int16)


def test_streams_graphs_and_repeats():
    """Two streams at once, and a graph replayed with other offsets and data between eager work, give the bits of
    eager calls."""
    cases = []
    for M, N, K, E in ((16, 1376, 512, 8), (300, 520, 1032, 5), (2048, 2048, 264, 3)):
        A, B, D = (torch.randn(*s, generator=gen(M + i), device="cuda").bfloat16() for i, s in enumerate(((M, K), (E, K, N), (M, N))))
        W = g.f8_quantize_weight(B.transpose(1, 2).contiguous())
        cases.append((A, B, D, W, offsets_of(ragged(M, E, M))))

    def run(c, out=None):
        A, B, D, (Wq, Sw), off = c
        return [g.grouped_matmul(A, B, off), *g.grouped_matmul_backward(D, A, B, off), g.f8_grouped_linear(A, Wq, Sw, off)]

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        outs = []
        for c in cases:
            for s in (s1, s2):
                with torch.cuda.stream(s):
                    outs.append(run(c))
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            for x, y in zip(o, want[i // 2]):
                assert torch.equal(bits(x), bits(y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [run(c) for c in cases]
    for turn in range(4):
        for c, w in zip(cases, want):
            c[0].copy_(torch.randn(c[0].shape, generator=gen(turn), device="cuda"))
            c[4].copy_(offsets_of(ragged(c[0].shape[0], c[4].numel() - 1, 100 + turn)))
        fresh = [run(c) for c in cases]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for h, f in zip(held, fresh):
            for x, y in zip(h, f):
                assert torch.equal(bits(x), bits(y))


def test_last_round_on_two_streams_and_in_a_graph():
    """Products whose last tiles are in pieces share a stream's workspace: two streams at once, and replays whose
    offsets make other numbers of pieces, or none."""
    M, N, K, E = 4096, 4352, 2184, 4
    A, B = torch.randn(M, K, generator=gen(1), device="cuda").bfloat16(), torch.randn(E, K, N, generator=gen(2), device="cuda").bfloat16()
    D = torch.randn(M, N, generator=gen(3), device="cuda").bfloat16()
    x, Wq, Sw = D[:, :4096], *g.f8_quantize_weight(torch.randn(N, 4096, generator=gen(4), device="cuda").bfloat16())
    off = offsets_of(even(M, E))

    def run():
        return [g.grouped_matmul(A, B, off), g.grouped_matmul_backward(D, A, B, off, need_dB=False)[0], g.f8_linear(x, Wq, Sw)]

    kinds = [even(M, E), [0, M, M, M, M], [0, 1, 2, 3, M], [0, 300, 1500, 2900, 4000], [5, 5, 5, 5, 5], even(M, E)]
    want = []
    for k in kinds:
        off.copy_(offsets_of(k))
        want.append(run())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(2):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append(run())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(bits(y), bits(z)) for y, z in zip(o, want[-1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for k, w in zip(kinds * 2, want * 2):
        off.copy_(offsets_of(k))
        fresh = run()
        graph.replay()
        torch.cuda.synchronize()
        for h, f, y in zip(held, fresh, w):
            assert torch.equal(bits(h), bits(y)) and torch.equal(bits(f), bits(y)), k


def test_memory_belongs_to_the_stream_given():
    import ctypes

    A, B, off = ints(1, 2048, 512).bfloat16(), ints(2, 4, 512, 256).bfloat16(), offsets_of(even(2048, 4))
    Wq, Sw = g.f8_quantize_weight(B.transpose(1, 2).contiguous())
    want, want8 = g.grouped_matmul(A, B, off), g.f8_grouped_linear(A, Wq, Sw, off)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    def owns(t):
        return any(s["stream"] == side.cuda_stream and s["address"] <= t.data_ptr() < s["address"] + s["total_size"]
                   for s in torch.cuda.memory_snapshot())

    here = torch.cuda.current_stream()
    C = g.grouped_matmul(A, B, off, stream=side.cuda_stream)
    dA, dB = g.grouped_matmul_backward(C, A, B, off, stream=ctypes.c_void_p(side.cuda_stream))
    Aq, Sa = g.f8_quantize(A, stream=side.cuda_stream)
    q, s = g.f8_quantize_weight(B, stream=side.cuda_stream)
    C8, L8 = g.f8_grouped_matmul(Aq, Sa, Wq, Sw, off, stream=side.cuda_stream), g.f8_grouped_linear(A, Wq, Sw, off, stream=side.cuda_stream)
    one = g.f8_matmul(Aq, Sa, Wq[0], Sw[0], stream=side.cuda_stream)
    for t in (C, dA, dB, Aq, Sa, q, s, C8, L8, one):
        assert owns(t)
    assert torch.cuda.current_stream() == here and not owns(g.grouped_matmul(A, B, off))
    torch.cuda.synchronize()
    assert torch.equal(C, want) and torch.equal(C8, want8) and torch.equal(L8, want8)


def test_refusals_on_the_device():
    A, B, off = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 8, 16, dtype=torch.bfloat16, device="cuda"), offsets_of([0, 2, 4])
    Wq, Sw = g.f8_quantize_weight(B.transpose(1, 2).contiguous())
    with pytest.raises(TypeError):
        g.grouped_matmul(A, B, off.long())
    for bad in (off[:2], off.cpu(), offsets_of([0, 0, 2, 0, 4])[::2], off.view(1, 3)):
        with pytest.raises(ValueError):
            g.grouped_matmul(A, B, bad)
        with pytest.raises(ValueError):
            g.f8_grouped_linear(A, Wq, Sw, bad)
        with pytest.raises(ValueError):
            g.grouped_matmul_backward(torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda"), A, B, bad)
    with pytest.raises(ValueError):
        g.grouped_matmul(A[:, :4], B, off)
    with pytest.raises(ValueError):
        g.grouped_matmul(A, B.transpose(1, 2), off)
    with pytest.raises(ValueError):
        g.grouped_matmul(A, B, off, out=A)
    with pytest.raises(ValueError):
        g.f8_grouped_linear(A, Wq, Sw[:1], off)
    with pytest.raises(ValueError):
        g.f8_grouped_linear(A, Wq[0], Sw[0], off)
    with pytest.raises(ValueError):
        g.f8_linear(A, Wq, Sw)
    with pytest.raises(g.GemmError):
        g.f8_grouped_linear(A, Wq, Sw, off, work=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_a_layer_of_experts():
    """Forward, backward and 8-bit serving together: gate and up products of a small mixture of experts sorted by
    expert, through autograd, against float64 of the same operands."""
    T, E, K, N = 150, 6, 128, 72

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, A, B, off):
            ctx.save_for_backward(A, B, off)
            return g.grouped_matmul(A, B, off)

        @staticmethod
        def backward(ctx, d):
            A, B, off = ctx.saved_tensors
            return (*g.grouped_matmul_backward(d.contiguous(), A, B, off, *ctx.needs_input_grad[:2]), None)

    x = torch.randn(T, K, generator=gen(1), device="cuda").bfloat16()
    expert = torch.randint(0, E - 1, (T, 2), generator=gen(2), device="cuda").flatten()   # the last has no tokens
    order = expert.argsort(stable=True)
    token = order // 2
    off = torch.searchsorted(expert[order].contiguous(), torch.arange(E + 1, device="cuda")).int()
    B = (torch.randn(E, K, N, generator=gen(3), device="cuda") * K**-0.5).bfloat16().requires_grad_()
    h = Experts.apply(x[token], B, off)
    weight = torch.rand(2 * T, 1, generator=gen(4), device="cuda")
    loss = (h.float() * weight).square().sum()
    loss.backward()
    Bd = B.detach().double().requires_grad_()
    rows = torch.cat([x[token][a:b].double() @ Bd[e] for e, a, b in spans(off.tolist(), 2 * T)])
    (rows * weight.double()).square().sum().backward()
    assert float((h.double() - rows).norm() / rows.norm()) < 2.0**-8
    # h, its gradient and dB are each rounded once
    assert float((B.grad.double() - Bd.grad).norm() / Bd.grad.norm()) < 3 * 2.0**-8
    assert not B.grad[E - 1].any()
    Wq, Sw = g.f8_quantize_weight(B.detach().transpose(1, 2).contiguous())
    y = g.f8_grouped_linear(x[token], Wq, Sw, off)
    # codes are off by 2^-4 of their value at most, on both sides, in independent directions: far below their sum
    assert float((y.double() - rows).norm() / rows.norm()) < 2 * 2.0**-4


@pytest.mark.parametrize("what", ["rows", "weights"])
def test_offsets_past_32_bits(what):
    """Rows, weights and outputs whose byte offsets pass 2^32: the last ones are the first ones."""
    if what == "rows":
        M, N, K = 1_100_000, 2056, 264
        A, B = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), ints(1, 2, K, N).bfloat16()
        A[:64] = ints(2, 64, K)
        A[-64:] = A[:64]
        B[1] = B[0]
        off = offsets_of([0, 64, M])
        C = g.grouped_matmul(A, B, off)
        assert C.numel() * 2 > 1 << 32
        same(C[:64], A[:64].double() @ B[0].double(), "first rows")
        assert torch.equal(C[-64:], C[:64]) and not C[64:-64].any()
        D = torch.zeros_like(C)
        D[:64] = C[:64].clamp(-2, 2)
        D[-64:] = D[:64]
        dA, dB = g.grouped_matmul_backward(D, A, B, off)
        same(dA[:64], D[:64].double() @ B[0].double().t(), "first rows of dA")
        assert torch.equal(dA[-64:], dA[:64]) and not dA[64:-64].any()
        same(dB[0], A[:64].double().t() @ D[:64].double(), "dB")
        assert torch.equal(dB[1], dB[0])
    else:
        E, N, K = 60, 4096, 11008
        B = torch.zeros(E, K, N, dtype=torch.bfloat16, device="cuda")
        B[0] = ints(1, K, N, top=1)
        B[-1] = B[0]
        A = ints(2, 32, K, top=1).bfloat16()
        A[16:] = A[:16]
        off = offsets_of([0, 16, *([16] * (E - 2)), 32])
        assert B[-1].data_ptr() - B.data_ptr() > 1 << 32
        C = g.grouped_matmul(A, B, off)
        same(C[:16], A[:16].double() @ B[0].double(), "first group")
        assert torch.equal(C[16:], C[:16])
        dA, dB = g.grouped_matmul_backward(C.clamp(-2, 2), A, B, off)
        same(dB[0], A[:16].double().t() @ C[:16].clamp(-2, 2).double(), "dB")
        assert torch.equal(dB[-1], dB[0]) and not dB[1:-1].any() and torch.equal(dA[16:], dA[:16])
        del dB
        Wq = torch.zeros(2 * E, N, K, dtype=F8, device="cuda")
        Wq[0] = B[0].t()
        Wq[-1] = Wq[0]
        del B
        Aq, Sa = g.f8_quantize(A)
        Sw = torch.ones(2 * E, N // 128, K // 128, device="cuda")
        C8 = g.f8_grouped_matmul(Aq, Sa, Wq, Sw, offsets_of([0, 16, *([16] * (2 * E - 2)), 32]))
        assert Wq[-1].data_ptr() - Wq.data_ptr() > 1 << 32
        assert torch.equal(C8[16:], C8[:16])
        assert float((C8.double() - C.double()).norm() / C.double().norm()) < 2.0**-7
