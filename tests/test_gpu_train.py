"""The training entry points on the GPU: gemm_bf16_bwd, gemm_bf16_swiglu_train and
gemm_bf16_swiglu_bwd against float64.

Tolerances. Products: the product check's |c - ref| <= 2^-8 |ref| + 2^-16 sum |a b|. The forward's C:
the oracle's bound for the fused gated product. dGU, element by element from bf16 inputs in float32:
sigmoid and 1 + g (1 - s) carry a few float32 roundings of terms of size 1 and |g|, so dg is within
2^-19 |d u| s (1 + |g|) and du within 2^-19 |d g| s of the exact value, before the rounding to bf16
(2^-8 of the result); a sigmoid below float32's normal range (g < -87) may come out as zero, which
the same sizes without s times 2^-126 cover. dA and dB are products of the dGU that the call wrote, and held to the product
check on those bits.
"""

import numpy as np
import pytest

import oracle
from oracle import bf16_to_f64
from oracle import swiglu as osw
from synth import matrix

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.set_device(0)
    g.gemm_init(0)
    yield


class Buf:
    """A bf16 matrix in device memory: `ld` columns a row, `offset` elements into its allocation."""

    def __init__(self, rows, cols, data=None, ld=None, offset=0):
        self.rows, self.cols, self.ld, self.offset = rows, cols, max(ld or cols, cols), offset
        host = np.full(max(offset + rows * self.ld, 1), 0x7FC0, np.uint16)  # NaN outside the matrix
        if data is not None:
            host[offset: offset + rows * self.ld].reshape(rows, self.ld)[:, :cols] = data
        self.t = torch.from_numpy(host.view(np.int16)).cuda()

    def ptr(self):
        return self.t.data_ptr() + 2 * self.offset

    def bits(self):
        h = self.t.cpu().numpy().view(np.uint16)
        body = h[self.offset: self.offset + self.rows * self.ld].reshape(self.rows, self.ld)
        assert (h[: self.offset] == 0x7FC0).all() and (body[:, self.cols:] == 0x7FC0).all(), "wrote outside"
        return np.ascontiguousarray(body[:, : self.cols])


def rows_of(M, n=48):
    return np.arange(M) if M <= n else np.unique(np.linspace(0, M - 1, n).astype(int))


def check_product(C, A, B, what):
    """C against A B (bf16 bits), on sampled rows when it is large."""
    r = rows_of(len(A), 4096 if A.shape[0] * A.shape[1] * B.shape[1] < 1 << 31 else 48)
    ref, sabs = oracle.gemm(np.ascontiguousarray(A[r]), np.ascontiguousarray(B), M=len(r), N=B.shape[1], K=A.shape[1])
    res = oracle.check(np.ascontiguousarray(C[r]), ref, sabs)
    assert res.ok, f"{what}: {res.summary()}"


# tokens x width out x width in: toy blocks, odd numbers of tokens, one token, both tile sizes, K split,
# products cut in two, a sum over fewer tokens than one k-step
SHAPES = [(1, 8, 8), (2, 16, 64), (31, 40, 24), (33, 520, 328), (64, 1000, 200), (65, 264, 136), (128, 128, 128),
          (257, 256, 512), (300, 520, 328), (509, 1376, 512), (1000, 1000, 1000), (4097, 520, 264),
          (200, 2048, 4096), (200, 4096, 2048), (640, 4352, 4096)]
LOOSE = [(3, 5, 7, 0, 0), (70, 100, 30, 0, 0), (65, 72, 40, 3, 0), (65, 72, 40, 0, 1), (130, 200, 96, 5, 1)]
PADDED = [(65, 264, 136, 8, 8), (300, 520, 328, 24, 16)]


@pytest.mark.parametrize("M,N,K,pad,offset", [(*s, 0, 0) for s in SHAPES] + LOOSE + PADDED)
def test_linear_backward(M, N, K, pad, offset):
    A, B = matrix("normal", M, K, seed=M + 1), matrix("normal", K, N, seed=N + 2, sigma=0.05)
    D = matrix("normal", M, N, seed=K + 3, sigma=0.01)
    D[rows_of(M)[::7]] = 0                                # tokens without a gradient
    bA, bB, bD = (Buf(*x.shape, x, x.shape[1] + pad, offset) for x in (A, B, D))
    dA, dB = Buf(M, K, ld=K + pad, offset=offset), Buf(K, N, ld=N + pad, offset=offset)
    s = g.current_stream_handle()
    g.gemm_bf16_bwd(M, N, K, bD.ptr(), bD.ld, bA.ptr(), bA.ld, bB.ptr(), bB.ld, dA.ptr(), dA.ld, dB.ptr(), dB.ld, s)
    torch.cuda.synchronize()
    plan = g.gemm_last_plan()
    assert plan["op"] == "grad_b" and (plan["M"], plan["N"], plan["K"]) == (K, N, M)
    check_product(dA.bits(), D, B.T, f"dA {M}x{N}x{K}")
    check_product(dB.bits(), np.ascontiguousarray(A.T), D, f"dB {M}x{N}x{K}")
    # either gradient alone: the same bits, the other's operand not read
    for need in ("A", "B"):
        d1 = Buf(M, K, ld=K + pad, offset=offset) if need == "A" else Buf(K, N, ld=N + pad, offset=offset)
        if need == "A":
            g.gemm_bf16_bwd(M, N, K, bD.ptr(), bD.ld, None, 0, bB.ptr(), bB.ld, d1.ptr(), d1.ld, None, 0, s)
        else:
            g.gemm_bf16_bwd(M, N, K, bD.ptr(), bD.ld, bA.ptr(), bA.ld, None, 0, None, 0, d1.ptr(), d1.ld, s)
        torch.cuda.synchronize()
        assert np.array_equal(d1.bits(), (dA if need == "A" else dB).bits())


def test_empty_sums_write_zeros():
    s = g.current_stream_handle()
    dA, dB = Buf(5, 8), Buf(8, 16)
    some = Buf(32, 32, np.ones((32, 32), np.uint16))
    g.gemm_bf16_bwd(5, 0, 8, None, 0, some.ptr(), 8, None, 0, dA.ptr(), 8, None, 0, s)   # N = 0
    g.gemm_bf16_bwd(0, 16, 8, None, 16, None, 8, some.ptr(), 16, dA.ptr(), 8, dB.ptr(), 16, s)  # M = 0
    torch.cuda.synchronize()
    assert (dA.bits() == 0).all() and (dB.bits() == 0).all()
    dA, dB = Buf(5, 8), Buf(8, 32)
    g.gemm_bf16_swiglu_bwd(5, 0, 8, None, 0, None, 0, some.ptr(), 8, None, 0, None, 0, dA.ptr(), 8, None, 0, s)
    g.gemm_bf16_swiglu_bwd(0, 16, 8, None, 16, None, 32, None, 8, some.ptr(), 32, None, 32, None, 8, dB.ptr(), 32, s)
    GU, C = Buf(5, 32), Buf(5, 16)
    g.gemm_bf16_swiglu_train(5, 16, 0, None, 0, None, 32, GU.ptr(), 32, C.ptr(), 16, s)
    torch.cuda.synchronize()
    for b in (dA, dB, GU, C):
        assert (b.bits() == 0).all()


@pytest.mark.parametrize("M,N,K,pad,offset", [(*s, 0, 0) for s in SHAPES] + LOOSE + PADDED)
def test_gated_forward(M, N, K, pad, offset):
    A, B = matrix("normal", M, K, seed=M + 11), matrix("normal", K, 2 * N, seed=N + 12, sigma=0.05)
    bA, bB = Buf(M, K, A, K + pad, offset), Buf(K, 2 * N, B, 2 * N + pad, offset)
    GU, C = Buf(M, 2 * N, ld=2 * N + pad, offset=offset), Buf(M, N, ld=N + pad, offset=offset)
    g.gemm_bf16_swiglu_train(M, N, K, bA.ptr(), bA.ld, bB.ptr(), bB.ld, GU.ptr(), GU.ld, C.ptr(), C.ld,
                             g.current_stream_handle())
    torch.cuda.synchronize()
    plan = g.gemm_last_plan()
    assert plan["op"] == "swiglu_train"
    check_product(GU.bits(), A, B, f"GU {M}x{N}x{K} {plan['reason']}")
    r = rows_of(M, 4096 if M * N * K < 1 << 30 else 48)
    h, slack = osw.swiglu(np.ascontiguousarray(A[r]), B, len(r), N, K)
    res = osw.check(np.ascontiguousarray(C.bits()[r]), h, slack)
    assert res.ok, f"C {M}x{N}x{K}: {res.summary()}"


def grad_formula(d, gate, up):
    """(dg, du, and the two bounds' sizes) in float64."""
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-gate))
    dg, du = d * up * sig * (1 + gate * (1 - sig)), d * gate * sig
    bare_g, bare_u = np.abs(d * up) * (1 + np.abs(gate)), np.abs(d * gate)
    return dg, du, bare_g * (sig + 2.0**-107), bare_u * (sig + 2.0**-107)


def check_dgu(got, D, GU, what):
    d, gu = bf16_to_f64(D), bf16_to_f64(GU)
    N = D.shape[1]
    dg, du, sg, su = grad_formula(d, gu[:, :N], gu[:, N:])
    ref, size = np.concatenate([dg, du], 1), np.concatenate([sg, su], 1)
    off = np.abs(bf16_to_f64(got) - ref) - (2.0**-8 * np.abs(ref) + (1 + 2.0**-8) * 2.0**-19 * size + 2.0**-126)
    assert (off <= 0).all(), f"{what}: {(off > 0).sum()} outside, worst {off.max()}"


@pytest.mark.parametrize("M,N,K,pad,offset", [(*s, 0, 0) for s in SHAPES] + LOOSE + PADDED)
def test_gated_backward(M, N, K, pad, offset):
    A, B = matrix("normal", M, K, seed=M + 21), matrix("normal", K, 2 * N, seed=N + 22, sigma=0.05)
    D, GU = matrix("normal", M, N, seed=K + 23, sigma=0.01), matrix("normal", M, 2 * N, seed=M + 24, sigma=3.0)
    D[rows_of(M)[::7]] = 0
    bA, bB = Buf(M, K, A, K + pad, offset), Buf(K, 2 * N, B, 2 * N + pad, offset)
    bD, bG = Buf(M, N, D, N + pad, offset), Buf(M, 2 * N, GU, 2 * N + pad, offset)
    out = []
    for inplace in (False, True):
        dG = bG if inplace else Buf(M, 2 * N, ld=2 * N + pad, offset=offset)
        dA, dB = Buf(M, K, ld=K + pad, offset=offset), Buf(K, 2 * N, ld=2 * N + pad, offset=offset)
        g.gemm_bf16_swiglu_bwd(M, N, K, bD.ptr(), bD.ld, bG.ptr(), bG.ld, bA.ptr(), bA.ld, bB.ptr(), bB.ld, dG.ptr(),
                               dG.ld, dA.ptr(), dA.ld, dB.ptr(), dB.ld, g.current_stream_handle())
        torch.cuda.synchronize()
        out.append((dG.bits(), dA.bits(), dB.bits()))
    for x, y in zip(*out):
        assert np.array_equal(x, y), "dGU in GU's memory gives other bits"
    dg, da, db = out[0]
    check_dgu(dg, D, GU, f"dGU {M}x{N}x{K}")
    check_product(da, dg, B.T, f"dA {M}x{N}x{K}")
    check_product(db, np.ascontiguousarray(A.T), dg, f"dB {M}x{N}x{K}")


def test_gate_gradient_at_extreme_gates():
    """Saturated gates, zeros and infinities: the limits of the formula, and no NaN at finite gates."""
    gates = np.array([0.0, -0.0, 1e-30, -1e-30, 20, -20, 88, -88, 89, -89, 200, -200, 3e38, -3e38], np.float32)
    M, N = 3, 24
    gu = np.ones((M, 2 * N), np.float32)
    gu[:, : len(gates)] = gates
    gu[:, N:] = 2.0
    D, GU = oracle.bf16_rne(np.full((M, N), 0.5)), oracle.bf16_rne(gu.astype(np.float64))
    bD, bG, dG = Buf(M, N, D), Buf(M, 2 * N, GU), Buf(M, 2 * N)
    g.gemm_bf16_swiglu_bwd(M, N, 8, bD.ptr(), N, bG.ptr(), 2 * N, None, 0, None, 0, dG.ptr(), 2 * N, None, 0, None, 0,
                           g.current_stream_handle())
    torch.cuda.synchronize()
    check_dgu(dG.bits(), D, GU, "extreme gates")


def test_gate_gradient_against_differences():
    """dGU element by element against central differences of the forward in float64: step 1e-4, whose
    own error is 1e-8 / 6 of the third derivative (at most 2 |d u|) and 1e-12 of rounding."""
    M, N = 37, 64
    D, GU = matrix("normal", M, N, seed=5, sigma=1.0), matrix("normal", M, 2 * N, seed=6, sigma=2.0)
    bD, bG, dG = Buf(M, N, D), Buf(M, 2 * N, GU), Buf(M, 2 * N)
    g.gemm_bf16_swiglu_bwd(M, N, 8, bD.ptr(), N, bG.ptr(), 2 * N, None, 0, None, 0, dG.ptr(), 2 * N, None, 0, None, 0,
                           g.current_stream_handle())
    torch.cuda.synchronize()
    d, gu = bf16_to_f64(D), bf16_to_f64(GU)
    gate, up, eps = gu[:, :N], gu[:, N:], 1e-4
    f = lambda a, b: d * osw.silu(a) * b  # noqa: E731
    fd = np.concatenate([(f(gate + eps, up) - f(gate - eps, up)) / (2 * eps),
                         (f(gate, up + eps) - f(gate, up - eps)) / (2 * eps)], 1)
    size = np.concatenate([np.abs(d * up) * (1 + np.abs(gate)), np.abs(d * gate)], 1)
    tol = 2.0**-8 * np.abs(fd) + 2.0**-18 * size + 1e-8 * np.tile((1 + np.abs(d)) * (1 + np.abs(gate) + np.abs(up)), 2)
    assert (np.abs(bf16_to_f64(dG.bits()) - fd) <= tol).all()


def test_block_gradient_against_differences():
    """dA and dB of the whole block against central differences of sum(dC * C) along random
    directions, in float64. A and B are small integers, so that g and u are exact in bf16 and the
    kernels' only errors are the roundings of dGU and of the gradients to bf16, 2^-8 of each at
    most, plus the products' 2^-16 of their absolute sums."""
    M, N, K = 40, 24, 8
    rng = np.random.default_rng(3)
    A, B = rng.integers(-1, 2, (M, K)).astype(np.float64), rng.integers(-1, 2, (K, 2 * N)).astype(np.float64)
    Db = oracle.bf16_rne(rng.normal(size=(M, N)))
    d = bf16_to_f64(Db)
    dev = lambda x: torch.from_numpy(oracle.bf16_rne(x).view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    tA, tB, tD = dev(A), dev(B), torch.from_numpy(Db.view(np.int16)).view(torch.bfloat16).cuda()
    C, GU = g.swiglu_forward(tA, tB)
    assert np.array_equal(GU.double().cpu().numpy(), A @ B)
    dA, dB, dGU = (x.double().cpu().numpy() for x in g.swiglu_backward(tD, GU, tA, tB))

    def loss(a, b):
        y = a @ b
        return (d * osw.silu(y[:, :N]) * y[:, N:]).sum()

    absD = np.abs(dGU)
    eA = 2.0**-7 * (absD @ np.abs(B).T) + 2.0**-8 * np.abs(dA)
    eB = 2.0**-7 * (np.abs(A).T @ absD) + 2.0**-8 * np.abs(dB)
    for _ in range(8):
        da, db, eps = rng.normal(size=A.shape), rng.normal(size=B.shape), 1e-5
        fd = (loss(A + eps * da, B + eps * db) - loss(A - eps * da, B - eps * db)) / (2 * eps)
        tol = (np.abs(da) * eA).sum() + (np.abs(db) * eB).sum() + 1e-6 * (1 + abs(fd))
        assert abs((dA * da).sum() + (dB * db).sum() - fd) <= tol


def test_infinities_stay_in_their_rows():
    """An infinity in one token reaches that token's dA only; in one output column's dC, only that
    column of dB. Rows and columns past the matrix do not mix in."""
    M, N, K = 130, 136, 264
    A, B = matrix("normal", M, K, seed=31), matrix("normal", K, N, seed=32, sigma=0.05)
    D = matrix("normal", M, N, seed=33, sigma=0.1)
    D[5, 9] = 0x7F80
    dA, dB = g.matmul_backward(*(torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() for x in (D, A, B)))
    fa, fb = torch.isfinite(dA).cpu().numpy(), torch.isfinite(dB).cpu().numpy()
    assert fa[np.arange(M) != 5].all() and fb[:, np.arange(N) != 9].all()
    assert not fa[5].all() and not fb[:, 9].all()


def test_streams_graphs_and_repeats():
    M, N, K = 300, 1000, 520
    t = lambda *s, sd=1.0: (torch.randn(*s, generator=torch.Generator().manual_seed(sum(s))) * sd).bfloat16().cuda()  # noqa: E731
    A, B, D = t(M, K), t(K, 2 * N, sd=0.05), t(M, N, sd=0.1)

    def step():
        C, GU = g.swiglu_forward(A, B)
        return (C, GU, *g.swiglu_backward(D, GU, A, B), *g.matmul_backward(D, A, B[:, :N]))

    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
        torch.cuda.synchronize()
        for outs in got:
            for x, y in zip(outs, want):
                assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        for x in outs:
            x.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_offsets_past_32_bits():
    """More than 2^32 bytes of activations and of g and u: only the first and last tokens are not zero,
    and both gradients are those of these tokens alone."""
    M, N, K = 540_001, 2056, 4104
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    few = torch.cat([torch.arange(64), torch.arange(M - 65, M)]).cuda()
    x, d, B = r(len(few), K).bfloat16(), (r(len(few), N) * 0.1).bfloat16(), (r(K, 2 * N) * 0.02).bfloat16()
    A = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    D = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    A[few], D[few] = x, d
    C, GU = g.swiglu_forward(A, B)
    c, gu = g.swiglu_forward(x, B)
    assert A.numel() * 2 > 1 << 32 and GU.numel() * 2 > 1 << 32
    err = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    # the same products in another order of sums, each rounded to bf16
    assert err(C[few], c) < 2.0**-8 and err(GU[few], gu) < 2.0**-8 and not C[64:-65].any()
    dA, dB, dGU = g.swiglu_backward(D, GU, A, B, inplace=True)
    da, db, dgu = g.swiglu_backward(d, gu, x, B)
    assert err(dGU[few], dgu) < 2.0**-7 and err(dA[few], da) < 2.0**-7 and err(dB, db) < 2.0**-7
    assert not dA[64:-65].any() and not dGU[64:-65].any()


def test_gates_below_the_normal_range():
    """Gates at which the sigmoid is below float32's normal range (g < -87.3) while g s, or g s u with a
    large u, is not. silu(g) carries 2^-20 of its size and, below 2^-126 itself, float32's smallest step
    2^-149; u multiplies both, and the rounding to bf16 adds 2^-8 of the result."""
    gates = np.array([-87.0, -87.5, -88.0, -88.5, -89.0, -91.0, -95.0, -100.0], np.float64)
    M, N, K = 70, 8, 8
    for scale in (2.0**100, 2.0**20):
        A, B = np.zeros((M, K)), np.zeros((K, 2 * N))
        A[:, 0], B[0, :N], B[0, N:] = 1, gates, scale
        dev = lambda x: torch.from_numpy(oracle.bf16_rne(x).view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
        # the matrix kernels, and the general one (rows without 16-byte alignment)
        for tA in (dev(A), dev(np.concatenate([A, A[:, :1]], 1))[:, :K]):
            C, GU = g.swiglu_forward(tA, dev(B))
            assert np.array_equal(GU.double().cpu().numpy(), A @ B)
            s = gates / (1 + np.exp(-gates))
            slack = 2.0**-8 * np.abs(s * scale) + (2.0**-20 * np.abs(s) + 2.0**-149) * scale + 2.0**-133
            off = np.abs(C.double().cpu().numpy() - s * scale) - slack
            assert (off <= 0).all(), (scale, gates[(off > 0).any(0)])
        # du = d silu(g), dg = d u s (1 + g (1 - s))
        D = dev(np.full((M, N), scale))
        GU = dev(np.concatenate([np.tile(gates, (M, 1)), np.ones((M, N))], 1))
        _, _, dGU = g.swiglu_backward(D, GU, dev(A), dev(B), need_dA=False, need_dB=False)
        sig = 1 / (1 + np.exp(-gates))
        ds = sig * (1 + gates * (1 - sig))
        want = np.concatenate([ds, s]) * scale
        size = np.concatenate([sig * (1 + np.abs(gates)), np.abs(s)])
        slack = 2.0**-8 * np.abs(want) + (2.0**-19 * size + 2.0**-149) * scale + 2.0**-133
        off = np.abs(dGU.double().cpu().numpy() - want) - slack
        assert (off <= 0).all(), (scale, np.argwhere((off > 0).any(0)).ravel())


def test_a_refused_call_leaves_gu_as_it_was():
    """dGU in GU's memory, and a weight gradient with more tiles than the general kernel's grid holds: the
    refusal comes before the pass that overwrites GU. (dB is never written: no such memory is needed.)"""
    K = 1 << 17
    bA = Buf(1, K, matrix("normal", 1, K, seed=7))
    wide = 1 << 22           # past the matrix kernels' leading dimensions; 2^11 x 2^16 tiles
    gu = Buf(1, wide, matrix("normal", 1, wide, seed=9))
    d = Buf(1, wide // 2, matrix("normal", 1, wide // 2, seed=8))
    before = gu.bits()
    st = g.lib().gemm_bf16_swiglu_bwd(1, wide // 2, K, d.ptr(), wide // 2, gu.ptr(), wide, bA.ptr(), K, None, wide, gu.ptr(),
                                      wide, None, K, 64, wide, g.current_stream_handle())
    torch.cuda.synchronize()
    assert st == g.GEMM_ERR_UNSUPPORTED
    assert np.array_equal(gu.bits(), before)


def test_a_call_without_a_workspace_leaves_gu_as_it_was():
    """The library keeps a workspace for each of 64 streams; the next stream whose product needs one is
    refused, before a dGU in GU's memory is written. The call then gives, on a stream that has one, the
    bits of an out-of-place call."""
    import ctypes

    L = g.lib()
    M, N, K = 64, 2048, 64          # dA sums over 4096: split
    bD, bG, bA, bB = (Buf(r, c, matrix("normal", r, c, seed=r + c)) for r, c in ((M, N), (M, 2 * N), (M, K), (K, 2 * N)))
    want, dA, dB = Buf(M, 2 * N), Buf(M, K), Buf(K, 2 * N)

    def call(dGU, stream):
        return L.gemm_bf16_swiglu_bwd(M, N, K, bD.ptr(), N, bG.ptr(), 2 * N, bA.ptr(), K, bB.ptr(), 2 * N, dGU.ptr(), 2 * N,
                                      dA.ptr(), K, dB.ptr(), 2 * N, stream)

    here = g.current_stream_handle()
    assert call(want, here) == g.GEMM_OK
    torch.cuda.synchronize()
    before, want = bG.bits(), want.bits()
    streams, refused = [], None
    x, y, z = Buf(64, 4096, matrix("normal", 64, 4096, seed=5)), Buf(64, 4096, matrix("normal", 64, 4096, seed=6)), Buf(64, 64)
    try:
        for _ in range(66):
            h = ctypes.c_void_p()
            assert L.hipStreamCreate(ctypes.byref(h)) == 0
            streams.append(h)
            # x y^T over 4096: split over K, so with partial sums
            st = L.gemm_bf16_bwd(64, 4096, 64, x.ptr(), 4096, None, 64, y.ptr(), 4096, z.ptr(), 64, None, 4096, h)
            torch.cuda.synchronize()
            if st != g.GEMM_OK:
                assert st == g.GEMM_ERR_UNSUPPORTED
                refused = h
                break
            assert g.gemm_last_plan()["splits"] > 1
        assert refused is not None
        assert call(bG, refused) == g.GEMM_ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert np.array_equal(bG.bits(), before)
        assert call(bG, here) == g.GEMM_OK
        torch.cuda.synchronize()
        assert np.array_equal(bG.bits(), want)
    finally:
        torch.cuda.synchronize()
        g.gemm_finalize()
        g.gemm_init(0)
        for h in streams:
            L.hipStreamDestroy(h)


def test_last_plan_names_both_gradients_of_one_launch():
    def t(*s):
        return torch.zeros(*s, dtype=torch.bfloat16, device="cuda")

    sizes = lambda p: (p["op"], p["M"], p["N"], p["K"])  # noqa: E731
    D, A, B = t(512, 264), t(512, 520), t(520, 264)
    g.matmul_backward(D, A, B)
    p = g.gemm_last_plan()
    assert sizes(p) == ("grad_b", 520, 264, 512) and sizes(p["with"]) == ("grad_a", 512, 520, 264)
    g.matmul_backward(D, A, B, need_dA=False)
    assert sizes(g.gemm_last_plan()) == ("grad_b", 520, 264, 512) and "with" not in g.gemm_last_plan()
    g.matmul_backward(D, A, B, need_dB=False)
    assert sizes(g.gemm_last_plan()) == ("grad_a", 512, 520, 264) and "with" not in g.gemm_last_plan()
    # a launch each: the plan is the second's
    g.matmul_backward(t(4096, 4096), t(4096, 4096), t(4096, 4096))
    assert g.gemm_last_plan()["op"] == "grad_b" and "with" not in g.gemm_last_plan()


def test_in_an_autograd_function():
    """The calls refuse tensors that require grad, and train inside a torch.autograd.Function, whose
    gradients are those of the calls by themselves."""

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            C, GU = g.swiglu_forward(x, w)
            ctx.save_for_backward(x, w, GU)
            return C

        @staticmethod
        def backward(ctx, dC):
            x, w, GU = ctx.saved_tensors
            return g.swiglu_backward(dC, GU, x, w)[:2]

    dev = lambda *s: (torch.randn(*s, generator=torch.Generator().manual_seed(s[0])) * 0.2).bfloat16().cuda()  # noqa: E731
    x, w, d = dev(70, 136).requires_grad_(), dev(136, 160).requires_grad_(), dev(70, 80)
    y, (q, s) = x.detach(), g.i8_quantize(w)
    sg = s.clone().requires_grad_()
    for call in (lambda: g.swiglu_forward(x, w.detach()), lambda: g.swiglu_forward(y, w),
                 lambda: g.matmul_backward(d, y, w[:, :80]), lambda: g.i8_linear(y[:, :160] @ y.new_zeros(136, 160), q, sg),
                 lambda: g.i8_linear(y, g.i8_quantize(y)[0], torch.ones(70, device="cuda"),
                                     out=torch.zeros(70, 70, dtype=torch.bfloat16, device="cuda").requires_grad_())):
        with pytest.raises(RuntimeError, match="requires grad"):
            call()
    C = Gated.apply(x, w)
    C.backward(d)
    want, GU = g.swiglu_forward(y, w.detach())
    dA, dB, _ = g.swiglu_backward(d, GU, y, w.detach())
    assert torch.equal(C, want) and torch.equal(x.grad, dA) and torch.equal(w.grad, dB)
    with torch.no_grad():
        assert torch.equal(g.swiglu_forward(x, w)[0], want)


def some_rows(M, n=64):
    """Rows of both halves of the first, of middle and of the last 256-row tiles, and both sides of a cut."""
    rng = np.random.default_rng(M)
    near = [r for t in range(0, M, 256) for r in (t, t + 127, t + 128, t + 255)] + [M - 1]
    return np.unique([r for r in near if r < M] + rng.integers(0, M, n).tolist())


def expect_large(plan, cut):
    assert plan["kernel"] == "tile" and plan["bm"] == 256, plan
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert plan.get("cut", {}).get("axis") == cut, plan


# 256 x 256 tiles in a partial wave and in full waves with the last one cut off across columns or rows,
# over odd (328, 336, 333: 11) and even (360: 12) numbers of k-steps that go round the five-slot rings
@pytest.mark.parametrize("M,N,K,cut", [(2300, 2040, 328, None), (2300, 2040, 360, None), (4096, 2176, 328, "n"),
                                       (4350, 2040, 360, "m")])
def test_large_tiles_forward(M, N, K, cut):
    A, B = matrix("normal", M, K, seed=M), matrix("normal", K, 2 * N, seed=N, sigma=0.05)
    bA, bB = Buf(M, K, A), Buf(K, 2 * N, B)
    GU, C = Buf(M, 2 * N, ld=2 * N + 8), Buf(M, N, ld=N + 16)
    g.gemm_bf16_swiglu_train(M, N, K, bA.ptr(), K, bB.ptr(), 2 * N, GU.ptr(), GU.ld, C.ptr(), C.ld, g.current_stream_handle())
    torch.cuda.synchronize()
    expect_large(g.gemm_last_plan(), cut)
    r = some_rows(M)
    a = np.ascontiguousarray(A[r])
    ref, sabs = oracle.gemm(a, B, M=len(r), N=2 * N, K=K)
    res = oracle.check(np.ascontiguousarray(GU.bits()[r]), ref, sabs)
    assert res.ok, res.summary()
    h, slack = osw.swiglu(a, B, len(r), N, K)
    res = osw.check(np.ascontiguousarray(C.bits()[r]), h, slack)
    assert res.ok, res.summary()


# rows of the output, its columns, the sum's length
@pytest.mark.parametrize("R,C,S,cut", [(2300, 4088, 336, None), (2300, 4088, 360, None), (4350, 4088, 360, "m"),
                                       (4090, 4352, 336, "n")])
def test_large_tiles_grad_a(R, C, S, cut):
    D, B = matrix("normal", R, S, seed=R, sigma=0.01), matrix("normal", C, S, seed=C, sigma=0.05)
    bD, bB, dA = Buf(R, S, D), Buf(C, S, B), Buf(R, C, ld=C + 8)
    g.gemm_bf16_bwd(R, S, C, bD.ptr(), S, None, C, bB.ptr(), S, dA.ptr(), dA.ld, None, S, g.current_stream_handle())
    torch.cuda.synchronize()
    expect_large(g.gemm_last_plan(), cut)
    r = some_rows(R)
    ref, sabs = oracle.gemm(np.ascontiguousarray(D[r]), np.ascontiguousarray(B.T), M=len(r), N=C, K=S)
    res = oracle.check(np.ascontiguousarray(dA.bits()[r]), ref, sabs)
    assert res.ok, res.summary()


@pytest.mark.parametrize("R,C,S,cut", [(2296, 4088, 333, None), (2296, 4088, 360, None), (4352, 4088, 360, "m"),
                                       (4088, 4352, 333, "n")])
def test_large_tiles_grad_b(R, C, S, cut):
    A, D = matrix("normal", S, R, seed=R), matrix("normal", S, C, seed=C, sigma=0.01)
    bA, bD, dB = Buf(S, R, A), Buf(S, C, D), Buf(R, C, ld=C + 8)
    g.gemm_bf16_bwd(S, C, R, bD.ptr(), C, bA.ptr(), R, None, C, None, R, dB.ptr(), dB.ld, g.current_stream_handle())
    torch.cuda.synchronize()
    expect_large(g.gemm_last_plan(), cut)
    r = some_rows(R)
    ref, sabs = oracle.gemm(np.ascontiguousarray(A.T[r]), D, M=len(r), N=C, K=S)
    res = oracle.check(np.ascontiguousarray(dB.bits()[r]), ref, sabs)
    assert res.ok, res.summary()


@pytest.mark.parametrize("R,C,S,splits", [(1400, 2032, 6440, 2), (1400, 2032, 4512, 1), (1400, 2032, 3872, 1)])
def test_two_pieces_on_most_cus(R, C, S, splits):
    """dA, dB and the forward on 176 tiles of 128 x 128, sums of 202, 141 and 121 k-steps: two pieces of dA
    from 200 and of the others from 120, an even number of k-steps in each."""
    whole_cus = torch.cuda.get_device_properties(0).multi_processor_count == 256

    def planned(splits, steps):
        p = g.gemm_last_plan()
        assert p["bm"] == 128
        if whole_cus:
            assert (p["splits"], p["kt_per_split"]) == ((2, (steps + 1) // 2 + (steps + 1) // 2 % 2) if splits == 2 else (1, steps))

    def check(out, X, Y):
        r = some_rows(len(X), 32)
        ref, sabs = oracle.gemm(np.ascontiguousarray(X[r]), Y, M=len(r), N=Y.shape[1], K=S)
        res = oracle.check(np.ascontiguousarray(out[r]), ref, sabs)
        assert res.ok, res.summary()

    steps, s = -(-S // 32), g.current_stream_handle()
    X, Y = matrix("normal", R, S, seed=1), matrix("normal", C, S, seed=2, sigma=0.05)
    bX, bY, out = Buf(R, S, X), Buf(C, S, Y), Buf(R, C)
    g.gemm_bf16_bwd(R, S, C, bX.ptr(), S, None, C, bY.ptr(), S, out.ptr(), C, None, S, s)
    torch.cuda.synchronize()
    planned(splits, steps)
    check(out.bits(), X, np.ascontiguousarray(Y.T))
    XT, YT = np.ascontiguousarray(X.T), np.ascontiguousarray(Y.T)
    bX, bY, out = Buf(S, R, XT), Buf(S, C, YT), Buf(R, C)
    g.gemm_bf16_bwd(S, C, R, bY.ptr(), C, bX.ptr(), R, None, C, None, R, out.ptr(), C, s)
    torch.cuda.synchronize()
    planned(2, steps)
    check(out.bits(), X, YT)
    bX, GU, h = Buf(R, S, X), Buf(R, C), Buf(R, C // 2)
    g.gemm_bf16_swiglu_train(R, C // 2, S, bX.ptr(), S, bY.ptr(), C, GU.ptr(), C, h.ptr(), C // 2, s)
    torch.cuda.synchronize()
    planned(2, steps)
    check(GU.bits(), X, YT)
