"""8-bit floating-point codes and products on the GPU: codes and scales bit for bit, products against float64
(the tolerances are those of the grouped products' tests)."""

import numpy as np
import pytest

from grouping import e4m3_round, e4m3_values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402
from test_gpu_grouped import CUT, bf, blocks, close, f8, gen, ints, powers, same, spread, strided4  # noqa: E402

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.set_device(0)
    g.gemm_init(0)
    yield


def codes_and_scales(x, axes, most):
    """Values of the codes and scales of blocks of float64 x, whose largest magnitude over `axes` is `most`."""
    tiny = most < 448 * 2.0**-126
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(tiny, x * 2.0**126, x * 448 / most)
        s = np.where(tiny, 2.0**-126, (most.astype(np.float32) / np.float32(448)).astype(np.float64))
    q = np.where((most == 0) | ~np.isfinite(most), 0.0, q)
    s = np.where(most == 0, 0.0, np.where(np.isfinite(most), s, np.nan))
    return e4m3_round(q), s


def reference_rows(x):
    """(R x K values of the codes, blocks x R scales) of float64 rows."""
    R, K = x.shape
    b = np.concatenate([x, np.zeros((R, -K % 128))], 1).reshape(R, -1, 128)
    q, s = codes_and_scales(b, 2, np.where(np.isnan(b).any(2), np.nan, np.abs(b).max(2))[:, :, None])
    return q.reshape(R, -1)[:, :K], s[:, :, 0].T


def check_rows(X, what):
    Q, S = g.f8_quantize(X)
    assert Q.dtype == F8 and Q.shape == X.shape and S.shape == (blocks(X.shape[1]), X.shape[0])
    q, s = reference_rows(X.double().cpu().numpy())
    assert np.array_equal(S.double().cpu().numpy(), s, equal_nan=True), f"{what}: scales"
    got = Q.float().double().cpu().numpy()
    assert np.array_equal(got, q), f"{what}: {np.argwhere(got != q)[:3].tolist()} {got[got != q][:3]} {q[got != q][:3]}"
    return Q, S


@pytest.mark.parametrize("R,K,pad,offset", [(1, 1, 0, 0), (1, 4096, 0, 0), (3, 129, 0, 0), (5, 127, 1, 0), (17, 1003, 0, 1),
                                            (16, 11008, 8, 8), (509, 1003, 3, 5), (4096, 520, 0, 0), (70, 20000, 0, 0),
                                            (2, 65, 0, 0), (33, 8, 5, 2), (9000, 40, 0, 0), (300, 4100, 4, 0)])
def test_quantize(R, K, pad, offset):
    x = torch.randn(R, K, generator=gen(R + K), device="cuda") * torch.exp2(4 * torch.randn(R, 1, generator=gen(K), device="cuda"))
    Q, _ = check_rows(bf(x, pad, offset), f"{R} x {K}")
    ld = -(-K // 16) * 16                                   # rows are padded with zeros
    assert Q.stride(0) == ld or R == 1
    assert not Q.as_strided((R, ld), (ld, 1)).view(torch.uint8)[:, K:].any()


def test_quantize_every_mantissa():
    """Every mantissa of the largest value against every mantissa of a value, over the exponents down to codes that
    round to zero: ties, and everything next to one."""
    big = (np.arange(128, 256, dtype=np.float64) / 128)[:, None, None]
    small = (np.arange(128, 256, dtype=np.float64) / 128)[None, None, :] * np.exp2(-np.arange(0, 20.0))[None, :, None]
    x = np.minimum(np.broadcast_to(small, (128, 20, 128)), np.broadcast_to(big, (128, 20, 128))).copy()
    x[:, :, 0] = big[:, :, 0]
    x[:, 1::2, 1:] *= -1
    for scale in (1.0, 2.0**-100, 2.0**100):
        check_rows(torch.from_numpy(x.reshape(-1, 128) * scale).cuda().bfloat16(), f"times {scale}")


def test_quantize_special_blocks():
    x = torch.randn(12, 300, generator=gen(1), device="cuda").bfloat16()
    x[0, :128] = 0
    x[1, 130] = float("inf")
    x[2, 299] = float("nan")
    x[3, :] = 0
    x[4, 5], x[4, 6] = float("-inf"), float("nan")
    x[5, 128:256] = 0
    x[5, 200] = 2.0**-133                                    # the smallest bf16
    x[6] = x[6].float().mul(2.0**-130).bfloat16()            # subnormal
    x[7] = x[7].float().mul(2.0**-117).bfloat16()            # about the smallest scale
    x[8, 0] = 3.3895313892515355e38                          # the largest bf16
    x[9] = x[9].float().mul(2.0**-120).bfloat16()
    x[10, :] = -0.0
    Q, S = check_rows(x, "special")
    assert torch.isnan(S[1, 1]) and torch.isnan(S[2, 2]) and torch.isnan(S[0, 4]) and not torch.isnan(S[0, 1])
    assert S[0, 3] == 0 and S[1, 5] == 2.0**-126


@pytest.mark.parametrize("E,N,K,pad,offset", [(None, 128, 128, 0, 0), (None, 1, 1, 0, 0), (None, 300, 129, 0, 0),
                                              (None, 2501, 1003, 5, 3), (3, 200, 300, 0, 0), (5, 129, 17, 3, 1), (2, 512, 4096, 8, 8)])
def test_quantize_weight(E, N, K, pad, offset):
    x = torch.randn(*((E,) if E else ()), N, K, generator=gen(N + K), device="cuda") * 0.02
    if N > 130:
        x[..., 128:, : min(K, 128)] = 0
    W = bf(x, pad, offset)
    Q, S = g.f8_quantize_weight(W)
    assert Q.shape == W.shape and S.shape == (*W.shape[:-2], blocks(N), blocks(K))
    for w, q, s in zip(W, Q, S) if E else ((W, Q, S),):
        b = np.zeros((blocks(N) * 128, blocks(K) * 128))
        b[:N, :K] = w.double().cpu().numpy()
        b = b.reshape(blocks(N), 128, blocks(K), 128)
        rq, rs = codes_and_scales(b, (1, 3), np.abs(b).max((1, 3), keepdims=True))
        assert np.array_equal(s.double().cpu().numpy(), rs[:, 0, :, 0])
        assert np.array_equal(q.float().double().cpu().numpy(), rq.reshape(blocks(N) * 128, -1)[:N, :K])


def reference(A, Sa, W, Sw):
    a = A.double() * Sa.double().t().repeat_interleave(128, 1)[:, : A.shape[1]]
    w = W.double() * spread(Sw.double(), *W.shape)
    return a @ w.t(), a.abs() @ w.abs().t()


SHAPES = [(1, 1, 1), (1, 11008, 4096), (1, 1000, 11008), (2, 17, 130), (3, 2352, 9118), (8, 4096, 4096), (16, 4096, 11008), (17, 520, 1003),
          (32, 1376, 512), (33, 64, 16), (64, 4096, 11008), (64, 1000, 2000), (65, 300, 129), (100, 129, 128), (257, 256, 512), (300, 520, 328),
          (509, 2501, 1003), (777, 1024, 2049), (1000, 1000, 1000), (2000, 4001, 257), (4096, 4096, 1024), (4097, 2056, 390),
          (640, 4352, 4096), (2048, 2048, 11008), (100, 72, 16448), (70, 64, 16385), (200, 130, 8300),
          (4096, 4352, 4096), (4353, 4096, 1104), (2176, 8200, 2064), (6000, 2900, 4100), (4100, 4352, 16500),
          (8192, 4352, 4736), (4609, 11000, 4130)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    A, W = ints(M, M, K), ints(N, N, K)
    Sa, Sw = powers(1, blocks(K), M), powers(2, blocks(N), blocks(K))
    ref, _ = reference(A, Sa, W, Sw)
    room = -K % 16
    same(g.f8_matmul(f8(A, room), Sa, f8(W, room), Sw), ref, "whole numbers")
    out = bf(torch.zeros(M, N), 3, 1)
    assert g.f8_matmul(f8(A, room + 16, 16), strided4(Sa, 1), f8(W, room + 32, 16), strided4(Sw, 2), out=out) is out
    same(out, ref, "padded rows")
    assert (out.as_strided((M, 3), (N + 3, 1), out.storage_offset() + N)[:-1].contiguous().view(torch.int16) == 0x7FC0).all()
    if M * N * K <= 1 << 30:
        same(g.f8_matmul(f8(A, 3, 1), Sa, f8(W, 5, 3), Sw), ref, "any alignment")


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    """From bf16: the codes and scales of the quantiser, in the same call."""
    x = torch.randn(M, K, generator=gen(M), device="cuda") * (1 + 15 * (torch.rand(K, generator=gen(1), device="cuda") < 0.01))
    Wq, Sw = g.f8_quantize_weight((0.02 * torch.randn(N, K, generator=gen(N), device="cuda")).bfloat16())
    A = bf(x, 8, 8)
    Aq, Sa = g.f8_quantize(A)
    ref, sabs = reference(Aq.float(), Sa, Wq.float(), Sw)
    C = g.f8_linear(A, Wq, Sw)
    close(C, ref, sabs, K, "linear", CUT)
    assert torch.equal(g.f8_matmul(Aq, Sa, Wq, Sw), C)
    assert torch.equal(g.f8_linear(bf(x, 3, 1), Wq, Sw), C)
    work = torch.full((g.gemm_f8_work_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(g.f8_linear(A, Wq, Sw, work=work), C)


@pytest.mark.parametrize("M,N,K", [(1, 64, 300), (40, 200, 300), (300, 264, 500)])
def test_every_code(M, N, K):
    """All finite codes, and NaN ones that spoil their own outputs alone."""
    finite = torch.from_numpy(np.flatnonzero(np.isfinite(e4m3_values())).astype(np.uint8)).cuda()
    pick = lambda seed, *s: finite[torch.randint(0, len(finite), s, generator=gen(seed), device="cuda")].view(F8)  # noqa: E731
    room = -K % 16
    A, W = (torch.cat([t.view(torch.uint8), torch.full((t.shape[0], room), 0x7F, dtype=torch.uint8, device="cuda")], 1).view(F8)[:, :K]
            for t in (pick(1, M, K), pick(2, N, K)))
    Sa, Sw = torch.rand(blocks(K), M, generator=gen(3), device="cuda") + 0.5, torch.rand(blocks(N), blocks(K), generator=gen(4), device="cuda") + 0.5
    ref, sabs = reference(A.float(), Sa, W.float(), Sw)
    close(g.f8_matmul(A, Sa, W, Sw), ref, sabs, K, "codes", CUT)
    A.view(torch.uint8)[0, 7] = 0x7F
    W.view(torch.uint8)[5, 290] = 0xFF
    C = g.f8_matmul(A, Sa, W, Sw)
    bad = torch.isnan(C)
    assert bad[0].all() and bad[:, 5].all()
    bad[0], bad[:, 5] = False, False
    assert not bad.any()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_what_the_matrix_instruction_keeps(M):
    """2^16 at one k, -2^16 at another and a product 2^gap times smaller at a third, of which the first two cancel. Up
    to gap 13 it is kept wherever the three lie, beyond where it has no large product among its eight; lost, it
    is off by less than 2^-13 of the largest."""
    gaps = range(0, 30)
    N = 4 * len(gaps)
    places = [(0, 1, 2), (0, 64, 127), (1, 2, 32), (7, 40, 90)]
    A, W, want = torch.zeros(M, 128, device="cuda"), torch.zeros(N, 128, device="cuda"), torch.zeros(N)
    for j, (a, b, c) in enumerate(places):
        for gap in gaps:
            e = 16 - gap
            n = len(gaps) * j + gap
            W[n, a], W[n, b], W[n, c] = 256.0, -256.0, 2.0 ** (e - 8) if e >= -1 else 0.0
            want[n] = 2.0**e if e >= -1 else 0.0
    A[:] = 256.0
    C = g.f8_matmul(A.to(F8), torch.ones(1, M, device="cuda"), W.to(F8), torch.ones(blocks(N), 1, device="cuda")).float().cpu()
    assert (C == C[0]).all()
    err = (C[0] - want).abs().view(4, -1)
    assert not err[:, :14].any() and (err < 2.0**3).all() and not err[1:].any()


def test_non_finite_values_spoil_their_rows_alone():
    A = torch.randn(70, 264, generator=gen(1), device="cuda").bfloat16()
    A[1, 3], A[65, 200] = float("inf"), float("nan")
    Wq, Sw = g.f8_quantize_weight((0.02 * torch.randn(40, 264, generator=gen(2), device="cuda")).bfloat16())
    for rows in (slice(0, 2), slice(1, 2), slice(0, 70)):
        C = g.f8_linear(A[rows], Wq, Sw)
        bad = torch.isnan(C).all(1).nonzero().flatten().tolist()
        assert bad == {2: [1], 1: [0], 70: [1, 65]}[C.shape[0]] and int(torch.isfinite(C).all(1).sum()) == C.shape[0] - len(bad)


def test_empty_sizes():
    Wq, Sw = g.f8_quantize_weight(torch.ones(24, 64, dtype=torch.bfloat16, device="cuda"))
    assert g.f8_linear(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), Wq, Sw).shape == (0, 24)
    assert g.f8_linear(torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), Wq[:0], Sw[:0]).shape == (4, 0)
    Wq, Sw = g.f8_quantize_weight(torch.ones(24, 0, dtype=torch.bfloat16, device="cuda"))
    assert not g.f8_linear(torch.ones(4, 0, dtype=torch.bfloat16, device="cuda"), Wq, Sw).any()


def test_streams_graphs_and_repeats():
    cases = []
    for M, N, K in ((1, 4096, 4096), (16, 4096, 11008), (64, 1000, 2056), (300, 520, 4096)):
        A = torch.randn(M, K, generator=gen(K), device="cuda").bfloat16()
        Wq, Sw = g.f8_quantize_weight((0.02 * torch.randn(N, K, generator=gen(N), device="cuda")).bfloat16())
        cases.append((A, Wq, Sw, g.f8_linear(A, Wq, Sw)))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        outs = []
        for A, Wq, Sw, _ in cases:
            for s in (s1, s2):
                with torch.cuda.stream(s):
                    outs.append(g.f8_linear(A, Wq, Sw))
        torch.cuda.synchronize()
        for i, y in enumerate(outs):
            assert torch.equal(y, cases[i // 2][3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [g.f8_linear(A, Wq, Sw) for A, Wq, Sw, _ in cases]
    for turn in range(4):
        for A, *_ in cases:
            A.copy_(torch.randn(A.shape, generator=gen(turn), device="cuda"))
        fresh = [g.f8_linear(A, Wq, Sw) for A, Wq, Sw, _ in cases]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, fresh):
            assert torch.equal(x, y)


def test_a_refused_call_leaves_its_work_buffer_as_it_was():
    A = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    Wq, Sw = g.f8_quantize_weight(torch.ones(24, 64, dtype=torch.bfloat16, device="cuda"))
    work = torch.full((4 * 64 + 4 * 4 - 1,), 0x5A, dtype=torch.uint8, device="cuda")
    with pytest.raises(g.GemmError):
        g.f8_linear(A, Wq, Sw, work=work)
    torch.cuda.synchronize()
    assert (work == 0x5A).all()


def test_offsets_past_32_bits():
    M, N, K = 1_060_003, 2056, 4104
    head = torch.randn(64, K, generator=gen(1), device="cuda").bfloat16()
    A = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    A[:64] = head
    A[-64:] = head
    Wq, Sw = g.f8_quantize_weight((0.02 * torch.randn(N, K, generator=gen(2), device="cuda")).bfloat16())
    Aq, Sa = g.f8_quantize(A)
    del A
    assert torch.equal(Aq[-64:].view(torch.uint8), Aq[:64].view(torch.uint8)) and torch.equal(Sa[:, -64:], Sa[:, :64])
    C = g.f8_matmul(Aq, Sa, Wq, Sw)
    assert C.numel() * 2 > 1 << 32 and Aq.numel() > 1 << 32
    assert torch.equal(C[-64:], C[:64]) and not C[64:-64].any()
    close(C[:64], *reference(Aq[:64].float(), Sa[:, :64], Wq.float(), Sw), K, "first rows", CUT)
