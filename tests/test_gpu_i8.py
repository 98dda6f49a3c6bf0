"""The 8-bit products on the GPU against integer sums and float64.

gemm_i8's result is pinned bit for bit: the 32-bit sum is exact, and its float32 conversion and two
multiplications by the scales are single IEEE operations that numpy repeats. The gated form is held
to a bound: g and u carry three float32 roundings each (3 * 2^-24, taken as 2^-22), which the slope of
silu (at most 1.1) passes on; evaluating silu and the product adds 2^-20 of the result, and the
rounding to bf16 2^-8 (as in the float product's check). Codes of gemm_i8_quantize are compared with
the definition's two float32 divisions, bit for bit.
"""

import ctypes

import numpy as np
import pytest

from oracle import bf16_to_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gemv_layers_amd as g  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.set_device(0)
    g.gemm_init(0)
    yield


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def codes(rows, k, ld, seed, full=False):
    """Random codes (with -128 when `full`), the padding between k and ld filled with them too."""
    rng = np.random.default_rng(seed)
    return rng.integers(-128 if full else -127, 128, (rows, max(ld, 1)), dtype=np.int8)[:, :ld]


def bf16_of(x32):
    """float32 -> bf16 bits, to nearest even (finite values)."""
    u = np.ascontiguousarray(x32, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def widen(h):
    """bf16 bits -> float64."""
    return bf16_to_f64(np.ascontiguousarray(h))


def place(a, offset=0):
    """A host array on the device, `offset` elements past the start of its allocation."""
    flat = np.concatenate([np.zeros(offset, a.dtype), a.ravel()])
    return torch.from_numpy(flat).cuda(), offset * a.dtype.itemsize


def poisoned(n):
    return torch.full((max(n, 1),), float("nan"), dtype=torch.bfloat16, device="cuda")


def product(M, N, K, lda=None, ldw=None, ldc=None, offset=0, c_offset=0, seed=0, full=False, glu=False, sa=None):
    """Runs gemm_i8 (or its gated form) and returns (C bits, exact sums, sa, sw, plan)."""
    lda = -(-K // 16) * 16 if lda is None else lda
    ldw = -(-K // 16) * 16 if ldw is None else ldw
    ldc = N if ldc is None else ldc
    rows = 2 * N if glu else N
    A, W = codes(M, K, lda, seed + 1, full), codes(rows, K, ldw, seed + 2, full)
    rng = np.random.default_rng(seed + 3)
    sa = rng.uniform(0.5, 2, M).astype(np.float32) / 127 if sa is None else sa
    sw = (rng.uniform(0.5, 2, rows) * 0.02 / 127 / max(K, 1) ** 0.5 * 30).astype(np.float32)
    (dA, oa), (dW, ow) = place(A, offset), place(W, offset)
    (dsa, _), (dsw, _) = place(sa), place(sw)
    C = poisoned(M * ldc + c_offset)
    fn = g.gemm_i8_swiglu if glu else g.gemm_i8
    fn(M, N, K, dA.data_ptr() + oa, lda, dsa.data_ptr(), dW.data_ptr() + ow, ldw, dsw.data_ptr(),
       C.data_ptr() + 2 * c_offset, ldc, g.current_stream_handle())
    torch.cuda.synchronize()
    out = bits(C)
    assert (out[:c_offset] == 0x7FC0).all() or c_offset == 0
    out = out[c_offset: c_offset + M * ldc].reshape(M, ldc)
    # columns past N keep the poison
    assert not (out[:, N:] != bits(poisoned(1))[0]).any(), "wrote past N"
    acc = A[:, :K].astype(np.float64) @ W[:, :K].astype(np.float64).T
    return out[:, :N], acc, sa, sw, g.gemm_last_plan()


def expect(acc, sa, sw):
    with np.errstate(invalid="ignore"):
        return bf16_of(acc.astype(np.float32) * sa[:, None] * sw[None, :])


# single tokens, decode batches, ragged widths, lengths of one, k-steps cut anywhere, both tile
# sizes, K split, and products cut in two
SHAPES = [(1, 1, 1), (1, 16, 64), (1, 520, 328), (2, 1000, 1000), (3, 17, 15), (5, 129, 4097), (16, 64, 2048),
          (17, 257, 33), (33, 2056, 520), (64, 1000, 200), (64, 4096, 1024), (65, 520, 328), (127, 129, 65),
          (128, 128, 64), (129, 127, 63), (256, 256, 256), (300, 1000, 1000), (509, 2501, 1003), (1000, 1000, 1000),
          (513, 1032, 2056), (128, 256, 11008), (1031, 4099, 129), (4097, 4104, 192), (4096, 4352, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_i8_bits(M, N, K):
    C, acc, sa, sw, plan = product(M, N, K, seed=M + N + K)
    want = expect(acc, sa, sw)
    bad = np.argwhere(C != want)
    assert bad.size == 0, f"{M}x{N}x{K} {plan}: {len(bad)} differ, first {bad[0].tolist()}"


@pytest.mark.parametrize("M,N,K", [(1, 11008, 4096), (16, 4096, 11008), (64, 11008, 4096), (64, 4096, 11008)])
def test_i8_decode_full(M, N, K):
    C, acc, sa, sw, plan = product(M, N, K, seed=7)
    assert np.array_equal(C, expect(acc, sa, sw)), plan


@pytest.mark.parametrize("M,N,K,lda,ldw,ldc,off,coff", [
    (5, 13, 7, 7, 7, 13, 1, 1),              # nothing aligned
    (70, 100, 30, 30, 31, 101, 0, 0),        # leading dimensions of no multiple
    (70, 100, 30, 48, 64, 104, 0, 0),        # padded rows
    (300, 264, 160, 176, 192, 264, 0, 3),    # C off 16-byte alignment
    (300, 264, 160, 176, 192, 265, 0, 0),    # an odd ldc
    (3, 264, 160, 176, 192, 272, 0, 1),
    (300, 264, 160, 176, 192, 264, 8, 0),    # codes off 16-byte alignment
    (64, 72, 1000, 1008, 1024, 80, 0, 0)])
def test_i8_layouts(M, N, K, lda, ldw, ldc, off, coff):
    for glu in (False, True):
        C, acc, sa, sw, plan = product(M, N, K, lda, ldw, ldc, off, coff, seed=3, full=True, glu=glu)
        if glu:
            check_glu(C, acc, sa, sw, plan)
        else:
            assert np.array_equal(C, expect(acc, sa, sw)), plan


def check_glu(C, acc, sa, sw, what):
    N = C.shape[1]
    y = acc * sa[:, None].astype(np.float64) * sw[None, :].astype(np.float64)
    gate, up = y[:, :N], y[:, N:]
    with np.errstate(over="ignore"):
        silu = gate / (1 + np.exp(-gate))
    h = silu * up
    e = 2.0**-22
    slack = 1.1 * e * np.abs(gate) * np.abs(up) + e * np.abs(h) + 2.0**-20 * np.abs(h) + 2.0**-8 * np.abs(h) + 1e-38
    off = np.abs(widen(C) - h) - slack
    assert np.isfinite(widen(C)).all() and (off <= 0).all(), f"{what}: {(off > 0).sum()} outside the bound"


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 520, 328), (3, 17, 15), (16, 4096, 4096), (33, 2056, 520),
                                   (64, 1000, 200), (65, 520, 328), (129, 127, 63), (300, 1000, 1000),
                                   (509, 1251, 1003), (128, 256, 4096), (1031, 2056, 129), (4096, 2176, 256)])
def test_i8_swiglu(M, N, K):
    C, acc, sa, sw, plan = product(M, N, K, seed=M + K, glu=True)
    check_glu(C, acc, sa, sw, plan)


def test_largest_sums_do_not_overflow():
    # 128 * 128 * 131071 is the largest sum that is taken
    M, N, K = 3, 24, 131071
    A = torch.full((M, K + 1), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(32, device="cuda")
    C = poisoned(M * N)
    g.gemm_i8(M, N, K, A.data_ptr(), K + 1, one.data_ptr(), torch.full((N, K + 1), -128, dtype=torch.int8,
              device="cuda").data_ptr(), K + 1, one.data_ptr(), C.data_ptr(), N, g.current_stream_handle())
    torch.cuda.synchronize()
    assert (bits(C) == bf16_of(np.float32([128 * 128 * K]))[0]).all()


def test_empty_and_k_zero():
    one = torch.ones(16, device="cuda")
    C = poisoned(12)
    s = g.current_stream_handle()
    for fn in (g.gemm_i8, g.gemm_i8_swiglu):
        fn(0, 4, 16, None, 16, None, C.data_ptr(), 16, one.data_ptr(), None, 4, s)
        fn(3, 0, 16, C.data_ptr(), 16, one.data_ptr(), None, 16, None, None, 0, s)
        torch.cuda.synchronize()
        assert (bits(C) == 0x7FC0).all()
    nan = torch.full((16,), float("nan"), device="cuda")
    for fn in (g.gemm_i8, g.gemm_i8_swiglu):
        C = poisoned(12)
        fn(3, 4, 0, None, 0, nan.data_ptr(), None, 0, nan.data_ptr(), C.data_ptr(), 4, s)
        torch.cuda.synchronize()
        assert (bits(C) == 0).all()


@pytest.mark.parametrize("M,N,K", [(2, 40, 64), (300, 264, 160)])
def test_scales_of_zero_inf_and_nan(M, N, K):
    sa = np.ones(M, np.float32)
    sa[0], sa[-1] = 0.0, np.nan
    C, acc, sa, sw, plan = product(M, N, K, seed=5, sa=sa)
    assert (widen(C[0]) == 0).all() and np.isnan(widen(C[-1])).all()
    assert np.array_equal(C[1:-1], expect(acc, sa, sw)[1:-1])


# ---- quantisation --------------------------------------------------------------------------------


def want_codes(x):
    """Codes and scales by the definition: s = max / 127 and round(x / s), each a float32 division."""
    x = x.astype(np.float32)
    amax = np.abs(x).max(1)
    s = amax / np.float32(127)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(amax[:, None] > 0, np.rint(x / s[:, None]), 0)
    bad = ~np.isfinite(amax)
    return np.where(bad[:, None], 0, q).astype(np.int8), np.where(bad, np.float32(np.nan), s)


def quantize(xbits, K, ldx, ldq, offset=0):
    R = len(xbits)
    dX, o = place(xbits, offset)
    Qd = torch.full((max(R * ldq, 1),), 99, dtype=torch.int8, device="cuda")
    S = torch.full((R,), -1.0, device="cuda")
    g.gemm_i8_quantize(R, K, dX.data_ptr() + o, ldx, Qd.data_ptr(), ldq, S.data_ptr(), g.current_stream_handle())
    torch.cuda.synchronize()
    return Qd.cpu().numpy()[: R * ldq].reshape(R, ldq), S.cpu().numpy()


@pytest.mark.parametrize("R,K,ldx,ldq,offset", [
    (1, 1, 1, 1, 0), (1, 1, 8, 16, 0), (3, 7, 8, 16, 0), (4, 64, 64, 64, 0), (5, 505, 512, 512, 0),
    (2, 1000, 1000, 1003, 0), (3, 2048, 2048, 2048, 0), (2, 4096, 4096, 4096, 0), (3, 11008, 11008, 11008, 0),
    (2, 16384, 16384, 16384, 0), (2, 16392, 16392, 16400, 0), (3, 1000, 1001, 1008, 1), (2, 40000, 40000, 40064, 0),
    (700, 200, 208, 256, 0), (4, 9118, 9118, 9120, 0), (600, 3711, 3711, 3712, 3), (3, 20001, 20001, 20016, 5),
    (3, 65529, 65531, 65536, 7), (2, 70000, 70001, 70016, 1)])
def test_quantize_codes(R, K, ldx, ldq, offset):
    rng = np.random.default_rng(R + K)
    x = rng.normal(size=(R, ldx)).astype(np.float32)
    x[:, K:] = np.nan                                   # padding is not read
    x[0, :K] *= 2.0**100
    if R > 1:
        x[1, :K] *= np.float32(2.0**-125)               # bf16 subnormals among them
    xb = bf16_of(x)
    xb[:, K:] = 0x7FC0
    q, s = quantize(xb, K, ldx, ldq, offset)
    wq, ws = want_codes(widen(xb[:, :K]))
    assert np.array_equal(q[:, :K], wq) and np.array_equal(s, ws)
    padded = min(ldq, -(-K // 16) * 16)
    assert (q[:, K:padded] == 0).all() and (q[:, padded:] == 99).all()


def test_quantize_ties_go_to_even():
    # max 127 * 2^e: the scale is a power of two and half codes are exact
    v = np.concatenate([[127.0], np.arange(-126.5, 127, 1)]).astype(np.float32)
    for e in (-20, 0, 30):
        xb = bf16_of((v * np.float32(2.0**e))[None])
        keep = widen(xb)[0] == v * np.float32(2.0**e)   # halves above 64 need more than bf16's 8 bits
        xb = np.ascontiguousarray(xb[:, keep])
        q, s = quantize(xb, xb.shape[1], xb.shape[1], xb.shape[1])
        assert s[0] == np.float32(2.0**e) and np.array_equal(q[0], np.rint(v[keep]).astype(np.int8))


def test_quantize_every_mantissa_and_halves():
    """Every bf16 mantissa as the row's maximum, against every mantissa at six exponents, half the
    maximum among them."""
    m = np.arange(128, 256, dtype=np.float64)
    x = np.concatenate([m * 2.0**-e for e in range(1, 7)] + [-m / 2])
    x = np.concatenate([m[:, None], np.broadcast_to(x, (128, len(x)))], 1)
    x = np.where(np.abs(x) <= m[:, None], x, 0)
    xb = bf16_of(x)
    assert (widen(xb) == x).all()
    q, s = quantize(xb, x.shape[1], x.shape[1], x.shape[1])
    wq, ws = want_codes(x)
    assert np.array_equal(q, wq) and np.array_equal(s, ws)


def test_quantize_zero_inf_nan_rows():
    x = np.zeros((6, 40), np.float32)
    x[1] = 1.0
    x[2, 3], x[2, 4] = np.inf, 1.0
    x[3, 3], x[3, 4] = -np.inf, 1.0
    x[4, 39] = np.nan
    x[5, 0] = -0.0
    q, s = quantize(bf16_of(x) | (np.isnan(x) * 0x7FC0).astype(np.uint16), 40, 40, 48)
    assert (q[[0, 2, 3, 4, 5], :] == 0).all() and (q[1, :40] == 127).all()
    assert s[0] == 0 and s[5] == 0 and np.isnan(s[[2, 3, 4]]).all() and s[1] == np.float32(1) / np.float32(127)


def test_quantize_empty():
    S = torch.full((3,), -1.0, device="cuda")
    g.gemm_i8_quantize(3, 0, None, 0, None, 0, S.data_ptr(), g.current_stream_handle())
    torch.cuda.synchronize()
    assert (S == 0).all()


# ---- products from bf16 activations ----------------------------------------------------------------


def act(M, K, seed, ld=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, ld or K, generator=gen)
    x[:, ::61] *= 20
    return x.bfloat16().cuda()[:, :K]


@pytest.mark.parametrize("M,N,K,ld", [(1, 520, 328, None), (2, 11008, 4096, None), (3, 40, 33, None), (5, 24, 1000, 1001),
                                      (16, 4096, 4096, None), (17, 264, 20000, None), (64, 1000, 4104, None),
                                      (300, 1000, 1000, 1008), (1100, 520, 328, None), (1, 17, 7, 8),
                                      (2, 40, 1000, 1008), (1, 1000, 16384, None), (2, 24, 16392, None),
                                      (2, 4096, 11008, None), (1, 72, 4104, 4112), (7, 75, 3711, None),
                                      (2, 520, 9118, None), (1, 75, 3711, None)])
def test_dynamic_equals_quantize_then_product(M, N, K, ld):
    A = act(M, K, M + K, ld)
    W = (torch.randn(2 * N, K, generator=torch.Generator().manual_seed(N)) * 0.02).bfloat16().cuda()
    Wq, Sw = g.i8_quantize(W)
    Aq, Sa = g.i8_quantize(A)
    for dyn, stat, w, s in ((g.i8_linear, g.i8_matmul, Wq[:N], Sw[:N]),
                            (g.i8_swiglu_linear, g.i8_swiglu_matmul, Wq, Sw)):
        want = stat(Aq, Sa, w, s)
        work = torch.full((g.gemm_i8_work_bytes(M, K) + 48,), 77, dtype=torch.uint8, device="cuda")
        for got in (dyn(A, w, s), dyn(A, w, s, work=work)):
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert (work[g.gemm_i8_work_bytes(M, K):] == 77).all()
    acc = Aq.cpu().numpy().astype(np.float64) @ Wq[:N].cpu().numpy().astype(np.float64).T
    got = g.i8_linear(A, Wq[:N], Sw[:N])
    assert np.array_equal(bits(got), expect(acc, Sa.cpu().numpy(), Sw[:N].cpu().numpy()))


def test_a_token_at_any_address():
    """One token whose row starts at an odd element: its bits are those of a copy."""
    A = act(8, 1001, 5)
    Wq, Sw = g.i8_quantize((torch.randn(520, 1001, generator=torch.Generator().manual_seed(6)) * 0.02).bfloat16().cuda())
    for r in range(8):
        for f in (g.i8_linear, g.i8_swiglu_linear):
            got, want = f(A[r : r + 1], Wq, Sw), f(A[r : r + 1].clone(), Wq, Sw)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_non_finite_token_gives_nan_outputs_only_in_its_row():
    for M in (3, 200):
        A = act(M, 264, 1)
        A[1, 7] = float("inf")
        W = (torch.randn(40, 264, generator=torch.Generator().manual_seed(2)) * 0.02).bfloat16().cuda()
        Wq, Sw = g.i8_quantize(W)
        y = g.i8_linear(A, Wq, Sw)
        assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def test_streams_graphs_and_repeats():
    """A side stream, two streams at once, and a replayed graph give the bits of an eager call."""
    cases = []
    for M, N, K in ((3, 4096, 4096), (64, 1000, 2056), (300, 520, 4096)):
        A = act(M, K, K)
        Wq, Sw = g.i8_quantize((torch.randn(2 * N, K, generator=torch.Generator().manual_seed(N)) * 0.02).bfloat16().cuda())
        out, work = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(
            g.gemm_i8_work_bytes(M, K), dtype=torch.uint8, device="cuda")
        cases.append((A, Wq, Sw, out, work, g.i8_swiglu_linear(A, Wq, Sw).clone()))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        outs = []
        for A, Wq, Sw, _, _, _ in cases:
            for s in (s1, s2):
                with torch.cuda.stream(s):
                    outs.append(g.i8_swiglu_linear(A, Wq, Sw))
        torch.cuda.synchronize()
        for i, y in enumerate(outs):
            assert torch.equal(y.view(torch.int16), cases[i // 2][5].view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for A, Wq, Sw, out, work, _ in cases:
            g.i8_swiglu_linear(A, Wq, Sw, out=out, work=work)
    for _ in range(4):
        for c in cases:
            c[3].fill_(float("nan"))
        g.i8_linear(cases[0][0], cases[0][1], cases[0][2])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for c in cases:
            assert torch.equal(c[3].view(torch.int16), c[5].view(torch.int16))


def test_refusals_on_the_device():
    A = act(4, 64, 1)
    Wq, Sw = g.i8_quantize(act(24, 64, 2))
    with pytest.raises(ValueError):
        g.i8_linear(A[:, :32], Wq, Sw)
    with pytest.raises(ValueError):
        g.i8_linear(A, Wq, Sw[:23])
    with pytest.raises(ValueError):
        g.i8_swiglu_linear(A, Wq[:23], Sw[:23])
    with pytest.raises(ValueError):
        g.i8_linear(A.t(), Wq, Sw)
    with pytest.raises(ValueError):
        g.i8_linear(A, Wq, Sw, out=torch.empty(4, 23, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(g.GemmError):
        g.i8_linear(A, Wq, Sw, work=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M,N", [(1 << 24, 1 << 12), (1 << 18, 1 << 18), (1 << 62, 1 << 61)])
def test_general_outputs_beyond_a_grid_are_refused(M, N):
    """Unaligned operands whose output has 2^24 or more 64 x 64 tiles: refused on the host, before a launch."""
    p, q = ctypes.c_void_p(66), ctypes.c_void_p(64)
    lib, s = g.lib(), g.current_stream_handle()
    assert lib.gemm_i8(M, N, 8, p, 9, q, p, 9, q, q, N, s) == g.GEMM_ERR_UNSUPPORTED
    assert lib.gemm_bf16_bwd(8, N, M, p, N + 1, p, M + 1, None, N, None, M, p, N + 1, s) == g.GEMM_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    """Activations, codes and outputs of more than 2^32 bytes: the last rows are the first ones."""
    M, N, K = 1_060_003, 2056, 4104
    gen = torch.Generator(device="cuda").manual_seed(1)
    head = torch.randn(64, K, generator=gen, device="cuda").bfloat16()
    A = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    A[:64] = head
    A[-64:] = head
    Wq, Sw = g.i8_quantize((torch.randn(N, K, generator=gen, device="cuda") * 0.02).bfloat16())
    Aq, Sa = g.i8_quantize(A)
    assert torch.equal(Aq[-64:], Aq[:64]) and torch.equal(Sa[-64:], Sa[:64])
    del A
    C = g.i8_matmul(Aq, Sa, Wq, Sw)
    assert C.numel() * 2 > 1 << 32 and Aq.numel() > 1 << 32
    assert torch.equal(C[-64:], C[:64]) and not C[64:-64].any()
    acc = Aq[:64].cpu().numpy().astype(np.float64) @ Wq.cpu().numpy().astype(np.float64).T
    assert np.array_equal(bits(C[:64]), expect(acc, Sa[:64].cpu().numpy(), Sw.cpu().numpy()))


def test_memory_belongs_to_the_stream_given():
    """With a stream's handle, new outputs and the work buffer come from that stream's memory: the work
    buffer is dropped when the call returns, and another stream's memory could be given out again then."""
    A, (Wq, Sw) = act(2048, 4096, 1), g.i8_quantize(act(24, 4096, 2))
    want = g.i8_linear(A, Wq, Sw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    def segments():
        return [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]

    def owns(t):
        return any(s["address"] <= t.data_ptr() < s["address"] + s["total_size"] for s in segments())

    assert not segments()
    here = torch.cuda.current_stream()
    out = torch.empty_like(want)
    C = g.i8_linear(A, Wq, Sw, out=out, stream=side.cuda_stream)
    assert C is out or C.data_ptr() == out.data_ptr()
    assert sum(s["total_size"] for s in segments()) >= g.gemm_i8_work_bytes(2048, 4096)
    D = g.i8_linear(A, Wq, Sw, stream=ctypes.c_void_p(side.cuda_stream))
    Aq, Sa = g.i8_quantize(A, stream=side.cuda_stream)
    E = g.i8_matmul(Aq, Sa, Wq, Sw, stream=side.cuda_stream)
    F, GU = g.swiglu_forward(A, A.view(4096, 2048), stream=side.cuda_stream)
    dA, dB, dGU = g.swiglu_backward(F, GU, A, A.view(4096, 2048), stream=side.cuda_stream)
    lA, lB = g.matmul_backward(C, A, A.view(4096, 2048)[:, :24], stream=side.cuda_stream)
    for t in (D, Aq, Sa, E, F, GU, dA, dB, dGU, lA, lB):
        assert owns(t)
    assert not owns(out) and torch.cuda.current_stream() == here
    assert not owns(g.i8_linear(A, Wq, Sw))  # and the current stream is what it was
    with pytest.raises(ValueError):
        g.i8_linear(A, Wq, Sw, out=out[:, :23], stream=side.cuda_stream)
    assert torch.cuda.current_stream() == here
    torch.cuda.synchronize()
    for t in (C, D, E):
        assert torch.equal(t.view(torch.int16), want.view(torch.int16))


def test_helpers_keep_references_and_take_streams():
    """The helpers neither leak nor lose a reference, and take a stream as a handle of either kind."""
    import sys

    A, (Wq, Sw) = act(3, 64, 1), g.i8_quantize(act(24, 64, 2))
    out = torch.empty(3, 24, dtype=torch.bfloat16, device="cuda")
    want = g.i8_linear(A, Wq, Sw)
    counts = [sys.getrefcount(x) for x in (A, Wq, Sw, out, None)]
    before = torch.cuda.memory_allocated()
    for _ in range(200):
        g.i8_linear(A, Wq, Sw)
        y = g.i8_linear(A, Wq, Sw, out=out)
        assert y is out
        with pytest.raises(ValueError):
            g.i8_linear(A, Wq, Sw[:5])
        with pytest.raises(g.GemmError):
            g.i8_linear(A, Wq, Sw, work=torch.empty(16, dtype=torch.uint8, device="cuda"))
    del y
    after = [sys.getrefcount(x) for x in (A, Wq, Sw, out, None)]
    assert after[:4] == counts[:4] and abs(after[4] - counts[4]) < 50
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side.cuda_stream, ctypes.c_void_p(side.cuda_stream)):
        out.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        g.i8_linear(A, Wq, Sw, out=out, stream=handle)
        side.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    with pytest.raises(AttributeError):
        g.i8_linear(A, Wq, Sw, stream="s")


@pytest.mark.parametrize("M", [1, 20, 130])
def test_gates_below_the_normal_range(M):
    """Gates at which the sigmoid is below float32's normal range (g < -87.3) while silu(g) u is not:
    silu(g) carries 2^-20 of its size and float32's smallest step 2^-149, which u multiplies; g is exact
    and the rounding to bf16 adds 2^-8 of the result."""
    gates = np.array([-87.0, -87.5, -88.0, -88.5, -89.0, -91.0, -95.0, -100.0])
    N, K, up = len(gates), 5, 2.0**100
    W = np.zeros((2 * N, 16), np.int8)
    W[:, 0] = 1
    sw = np.concatenate([gates, np.full(N, up)]).astype(np.float32)   # codes of one: the scale is the product
    sa = np.ones(M, np.float32)
    s = gates / (1 + np.exp(-gates))
    slack = 2.0**-8 * np.abs(s * up) + (2.0**-20 * np.abs(s) + 2.0**-149) * up
    for ld in (16, 17):     # the matrix kernels, and the general one
        A = np.zeros((M, ld), np.int8)
        A[:, 0] = 1
        (dA, _), (dW, _), (dsa, _), (dsw, _) = place(A), place(W), place(sa), place(sw)
        C = poisoned(M * N)
        g.gemm_i8_swiglu(M, N, K, dA.data_ptr(), ld, dsa.data_ptr(), dW.data_ptr(), 16, dsw.data_ptr(), C.data_ptr(), N,
                         g.current_stream_handle())
        torch.cuda.synchronize()
        off = np.abs(widen(bits(C)).reshape(M, N) - s * up) - slack
        assert (off <= 0).all(), (g.gemm_last_plan()["kernel"], gates[(off > 0).any(0)])


def test_a_refused_call_leaves_its_work_buffer_as_it_was():
    """A product that the general kernel's grid does not hold: refused before the activations are quantised."""
    M, N = 1 << 23, 1 << 13
    A, W = torch.ones(M, 1, dtype=torch.bfloat16, device="cuda"), torch.ones(N, 1, dtype=torch.int8, device="cuda")
    Sw = torch.ones(N, device="cuda")
    work = torch.full((g.gemm_i8_work_bytes(M, 1),), 77, dtype=torch.uint8, device="cuda")
    st = g.lib().gemm_i8_bf16(M, N, 1, A.data_ptr(), 1, W.data_ptr(), 1, Sw.data_ptr(), 64, N, work.data_ptr(), work.numel(),
                              g.current_stream_handle())
    torch.cuda.synchronize()
    assert st == g.GEMM_ERR_UNSUPPORTED and bool((work == 77).all())


def test_quantize_rows_past_one_grid():
    """2^22 + 3 rows of more than 16384 elements, 1024 threads each: more threads than one launch holds. Rows
    on both sides of every launch's end get their codes; the others, zeros, get zeros."""
    R, K = (1 << 22) + 3, 16385
    ld = 16392
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 220 << 30:
        pytest.skip("needs 206 GB of device memory")
    some = [0, 1, (1 << 22) - 2, (1 << 22) - 1, 1 << 22, R - 1]
    rng = np.random.default_rng(1)
    xb = bf16_of(rng.normal(size=(len(some), K)))
    wq, ws = want_codes(widen(xb))
    X = torch.zeros(R, ld, dtype=torch.bfloat16, device="cuda")
    X[some, :K] = torch.from_numpy(xb.view(np.int16)).view(torch.bfloat16).cuda()
    Q = torch.full((R, ld), 99, dtype=torch.int8, device="cuda")
    S = torch.full((R,), -1.0, device="cuda")
    g.gemm_i8_quantize(R, K, X.data_ptr(), ld, Q.data_ptr(), ld, S.data_ptr(), g.current_stream_handle())
    torch.cuda.synchronize()
    assert np.array_equal(Q[some, :K].cpu().numpy(), wq) and np.array_equal(S[some].cpu().numpy(), ws)
    assert int((S != 0).sum()) == len(some) and not Q[some, K:].any()
    for r in range(0, R, 1 << 19):
        rows = Q[r: r + (1 << 19)].view(torch.int64).any(1)
        assert [r + i for i in rows.nonzero().flatten().tolist()] == [i for i in some if r <= i < r + (1 << 19)]
    del X, Q, S
    torch.cuda.empty_cache()


def test_an_output_that_does_not_fit_raises_what_torch_raises():
    """torch.OutOfMemoryError, which callers catch to free memory and try again; the next call runs."""
    n = 1 << 20                                            # outputs of 2^41 bytes
    q, s = torch.ones(n, 16, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda")
    x = torch.ones(n, 16, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: g.i8_matmul(q, s, q, s), lambda: g.i8_linear(x, q, s), lambda: g.i8_swiglu_linear(x, q, s),
                 lambda: g.swiglu_forward(x, x.view(16, n))):
        with pytest.raises(torch.OutOfMemoryError):
            call()
    assert bool((g.i8_matmul(q[:2], s[:2], q, s) == 16).all())


# M, N, K, gated, and the streaming kernel it takes on 256 CUs: (16-row tiles of M, weight tiles a
# workgroup, waves), each with K whole and in pieces where a shape can have both
STREAMED = [
    (2, 40, 100, False, (1, 1, 4)), (5, 520, 2100, False, (1, 1, 4)), (4, 4100, 8200, False, (1, 1, 8)),
    (4, 1000, 9001, False, (1, 1, 8)), (16, 8300, 1000, False, (1, 4, 4)), (9, 9000, 1021, False, (1, 4, 4)),
    (3, 1000, 1030, True, (1, 2, 4)), (16, 200, 4100, True, (1, 2, 4)),
    (17, 300, 1000, False, (2, 1, 4)), (31, 200, 4099, False, (2, 1, 4)), (20, 333, 8200, False, (2, 1, 8)),
    (17, 2000, 5000, False, (2, 2, 4)), (32, 11000, 900, False, (2, 2, 4)), (17, 5120, 4100, False, (2, 4, 8)),
    (32, 20001, 1100, False, (2, 4, 8)),
    (33, 300, 1000, False, (3, 1, 4)), (47, 200, 4099, False, (3, 1, 4)), (40, 333, 8200, False, (3, 1, 8)),
    (33, 1500, 6001, False, (3, 2, 4)), (40, 9000, 1000, False, (3, 2, 4)), (33, 3000, 10001, False, (3, 4, 8)),
    (48, 20500, 1040, False, (3, 4, 8)),
    (49, 300, 1000, False, (4, 1, 4)), (64, 200, 4099, False, (4, 1, 4)), (60, 333, 8200, False, (4, 1, 8)),
    (49, 1400, 9001, False, (4, 2, 4)), (64, 10000, 1000, False, (4, 2, 4)), (61, 2056, 10500, False, (4, 4, 8)),
    (64, 20501, 1040, False, (4, 4, 8)),
    (17, 100, 3000, True, (2, 2, 4)), (30, 2000, 500, True, (2, 2, 4)), (17, 2056, 8200, True, (2, 4, 4)),
    (32, 10300, 1040, True, (2, 4, 4)), (33, 100, 3000, True, (3, 2, 4)), (48, 2000, 500, True, (3, 2, 4)),
    (33, 2056, 8200, True, (3, 4, 4)), (48, 10301, 1040, True, (3, 4, 4)), (49, 100, 3000, True, (4, 2, 4)),
    (64, 2000, 500, True, (4, 2, 4)), (49, 1400, 9001, True, (4, 4, 4)), (64, 10300, 1040, True, (4, 4, 4))]


@pytest.mark.parametrize("M,N,K,glu,kernel", STREAMED)
def test_every_streaming_kernel(M, N, K, glu, kernel):
    C, acc, sa, sw, plan = product(M, N, K, ldc=N + 3, seed=M + N, full=True, glu=glu)
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert (plan["kernel"], plan["mtiles"], plan["strip"] // 16, plan["threads"] // 64) == ("i8_decode", *kernel)
    if glu:
        check_glu(C, acc, sa, sw, plan)
    else:
        assert np.array_equal(C, expect(acc, sa, sw)), plan


# 256 x 256 tiles in a partial wave and in full waves with the last one cut off across columns or rows,
# ragged in every size, over odd and even numbers of k-steps that go round the five-slot rings
LARGE = [(2300, 4090, 700, None), (2300, 4090, 1000, None), (4090, 4350, 1000, "n"), (4350, 4090, 1000, "m")]


@pytest.mark.parametrize("M,N,K,cut", LARGE)
@pytest.mark.parametrize("glu", [False, True])
def test_large_tiles_over_many_steps(M, N, K, cut, glu):
    C, acc, sa, sw, plan = product(M, N // 2 if glu else N, K, seed=K + M, glu=glu)
    assert plan["kernel"] == "tile" and plan["bm"] == 256
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert plan.get("cut", {}).get("axis") == cut, plan
    if glu:
        check_glu(C, acc, sa, sw, plan)
    else:
        assert np.array_equal(C, expect(acc, sa, sw)), plan


@pytest.mark.parametrize("M,N,K", [(1400, 2040, 12900), (1400, 2040, 9000)])
def test_two_pieces_on_most_cus(M, N, K):
    """176 tiles of 128 x 128: two pieces of 102 k-steps for 202 of them, whole for 141."""
    for glu in (False, True):
        C, acc, sa, sw, plan = product(M, N // 2 if glu else N, K, seed=K, glu=glu)
        assert plan["bm"] == 128
        if torch.cuda.get_device_properties(0).multi_processor_count == 256:
            assert (plan["splits"], plan["kt_per_split"]) == ((2, 102) if K == 12900 else (1, 141))
        if glu:
            check_glu(C, acc, sa, sw, plan)
        else:
            assert np.array_equal(C, expect(acc, sa, sw)), plan
