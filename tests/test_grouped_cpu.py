"""The 8-bit floating-point and grouped entry points on a machine without a GPU: refusals are made on the host
before any HIP call, empty outputs are accepted, and the binding's helpers check their tensors."""

import ctypes

import numpy as np
import pytest

import gemv_layers_amd as g
from grouping import e4m3_round, e4m3_values, spans

OK, BAD, UNSUP, NOINIT = (g.GEMM_OK, g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED,
                          g.GEMM_ERR_NOT_INITIALIZED)
P = ctypes.c_void_p(64)  # a non-null, aligned stand-in; never dereferenced here
Q = ctypes.c_void_p(66)  # 2-byte aligned only
X = ctypes.c_void_p(65)  # odd


@pytest.mark.parametrize("args,status", [
    # R, K, X, ldx, Q, ldq, S, lds
    ((-1, 8, P, 8, P, 8, P, 4), BAD),
    ((4, -8, P, 8, P, 8, P, 4), BAD),
    ((4, 8, P, 7, P, 8, P, 4), BAD),
    ((4, 8, P, 8, P, 7, P, 4), BAD),
    ((4, 8, P, 8, P, 8, P, 3), BAD),          # lds < R
    ((4, 8, None, 8, P, 8, P, 4), BAD),
    ((4, 8, P, 8, None, 8, P, 4), BAD),
    ((4, 8, P, 8, P, 8, None, 4), BAD),
    ((4, 8, P, 8, P, 8, Q, 4), BAD),          # scales not 4-byte aligned
    ((4, 8, X, 8, P, 8, P, 4), BAD),          # bf16 at an odd address
    ((1 << 24, 8, P, 8, P, 8, P, 1 << 24), UNSUP),
    ((4, (1 << 30) + 1, P, 1 << 31, P, 1 << 31, P, 4), UNSUP),
    ((0, 8, None, 8, None, 8, None, 0), OK),
    ((4, 0, None, 0, None, 0, None, 4), OK),
    ((4, 8, Q, 8, X, 8, P, 4), NOINIT),       # any alignment of codes is taken
])
def test_quantize_refusals(args, status):
    assert g.lib().gemm_f8_quantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # E, N, K, W, ldw, stride_w, Q, ldq, stride_q, S, lds, stride_s
    ((2, 200, 300, P, 300, 60000, P, 304, 60800, P, 3, 6), NOINIT),
    ((2, 200, 300, P, 300, 0, P, 304, 60800, P, 3, 6), NOINIT),       # one weight twice
    ((2, 200, 300, P, 300, 60000, P, 304, 60799, P, 3, 6), BAD),      # the codes would meet
    ((2, 200, 300, P, 300, 60000, P, 304, 60800, P, 3, 5), BAD),      # the scales would meet
    ((1, 200, 300, P, 300, 0, P, 304, 0, P, 3, 0), NOINIT),
    ((2, 200, 300, P, 300, -1, P, 304, 60800, P, 3, 6), BAD),
    ((2, 200, 300, P, 299, 60000, P, 304, 60800, P, 3, 6), BAD),
    ((2, 200, 300, P, 300, 60000, P, 299, 60800, P, 3, 6), BAD),
    ((2, 200, 300, P, 300, 60000, P, 304, 60800, P, 2, 6), BAD),
    ((-1, 200, 300, P, 300, 60000, P, 304, 60800, P, 3, 6), BAD),
    ((2, 200, 300, None, 300, 60000, P, 304, 60800, P, 3, 6), BAD),
    ((2, 200, 300, X, 300, 60000, P, 304, 60800, P, 3, 6), BAD),
    ((2, 200, 300, P, 300, 60000, P, 304, 60800, Q, 3, 6), BAD),
    ((65537, 1, 1, P, 1, 1, P, 1, 1, P, 1, 1), UNSUP),
    ((1, 1 << 24, 8, P, 8, 0, P, 8, 0, P, 1, 0), UNSUP),
    ((0, 200, 300, None, 300, 0, None, 304, 0, None, 3, 0), OK),
])
def test_quantize_weight_refusals(args, status):
    assert g.lib().gemm_f8_quantize_weight(*args, None) == status


F8 = [
    # M, N, K, Aq, ldaq, Sa, ldsa, Wq, ldwq, Sw, ldsw, C, ldc
    ((8, 8, 200, P, 208, P, 8, P, 208, P, 2, P, 8), NOINIT),
    ((8, 8, 200, X, 201, P, 8, X, 203, P, 2, Q, 8), NOINIT),     # any alignment of codes is taken
    ((-1, 8, 200, P, 208, P, 8, P, 208, P, 2, P, 8), BAD),
    ((8, -1, 200, P, 208, P, 8, P, 208, P, 2, P, 8), BAD),
    ((8, 8, -1, P, 208, P, 8, P, 208, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 199, P, 8, P, 208, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 7, P, 208, P, 2, P, 8), BAD),        # ldsa < M
    ((8, 8, 200, P, 208, P, 8, P, 199, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 8, P, 208, P, 1, P, 8), BAD),        # ldsw < 2 blocks
    ((8, 8, 200, P, 208, P, 8, P, 208, P, 2, P, 7), BAD),
    ((8, 8, 200, None, 208, P, 8, P, 208, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, None, 8, P, 208, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 8, None, 208, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 8, P, 208, None, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 8, P, 208, P, 2, None, 8), BAD),
    ((8, 8, 200, P, 208, Q, 8, P, 208, P, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 8, P, 208, Q, 2, P, 8), BAD),
    ((8, 8, 200, P, 208, P, 8, P, 208, P, 2, X, 8), BAD),
    ((1 << 24, 8, 200, P, 208, P, 1 << 24, P, 208, P, 2, P, 8), UNSUP),
    ((8, 8, (1 << 30) + 1, P, 1 << 31, P, 8, P, 1 << 31, P, 1 << 24, P, 8), UNSUP),
    ((0, 8, 200, None, 208, None, 0, P, 208, P, 2, None, 8), OK),
    ((8, 0, 200, P, 208, P, 8, None, 208, None, 2, None, 0), OK),
    ((8, 8, 0, None, 0, None, 8, None, 0, None, 0, P, 8), NOINIT),
]


@pytest.mark.parametrize("args,status", F8)
def test_f8_refusals(args, status):
    assert g.lib().gemm_f8(*args, None) == status


@pytest.mark.parametrize("args,status", F8)
@pytest.mark.parametrize("E", [1, 7])
def test_f8_grouped_refusals(args, status, E):
    M, N, K, Aq, ldaq, Sa, ldsa, Wq, ldwq, Sw, ldsw, C, ldc = args
    assert g.lib().gemm_f8_grouped(M, N, K, E, Aq, ldaq, Sa, ldsa, Wq, ldwq, 8 * 208, Sw, ldsw, 2, P, C, ldc,
                                   None) == status


GROUPS = [
    # E, stride of the weights, offsets
    ((3, 64, P), NOINIT), ((3, 0, P), NOINIT), ((-1, 64, P), BAD), ((3, -8, P), BAD), ((3, 64, None), BAD),
    ((3, 64, Q), BAD), ((65536, 64, P), NOINIT), ((65537, 64, P), UNSUP),
]


@pytest.mark.parametrize("groups,status", GROUPS)
def test_group_refusals(groups, status):
    E, stride, offsets = groups
    L = g.lib()
    assert L.gemm_bf16_grouped(8, 8, 8, E, P, 8, P, 8, stride, offsets, P, 8, None) == status
    assert L.gemm_bf16_grouped_bwd(8, 8, 8, E, P, 8, P, 8, P, 8, stride, offsets, P, 8, P, 8, 64, None) == status
    assert L.gemm_f8_grouped(8, 8, 8, E, P, 16, P, 8, P, 16, stride, P, 1, 1, offsets, P, 8, None) == status
    assert L.gemm_f8_grouped_bf16(8, 8, 8, E, P, 8, P, 16, stride, P, 1, 1, offsets, P, 8, P, 1 << 20, None) == status


@pytest.mark.parametrize("args,status", [
    # M, N, K, A, lda, B, ldb, C, ldc
    ((-1, 8, 8, P, 8, P, 8, P, 8), BAD), ((8, -1, 8, P, 8, P, 8, P, 8), BAD), ((8, 8, -1, P, 8, P, 8, P, 8), BAD),
    ((8, 8, 8, P, 7, P, 8, P, 8), BAD), ((8, 8, 8, P, 8, P, 7, P, 8), BAD), ((8, 8, 8, P, 8, P, 8, P, 7), BAD),
    ((8, 8, 8, None, 8, P, 8, P, 8), BAD), ((8, 8, 8, P, 8, None, 8, P, 8), BAD), ((8, 8, 8, P, 8, P, 8, None, 8), BAD),
    ((8, 8, 8, X, 8, P, 8, P, 8), BAD), ((8, 8, 8, P, 8, X, 8, P, 8), BAD), ((8, 8, 8, P, 8, P, 8, X, 8), BAD),
    ((8, 8, 8, Q, 9, Q, 11, Q, 13), NOINIT), ((1 << 24, 8, 8, P, 8, P, 8, P, 8), UNSUP),
    ((8, 8, (1 << 30) + 1, P, 1 << 31, P, 8, P, 8), UNSUP),
    ((0, 8, 8, None, 8, P, 8, None, 8), OK), ((8, 0, 8, P, 8, None, 0, None, 0), OK),
    ((8, 8, 0, None, 0, None, 8, P, 8), NOINIT),
])
def test_grouped_refusals(args, status):
    M, N, K, A, lda, B, ldb, C, ldc = args
    assert g.lib().gemm_bf16_grouped(M, N, K, 3, A, lda, B, ldb, 64, P, C, ldc, None) == status


@pytest.mark.parametrize("args,status", [
    # M, N, K, E, dC, lddc, A, lda, B, ldb, stride_b, offsets, dA, ldda, dB, lddb, stride_db
    ((8, 8, 8, 3, P, 8, P, 8, P, 8, 64, P, P, 8, P, 8, 64), NOINIT),
    ((8, 8, 8, 3, P, 7, P, 8, P, 8, 64, P, P, 8, P, 8, 64), BAD),
    ((8, 8, 8, 3, None, 8, P, 8, P, 8, 64, P, P, 8, P, 8, 64), BAD),
    ((8, 8, 8, 3, P, 8, None, 8, P, 8, 64, P, P, 8, P, 8, 64), BAD),
    ((8, 8, 8, 3, P, 8, P, 8, None, 8, 64, P, P, 8, P, 8, 64), BAD),
    ((8, 8, 8, 3, P, 8, P, 8, P, 8, 64, P, P, 7, P, 8, 64), BAD),
    ((8, 8, 8, 3, P, 8, P, 8, P, 8, 64, P, P, 8, P, 7, 64), BAD),
    ((8, 8, 8, 3, P, 8, P, 8, P, 8, 64, P, P, 8, P, 8, 63), BAD),           # the gradients would meet
    ((8, 8, 8, 1, P, 8, P, 8, P, 8, 64, P, P, 8, P, 8, 0), NOINIT),
    ((8, 8, 8, 3, P, 8, None, 0, P, 8, 64, P, P, 8, None, 0, 0), NOINIT),   # dA alone: A is not read
    ((8, 8, 8, 3, P, 8, P, 8, None, 0, 64, P, None, 0, P, 8, 64), NOINIT),  # dB alone: B is not read
    ((8, 8, 8, 3, P, 8, None, 0, None, 0, 64, P, None, 0, None, 0, 0), OK),
    ((8, 8, 8, 3, X, 8, P, 8, P, 8, 64, P, P, 8, P, 8, 64), BAD),
    ((8, 8, 8, 3, P, 8, P, 8, P, 8, 64, P, X, 8, P, 8, 64), BAD),
    ((8, 8, 8, 3, P, 8, P, 8, P, 8, 64, P, P, 8, X, 8, 64), BAD),
    ((0, 8, 8, 3, None, 8, None, 8, P, 8, 64, None, P, 8, P, 8, 64), NOINIT),  # dB is zero
    ((8, 0, 8, 3, None, 0, P, 8, None, 0, 64, P, P, 8, P, 0, 64), NOINIT),     # dA is zero
    ((8, 8, 0, 3, P, 8, None, 0, None, 8, 64, P, P, 0, P, 8, 64), OK),
    ((8, 8, 8, 0, P, 8, P, 8, None, 8, 64, None, P, 8, P, 8, 64), NOINIT),     # no groups: dA is zero
])
def test_grouped_bwd_refusals(args, status):
    assert g.lib().gemm_bf16_grouped_bwd(*args, None) == status


@pytest.mark.parametrize("work,size,status", [(P, 5 * 16 + 5 * 4, NOINIT), (P, 5 * 16 + 5 * 4 - 1, BAD), (None, 1 << 20, BAD),
                                              (ctypes.c_void_p(72), 1 << 20, BAD)])
def test_work_buffer(work, size, status):
    L = g.lib()
    assert L.gemm_f8_bf16(5, 8, 8, P, 8, P, 16, P, 1, P, 8, work, size, None) == status
    assert L.gemm_f8_grouped_bf16(5, 8, 8, 2, P, 8, P, 16, 128, P, 1, 1, P, P, 8, work, size, None) == status
    assert L.gemm_f8_bf16(5, 8, 8, X, 8, P, 16, P, 1, P, 8, P, 1 << 20, None) == BAD    # bf16 at an odd address
    assert L.gemm_f8_bf16(0, 8, 8, None, 8, P, 16, P, 1, None, 8, None, 0, None) == OK


def test_work_bytes():
    assert g.gemm_f8_work_bytes(4, 8) == 4 * 16 + 4 * 4
    assert g.gemm_f8_work_bytes(3, 257) == 3 * 272 + 3 * 3 * 4
    assert g.gemm_f8_work_bytes(0, 8) == 0
    n = ctypes.c_int64()
    L = g.lib()
    assert L.gemm_f8_work_bytes(-1, 8, ctypes.byref(n)) == BAD
    assert L.gemm_f8_work_bytes(1, 8, None) == BAD
    assert L.gemm_f8_work_bytes(1 << 24, 8, ctypes.byref(n)) == UNSUP
    assert L.gemm_f8_work_bytes(1, (1 << 30) + 1, ctypes.byref(n)) == UNSUP


def test_spans_of_any_offsets():
    assert spans([0, 3, 3, 8], 8) == [(0, 0, 3), (1, 3, 3), (2, 3, 8)]
    assert spans([2, 5, 7], 9) == [(0, 2, 5), (1, 5, 7)]
    assert spans([-4, 6, 2, 99], 8) == [(0, 0, 6), (1, 6, 6), (2, 6, 8)]


def test_e4m3_of_the_tests():
    torch = pytest.importorskip("torch")
    v = e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(v, t, equal_nan=True)
    x = np.random.default_rng(0).uniform(-448, 448, 10000) * np.exp2(-np.random.default_rng(1).integers(0, 18, 10000))
    x = np.concatenate([x, (v[1:127] + v[:126]) / 2])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(e4m3_round(x.astype(np.float32).astype(np.float64)), want)


# ---- helpers ------------------------------------------------------------------------------------------

torch = pytest.importorskip("torch")
BF = torch.zeros(4, 8, dtype=torch.bfloat16)
BF3 = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
F = torch.zeros(4, 8).to(torch.float8_e4m3fn)
F3 = torch.zeros(2, 4, 8).to(torch.float8_e4m3fn)
SA, SW, SW3 = torch.zeros(1, 4), torch.zeros(1, 1), torch.zeros(2, 1, 1)
OFF = torch.zeros(3, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: g.f8_quantize(F), lambda: g.f8_quantize(None), lambda: g.f8_quantize_weight(BF.float()),
    lambda: g.f8_matmul(BF, SA, F, SW), lambda: g.f8_matmul("x", SA, F, SW), lambda: g.f8_linear(F, F, SW),
    lambda: g.grouped_matmul(BF.half(), BF3, OFF), lambda: g.grouped_matmul(3, BF3, OFF),
    lambda: g.grouped_matmul_backward(BF, BF.float(), BF3, OFF), lambda: g.f8_grouped_matmul(BF, SA, F3, SW3, OFF),
    lambda: g.f8_grouped_linear(BF.float(), F3, SW3, OFF)])
def test_types(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call", [
    lambda: g.f8_quantize(BF), lambda: g.f8_quantize(BF[0]), lambda: g.f8_quantize_weight(BF),
    lambda: g.f8_quantize_weight(BF3), lambda: g.f8_quantize_weight(BF[0]), lambda: g.f8_matmul(F, SA, F, SW),
    lambda: g.f8_linear(BF, F, SW), lambda: g.grouped_matmul(BF, BF3, OFF),
    lambda: g.grouped_matmul_backward(BF, BF, BF3, OFF), lambda: g.f8_grouped_matmul(F, SA, F3, SW3, OFF),
    lambda: g.f8_grouped_linear(BF, F3, SW3, OFF)])
def test_host_tensors_and_shapes(call):
    with pytest.raises(ValueError):
        call()


def grad(t):
    return t.clone().requires_grad_()


@pytest.mark.parametrize("call,name", [
    (lambda: g.grouped_matmul(grad(BF), BF3, OFF), "A"), (lambda: g.f8_linear(grad(BF), F, SW), "A"),
    (lambda: g.grouped_matmul_backward(BF, grad(BF), BF3, OFF), "A"),
    (lambda: g.f8_grouped_linear(grad(BF), F3, SW3, OFF), "A")])
def test_a_graph_is_not_lost_without_a_word(call, name):
    with pytest.raises(RuntimeError, match=f"{name} requires grad"):
        call()


def test_argument_counts():
    m = g._load_ops()
    for name, n in (("f8_quantize", 2), ("f8_quantize_weight", 2), ("f8", 7), ("f8_dynamic", 7), ("grouped", 5),
                    ("grouped_bwd", 7), ("bind_grouped", 8)):
        with pytest.raises(TypeError):
            getattr(m, name)(*[None] * (n - 1))
        with pytest.raises(TypeError):
            getattr(m, name)(*[None] * (n + 1))
