"""The 8-bit and training entry points on a machine without a GPU: refusals are made on the host
before any HIP call, empty outputs are accepted, and the binding's helpers check their tensors."""

import ctypes

import pytest

import gemv_layers_amd as g

OK, BAD, UNSUP, NOINIT = (g.GEMM_OK, g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED,
                          g.GEMM_ERR_NOT_INITIALIZED)
P = ctypes.c_void_p(64)  # a non-null, aligned stand-in; never dereferenced here
Q = ctypes.c_void_p(66)  # 2-byte aligned only
X = ctypes.c_void_p(65)  # odd


@pytest.mark.parametrize("args,status", [
    ((-1, 8, P, 8, P, 8, P), BAD),
    ((4, -8, P, 8, P, 8, P), BAD),
    ((4, 8, P, 7, P, 8, P), BAD),          # ldx < K
    ((4, 8, P, 8, P, 7, P), BAD),          # ldq < K
    ((4, 8, None, 8, P, 8, P), BAD),
    ((4, 8, P, 8, None, 8, P), BAD),
    ((4, 8, P, 8, P, 8, None), BAD),
    ((4, 8, P, 8, P, 8, Q), BAD),          # scales not 4-byte aligned
    ((4, 8, X, 8, P, 8, P), BAD),          # bf16 at an odd address
    ((1 << 24, 8, P, 8, P, 8, P), UNSUP),
    ((0, 8, None, 8, None, 8, None), OK),
    ((4, 8, Q, 8, X, 8, P), NOINIT),       # any alignment of codes is taken
    ((4, 0, None, 0, None, 0, P), NOINIT),
])
def test_quantize_refusals(args, status):
    assert g.lib().gemm_i8_quantize(*args, None) == status


I8 = [
    ((-1, 8, 8, P, 8, P, P, 8, P, P, 8), BAD),
    ((8, -1, 8, P, 8, P, P, 8, P, P, 8), BAD),
    ((8, 8, -1, P, 8, P, P, 8, P, P, 8), BAD),
    ((8, 8, 16, P, 8, P, P, 16, P, P, 8), BAD),      # ldaq < K
    ((8, 8, 16, P, 16, P, P, 8, P, P, 8), BAD),      # ldwq < K
    ((8, 8, 8, P, 8, P, P, 8, P, P, 7), BAD),        # ldc < N
    ((8, 8, 8, None, 8, P, P, 8, P, P, 8), BAD),
    ((8, 8, 8, P, 8, None, P, 8, P, P, 8), BAD),
    ((8, 8, 8, P, 8, P, None, 8, P, P, 8), BAD),
    ((8, 8, 8, P, 8, P, P, 8, None, P, 8), BAD),
    ((8, 8, 8, P, 8, P, P, 8, P, None, 8), BAD),
    ((8, 8, 8, P, 8, Q, P, 8, P, P, 8), BAD),        # scales not 4-byte aligned
    ((8, 8, 8, P, 8, P, P, 8, Q, P, 8), BAD),
    ((8, 8, 8, P, 8, P, P, 8, P, X, 8), BAD),        # C at an odd address
    ((8, 8, 131072, P, 1 << 17, P, P, 1 << 17, P, P, 8), UNSUP),  # 32-bit sums could overflow
    ((8, 8, 131071, P, 1 << 17, P, P, 1 << 17, P, P, 8), NOINIT),
    ((0, 8, 8, None, 8, None, P, 8, P, None, 8), OK),
    ((8, 0, 8, P, 8, P, None, 8, None, None, 0), OK),
    ((8, 8, 0, None, 0, P, None, 0, P, P, 8), NOINIT),
    ((8, 8, 8, X, 8, P, X, 8, P, Q, 8), NOINIT),     # any alignment of codes is taken
]


@pytest.mark.parametrize("name", ["gemm_i8", "gemm_i8_swiglu"])
@pytest.mark.parametrize("args,status", I8)
def test_i8_refusals(name, args, status):
    assert getattr(g.lib(), name)(*args, None) == status


@pytest.mark.parametrize("name", ["gemm_i8_bf16", "gemm_i8_swiglu_bf16"])
@pytest.mark.parametrize("args,status", [
    ((4, 8, 8, P, 8, P, 8, P, P, 8, P, 80), NOINIT),         # 4 rows of 16 codes and 4 scales
    ((4, 8, 8, P, 8, P, 8, P, P, 8, P, 79), BAD),            # work too small
    ((4, 8, 8, P, 8, P, 8, P, P, 8, None, 80), BAD),
    ((4, 8, 8, P, 8, P, 8, P, P, 8, ctypes.c_void_p(72), 80), BAD),  # work not 16-byte aligned
    ((4, 8, 8, P, 7, P, 8, P, P, 8, P, 80), BAD),            # lda < K
    ((4, 8, 8, X, 8, P, 8, P, P, 8, P, 80), BAD),            # bf16 at an odd address
    ((4, 8, 8, None, 8, P, 8, P, P, 8, P, 80), BAD),
    ((4, 8, 131072, P, 1 << 17, P, 1 << 17, P, P, 8, P, 1 << 20), UNSUP),
    ((1 << 24, 8, 8, P, 8, P, 8, P, P, 8, P, 1 << 40), UNSUP),
    ((0, 8, 8, None, 8, P, 8, P, None, 8, None, 0), OK),
    ((4, 0, 8, P, 8, None, 8, None, None, 0, None, 0), OK),
])
def test_i8_bf16_refusals(name, args, status):
    assert getattr(g.lib(), name)(*args, None) == status


def test_i8_work_bytes():
    assert g.gemm_i8_work_bytes(4, 8) == 4 * 16 + 16
    assert g.gemm_i8_work_bytes(3, 33) == 3 * 48 + 12
    assert g.gemm_i8_work_bytes(0, 8) == 0
    n = ctypes.c_int64()
    L = g.lib()
    assert L.gemm_i8_work_bytes(-1, 8, ctypes.byref(n)) == BAD
    assert L.gemm_i8_work_bytes(1, 8, None) == BAD
    assert L.gemm_i8_work_bytes(1, 131072, ctypes.byref(n)) == UNSUP
    assert L.gemm_i8_work_bytes(1 << 24, 8, ctypes.byref(n)) == UNSUP


@pytest.mark.parametrize("args,status", [
    # M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb
    ((-1, 8, 8, P, 8, P, 8, P, 8, P, 8, P, 8), BAD),
    ((8, 8, 8, P, 7, P, 8, P, 8, P, 8, P, 8), BAD),
    ((8, 8, 8, None, 8, P, 8, P, 8, P, 8, P, 8), BAD),
    ((8, 8, 8, X, 8, P, 8, P, 8, P, 8, P, 8), BAD),
    ((8, 8, 8, P, 8, None, 8, P, 8, P, 8, P, 8), BAD),       # dB needs A
    ((8, 8, 8, P, 8, P, 8, None, 8, P, 8, P, 8), BAD),       # dA needs B
    ((8, 8, 8, P, 8, P, 7, P, 8, P, 8, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 8, P, 7, P, 8, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 8, P, 8, P, 7, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 8, P, 8, P, 8, P, 7), BAD),
    ((8, 8, 8, P, 8, P, 8, P, 8, X, 8, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 8, P, 8, P, 8, P, 8), NOINIT),
    ((8, 8, 8, P, 8, None, 0, P, 8, P, 8, None, 0), NOINIT),  # dA alone: A is not read
    ((8, 8, 8, P, 8, P, 8, None, 0, None, 0, P, 8), NOINIT),  # dB alone: B is not read
    ((8, 8, 8, P, 8, None, 0, None, 0, None, 0, None, 0), OK),
    ((8, 8, 0, P, 8, P, 0, P, 8, P, 0, P, 8), OK),
    ((0, 8, 8, None, 8, None, 8, P, 8, P, 8, P, 8), NOINIT),  # dB is a zero K x N matrix
])
def test_bwd_refusals(args, status):
    assert g.lib().gemm_bf16_bwd(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # M, N, K, A, lda, B, ldb, GU, ldgu, C, ldc
    ((8, 8, 8, P, 8, P, 16, P, 16, P, 8), NOINIT),
    ((8, 8, 8, P, 8, P, 15, P, 16, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 15, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 16, P, 7), BAD),
    ((8, 8, 8, P, 7, P, 16, P, 16, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 16, None, 16, P, 8), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 16, None, 8), BAD),
    ((8, 8, 8, X, 8, P, 16, P, 16, P, 8), BAD),
    ((8, 2**62, 8, P, 8, P, 2**63 - 1, P, 2**63 - 1, P, 2**62), BAD),  # 2N overflows
    ((0, 8, 8, None, 8, P, 16, None, 16, None, 8), OK),
])
def test_swiglu_train_refusals(args, status):
    assert g.lib().gemm_bf16_swiglu_train(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # M, N, K, dC, lddc, GU, ldgu, A, lda, B, ldb, dGU, lddgu, dA, ldda, dB, lddb
    ((8, 8, 8, P, 8, P, 16, P, 8, P, 16, P, 16, P, 8, P, 16), NOINIT),
    ((8, 8, 8, P, 7, P, 16, P, 8, P, 16, P, 16, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, P, 15, P, 8, P, 16, P, 16, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 8, P, 16, P, 15, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 8, P, 15, P, 16, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 8, P, 16, P, 16, P, 8, P, 15), BAD),
    ((8, 8, 8, None, 8, P, 16, P, 8, P, 16, P, 16, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, None, 16, P, 8, P, 16, P, 16, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, P, 16, P, 8, P, 16, None, 16, P, 8, P, 16), BAD),
    ((8, 8, 8, P, 8, P, 16, None, 0, None, 0, P, 16, None, 0, None, 0), NOINIT),  # dGU alone
    ((0, 8, 0, None, 8, None, 16, None, 0, P, 16, None, 16, None, 0, None, 16), OK),
])
def test_swiglu_bwd_refusals(args, status):
    assert g.lib().gemm_bf16_swiglu_bwd(*args, None) == status


def test_helpers_check_their_tensors():
    torch = pytest.importorskip("torch")
    A = torch.zeros(4, 8, dtype=torch.bfloat16)
    q = torch.zeros(4, 8, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError):
        g.i8_quantize(A)                      # not on a device
    with pytest.raises(TypeError):
        g.i8_quantize(A.float())
    with pytest.raises(TypeError):
        g.i8_matmul(A, s, q, s)
    with pytest.raises(ValueError):
        g.i8_matmul(q, s, q, s)
    with pytest.raises(TypeError):
        g.i8_linear(q, q, s)
    with pytest.raises(TypeError):
        g.swiglu_forward(A.float(), A)
    with pytest.raises(ValueError):
        g.matmul_backward(A, A, A)
