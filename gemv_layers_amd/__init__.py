"""Python binding of libgemm_bf16.so, the gfx950 bf16 GEMM library (include/gemm_bf16.h).

Argument marshalling only: every function forwards to the C ABI function of the same name, and
every step of the product runs in the library's HIP kernels. There is no CPU or PyTorch
fallback: if the library is not built, or a call fails, an exception is raised.

The ``matmul`` helper takes PyTorch bf16 tensors (PyTorch is used for device memory and streams
only) and passes their device pointers, leading dimensions and the current stream.
"""

from __future__ import annotations

import ctypes
import json
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemm_bf16.so")

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_UNSUPPORTED = 2
GEMM_ERR_NOT_INITIALIZED = 3
GEMM_ERR_HIP = 4

GEMM_PLAN_SKINNY = 1
GEMM_PLAN_SWIGLU = 2
GEMM_PLAN_MX = 4
GEMM_PLAN_PACKED = 8

# every symbol include/gemm_bf16.h declares
EXPORTS = (
    "gemm_init", "gemm_bf16", "gemm_bf16_noalloc", "gemm_bf16_skinny", "gemm_bf16_tiled", "gemm_bf16_swiglu",
    "gemm_plan_describe",
    "gemm_wave_efficiency", "gemm_last_plan", "gemm_status_string", "gemm_finalize",
    "gemm_peak_mfma_launch", "gemm_peak_mfma_data_launch", "gemm_peak_copy_launch", "gemm_peak_read_launch",
    "gemm_peak_clock_launch", "gemm_peak_xcc_launch",
    "gemm_peak_empty_launch", "gemm_fill_launch",
    "gemm_mx_packed_sizes", "gemm_mx_pack_weight", "gemm_mx_quantize_act", "gemm_mx_decode",
    "gemm_mx_decode_bf16", "gemm_pack_weight_bf16", "gemm_bf16_packed",
    "gemm_i8_quantize", "gemm_i8", "gemm_i8_swiglu", "gemm_i8_work_bytes", "gemm_i8_bf16",
    "gemm_i8_swiglu_bf16", "gemm_bf16_bwd", "gemm_bf16_swiglu_train", "gemm_bf16_swiglu_bwd",
    "gemm_f8_quantize", "gemm_f8_quantize_weight", "gemm_f8", "gemm_f8_work_bytes", "gemm_f8_bf16",
    "gemm_bf16_grouped", "gemm_bf16_grouped_bwd", "gemm_f8_grouped", "gemm_f8_grouped_bf16",
)


class GemmError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} failed: {status_string(status)} ({status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load the in-tree library (built by gemv_layers_amd.build); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m gemv_layers_amd.build` "
                           "(there is no fallback path)")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, p, u32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_uint32
    gemm_sig = [i64, i64, i64, p, i64, p, i64, p, i64, p]
    for name in ("gemm_bf16", "gemm_bf16_noalloc", "gemm_bf16_skinny", "gemm_bf16_tiled", "gemm_bf16_swiglu"):
        getattr(L, name).argtypes = gemm_sig
        getattr(L, name).restype = i32
    L.gemm_init.argtypes = [i32]
    L.gemm_init.restype = i32
    L.gemm_plan_describe.argtypes = [i64, i64, i64, i32, i32, ctypes.c_char_p, i32]
    L.gemm_plan_describe.restype = i32
    L.gemm_wave_efficiency.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_int64)]
    L.gemm_wave_efficiency.restype = i32
    L.gemm_last_plan.argtypes = [ctypes.c_char_p, i32]
    L.gemm_last_plan.restype = i32
    L.gemm_status_string.argtypes = [i32]
    L.gemm_status_string.restype = ctypes.c_char_p
    L.gemm_finalize.argtypes = []
    L.gemm_finalize.restype = i32
    L.gemm_peak_mfma_launch.argtypes = [i64, i32, p, p, p]
    L.gemm_peak_mfma_launch.restype = i32
    L.gemm_peak_mfma_data_launch.argtypes = [p, i64, i32, p, p, p]
    L.gemm_peak_mfma_data_launch.restype = i32
    L.gemm_peak_copy_launch.argtypes = [p, p, i64, p]
    L.gemm_peak_copy_launch.restype = i32
    L.gemm_peak_read_launch.argtypes = [p, i64, p, p]
    L.gemm_peak_read_launch.restype = i32
    L.gemm_peak_clock_launch.argtypes = [i64, i32, p, p]
    L.gemm_peak_clock_launch.restype = i32
    L.gemm_peak_xcc_launch.argtypes = [i32, p, p]
    L.gemm_peak_xcc_launch.restype = i32
    L.gemm_peak_empty_launch.argtypes = [p]
    L.gemm_peak_empty_launch.restype = i32
    L.gemm_fill_launch.argtypes = [p, i64, u32, p]
    L.gemm_fill_launch.restype = i32
    L.gemm_mx_packed_sizes.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
    L.gemm_mx_packed_sizes.restype = i32
    L.gemm_mx_pack_weight.argtypes = [i64, i64, p, i64, p, p, p]
    L.gemm_mx_pack_weight.restype = i32
    L.gemm_mx_quantize_act.argtypes = [i64, i64, p, i64, p, i64, p, i64, p]
    L.gemm_mx_quantize_act.restype = i32
    L.gemm_mx_decode.argtypes = [i64, i64, i64, p, i64, p, i64, p, p, p, i64, p]
    L.gemm_mx_decode.restype = i32
    L.gemm_mx_decode_bf16.argtypes = [i64, i64, i64, p, i64, p, p, p, i64, p]
    L.gemm_mx_decode_bf16.restype = i32
    L.gemm_pack_weight_bf16.argtypes = [i64, i64, p, i64, p, p]
    L.gemm_pack_weight_bf16.restype = i32
    L.gemm_bf16_packed.argtypes = [i64, i64, i64, p, i64, p, p, i64, p]
    L.gemm_bf16_packed.restype = i32
    L.gemm_i8_quantize.argtypes = [i64, i64, p, i64, p, i64, p, p]
    L.gemm_i8_work_bytes.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_int64)]
    for name in ("gemm_i8", "gemm_i8_swiglu"):
        getattr(L, name).argtypes = [i64, i64, i64, p, i64, p, p, i64, p, p, i64, p]
    for name in ("gemm_i8_bf16", "gemm_i8_swiglu_bf16"):
        getattr(L, name).argtypes = [i64, i64, i64, p, i64, p, i64, p, p, i64, p, i64, p]
    L.gemm_bf16_bwd.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p]
    L.gemm_bf16_swiglu_train.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p]
    L.gemm_bf16_swiglu_bwd.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p]
    for name in ("gemm_i8_quantize", "gemm_i8_work_bytes", "gemm_i8", "gemm_i8_swiglu", "gemm_i8_bf16",
                 "gemm_i8_swiglu_bf16", "gemm_bf16_bwd", "gemm_bf16_swiglu_train", "gemm_bf16_swiglu_bwd"):
        getattr(L, name).restype = i32
    L.gemm_f8_quantize.argtypes = [i64, i64, p, i64, p, i64, p, i64, p]
    L.gemm_f8_quantize_weight.argtypes = [i64, i64, i64, p, i64, i64, p, i64, i64, p, i64, i64, p]
    L.gemm_f8.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p]
    L.gemm_f8_work_bytes.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_int64)]
    L.gemm_f8_bf16.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p]
    L.gemm_bf16_grouped.argtypes = [i64, i64, i64, i64, p, i64, p, i64, i64, p, p, i64, p]
    L.gemm_bf16_grouped_bwd.argtypes = [i64, i64, i64, i64, p, i64, p, i64, p, i64, i64, p, p, i64, p, i64, i64, p]
    L.gemm_f8_grouped.argtypes = [i64, i64, i64, i64, p, i64, p, i64, p, i64, i64, p, i64, i64, p, p, i64, p]
    L.gemm_f8_grouped_bf16.argtypes = [i64, i64, i64, i64, p, i64, p, i64, i64, p, i64, i64, p, p, i64, p, i64, p]
    for name in ("gemm_f8_quantize", "gemm_f8_quantize_weight", "gemm_f8", "gemm_f8_work_bytes", "gemm_f8_bf16",
                 "gemm_bf16_grouped", "gemm_bf16_grouped_bwd", "gemm_f8_grouped", "gemm_f8_grouped_bf16"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def _check(func: str, status: int) -> None:
    if status != GEMM_OK:
        raise GemmError(func, status)


def status_string(status: int) -> str:
    return lib().gemm_status_string(int(status)).decode()


gemm_status_string = status_string


def gemm_init(device: int = 0) -> None:
    _check("gemm_init", lib().gemm_init(int(device)))


def gemm_finalize() -> None:
    _check("gemm_finalize", lib().gemm_finalize())


def _call(name, M, N, K, A, lda, B, ldb, C, ldc, stream):
    st = getattr(lib(), name)(int(M), int(N), int(K), A, int(lda), B, int(ldb), C, int(ldc), stream)
    _check(name, st)


def gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = A * B on raw device pointers (ints); see include/gemm_bf16.h."""
    _call("gemm_bf16", M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """gemm_bf16 with the library's fixed scratch array as workspace (never allocates)."""
    _call("gemm_bf16_noalloc", M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_skinny(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    _call("gemm_bf16_skinny", M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_tiled(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    _call("gemm_bf16_tiled", M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_swiglu(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = silu(A * B[:, :N]) * (A * B[:, N:2N]) on raw device pointers; B is K x 2N."""
    _call("gemm_bf16_swiglu", M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_plan_describe(M: int, N: int, K: int, cus: int = 256, skinny: bool = False,
                       swiglu: bool = False, mx: bool = False, packed: bool = False) -> dict:
    buf = ctypes.create_string_buffer(4096)
    flags = ((GEMM_PLAN_SKINNY if skinny else 0) | (GEMM_PLAN_SWIGLU if swiglu else 0)
             | (GEMM_PLAN_MX if mx else 0) | (GEMM_PLAN_PACKED if packed else 0))
    _check("gemm_plan_describe", lib().gemm_plan_describe(M, N, K, cus, flags, buf, 4096))
    return json.loads(buf.value.decode())


def gemm_mx_packed_sizes(N: int, K: int) -> tuple[int, int]:
    """(code bytes, scale bytes) of the packed MXFP4 form of an N x K weight."""
    w, s = ctypes.c_int64(), ctypes.c_int64()
    _check("gemm_mx_packed_sizes", lib().gemm_mx_packed_sizes(N, K, ctypes.byref(w), ctypes.byref(s)))
    return w.value, s.value


def gemm_mx_pack_weight(N, K, W, ldw, Wp, Sp, stream=None) -> None:
    _check("gemm_mx_pack_weight", lib().gemm_mx_pack_weight(N, K, W, ldw, Wp, Sp, stream))


def gemm_mx_quantize_act(M, K, A, lda, Aq, ldaq, As, ldas, stream=None) -> None:
    _check("gemm_mx_quantize_act", lib().gemm_mx_quantize_act(M, K, A, lda, Aq, ldaq, As, ldas, stream))


def gemm_mx_decode(M, N, K, Aq, ldaq, As, ldas, Wp, Sp, C, ldc, stream=None) -> None:
    _check("gemm_mx_decode", lib().gemm_mx_decode(M, N, K, Aq, ldaq, As, ldas, Wp, Sp, C, ldc, stream))


def gemm_mx_decode_bf16(M, N, K, A, lda, Wp, Sp, C, ldc, stream=None) -> None:
    _check("gemm_mx_decode_bf16", lib().gemm_mx_decode_bf16(M, N, K, A, lda, Wp, Sp, C, ldc, stream))


def gemm_pack_weight_bf16(K, N, B, ldb, Bp, stream=None) -> None:
    _check("gemm_pack_weight_bf16", lib().gemm_pack_weight_bf16(K, N, B, ldb, Bp, stream))


def gemm_bf16_packed(M, N, K, A, lda, Bp, C, ldc, stream=None) -> None:
    _check("gemm_bf16_packed", lib().gemm_bf16_packed(M, N, K, A, lda, Bp, C, ldc, stream))


def gemm_i8_quantize(R, K, X, ldx, Q, ldq, S, stream=None) -> None:
    _check("gemm_i8_quantize", lib().gemm_i8_quantize(R, K, X, ldx, Q, ldq, S, stream))


def gemm_i8(M, N, K, Aq, ldaq, Sa, Wq, ldwq, Sw, C, ldc, stream=None) -> None:
    _check("gemm_i8", lib().gemm_i8(M, N, K, Aq, ldaq, Sa, Wq, ldwq, Sw, C, ldc, stream))


def gemm_i8_swiglu(M, N, K, Aq, ldaq, Sa, Wq, ldwq, Sw, C, ldc, stream=None) -> None:
    _check("gemm_i8_swiglu", lib().gemm_i8_swiglu(M, N, K, Aq, ldaq, Sa, Wq, ldwq, Sw, C, ldc, stream))


def gemm_i8_work_bytes(M: int, K: int) -> int:
    """Bytes of the work buffer of gemm_i8_bf16 and gemm_i8_swiglu_bf16."""
    n = ctypes.c_int64()
    _check("gemm_i8_work_bytes", lib().gemm_i8_work_bytes(M, K, ctypes.byref(n)))
    return n.value


def gemm_i8_bf16(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, work, work_bytes, stream=None) -> None:
    _check("gemm_i8_bf16", lib().gemm_i8_bf16(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, work, work_bytes, stream))


def gemm_i8_swiglu_bf16(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, work, work_bytes, stream=None) -> None:
    _check("gemm_i8_swiglu_bf16",
           lib().gemm_i8_swiglu_bf16(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, work, work_bytes, stream))


def gemm_bf16_bwd(M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb, stream=None) -> None:
    _check("gemm_bf16_bwd", lib().gemm_bf16_bwd(M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb, stream))


def gemm_bf16_swiglu_train(M, N, K, A, lda, B, ldb, GU, ldgu, C, ldc, stream=None) -> None:
    _check("gemm_bf16_swiglu_train",
           lib().gemm_bf16_swiglu_train(M, N, K, A, lda, B, ldb, GU, ldgu, C, ldc, stream))


def gemm_bf16_swiglu_bwd(M, N, K, dC, lddc, GU, ldgu, A, lda, B, ldb, dGU, lddgu, dA, ldda, dB, lddb,
                         stream=None) -> None:
    _check("gemm_bf16_swiglu_bwd",
           lib().gemm_bf16_swiglu_bwd(M, N, K, dC, lddc, GU, ldgu, A, lda, B, ldb, dGU, lddgu, dA, ldda, dB, lddb,
                                      stream))


def gemm_f8_quantize(R, K, X, ldx, Q, ldq, S, lds, stream=None) -> None:
    _check("gemm_f8_quantize", lib().gemm_f8_quantize(R, K, X, ldx, Q, ldq, S, lds, stream))


def gemm_f8_quantize_weight(E, N, K, W, ldw, stride_w, Q, ldq, stride_q, S, lds, stride_s, stream=None) -> None:
    _check("gemm_f8_quantize_weight",
           lib().gemm_f8_quantize_weight(E, N, K, W, ldw, stride_w, Q, ldq, stride_q, S, lds, stride_s, stream))


def gemm_f8(M, N, K, Aq, ldaq, Sa, ldsa, Wq, ldwq, Sw, ldsw, C, ldc, stream=None) -> None:
    _check("gemm_f8", lib().gemm_f8(M, N, K, Aq, ldaq, Sa, ldsa, Wq, ldwq, Sw, ldsw, C, ldc, stream))


def gemm_f8_work_bytes(M: int, K: int) -> int:
    """Bytes of the work buffer of gemm_f8_bf16 and gemm_f8_grouped_bf16."""
    n = ctypes.c_int64()
    _check("gemm_f8_work_bytes", lib().gemm_f8_work_bytes(M, K, ctypes.byref(n)))
    return n.value


def gemm_f8_bf16(M, N, K, A, lda, Wq, ldwq, Sw, ldsw, C, ldc, work, work_bytes, stream=None) -> None:
    _check("gemm_f8_bf16", lib().gemm_f8_bf16(M, N, K, A, lda, Wq, ldwq, Sw, ldsw, C, ldc, work, work_bytes, stream))


def gemm_bf16_grouped(M, N, K, E, A, lda, B, ldb, stride_b, offsets, C, ldc, stream=None) -> None:
    _check("gemm_bf16_grouped", lib().gemm_bf16_grouped(M, N, K, E, A, lda, B, ldb, stride_b, offsets, C, ldc, stream))


def gemm_bf16_grouped_bwd(M, N, K, E, dC, lddc, A, lda, B, ldb, stride_b, offsets, dA, ldda, dB, lddb, stride_db,
                          stream=None) -> None:
    _check("gemm_bf16_grouped_bwd",
           lib().gemm_bf16_grouped_bwd(M, N, K, E, dC, lddc, A, lda, B, ldb, stride_b, offsets, dA, ldda, dB, lddb,
                                       stride_db, stream))


def gemm_f8_grouped(M, N, K, E, Aq, ldaq, Sa, ldsa, Wq, ldwq, stride_wq, Sw, ldsw, stride_sw, offsets, C, ldc,
                    stream=None) -> None:
    _check("gemm_f8_grouped",
           lib().gemm_f8_grouped(M, N, K, E, Aq, ldaq, Sa, ldsa, Wq, ldwq, stride_wq, Sw, ldsw, stride_sw, offsets, C,
                                 ldc, stream))


def gemm_f8_grouped_bf16(M, N, K, E, A, lda, Wq, ldwq, stride_wq, Sw, ldsw, stride_sw, offsets, C, ldc, work,
                         work_bytes, stream=None) -> None:
    _check("gemm_f8_grouped_bf16",
           lib().gemm_f8_grouped_bf16(M, N, K, E, A, lda, Wq, ldwq, stride_wq, Sw, ldsw, stride_sw, offsets, C, ldc,
                                      work, work_bytes, stream))


def gemm_wave_efficiency(ctas: int, slots: int):
    eff, waves = ctypes.c_double(), ctypes.c_int64()
    _check("gemm_wave_efficiency", lib().gemm_wave_efficiency(ctas, slots, ctypes.byref(eff),
                                                              ctypes.byref(waves)))
    return eff.value, waves.value


def gemm_last_plan() -> dict:
    buf = ctypes.create_string_buffer(4096)
    _check("gemm_last_plan", lib().gemm_last_plan(buf, 4096))
    return json.loads(buf.value.decode())


def gemm_peak_mfma_launch(iters, blocks, sink, cycles, stream=None) -> None:
    _check("gemm_peak_mfma_launch", lib().gemm_peak_mfma_launch(iters, blocks, sink, cycles, stream))


def gemm_peak_copy_launch(src, dst, nbytes, stream=None) -> None:
    _check("gemm_peak_copy_launch", lib().gemm_peak_copy_launch(src, dst, nbytes, stream))


def gemm_peak_read_launch(src, nbytes, sink, stream=None) -> None:
    _check("gemm_peak_read_launch", lib().gemm_peak_read_launch(src, nbytes, sink, stream))


def gemm_peak_clock_launch(iters, blocks, out, stream=None) -> None:
    _check("gemm_peak_clock_launch", lib().gemm_peak_clock_launch(iters, blocks, out, stream))


def gemm_peak_mfma_data_launch(ops, iters, blocks, sink, cycles, stream=None) -> None:
    _check("gemm_peak_mfma_data_launch",
           lib().gemm_peak_mfma_data_launch(ops, iters, blocks, sink, cycles, stream))


def gemm_peak_xcc_launch(blocks, out, stream=None) -> None:
    _check("gemm_peak_xcc_launch", lib().gemm_peak_xcc_launch(blocks, out, stream))


def gemm_peak_empty_launch(stream=None) -> None:
    _check("gemm_peak_empty_launch", lib().gemm_peak_empty_launch(stream))


def gemm_fill_launch(dst, nbytes, value, stream=None) -> None:
    _check("gemm_fill_launch", lib().gemm_fill_launch(dst, nbytes, value & 0xFFFFFFFF, stream))


# ---- PyTorch marshalling helpers ----------------------------------------------------------

def current_stream_handle():
    import torch

    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_ENTRY = {"auto": "gemm_bf16", "skinny": "gemm_bf16_skinny", "tiled": "gemm_bf16_tiled"}


def matmul(A, B, out=None, entry: str = "auto", stream=None):
    """C = A @ B for 2-D bf16 CUDA tensors with unit column stride; returns C (bf16)."""
    import torch

    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError("shapes do not form a matrix product")
    if not (A.is_cuda and B.is_cuda):
        raise ValueError("A and B must be device tensors")
    M, K = A.shape
    N = B.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    for t in (A, B, out):
        if t.numel() and t.stride(1) != 1:
            raise ValueError("unit column stride required")
    st = stream if stream is not None else current_stream_handle()
    _call(_ENTRY[entry], M, N, K, ctypes.c_void_p(A.data_ptr()), max(A.stride(0), K),
          ctypes.c_void_p(B.data_ptr()), max(B.stride(0), N), ctypes.c_void_p(out.data_ptr()),
          max(out.stride(0), N), st)
    return out


def swiglu_matmul(A, B, out=None, stream=None):
    """silu(A @ B[:, :N]) * (A @ B[:, N:]) for bf16 CUDA tensors, B of shape (K, 2N): the gate
    and up weights side by side. Returns the (M, N) bf16 result."""
    import torch

    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0] or B.shape[1] % 2:
        raise ValueError("B must be K x 2N for A of shape M x K")
    if not (A.is_cuda and B.is_cuda):
        raise ValueError("A and B must be device tensors")
    M, K = A.shape
    N = B.shape[1] // 2
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    for t in (A, B, out):
        if t.numel() and t.stride(1) != 1:
            raise ValueError("unit column stride required")
    st = stream if stream is not None else current_stream_handle()
    _call("gemm_bf16_swiglu", M, N, K, ctypes.c_void_p(A.data_ptr()), max(A.stride(0), K),
          ctypes.c_void_p(B.data_ptr()), max(B.stride(0), 2 * N), ctypes.c_void_p(out.data_ptr()),
          max(out.stride(0), N), st)
    return out


# ---- 8-bit and grouped products, training: PyTorch marshalling ----------------------------------------
#
# A small product takes the GPU a few microseconds, so the tensors are checked, and the outputs made,
# in a C++ module (_torch_ops). The functions below name its arguments. With `stream`, a handle, a call
# runs as under torch.cuda.stream of it: its outputs belong to that stream. They record no graph: a
# tensor that requires grad, with grad mode on, is refused (RuntimeError) by all but i8_quantize and
# f8_quantize(_weight), whose codes have no gradient. Wrap swiglu_forward and swiglu_backward, or grouped_matmul
# and grouped_matmul_backward, in a torch.autograd.Function to train with autograd.

_ops = None


def _load_ops():
    """The marshalling module (built by gemv_layers_amd.build), with the library's addresses in it."""
    global _ops
    if _ops is None:
        import torch  # noqa: F401  (the module links to it)

        L = lib()
        try:
            from . import _torch_ops as m
        except ImportError as e:
            raise RuntimeError(f"_torch_ops.so is not built or does not fit this PyTorch ({e}); run "
                               "`python -m gemv_layers_amd.build` (there is no fallback path)") from e
        m.bind(_check, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "gemm_i8_quantize", "gemm_i8", "gemm_i8_swiglu", "gemm_i8_bf16", "gemm_i8_swiglu_bf16", "gemm_bf16_bwd",
            "gemm_bf16_swiglu_train", "gemm_bf16_swiglu_bwd")))
        m.bind_grouped(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "gemm_f8_quantize", "gemm_f8_quantize_weight", "gemm_f8", "gemm_f8_bf16", "gemm_f8_grouped",
            "gemm_f8_grouped_bf16", "gemm_bf16_grouped", "gemm_bf16_grouped_bwd")))
        _ops = m
    return _ops


def i8_quantize(X, stream=None):
    """8-bit codes and scales of each row of a bf16 matrix: (Q int8 of X's shape, S float32).
    Q's rows are padded to 16 bytes in memory, as the matrix kernels want them. For an nn.Linear
    weight the rows are output channels; for activations they are tokens."""
    return (_ops or _load_ops()).quantize(X, stream)


def i8_matmul(Aq, Sa, Wq, Sw, out=None, stream=None):
    """(Aq @ Wq.T) * Sa[:, None] * Sw as bf16: int8 codes Aq (M x K) and Wq (N x K), float32 scales."""
    return (_ops or _load_ops()).i8(Aq, Sa, Wq, Sw, out, stream, False)


def i8_swiglu_matmul(Aq, Sa, Wq, Sw, out=None, stream=None):
    """silu(g) * u of the 8-bit product with a 2N x K gate/up weight (gate rows first); M x N bf16."""
    return (_ops or _load_ops()).i8(Aq, Sa, Wq, Sw, out, stream, True)


def i8_linear(A, Wq, Sw, out=None, work=None, stream=None):
    """The 8-bit product of bf16 activations A (M x K), quantised row by row in the call, with an
    8-bit weight (N x K codes, N scales); M x N bf16. `work`: a uint8 tensor of
    gemm_i8_work_bytes(M, K) bytes to reuse, else one is allocated."""
    return (_ops or _load_ops()).i8_dynamic(A, Wq, Sw, out, work, stream, False)


def i8_swiglu_linear(A, Wq, Sw, out=None, work=None, stream=None):
    """silu(g) * u of the 8-bit product of bf16 activations with a 2N x K gate/up weight."""
    return (_ops or _load_ops()).i8_dynamic(A, Wq, Sw, out, work, stream, True)


def matmul_backward(dC, A, B, need_dA=True, need_dB=True, stream=None):
    """(dA, dB) = (dC @ B.T, A.T @ dC), the gradients of matmul(A, B); None for one not needed."""
    return (_ops or _load_ops()).bwd(dC, A, B, need_dA, need_dB, stream)


def swiglu_forward(A, B, stream=None):
    """(C, GU) of the gated block for training: GU = A @ B (M x 2N, gate then up), C = silu(g) * u."""
    return (_ops or _load_ops()).train(A, B, stream)


def swiglu_backward(dC, GU, A, B, need_dA=True, need_dB=True, inplace=False, stream=None):
    """(dA, dB, dGU): the gradients of swiglu_forward's C. With `inplace`, dGU takes GU's memory."""
    return (_ops or _load_ops()).swiglu_bwd(dC, GU, A, B, need_dA, need_dB, inplace, stream)


# 8-bit floating point: codes are torch.float8_e4m3fn, scales float32 over blocks of 128 inputs.

def f8_quantize(X, stream=None):
    """e4m3 codes and scales of each block of 128 columns of each row of a bf16 matrix: (Q float8_e4m3fn of X's
    shape, S float32 of ceil(K / 128) x rows, S[b, r] the scale of row r's block b). Q's rows are padded to 16
    bytes in memory, as the matrix kernels want them."""
    return (_ops or _load_ops()).f8_quantize(X, stream)


def f8_quantize_weight(W, stream=None):
    """e4m3 codes and scales of each 128 x 128 block of a bf16 weight (N x K, the nn.Linear layout) or of a stack
    of them (E x N x K): (Q of W's shape, S float32 of [E x] ceil(N / 128) x ceil(K / 128))."""
    return (_ops or _load_ops()).f8_quantize_weight(W, stream)


def f8_matmul(Aq, Sa, Wq, Sw, out=None, stream=None):
    """The product of e4m3 codes Aq (M x K) and Wq (N x K) with their block scales (f8_quantize's and
    f8_quantize_weight's): Aq @ Wq.T with every block of 128 inputs scaled, as M x N bf16."""
    return (_ops or _load_ops()).f8(Aq, Sa, Wq, Sw, None, out, stream)


def f8_linear(A, Wq, Sw, out=None, work=None, stream=None):
    """f8_matmul of bf16 activations A (M x K), quantised in the call. `work`: a uint8 tensor of
    gemm_f8_work_bytes(M, K) bytes to reuse, else one is allocated."""
    return (_ops or _load_ops()).f8_dynamic(A, Wq, Sw, None, out, work, stream)


# Grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 belong to group e, `offsets` an int32 device tensor of
# E + 1 values that only the kernels read, and that stay as they are until the call's work is done. Rows of no
# group come out as zeros.

def grouped_matmul(A, B, offsets, out=None, stream=None):
    """Each group's rows of A (M x K, bf16) times its own B[e] (E x K x N): M x N bf16."""
    return (_ops or _load_ops()).grouped(A, B, offsets, out, stream)


def grouped_matmul_backward(dC, A, B, offsets, need_dA=True, need_dB=True, stream=None):
    """(dA, dB): the gradients of grouped_matmul(A, B, offsets); None for one not needed. dB is E x K x N, zero for
    groups without rows."""
    return (_ops or _load_ops()).grouped_bwd(dC, A, B, offsets, need_dA, need_dB, stream)


def f8_grouped_matmul(Aq, Sa, Wq, Sw, offsets, out=None, stream=None):
    """f8_matmul with each group's own weight: Wq E x N x K codes, Sw E x ceil(N / 128) x ceil(K / 128) scales."""
    return (_ops or _load_ops()).f8(Aq, Sa, Wq, Sw, offsets, out, stream)


def f8_grouped_linear(A, Wq, Sw, offsets, out=None, work=None, stream=None):
    """f8_grouped_matmul of bf16 activations A (M x K), quantised in the call."""
    return (_ops or _load_ops()).f8_dynamic(A, Wq, Sw, offsets, out, work, stream)
