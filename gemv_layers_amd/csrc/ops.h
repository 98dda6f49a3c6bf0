// Launch interfaces of the 8-bit and training kernels (internal header).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glk {

// Which product a kernel computes. "Contiguous" operands hold the summed index contiguous in
// memory, "strided" ones hold it as their row index.
enum OpMode : int {
    kOpI8 = 0,     // C = (A W^T) sa sw: 8-bit codes, both operands contiguous (W is N x K)
    kOpAbt = 1,    // C = A B^T: bf16, both operands contiguous (B is N x K)
    kOpAtb = 2,    // C = A^T B: bf16, both operands strided (A is K x M, B is K x N)
    kOpTrain = 3,  // GU = A B, C = silu(g) u: bf16, A contiguous, B (K x 2N) strided; gated
};

// One product: an M x N output summed over K. Sizes and leading dimensions are in elements.
struct OpArgs {
    const void* A;
    const void* B;
    uint16_t* C;
    uint16_t* GU;     // kOpTrain: M x 2N
    const float* sa;  // kOpI8: M
    const float* sb;  // kOpI8: N, or 2N gated
    int64_t M, N, K;
    int64_t lda, ldb, ldc, ldgu;
};

// ---- general kernel (any alignment, leading dimension or size) -------------------------------
hipError_t launch_op_generic(int mode, bool glu, const OpArgs& a, hipStream_t s);

// ---- MFMA tiles ---------------------------------------------------------------------------------
// One launch over an M x N output (or a rectangle of it), sizes in elements.
struct OpTileArgs {
    const void* A;
    const void* B;
    uint16_t* C;
    uint16_t* GU;
    const float* sa;
    const float* sb;
    int M, N, K;
    int lda, ldb, ldc, ldgu;
    int up;              // gated: where the up half starts in the weight, its scales and GU
    int vec;             // C takes aligned 16-byte stores
    int tiles_m, tiles_n, group_m, nxcd;
    int splits, kt_per_split;  // pieces of K per tile, 64-byte k-steps in each (128 x 128 tiles)
    float* ws;
    uint32_t* counters;
};
// tile: 256, 128 or 64 rows and (weight) columns; the gated forms make half as many output columns
hipError_t launch_op_tile(int mode, bool glu, int tile, const OpTileArgs& a, int grid, hipStream_t s);
// kOpAbt on `a` and kOpAtb on `b` in one launch, tiles of 128 or 64
hipError_t launch_op_pair(int tile, const OpTileArgs& a, const OpTileArgs& b, int grid, hipStream_t s);
hipError_t configure_op_kernels();

// ---- 8-bit product of few tokens -------------------------------------------------------------------
constexpr int kI8FusedK = 16384;  // the longest row that the fused form quantises
struct I8DecodeArgs {
    const int8_t* A;      // M rows of codes, with scales sa; or, fused, null and
    const uint16_t* A16;  // one row of bf16, quantised in the kernel
    const int8_t* W;
    uint16_t* C;
    const float* sa;
    const float* sb;     // N scales, or 2N gated
    int M, N, K;         // M <= 64
    int lda, ldw, ldc;
    int pieces;          // of K, one workgroup each
    int32_t* ws;         // pieces > 1: groups * pieces * tn * mt * 256
    uint32_t* counters;  // one per group, zero between launches
};
// mt: 16-row tiles of M; tn: 16-row weight tiles per workgroup (gated: half gate, half up); nw waves
hipError_t launch_i8_decode(bool glu, int mt, int tn, int nw, const I8DecodeArgs& a, int grid, hipStream_t s);
hipError_t configure_i8_decode();

// ---- row kernels --------------------------------------------------------------------------------
// symmetric 8-bit codes of each row: see gemm_i8_quantize
hipError_t launch_i8_quantize(const uint16_t* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq,
                              float* S, hipStream_t s);
// dGU from dC and GU: see gemm_bf16_swiglu_bwd
hipError_t launch_swiglu_grad(const uint16_t* dC, int64_t lddc, const uint16_t* GU, int64_t ldgu, uint16_t* dGU,
                              int64_t lddgu, int64_t M, int64_t N, hipStream_t s);

}  // namespace glk
