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
    kOpAb = 4,     // C = A B: bf16, A contiguous, B (K x N) strided
    kOpF8 = 5,     // C = sum over blocks of 128 k of (A W^T) sa sw: e4m3 codes, both contiguous (W is N x K)
};

// One product: an M x N output summed over K. Sizes and leading dimensions are in elements.
struct OpArgs {
    const void* A;
    const void* B;
    uint16_t* C;
    uint16_t* GU;     // kOpTrain: M x 2N
    const float* sa;  // kOpI8: M; kOpF8: ceil(K / 128) x M
    const float* sb;  // kOpI8: N, or 2N gated; kOpF8: ceil(N / 128) x ceil(K / 128)
    int64_t M, N, K;
    int64_t lda, ldb, ldc, ldgu;
    int64_t ldsa = 0, ldsb = 0;  // kOpF8
};

// The groups of a product whose rows belong to groups with a B of their own. Rows are those of A and C, or
// of A and B (dC) where the rows are summed over (kOpAtb).
struct GroupArgs {
    const int32_t* offsets;  // groups + 1 row offsets on the device, or null: one group of all rows
    int groups;
    int rows;                // of all groups and of none
    int64_t stride_b;        // elements from one group's B to the next's (kOpAb, kOpAbt, kOpF8)
    int64_t stride_c;        // and from one's C (kOpAtb)
    int64_t stride_sb;       // and from one's scales (kOpF8)
    // 256 x 256 tiles: the CUs, and the most pieces of K and slots of the workspace for the tiles of a last round, which are
    // cut where both have two for each
    int cus = 1, tail = 1, slots = 0;
};

// ---- general kernel (any alignment, leading dimension or size) -------------------------------
hipError_t launch_op_generic(int mode, bool glu, const OpArgs& a, hipStream_t s);

// The same element by element for products grouped by rows and for kOpF8. a.M is all rows, or A's width
// (kOpAtb, where a.K is not read).
hipError_t launch_group_generic(int mode, const OpArgs& a, const GroupArgs& g, hipStream_t s);
constexpr int kMaxGroups = 65536;
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
struct F8TileArgs : OpTileArgs {
    int64_t ldsa, ldsb;
};
// tile: 256, 128 or 64 rows and (weight) columns; the gated forms make half as many output columns
hipError_t launch_op_tile(int mode, bool glu, int tile, const OpTileArgs& a, int grid, hipStream_t s);
// kOpAbt on `a` and kOpAtb on `b` in one launch, tiles of 128 or 64
hipError_t launch_op_pair(int tile, const OpTileArgs& a, const OpTileArgs& b, int grid, hipStream_t s);
hipError_t configure_op_kernels();
// the same tiles over grouped rows, their sizes read from the offsets (kOpAb, kOpAbt, kOpAtb). a.M is all rows,
// a.tiles_m not read; for kOpAtb a.M is A's width, a.K and a.kt_per_split are not read and the tiles are those of
// one group. `grid`: the most units that any offsets make.
hipError_t launch_group_tile(int mode, int tile, const OpTileArgs& a, const GroupArgs& g, int grid, hipStream_t s);
// kOpAbt on `a`, its first `grid_a` workgroups, and kOpAtb on `b` in one launch, tiles of 128 or 64
hipError_t launch_group_pair(int tile, const OpTileArgs& a, const GroupArgs& ga, int grid_a, const OpTileArgs& b,
                             const GroupArgs& gb, int grid_b, hipStream_t s);
hipError_t configure_group_kernels();
// kOpF8: as launch_group_tile; a.kt_per_split is even
hipError_t launch_f8_tile(int tile, const F8TileArgs& a, const GroupArgs& g, int grid, hipStream_t s);
hipError_t configure_f8_kernels();

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

// ---- 8-bit floating-point product of few rows ------------------------------------------------------
constexpr int kF8FusedK = 16384;  // the longest row that the fused form quantises
struct F8DecodeArgs {
    const uint8_t* A;     // rows of codes, with scales sa (block by block); or, fused, null and
    const uint16_t* A16;  // one row of bf16, quantised in the kernel
    const uint8_t* W;
    uint16_t* C;
    const float* sa;
    const float* sb;
    int N, K;
    int lda, ldw, ldc;
    int strips;           // of tn 16-row weight tiles
    int pieces;           // of K, one workgroup each
    int nxcd;             // XCDs the hardware deals workgroups over (1 = no remap)
    float* ws;            // pieces > 1: row tiles * strips * pieces * tn * mt * 256
    uint32_t* counters;   // one per row tile and strip, zero between launches
    int64_t ldsa, ldsb;
};
// mt: 16-row tiles in a row tile (1, 2 or 4); tn: 16-row weight tiles per workgroup (1, 2 or 4) of four waves
hipError_t launch_f8_decode(int mt, int tn, const F8DecodeArgs& a, const GroupArgs& g, int grid, hipStream_t s);

// ---- row kernels --------------------------------------------------------------------------------
// symmetric 8-bit codes of each row: see gemm_i8_quantize
hipError_t launch_i8_quantize(const uint16_t* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq,
                              float* S, hipStream_t s);
// e4m3 codes and a scale for each block of 128 values of each row, S[block * lds + row]: see gemm_f8_quantize
hipError_t launch_f8_quantize(const uint16_t* X, int64_t R, int64_t K, int64_t ldx, uint8_t* Q, int64_t ldq,
                              float* S, int64_t lds, hipStream_t s);
// the same for each 128 x 128 block of E matrices: see gemm_f8_quantize_weight
struct F8WeightArgs {
    const uint16_t* W;
    uint8_t* Q;
    float* S;
    int64_t E, N, K, ldw, stride_w, ldq, stride_q, lds, stride_s;
};
hipError_t launch_f8_quantize_weight(const F8WeightArgs& a, hipStream_t s);
// dGU from dC and GU: see gemm_bf16_swiglu_bwd
hipError_t launch_swiglu_grad(const uint16_t* dC, int64_t lddc, const uint16_t* GU, int64_t ldgu, uint16_t* dGU,
                              int64_t lddgu, int64_t M, int64_t N, hipStream_t s);

}  // namespace glk
