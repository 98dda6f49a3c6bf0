// Matrix kernels of the 8-bit and training products for gfx950, on MFMA tiles.
//
// One k-step is 64 bytes of the summed index: 64 codes or 32 bf16 values, one
// v_mfma_i32_16x16x64_i8 or v_mfma_f32_16x16x32_bf16 for each 16 x 16 output block (16 bytes of each
// operand per lane, the same cycles, the same accumulator layout). An operand comes in one of two
// forms, and every product is a pair of them:
//   contiguous: the summed index is contiguous in memory (codes; dC and B of dA = dC B^T). A slot of
//     its LDS ring holds half of the tile's rows, 128 bytes (two k-steps) of each, so that copies
//     read whole lines: with one k-step of all rows, 64-byte rows, every line crossed the L1 twice
//     (8-bit 4096 x 4096 x 11008: 152 us against 124). 16-byte chunk c of row r is stored at c ^
//     ((r >> 1) & 7): the 16 rows that one cycle of a ds_read_b128 serves cover all 64 banks.
//   strided: the summed index is the row (A and dC of dB = A^T dC; B of the forward). A slot holds one
//     k-step, 32 rows of R elements, and ds_read_b64_tr_b16 transposes 4 x 16 blocks on the way to
//     registers; the 32-byte column groups of row k are stored at group ^ s(k), s(k) = (k & 3) | ((k >>
//     1) & 4).
// Both take 64 R bytes a slot. Slots are filled HBM -> LDS without registers, in rings of 5 for each
// operand: 160 KB for the 256 x 256 tile, 80 KB (two workgroups a CU) for 128 x 128, 40 KB for 64 x 64.
//
// Schedules. 256 x 256 (op_pp_kernel): two groups of four waves, one of each group on every SIMD; in
// turn one group reads its operands and issues copies while the other runs 32 MFMAs back to back, and
// they swap at each barrier. 128 x 128 and 64 x 64 (op_small): four waves in step, operands double-buffered
// in registers, K split over idle CUs with partial sums in a workspace that the last arriver adds in
// order (the same bits on every run; integer sums are exact in any order).
//
// Epilogues round once to bf16, staged through LDS so that each row segment is written by one
// instruction. Codes: the 32-bit sum times the row's and the column's scale in float32, and for the
// gated form silu(g) u. Training forward: g and u, then silu(g) u from their float32 values.
// Codes past K in the last 16-byte chunk of a row are whatever the caller's padding holds: they are
// cleared in the A operand, which is enough, as 0 times any code is 0.
//
// Measured, 256 x 256 tiles, medians of the kernel once the clock has settled: 8-bit 4096 x 4096 x 11008
// 127 us, 2.9 POP/s of the 4.0 that the matrix cores reach on random codes in registers; dA = dC B^T 4096
// x 4096 x 22016 484 us, 1.53 PFLOP/s of 2.0; of dB = A^T dC 4096 x 22016 x 4096 the 1280 tiles of its full
// waves 558 us, 1.23, and as many of the forward 542 us, 1.27 (after an idle spell 130, 486, 577 and 578). What bounds them, from timing-only
// copies that leave one part out (us, in that order, the whole 124, 470, 556, and 666 for the forward's
// 1376 tiles): without the copies 105, 362, 443, 478; without the operand reads 113, 469, 451, 641;
// without the MFMAs 84, 430, 360, 474; the operand reads alone 59, 187, 280, 273. dA waits
// mostly for its copies (32 KB a k-step from the L2 into each CU); in the others copies and MFMAs weigh
// alike, and in dB the reads too: a transposing read of a k-step's operands takes 0.44 us, a plain one 0.27.
// Where the copied lines come from does not matter (all tiles on the same panels: dA 459, dB 552), nor
// do wave priorities, copies issued before the reads, or tile rows walked in groups of 8 for 4 (all
// within 1%). Four waves of 128 x 128, which read a third less from LDS, gained nothing (dB 597-608
// against 599).

#include "ops_tile.h"

namespace glk {

template <int MODE, bool GLU>
__global__ void __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2, 2)))
op_pp_kernel(OpTileArgs p) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    op_pp<MODE, GLU>(p, op_place<256, GLU ? 128 : 256>(p, (int)blockIdx.x), lds);
}

template <int BT, int MODE, bool GLU>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
op_small_kernel(OpTileArgs p) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    op_small<BT, MODE, GLU>(p, op_place<BT, GLU ? BT / 2 : BT>(p, (int)blockIdx.x), lds);
}

// Both gradients of a product in one launch: dA = dC B^T first, dB = A^T dC after. They share dC and
// neither fills the card when it is small.
template <int BT>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
op_pair_kernel(OpTileArgs pa, OpTileArgs pb) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int first = pa.tiles_m * pa.tiles_n * pa.splits;
    if ((int)blockIdx.x < first)
        op_small<BT, kOpAbt, false>(pa, op_place<BT, BT>(pa, (int)blockIdx.x), lds);
    else
        op_small<BT, kOpAtb, false>(pb, op_place<BT, BT>(pb, (int)blockIdx.x - first), lds);
}

template <int MODE, bool GLU>
static hipError_t launch_mode(int tile, const OpTileArgs& a, int grid, hipStream_t s) {
    if (tile == 256) {
        if (a.splits != 1) return hipErrorInvalidValue;
        op_pp_kernel<MODE, GLU><<<grid, 512, OpTile<256, 256, 2, 4, MODE>::LDS_BYTES, s>>>(a);
    } else if (tile == 128) {
        op_small_kernel<128, MODE, GLU><<<grid, 256, OpTile<128, 128, 2, 2, MODE>::LDS_BYTES, s>>>(a);
    } else {
        op_small_kernel<64, MODE, GLU><<<grid, 256, OpTile<64, 64, 2, 2, MODE>::LDS_BYTES, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_op_tile(int mode, bool glu, int tile, const OpTileArgs& a, int grid, hipStream_t s) {
    switch (mode) {
        case kOpI8: return glu ? launch_mode<kOpI8, true>(tile, a, grid, s) : launch_mode<kOpI8, false>(tile, a, grid, s);
        case kOpAbt: return launch_mode<kOpAbt, false>(tile, a, grid, s);
        case kOpAtb: return launch_mode<kOpAtb, false>(tile, a, grid, s);
        case kOpTrain: return launch_mode<kOpTrain, true>(tile, a, grid, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_op_pair(int tile, const OpTileArgs& a, const OpTileArgs& b, int grid, hipStream_t s) {
    if (tile == 128)
        op_pair_kernel<128><<<grid, 256, OpTile<128, 128, 2, 2, kOpAbt>::LDS_BYTES, s>>>(a, b);
    else
        op_pair_kernel<64><<<grid, 256, OpTile<64, 64, 2, 2, kOpAbt>::LDS_BYTES, s>>>(a, b);
    return hipGetLastError();
}

static hipError_t set_lds(const void* kernel, int bytes) {
    return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// (the 64 x 64 kernels ask for 40 KB, which needs no setting)
template <int MODE, bool GLU>
static hipError_t configure_mode() {
    hipError_t e = set_lds((const void*)op_pp_kernel<MODE, GLU>, OpTile<256, 256, 2, 4, MODE>::LDS_BYTES);
    if (e == hipSuccess)
        e = set_lds((const void*)op_small_kernel<128, MODE, GLU>, OpTile<128, 128, 2, 2, MODE>::LDS_BYTES);
    return e;
}

hipError_t configure_op_kernels() {
    hipError_t e = configure_mode<kOpI8, false>();
    if (e == hipSuccess) e = configure_mode<kOpI8, true>();
    if (e == hipSuccess) e = configure_mode<kOpAbt, false>();
    if (e == hipSuccess) e = configure_mode<kOpAtb, false>();
    if (e == hipSuccess) e = configure_mode<kOpTrain, true>();
    if (e == hipSuccess) e = set_lds((const void*)op_pair_kernel<128>, OpTile<128, 128, 2, 2, kOpAbt>::LDS_BYTES);
    return e;
}

}  // namespace glk
