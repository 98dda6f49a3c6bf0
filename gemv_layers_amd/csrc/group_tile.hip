// Matrix kernels of the bf16 products grouped by expert for gfx950: the tiles, copies, schedules and epilogue of
// ops_tile.h, each workgroup finding its group and tile in the row offsets on the device (group.h).
//
// C_e = A_e B_e and dA_e = dC_e B_e^T have row tiles of any group; dB_e = A_e^T dC_e has every group's tiles, summed over
// its rows. A last row tile of a group works for as many rows as it holds and takes as long as a full one, and tiles of
// uneven groups leave CUs idle in the last round: 8192 rows, 4096 to 11008, as one product 558 us (1.32 PFLOP/s), dA 477,
// dB 590; in 8 even groups 605, 524 and 677; as an uneven router left them 635, 600 and 690 (1.16, 1.23, 1.07). Beyond that they
// are bound as op_pp is: copies, L2 to LDS, and matrix cores alike, at the power limit.
// Few rows are a stream of weights in 64 x 64 tiles: 16 rows, 7 of 8 groups, 4096 to 1376, 79 MB, 17.8 us (4.4 TB/s).
// Small products are one launch and the latency of their k-steps: 600 rows in 8 groups, 328 to 520, 5.6 us; both gradients
// of 1018 rows, 512 to 1376, 14.2 in one launch and 9.7 + 7.8 in two.

#include "group_tile.h"

namespace glk {

template <int MODE>
__global__ void __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2, 2)))
group_pp_kernel(OpTileArgs p, GroupArgs g) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    OpPlace at;
    if (group_tile<MODE, 256>(p, g, (int)blockIdx.x, &at)) op_pp<MODE, false, MODE != kOpAtb>(p, at, lds);
}

template <int BT, int MODE>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
group_small_kernel(OpTileArgs p, GroupArgs g) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    OpPlace at;
    if (group_tile<MODE, BT>(p, g, (int)blockIdx.x, &at)) op_small<BT, MODE, false>(p, at, lds);
}

// Both gradients in one launch: dA = dC B^T first, dB = A^T dC after.
template <int BT>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
group_pair_kernel(OpTileArgs pa, GroupArgs ga, int grid_a, OpTileArgs pb, GroupArgs gb) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    OpPlace at;
    if ((int)blockIdx.x < grid_a) {
        if (group_tile<kOpAbt, BT>(pa, ga, (int)blockIdx.x, &at)) op_small<BT, kOpAbt, false>(pa, at, lds);
    } else {
        if (group_tile<kOpAtb, BT>(pb, gb, (int)blockIdx.x - grid_a, &at)) op_small<BT, kOpAtb, false>(pb, at, lds);
    }
}

template <int MODE>
static hipError_t launch_mode(int tile, const OpTileArgs& a, const GroupArgs& g, int grid, hipStream_t s) {
    if (tile == 256) {
        if (a.splits != 1) return hipErrorInvalidValue;
        group_pp_kernel<MODE><<<grid, 512, OpTile<256, 256, 2, 4, MODE>::LDS_BYTES, s>>>(a, g);
    } else if (tile == 128) {
        group_small_kernel<128, MODE><<<grid, 256, OpTile<128, 128, 2, 2, MODE>::LDS_BYTES, s>>>(a, g);
    } else {
        group_small_kernel<64, MODE><<<grid, 256, OpTile<64, 64, 2, 2, MODE>::LDS_BYTES, s>>>(a, g);
    }
    return hipGetLastError();
}

hipError_t launch_group_tile(int mode, int tile, const OpTileArgs& a, const GroupArgs& g, int grid, hipStream_t s) {
    switch (mode) {
        case kOpAb: return launch_mode<kOpAb>(tile, a, g, grid, s);
        case kOpAbt: return launch_mode<kOpAbt>(tile, a, g, grid, s);
        case kOpAtb: return launch_mode<kOpAtb>(tile, a, g, grid, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_group_pair(int tile, const OpTileArgs& a, const GroupArgs& ga, int grid_a, const OpTileArgs& b,
                             const GroupArgs& gb, int grid_b, hipStream_t s) {
    if (tile == 128)
        group_pair_kernel<128><<<grid_a + grid_b, 256, OpTile<128, 128, 2, 2, kOpAbt>::LDS_BYTES, s>>>(a, ga, grid_a, b, gb);
    else
        group_pair_kernel<64><<<grid_a + grid_b, 256, OpTile<64, 64, 2, 2, kOpAbt>::LDS_BYTES, s>>>(a, ga, grid_a, b, gb);
    return hipGetLastError();
}

static hipError_t set_lds(const void* kernel, int bytes) {
    return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// (the 64 x 64 kernels ask for 40 KB, which needs no setting)
template <int MODE>
static hipError_t configure_mode() {
    hipError_t e = set_lds((const void*)group_pp_kernel<MODE>, OpTile<256, 256, 2, 4, MODE>::LDS_BYTES);
    if (e == hipSuccess)
        e = set_lds((const void*)group_small_kernel<128, MODE>, OpTile<128, 128, 2, 2, MODE>::LDS_BYTES);
    return e;
}

hipError_t configure_group_kernels() {
    hipError_t e = configure_mode<kOpAb>();
    if (e == hipSuccess) e = configure_mode<kOpAbt>();
    if (e == hipSuccess) e = configure_mode<kOpAtb>();
    if (e == hipSuccess) e = set_lds((const void*)group_pair_kernel<128>, OpTile<128, 128, 2, 2, kOpAbt>::LDS_BYTES);
    return e;
}

}  // namespace glk
