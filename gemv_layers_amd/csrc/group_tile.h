// Where a workgroup of a grouped product on MFMA tiles works (device side).
#pragma once

#include "group.h"
#include "ops_tile.h"

namespace glk {

// Narrows p to the group and tile of workgroup `block`; false where there is none. Rows of no group are a product
// over nothing, which writes zeros.
template <int MODE, int BT>
__device__ __forceinline__ bool group_tile(OpTileArgs& p, const GroupArgs& g, int block, OpPlace* at) {
    constexpr int ES = MODE == kOpF8 ? 1 : 2;
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    if constexpr (MODE == kOpAtb) {
        // groups in turn, each over all XCDs: with an XCD's contiguous share of all groups' tiles, the one of the
        // largest group worked longest (8192 rows in 8 uneven groups, 4096 x 11008: 963 us against 677 of even ones)
        const int tiles = p.tiles_m * p.tiles_n, per = tiles * p.splits, group = uni(block / per);
        int first, rows;
        group_rows(g, group, &first, &rows);
        *at = op_place_unit<BT, BT>(p, xcd_remap(block - group * per, per, p.nxcd));
        at->tile += group * tiles;
        p.A = static_cast<const char*>(p.A) + (int64_t)first * p.lda * ES;
        p.B = static_cast<const char*>(p.B) + (int64_t)first * p.ldb * ES;
        p.C += group * g.stride_c;
        p.K = rows;
        const int steps = (rows + 31) / 32;
        p.kt_per_split = uni((steps + p.splits - 1) / p.splits);
    } else {
        GroupSpan s;
        if (!find_span(g, BT, p.tiles_n * p.splits, p.nxcd, block, &s)) return false;
        p.tiles_m = s.tiles;
        *at = op_place_unit<BT, BT>(p, s.unit);
        at->tile += s.tile * p.tiles_n;
        p.A = static_cast<const char*>(p.A) + (int64_t)s.first * p.lda * ES;
        p.C += (int64_t)s.first * p.ldc;
        p.M = s.rows;
        if (s.group < 0)
            p.K = 0;
        else
            p.B = static_cast<const char*>(p.B) + s.group * g.stride_b * ES;
        if constexpr (MODE == kOpF8) {
            p.sa += s.first;
            p.sb += max(s.group, 0) * g.stride_sb;
        }
    }
    return true;
}

}  // namespace glk
