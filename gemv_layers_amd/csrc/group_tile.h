// Where a workgroup of a grouped product on MFMA tiles works (device side).
#pragma once

#include "group.h"
#include "k_piece.h"
#include "ops_tile.h"

namespace glk {

// 256 x 256 tiles, one a CU: the tiles of whole rounds, then those of a last round, where there are at least two slots of the
// workspace and two CUs for each, in up to g.tail pieces of K as far as both go. 32 MiB are 128 slots of 256 KB: of 256 CUs a
// last round of at most 64 tiles, a quarter, is cut, and fills at most half of them. The host cannot tell how many tiles
// the groups make. 8192 rows in 8 groups, 4096 to 11008: 1548 tiles, 12 past six rounds, 666 us whole and 640 in pieces;
// the gradient of its rows, 576 tiles, 64 past two rounds, 680 and 605.
struct TailUnits {
    const GroupArgs& g;
    int block, nxcd;
    int tile = 0, piece = 0, pieces = 1;  // of a tile in pieces: which, and of how many
    __device__ __forceinline__ bool operator()(int total, int* unit) {
        const int rest = total % g.cus;
        pieces = rest > 0 ? min(min(g.slots / rest, g.cus / rest), g.tail) : 1;
        if (pieces < 2) {
            pieces = 1;
            return EvenUnits{block, nxcd}(total, unit);
        }
        const int whole = total - rest, at = block - whole;
        if (at < 0) {
            pieces = 1;
            return EvenUnits{block, nxcd}(whole, unit);
        }
        if (at >= rest * pieces) return false;
        tile = at / pieces;
        piece = at - tile * pieces;
        *unit = whole + tile;
        return true;
    }
};

// Narrows p to the group and tile of workgroup `block`; false where there is none. Rows of no group are a product
// over nothing, which writes zeros.
template <int MODE, int BT, class Args>
__device__ __forceinline__ bool group_tile(Args& p, const GroupArgs& g, int block, OpPlace* at) {
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
        TailUnits tail{g, block, p.nxcd};
        if constexpr (BT == 256) {
            if (!find_span(g, BT, p.tiles_n, tail, &s)) return false;
        } else {
            if (!find_span(g, BT, p.tiles_n * p.splits, EvenUnits{block, p.nxcd}, &s)) return false;
        }
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
        if (BT == 256 && tail.pieces > 1) {  // whole 128-byte lines of a contiguous operand
            const KPiece piece = k_piece(p.K, 128 / ES, tail.pieces, tail.piece);
            const int k0 = uni(piece.first);
            p.K = uni(piece.count);
            if (p.K > 0) {
                p.A = static_cast<const char*>(p.A) + (int64_t)k0 * ES;
                p.B = static_cast<const char*>(p.B) + (MODE == kOpAb ? (int64_t)k0 * p.ldb : (int64_t)k0) * ES;
                if constexpr (MODE == kOpF8) {
                    p.sa += k0 / 128 * p.ldsa;
                    p.sb += k0 / 128;
                }
            }
            p.splits = uni(tail.pieces);
            at->tile = uni(tail.tile);
            at->piece = uni(tail.piece);
        }
    }
    return true;
}

}  // namespace glk
