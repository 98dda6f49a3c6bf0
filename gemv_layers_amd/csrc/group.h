// Which rows a workgroup of a grouped product takes (device side). The groups' row offsets are data on the
// device: the host sizes a grid for the most tiles that any offsets could make, and every workgroup finds
// its tile in them.
//
// The rows 0 .. rows - 1 are cut into spans: those before the first offset, each group's, and those after the
// last offset. An offset counts as the largest of itself, the ones before it and 0, and as `rows` beyond that:
// the spans are disjoint and in range whatever the offsets hold. A wave reads 64 offsets, or 256 at a time where
// there are more, and their running maximum and the sum of the spans' tiles are scans over the lanes (six data-parallel
// steps each, no LDS and no barrier): about 0.5 us with the load, against a launch more for a table of tiles. Four offsets
// a lane cost 0.2 us more than one and save passes: 600 rows in 8 groups, 520 x 328, 5.6 us with one and 5.8 with four;
// 8192 in 256, 2048 to 768 in codes, 96.5 and 93.3.
#pragma once

#include "common.h"
#include "ops.h"

namespace glk {

// v with lane i's operand from lane i - SHIFT's scan: the inclusive scan of 64 lanes by `f`, `id` its identity
template <class F>
__device__ __forceinline__ int wave_scan(int v, int id, F f) {
#define GLK_SCAN(ctrl, rows) v = f(v, __builtin_amdgcn_update_dpp(id, v, ctrl, rows, 0xF, false))
    GLK_SCAN(0x111, 0xF);  // row_shr 1, 2, 4, 8 within rows of 16 lanes
    GLK_SCAN(0x112, 0xF);
    GLK_SCAN(0x114, 0xF);
    GLK_SCAN(0x118, 0xF);
    GLK_SCAN(0x142, 0xA);  // row_bcast15 into rows 1 and 3, row_bcast31 into rows 2 and 3
    GLK_SCAN(0x143, 0xC);
#undef GLK_SCAN
    return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {
    return wave_scan(v, 0, [](int a, int b) { return max(a, b); });  // (values of 0 and more)
}
__device__ __forceinline__ int wave_scan_add(int v) {
    return wave_scan(v, 0, [](int a, int b) { return a + b; });
}

struct GroupSpan {
    int group;        // -1: rows of no group
    int first, rows;
    int tiles, tile;  // row tiles of this span, and of all before it
    int unit;         // the workgroup's unit among the span's tiles * per
};

// Which unit of `total` workgroup `block` takes, or false for none: each XCD a contiguous share.
struct EvenUnits {
    int block, nxcd;
    __device__ __forceinline__ bool operator()(int total, int* unit) const {
        if (block >= total) return false;
        *unit = xcd_remap(block, total, nxcd);
        return true;
    }
};

template <int R, class Which>
__device__ __forceinline__ bool search_spans(const GroupArgs& g, int bm, int per, Which&& which, GroupSpan* out) {
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    int unit;
    const int lane = threadIdx.x & 63, spans = g.groups + 2;
    constexpr int WAVE = 64 * R;  // spans of a pass, whose loads are in flight together
    // of spans s0 + R * lane + j: their ends and the tiles up to them; the next pass starts at row, tiles
    struct Part {
        int before, end[R], base, upto[R];
    };
    auto part = [&](int s0, int& row, int& tiles) {
        Part p;
        int local[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int s = s0 + R * lane + j;
            p.end[j] = s <= g.groups ? g.offsets[s] : g.rows;
        }
#pragma unroll
        for (int j = 0; j < R; ++j) p.end[j] = max(min(max(p.end[j], 0), g.rows), j ? p.end[j - 1] : 0);
        const int most = wave_scan_max(p.end[R - 1]);
        p.before = max(__builtin_amdgcn_update_dpp(0, most, 0x138, 0xF, 0xF, false), row);  // wave_shr 1
#pragma unroll
        for (int j = 0; j < R; ++j) {
            p.end[j] = max(p.end[j], p.before);
            local[j] = (p.end[j] - (j ? p.end[j - 1] : p.before) + bm - 1) / bm + (j ? local[j - 1] : 0);
        }
        p.base = wave_scan_add(local[R - 1]) - local[R - 1] + tiles;
#pragma unroll
        for (int j = 0; j < R; ++j) p.upto[j] = p.base + local[j];
        row = __builtin_amdgcn_readlane(p.end[R - 1], 63);
        tiles = __builtin_amdgcn_readlane(p.upto[R - 1], 63);
        return p;
    };
    int row = 0, total = 0;
    Part p = part(0, row, total);
    for (int s0 = WAVE; s0 < spans; s0 += WAVE) part(s0, row, total);
    if (!which(total * per, &unit)) return false;
    unit = uni(unit);
    const int tile = uni(unit / per);
    int s0 = 0, upto = 0;
    row = 0;
    if (spans > WAVE) p = part(0, row, upto);
    uint64_t hit;
    while (!(hit = __ballot(tile < p.upto[R - 1]))) {
        s0 += WAVE;
        if (s0 >= spans) return false;  // (offsets that changed since the first pass)
        p = part(s0, row, upto);
    }
    const int at = __builtin_ctzll(hit);
    // of that lane's spans the first whose tiles go past it
    int j = 0, first = p.before, last = p.end[0], from = p.base, to = p.upto[0];
#pragma unroll
    for (int i = 1; i < R; ++i) {
        const bool past = tile >= p.upto[i - 1];
        j = past ? i : j;
        first = past ? p.end[i - 1] : first;
        last = past ? p.end[i] : last;
        from = past ? p.upto[i - 1] : from;
        to = past ? p.upto[i] : to;
    }
    const int s = s0 + R * at + __builtin_amdgcn_readlane(j, at);
    GroupSpan r;
    r.group = s >= 1 && s <= g.groups ? s - 1 : -1;
    r.first = __builtin_amdgcn_readlane(first, at);
    r.rows = __builtin_amdgcn_readlane(last, at) - r.first;
    r.tile = __builtin_amdgcn_readlane(from, at);
    r.tiles = __builtin_amdgcn_readlane(to, at) - r.tile;
    r.unit = unit - r.tile * per;
    *out = r;
    return true;
}

// The span and unit of a workgroup for row tiles of `bm` rows, each of `per` units, as `which` picks the unit of all in
// order of rows, or false where it picks none. Every lane of the wave calls it.
template <class Which>
__device__ __forceinline__ bool find_span(const GroupArgs& g, int bm, int per, Which&& which, GroupSpan* out) {
    if (!g.offsets) {
        const int tiles = (g.rows - 1) / bm + 1;
        int unit;
        if (!which(tiles * per, &unit)) return false;
        *out = GroupSpan{0, 0, g.rows, __builtin_amdgcn_readfirstlane(tiles), 0, __builtin_amdgcn_readfirstlane(unit)};
        return true;
    }
    if (g.groups + 2 <= 64) return search_spans<1>(g, bm, per, which, out);
    return search_spans<4>(g, bm, per, which, out);
}

// The rows of group `e` (as find_span cuts them). Every lane of the wave calls it.
__device__ __forceinline__ void group_rows(const GroupArgs& g, int e, int* first, int* rows) {
    if (!g.offsets) {
        *first = 0;
        *rows = g.rows;
        return;
    }
    const int lane = threadIdx.x & 63;
    int most = 0;
    for (int i = lane; i <= e; i += 64) most = max(most, g.offsets[i]);
    const int end = g.offsets[e + 1];
    const int start = min(__builtin_amdgcn_readlane(wave_scan_max(most), 63), g.rows);
    *first = start;
    *rows = __builtin_amdgcn_readfirstlane(max(min(end, g.rows), start)) - start;
}

}  // namespace glk
