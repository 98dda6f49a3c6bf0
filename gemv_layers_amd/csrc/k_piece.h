// The pieces of a tile's summed index where its product is cut in equal shares of whole lines. Plain C++ with no GPU
// dependency, so host code and tests use the same function.
#pragma once

#include "stream_k.h"

namespace glk {

struct KPiece {
    int32_t first, count;
};

// Piece `piece` of `pieces` of an index of K elements: whole lines of `line` elements each (a short one last). Shares are
// rounded up, so that a last piece may start past the end: it is empty, at 0. (K at most 2^26, pieces at most 16.)
GLK_HD inline KPiece k_piece(int32_t K, int32_t line, int32_t pieces, int32_t piece) {
    const int32_t lines = K / line + (K % line != 0), share = (lines + pieces - 1) / pieces * line;
    const int32_t first = piece * share, left = K - first;
    if (left <= 0) return KPiece{0, 0};
    return KPiece{first, left < share ? left : share};
}

}  // namespace glk
