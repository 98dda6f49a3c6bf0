// Checks that the pieces of a summed index hold every element of it once, in order and in whole lines. Prints "ok" and
// exits 0, or prints the first mismatch and exits 1.
#include <stdint.h>
#include <stdio.h>

#include "k_piece.h"

static bool check(int32_t K, int32_t line, int32_t pieces) {
    int64_t end = 0;
    bool over = false;
    for (int32_t i = 0; i < pieces; ++i) {
        const glk::KPiece p = glk::k_piece(K, line, pieces, i);
        const bool empty = p.count == 0;
        if (p.count < 0 || (empty && p.first != 0) || (!empty && (over || p.first != end || p.first % line || p.first + int64_t(p.count) > K))) {
            printf("K=%d line=%d pieces=%d: piece %d is %d elements from %d, after %lld\n", K, line, pieces, i, p.count, p.first,
                   (long long)end);
            return false;
        }
        over = over || empty;
        end += p.count;
    }
    if (end != K) printf("K=%d line=%d pieces=%d: %lld elements in all\n", K, line, pieces, (long long)end);
    return end == K;
}

int main() {
    for (int32_t line = 64; line <= 128; line += 64)
        for (int32_t pieces = 1; pieces <= 16; ++pieces) {
            for (int32_t K = 0; K <= 5000; ++K)
                if (!check(K, line, pieces)) return 1;
            for (int32_t K = (1 << 26) - 5000; K <= 1 << 26; ++K)
                if (!check(K, line, pieces)) return 1;
        }
    printf("ok\n");
}
