// Prints plans of the 8-bit and training products: for each line "tile M N K cus glu contiguous" or "decode M N
// K cus glu 0" of the input, one JSON line {"plan": ..., "counters": ..., "fits": ...}. Linked to the library.
#include <iostream>
#include <string>

#include "plan.h"

int main() {
    std::string kind;
    int64_t M, N, K;
    int cus, glu, contiguous;
    while (std::cin >> kind >> M >> N >> K >> cus >> glu >> contiguous) {
        glk::DeviceInfo dev;
        dev.cus = cus;
        dev.nxcd = cus % 8 == 0 ? 8 : 1;
        dev.ws_floats = int64_t(8) << 20;
        dev.ws_counters = int64_t(1) << 16;
        const bool tile = kind == "tile";
        const glk::Plan p = tile ? glk::make_op_plan(M, N, K, dev, glu != 0, contiguous != 0)
                                 : glk::make_i8_decode_plan(M, N, K, dev, glu != 0);
        std::cout << "{\"plan\": " << glk::plan_json(p, M, N, K) << ", \"counters\": " << p.counters
                  << ", \"fits\": " << (!tile && glk::i8_decode_fits(M, K, p) ? "true" : "false") << "}\n";
    }
}
