// Prints plans of the products grouped by rows: for each line "tile rows groups M N K summed pairs strided cus" or
// "decode rows groups 0 N K 0 0 0 cus" of the input, one JSON line {"plan": ..., "counters": ..., "tail": ..., "fits": ...}. Linked to the library.
#include <iostream>
#include <string>

#include "plan.h"

int main() {
    std::string kind;
    glk::GroupShape g;
    int cus, summed, pairs, strided;
    while (std::cin >> kind >> g.rows >> g.groups >> g.M >> g.N >> g.K >> summed >> pairs >> strided >> cus) {
        glk::DeviceInfo dev;
        dev.cus = cus;
        dev.nxcd = cus % 8 == 0 ? 8 : 1;
        dev.ws_floats = int64_t(8) << 20;
        dev.ws_counters = int64_t(1) << 16;
        g.summed = summed != 0;
        g.pairs = pairs != 0;
        g.strided = strided != 0;
        const glk::Plan p = kind == "tile" ? glk::make_group_plan(g, dev) : glk::make_f8_decode_plan(g.rows, g.N, g.K, g.groups, dev);
        std::cout << "{\"plan\": " << glk::plan_json(p, g.M, g.N, g.K) << ", \"counters\": " << p.counters << ", \"tail\": " << p.tail
                  << ", \"fits\": " << (glk::f8_decode_fits(g.rows, g.groups) ? "true" : "false") << "}\n";
    }
}
