// The tile and the split of the sums that the 8-bit floating point product chooses (f8_plan.h, product.h), for the
// sizes on standard input: a line "M N k direct pitch" gives a line "bm bn tiles splits bytes".  Built for the
// host alone; no kernel is instantiated.
#include <cstdio>

#include "f8_plan.h"

using namespace ltx3drope;

int main() {
    int direct;
    unsigned M, N, k;
    unsigned long long pitch;
    while (std::scanf("%u %u %u %d %llu", &M, &N, &k, &direct, &pitch) == 5) {
        const Plan p = plan_product<OpF8, false, false>(M, N, k, direct != 0, pitch);
        std::printf("%u %u %u %u %zu\n", p.bm, p.bn, p.tiles, p.splits, p.partial_bytes);
    }
    return 0;
}
