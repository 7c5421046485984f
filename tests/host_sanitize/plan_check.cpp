// The tile, the split of the sums and the way of the operands that the block's matrix products choose
// (product.h), for the sizes on standard input: a line "op gated outer M N k direct pitch" gives a line
// "bm bn tiles splits bytes".  Built for the host alone; no kernel is instantiated.
#include <cstdio>
#include <cstring>

#include "product.h"

using namespace ltx3drope;

namespace {

template <class Op>
Plan plan(int gated, int outer, uint32_t M, uint32_t N, uint32_t k, bool direct, uint64_t pitch) {
    if (gated) return plan_product<Op, true, false>(M, N, k, direct, pitch);
    return outer ? plan_product<Op, false, true>(M, N, k, direct, pitch)
                 : plan_product<Op, false, false>(M, N, k, direct, pitch);
}

}  // namespace

int main() {
    char op[8];
    int gated, outer, direct;
    unsigned M, N, k;
    unsigned long long pitch;
    while (std::scanf("%7s %d %d %u %u %u %d %llu", op, &gated, &outer, &M, &N, &k, &direct, &pitch) == 8) {
        Plan p{};
        if (std::strcmp(op, "bf16") == 0) p = plan<OpBf16>(gated, outer, M, N, k, direct != 0, pitch);
        else if (std::strcmp(op, "f32") == 0) p = plan<OpF32>(gated, outer, M, N, k, direct != 0, pitch);
        else if (std::strcmp(op, "int8") == 0) p = plan<OpI8>(gated, outer, M, N, k, direct != 0, pitch);
        else return 1;
        std::printf("%u %u %u %u %zu\n", p.bm, p.bn, p.tiles, p.splits, p.partial_bytes);
    }
    return 0;
}
