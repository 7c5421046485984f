// Sine and cosine of csrc/axes_math.h on the host: for each fraction of a turn on standard input (the bits of a
// double in hexadecimal) a line of the bits of its cosine and sine.  Build with __host__ and __device__ empty.
#include <cinttypes>
#include <cstdio>

#include "axes_math.h"

int main() {
    uint64_t bits;
    while (std::scanf("%" SCNx64, &bits) == 1) {
        const ltx3drope::CosSin v = ltx3drope::cos_sin_of_turn(__builtin_bit_cast(double, bits));
        std::printf("%08x %08x\n", __builtin_bit_cast(uint32_t, v.c), __builtin_bit_cast(uint32_t, v.s));
    }
    return 0;
}
