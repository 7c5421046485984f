// Sine and cosine of the rotation with several axes, from the fraction of a turn.
//
// Four times the fraction is split into a whole number of quarters and a rest r of at most half a quarter, exactly;
// sine and cosine of r quarters are polynomials of degree 7 and 8 in fp32, fitted to the least largest error.  With the
// coefficients rounded to fp32 they are off by 3.1e-9 and 6.7e-9; r's own rounding to fp32 moves the angle by up to
// 2.3e-8, and with the roundings on the way the results are within 9.4e-8 (7.3e-8 over two million fractions).
//
// Only IEEE operations and explicit fused multiply-adds, so that a host program that defines the two
// qualifiers empty gets the device's bits.
#pragma once

#include <stdint.h>

namespace ltx3drope {

struct CosSin {
    float c, s;
};

// part: 0 <= part < 1 of a turn.  Adding 1.5 * 2^52 leaves the quarters in the sum's low bits.
__host__ __device__ inline CosSin cos_sin_of_turn(double part) {
    const double shifted = __builtin_fma(part, 4.0, 0x1.8p52);
    const uint32_t k = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, shifted));  // 0 to 4
    const float r = static_cast<float>(__builtin_fma(part, 4.0, 0x1.8p52 - shifted));  // quarters, |r| <= 1/2
    const float z = r * r;
    float p = __builtin_fmaf(z, -4.5922891e-3f, 7.9675903e-2f);
    p = __builtin_fmaf(z, __builtin_fmaf(z, p, -6.4596294e-1f), -6.5420830e-8f);
    const float s = __builtin_fmaf(r, 1.57079637f, r * p);
    float c = __builtin_fmaf(z, 9.0402167e-4f, -2.0860289e-2f);
    c = __builtin_fmaf(z, __builtin_fmaf(z, __builtin_fmaf(z, c, 2.5366924e-1f), -1.2337005f), 1.f);
    // a quarter more: (c, s) -> (-s, c)
    const float a = k & 1 ? s : c, b = k & 1 ? c : s;
    return CosSin{__builtin_bit_cast(float, __builtin_bit_cast(uint32_t, a) ^ ((k + 1) << 30 & 0x80000000u)),
                  __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, b) ^ (k << 30 & 0x80000000u))};
}

}  // namespace ltx3drope
