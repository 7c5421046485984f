// The tiles of the 8-bit floating point product (f8.hip) and what they cost, for plan_product.
#pragma once

#include "product.h"

namespace ltx3drope {

struct OpF8 {
    using Acc = f32x4;
    using Sum = float;
    static constexpr int kElem = 1;
};

// Fitted to products in us (bf16 out; whole calls), each tile with its best split:
//                            256x256  256x128  128x64  64x64
//     4096 x  4096, k 4096     68.6     78.4   102.8   146.4
//     2048 x  4096, k 4096     56.5     40.1    60.3    80.4
//     1024 x  4096, k 4096     37.8     34.7    33.7    41.7
//      512 x  8192, k 2048     32.5     22.3    19.5    24.8
//      128 x 10240, k 4096     27.7     24.0    25.2    21.2
//      300 x  1000, k 5696     23.9     20.9    18.7    16.3
//     4095 x   576, k 4672     38.0     31.7    32.8    38.7
// Outputs in fp32 (bf16's instructions) have the same order but for the wide tiles, which are 4 to 20 % apart.
template <>
inline constexpr TileCost kTileCosts<OpF8>[4] = {
    {256, 256, 1.9f, 1.9f, 1.0f, 1.1f, 7.0f},
    {256, 128, 0.75f, 1.1f, 1.0f, 1.2f, 4.0f},
    {128, 64, 0.65f, 0.36f, 1.0f, 1.42f, 1.2f},
    {64, 64, 0.32f, 0.26f, 1.0f, 1.5f, 0.8f},
};

}  // namespace ltx3drope
