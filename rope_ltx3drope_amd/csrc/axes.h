// Rotary positions with several axes: what the host side (axes_api.cpp) hands to the kernel's launcher (axes.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ltx3drope {

struct AxesTensor {  // [batch, tokens, heads, head_dim], head_dim innermost, strides in elements
    const char* in;
    char* out;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;
    uint32_t heads;
};

struct AxesProblem {
    AxesTensor q, k;
    const void* positions;  // strides in elements
    int64_t position_axis, position_batch, position_token;
    const void* frequencies;  // [pairs], radians a unit of position
    const uint8_t* axis;      // [pairs]
    uint32_t batch, tokens, head_dim, pairs, axes;
    uint32_t first_token;  // of a launch's tokens
    bool f32, halves, inverse, frequency_f32;
    uint32_t vector;    // elements of an access: 16 bytes, 2 elements or 1
    int position_type;  // LTX3DROPE_POSITION_*
};

constexpr int64_t kAxesMaxWidth = 65536;  // head_dim
constexpr int64_t kAxesMaxHeads = 65536;  // of q and of k
constexpr int64_t kAxesMaxBatch = 65535;  // one grid plane a sample

// Whether accesses of v elements cover the channels: whole accesses of rotated and of passed-through channels.  The
// pointers' and strides' alignment is checked by the host.
inline bool axes_vector_widths(uint32_t v, bool halves, uint32_t head_dim, uint32_t pairs) {
    return (halves ? pairs : 2 * pairs) % v == 0 && (head_dim - 2 * pairs) % v == 0;
}

hipError_t launch_axes(const AxesProblem& p, hipStream_t stream);

}  // namespace ltx3drope
