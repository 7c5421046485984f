// Rotary positions with several axes: what the host side (axes_api.cpp) hands to the kernel's launcher (axes.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "fastdiv.h"

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

// Accesses of `vector` elements: the pairs of a lane's unit, the registers of one access, and the rounds of a wavefront
// (16 registers of channels a lane, as many bytes on their way).
constexpr uint32_t axes_unit_accesses(bool halves, uint32_t vector) { return halves || vector == 1 ? 2 : 1; }
constexpr uint32_t axes_unit_pairs(bool halves, uint32_t vector) { return halves || vector == 1 ? vector : vector / 2; }
constexpr uint32_t axes_access_words(bool f32, uint32_t vector) { return f32 ? vector : (vector + 1) / 2; }
constexpr uint32_t axes_rounds(bool f32, bool halves, uint32_t vector) {
    const uint32_t r = 16 / (axes_unit_accesses(halves, vector) * axes_access_words(f32, vector));
    return r < 16 ? r : 16;
}

// The shape of a launch (axes.hip says what it is made of).
struct AxesShape {
    uint32_t segments;   // of pairs
    uint32_t copies;     // segments of channels that pass through, 0: they belong to the last one of pairs
    uint32_t seg_pairs;  // pairs of a segment (the last may have fewer)
    uint32_t slots;      // most heads side by side in a wavefront
    uint32_t q_rounds;
    uint32_t rounds;     // of q and k
    uint32_t together;   // tokens whose rounds are one wavefront's; 0: a token has groups of rounds, q's
    uint32_t q_groups;   // before k's in the grid
    uint32_t k_groups;
    FastDiv by_planes, by_q_groups, by_k_groups, by_axes, by_pairs;
};

constexpr uint32_t kMostAngles = 512;  // of several tokens

inline AxesShape axes_shape(const AxesProblem& p) {
    const uint32_t kPairs = axes_unit_pairs(p.halves, p.vector), kRounds = axes_rounds(p.f32, p.halves, p.vector);
    const uint32_t kElem = p.f32 ? 4 : 2;
    AxesShape s;
    const uint32_t tail = (p.head_dim - 2 * p.pairs) / p.vector, most_pairs = 64 * kPairs;
    s.segments = (p.pairs + most_pairs - 1) / most_pairs;
    s.seg_pairs = p.pairs < most_pairs ? p.pairs : most_pairs;
    const uint32_t last = p.pairs - (s.segments - 1) * s.seg_pairs;
    s.copies = last / kPairs + tail <= 64 ? 0 : (tail + 63) / 64;
    const uint32_t planes = s.segments + s.copies;
    // heads side by side, as many as fit in every segment; what a lane adds to the first one's address stays below 2^31
    int64_t head = 1;
    for (const AxesTensor* t : {&p.q, &p.k}) {
        head = head > t->in_head ? head : t->in_head;
        head = head > t->out_head ? head : t->out_head;
    }
    const int64_t reach = (int64_t(1) << 30) / (head * kElem);
    const uint32_t units = planes > 1 ? 64 : s.seg_pairs / kPairs + tail;
    s.slots = reach < 63 && static_cast<uint32_t>(reach) + 1 < 64 / units ? static_cast<uint32_t>(reach) + 1 : 64 / units;
    s.q_rounds = (p.q.heads + s.slots - 1) / s.slots;
    s.rounds = s.q_rounds + (p.k.heads + s.slots - 1) / s.slots;
    s.together = s.rounds <= kRounds ? 1 : 0;
    if (s.together && static_cast<uint64_t>(p.tokens) * p.batch * planes >= 16384) {
        // several tokens, if that leaves wavefronts enough to fill the chip
        const uint32_t rows = kMostAngles / s.seg_pairs, places = 64 / p.axes;
        uint32_t t = kRounds / s.rounds;
        t = t < rows ? t : rows;
        t = t < places ? t : places;
        s.together = t > 1 ? t : 1;
    }
    s.q_groups = (s.q_rounds + kRounds - 1) / kRounds;
    s.k_groups = (s.rounds - s.q_rounds + kRounds - 1) / kRounds;
    s.by_planes = make_fastdiv(planes);
    s.by_q_groups = make_fastdiv(s.q_groups ? s.q_groups : 1);
    s.by_k_groups = make_fastdiv(s.k_groups ? s.k_groups : 1);
    s.by_axes = make_fastdiv(p.axes);
    s.by_pairs = make_fastdiv(s.seg_pairs);
    return s;
}

// Workgroups of one token, or of `together` tokens: 2^25 at most (65536 + 65536 heads of 65536 channels).
inline uint32_t axes_jobs(const AxesShape& s) {
    return (s.segments + s.copies) * (s.together ? 1 : s.q_groups + s.k_groups);
}

// Tokens of one launch, one at the least: its workgroups of 64 threads have fewer than 2^32 threads between them.
inline uint32_t axes_launch_tokens(const AxesShape& s) { return ((uint32_t(1) << 26) - 1) / axes_jobs(s); }

// Workgroups of a launch of `tokens` tokens.
inline uint32_t axes_launch_groups(const AxesShape& s, uint32_t tokens) {
    return (s.together > 1 ? (tokens + s.together - 1) / s.together : tokens) * axes_jobs(s);
}

hipError_t launch_axes(const AxesProblem& p, hipStream_t stream);

}  // namespace ltx3drope
