// Rotary positions with several axes: pair i of a head is turned by
//     angle = position[axis(i)][token] * frequency(i)
// whatever the token's positions are, and every head of q and k by the same angles:
//     e' = e cos - o sin,  o' = e sin + o cos         (inverse: by -angle, which is the gradient's way back)
// with (e, o) = (x[2i], x[2i+1]) or, in halves, (x[i], x[i + pairs]).
//
// Angles are formed in 64 bits: a position of 100000 times a frequency near 1 leaves fp32 0.004 of a radian.
// The angle is taken in turns, a whole number of quarters is split off (exactly), and sine and cosine of the
// rest, |x| <= pi/4, are their Taylor sums in fp32 up to x^9 and x^10 (the next terms are below 2e-9).
//
// Bound: HBM.  Each channel is read and written once; an angle costs about 35 operations and is used by all heads, so
// a workgroup forms the (cos, sin) of its tokens once, one or a few a thread, into LDS, and then streams
// the heads past them, 16 bytes a thread.  A thread keeps its place in the head, and a token's cosines in
// registers for all its heads.  The tokens' cosines lie in two LDS buffers in turn, so one barrier a step is
// enough, and the next step's positions travel while this one streams.
#include <hip/hip_runtime.h>

#include "axes.h"
#include "ltx3drope.h"

namespace ltx3drope {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kThreads = 256;
constexpr uint32_t kMaxSteps = 4;  // angles a thread forms a step

__device__ __forceinline__ f32x2 cos_sin(double position, double frequency) {
    const double turns = position * frequency * 0.15915494309189533577;  // 1 / (2 pi)
    const double part = turns - floor(turns);
    const double quarters = rint(part * 4.0);
    const float x = static_cast<float>(fma(quarters, -0.25, part) * 6.283185307179586477);
    const float z = x * x;
    const float s = fmaf(fmaf(fmaf(fmaf(2.7557319e-6f, z, -1.9841270e-4f), z, 8.3333333e-3f), z, -1.6666667e-1f) * z, x, x);
    const float c = fmaf(fmaf(fmaf(fmaf(fmaf(-2.7557319e-7f, z, 2.4801587e-5f), z, -1.3888889e-3f), z, 4.1666667e-2f), z,
                              -0.5f), z, 1.f);
    const int k = static_cast<int>(quarters);  // 0 to 4
    const float a = k & 1 ? s : c, b = k & 1 ? c : s;
    // a quarter more: (c, s) -> (-s, c)
    return f32x2{(k + 1) & 2 ? -a : a, k & 2 ? -b : b};
}

__device__ __forceinline__ double position_at(const AxesProblem& p, uint32_t axis, uint32_t b, uint32_t n) {
    const int64_t at = axis * p.position_axis + b * p.position_batch + n * p.position_token;
    if (p.position_type == LTX3DROPE_POSITION_F32) return static_cast<const float*>(p.positions)[at];
    if (p.position_type == LTX3DROPE_POSITION_I32) return static_cast<const int32_t*>(p.positions)[at];
    return static_cast<double>(static_cast<const int64_t*>(p.positions)[at]);
}

// A thread's channels of one head: U pairs of a rotated unit, or V channels that pass through.
template <bool F32, bool HALVES, bool VEC>
struct Unit {
    static constexpr int V = VEC ? (F32 ? 4 : 8) : 1;                // elements of an access
    static constexpr int U = VEC ? (HALVES ? V : 4) : 1;             // pairs
    static constexpr int N = VEC && !F32 && !HALVES ? 1 : 2;         // accesses
    static constexpr int kElem = F32 ? 4 : 2;
    static constexpr int kWords = VEC ? 4 : 1;
    uint32_t w[N][kWords];

    // byte offset of the second access from the first
    static __device__ __forceinline__ uint32_t second(uint32_t pairs) {
        return (HALVES ? pairs : VEC ? 4u : 1u) * kElem;
    }
    __device__ __forceinline__ void load(const char* at, uint32_t next, bool both) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i == 1 && !both) break;
            const char* a = at + (i ? next : 0);
            if constexpr (VEC) {
                const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a));
#pragma unroll
                for (int j = 0; j < 4; ++j) w[i][j] = v[j];
            } else if constexpr (F32) {
                w[i][0] = *reinterpret_cast<const uint32_t*>(a);
            } else {
                w[i][0] = *reinterpret_cast<const uint16_t*>(a);
            }
        }
    }
    __device__ __forceinline__ void store(char* at, uint32_t next, bool both) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i == 1 && !both) break;
            char* a = at + (i ? next : 0);
            if constexpr (VEC) {
                __builtin_nontemporal_store(u32x4{w[i][0], w[i][1], w[i][2], w[i][3]}, reinterpret_cast<u32x4*>(a));
            } else if constexpr (F32) {
                *reinterpret_cast<uint32_t*>(a) = w[i][0];
            } else {
                *reinterpret_cast<uint16_t*>(a) = static_cast<uint16_t>(w[i][0]);
            }
        }
    }
    static __device__ __forceinline__ float low(uint32_t v) { return __uint_as_float(v << 16); }
    static __device__ __forceinline__ float high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
    }
    static __device__ __forceinline__ void turn(float& e, float& o, float c, float s) {
        const float x = fmaf(e, c, -(o * s));
        o = fmaf(e, s, o * c);
        e = x;
    }
    // keep: a bit for each pair that stays as it is
    __device__ __forceinline__ void rotate(const float (&c)[U], const float (&s)[U], uint32_t keep) {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                // pair j's words: the two accesses' word j, or neighbours
                uint32_t& we = HALVES || !VEC ? w[0][j % kWords] : w[(2 * j) / kWords][(2 * j) % kWords];
                uint32_t& wo = HALVES || !VEC ? w[N - 1][j % kWords] : w[(2 * j + 1) / kWords][(2 * j + 1) % kWords];
                float e = __uint_as_float(we), o = __uint_as_float(wo);
                turn(e, o, c[j], s[j]);
                if (!(keep >> j & 1)) {
                    we = __float_as_uint(e);
                    wo = __float_as_uint(o);
                }
            }
        } else if constexpr (!VEC) {
            float e = low(w[0][0]), o = low(w[N - 1][0]);
            turn(e, o, c[0], s[0]);
            if (!keep) {
                w[0][0] = pack(e, 0.f);
                w[N - 1][0] = pack(o, 0.f);
            }
        } else if constexpr (HALVES) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float e0 = low(w[0][j]), o0 = low(w[N - 1][j]), e1 = high(w[0][j]), o1 = high(w[N - 1][j]);
                turn(e0, o0, c[(2 * j) % U], s[(2 * j) % U]);
                turn(e1, o1, c[(2 * j + 1) % U], s[(2 * j + 1) % U]);
                const uint32_t mask = (keep >> (2 * j) & 1 ? 0xffffu : 0u) | (keep >> (2 * j + 1) & 1 ? 0xffff0000u : 0u);
                w[0][j] = (w[0][j] & mask) | (pack(e0, e1) & ~mask);
                w[N - 1][j] = (w[N - 1][j] & mask) | (pack(o0, o1) & ~mask);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float e = low(w[0][j]), o = high(w[0][j]);
                turn(e, o, c[j % U], s[j % U]);
                if (!(keep >> j & 1)) w[0][j] = pack(e, o);
            }
        }
    }
};

// What a workgroup covers: a segment of the head's pairs (and, in the last one, the channels that pass
// through), or of the channels that pass through alone.
struct AxesShape {
    uint32_t segments;      // of pairs
    uint32_t copies;        // segments of channels that pass through, 0: they belong to the last one of pairs
    uint32_t seg_pairs;     // pairs of a segment (the last may have fewer)
    uint32_t steps;         // tokens a step: those that the threads cover once, times this
    uint32_t head_splits;   // workgroups that share out a token's heads
};

template <bool F32, bool HALVES, bool VEC>
__global__ __launch_bounds__(256) void axes_rotate(AxesProblem p, AxesShape shape) {
    using T = Unit<F32, HALVES, VEC>;
    constexpr uint32_t U = T::U, V = T::V, kElem = T::kElem;
    extern __shared__ __align__(16) f32x2 turns[];  // [2][tokens a step][pairs of the segment]
    const uint32_t tid = threadIdx.x;
    const uint32_t seg = blockIdx.y / shape.head_splits, split = blockIdx.y % shape.head_splits, b = blockIdx.z;
    const uint32_t first = seg * shape.seg_pairs;  // pair
    const uint32_t P = seg >= shape.segments ? 0u
                       : p.pairs - first < shape.seg_pairs ? p.pairs - first : shape.seg_pairs;

    // this thread's place in the head, and its slot among the threads that take heads in turn
    const uint32_t all_tail = (p.head_dim - 2 * p.pairs) / V, rot = P / U;
    uint32_t tail = 0, tail0 = 0;  // units that pass through, and the first of them
    if (shape.copies == 0) {
        if (seg + 1 == shape.segments || shape.segments == 0) tail = all_tail;
    } else if (seg >= shape.segments) {
        tail0 = (seg - shape.segments) * kThreads;
        tail = all_tail - tail0 < kThreads ? all_tail - tail0 : kThreads;
    }
    const uint32_t units = rot + tail, slots = kThreads / units;
    const uint32_t unit = tid % units, slot = tid / units;
    const uint32_t heads = p.q.heads + p.k.heads;
    const uint32_t head_slots = slots < heads ? slots : heads, token_slots = slots / head_slots;
    const uint32_t head_slot = slot % head_slots, token_slot = slot / head_slots;
    const bool rotated = unit < rot, working = token_slot < token_slots;
    const uint32_t pair = first + unit * U;
    const uint32_t channel = rotated ? (HALVES ? pair : 2 * pair) : 2 * p.pairs + (tail0 + unit - rot) * V;
    const uint32_t next = T::second(p.pairs);
    const bool both = rotated;
    uint32_t keep = 0;
    if (rotated)
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) keep |= (p.axis[pair + j] >= p.axes ? 1u : 0u) << j;

    // the pair whose angles this thread forms
    const uint32_t lanes = P ? kThreads / P : 0u;  // tokens that the threads cover once
    const uint32_t my_pair = P ? tid % P : 0u, my_token = P ? tid / P : 0u;
    const bool forms = P && my_token < lanes;
    const uint32_t step_tokens = P ? lanes * shape.steps : shape.steps;
    uint32_t my_axis = 0xff;
    double my_frequency = 0.0;
    if (forms) {
        my_axis = p.axis[first + my_pair];
        my_frequency = p.frequency_f32 ? static_cast<const float*>(p.frequencies)[first + my_pair]
                                       : static_cast<const double*>(p.frequencies)[first + my_pair];
    }
    const bool turned = forms && my_axis < p.axes;
    double at[kMaxSteps];
    auto fetch = [&](uint32_t n0) {
#pragma unroll
        for (uint32_t i = 0; i < kMaxSteps; ++i) {
            const uint32_t n = n0 + i * lanes + my_token;
            at[i] = 0.0;
            if (i < shape.steps && turned && n < p.tokens) at[i] = position_at(p, my_axis, b, n);
        }
    };

    const uint32_t stride = gridDim.x * step_tokens;
    uint32_t phase = 0;
    uint32_t n0 = blockIdx.x * step_tokens;
    fetch(n0);
    for (; n0 < p.tokens; n0 += stride, phase ^= 1) {
        f32x2* mine = turns + phase * step_tokens * P;
        if (P) {
#pragma unroll
            for (uint32_t i = 0; i < kMaxSteps; ++i) {
                if (i >= shape.steps || !forms) break;
                f32x2 cs = cos_sin(at[i], my_frequency);
                if (p.inverse) cs[1] = -cs[1];
                mine[(i * lanes + my_token) * P + my_pair] = cs;
            }
            if (n0 + stride < p.tokens) fetch(n0 + stride);
            __syncthreads();
        }
        const uint32_t some = p.tokens - n0 < step_tokens ? p.tokens - n0 : step_tokens;
        if (!working) continue;
        for (uint32_t t = token_slot; t < some; t += token_slots) {
            const uint32_t n = n0 + t;
            float c[U], s[U];
            if (rotated) {
                const f32x2* cs = mine + t * P + unit * U;
                if constexpr (VEC) {  // P and U are multiples of 4
#pragma unroll
                    for (uint32_t j = 0; j < U; j += 2) {
                        const f32x4 two = *reinterpret_cast<const f32x4*>(cs + j);
                        c[j] = two[0];
                        s[j] = two[1];
                        c[j + 1] = two[2];
                        s[j + 1] = two[3];
                    }
                } else {
                    c[0] = cs[0][0];
                    s[0] = cs[0][1];
                }
            }
            const char* q_in = p.q.in + (b * p.q.in_batch + n * p.q.in_token + channel) * kElem;
            const char* k_in = p.k.in + (b * p.k.in_batch + n * p.k.in_token + channel) * kElem;
            char* q_out = p.q.out + (b * p.q.out_batch + n * p.q.out_token + channel) * kElem;
            char* k_out = p.k.out + (b * p.k.out_batch + n * p.k.out_token + channel) * kElem;
            auto place = [&](uint32_t h, const char*& in, char*& out) {
                const bool is_q = h < p.q.heads;
                const uint32_t hk = h - p.q.heads;
                in = is_q ? q_in + h * p.q.in_head * kElem : k_in + hk * p.k.in_head * kElem;
                out = is_q ? q_out + h * p.q.out_head * kElem : k_out + hk * p.k.out_head * kElem;
            };
            const uint32_t h_step = head_slots * shape.head_splits;
            for (uint32_t h = split * head_slots + head_slot; h < heads; h += 2 * h_step) {
                const bool more = h + h_step < heads;
                const char *in0, *in1;
                char *out0, *out1;
                T x, y;
                place(h, in0, out0);
                place(more ? h + h_step : h, in1, out1);
                x.load(in0, next, both);
                if (more) y.load(in1, next, both);
                if (rotated) x.rotate(c, s, keep);
                x.store(out0, next, both);
                if (more) {
                    if (rotated) y.rotate(c, s, keep);
                    y.store(out1, next, both);
                }
            }
        }
    }
}

template <bool F32, bool HALVES, bool VEC>
hipError_t launch(const AxesProblem& p, hipStream_t stream) {
    using T = Unit<F32, HALVES, VEC>;
    AxesShape s;
    const uint32_t tail = (p.head_dim - 2 * p.pairs) / T::V, heads = p.q.heads + p.k.heads;
    // as many pairs a segment as threads form at once
    s.segments = (p.pairs + kThreads - 1) / kThreads;
    s.seg_pairs = p.pairs < kThreads ? (p.pairs ? p.pairs : 1) : kThreads;
    const uint32_t last = p.pairs - (s.segments ? s.segments - 1 : 0) * s.seg_pairs;
    s.copies = last / T::U + tail <= kThreads ? 0 : (tail + kThreads - 1) / kThreads;
    const uint32_t lanes = kThreads / s.seg_pairs;
    const uint32_t units = s.seg_pairs / T::U, slots = units < kThreads ? kThreads / units : 1;
    const uint32_t token_slots = slots > heads ? slots / heads : 1;
    const uint32_t rounds = (heads + slots - 1) / slots;  // heads a thread takes of one token
    const uint32_t planes = (s.segments + s.copies > 0 ? s.segments + s.copies : 1) * p.batch;
    // Steps long enough that a thread moves 8 units between barriers, while the chip stays filled
    s.steps = 1;
    while (s.steps < kMaxSteps && s.steps * lanes * rounds < 8 * token_slots &&
           static_cast<uint64_t>(planes) * (p.tokens / (2 * s.steps * lanes)) >= 2048)
        s.steps *= 2;
    const uint32_t groups = (p.tokens + s.steps * lanes - 1) / (s.steps * lanes);
    const uint64_t blocks = static_cast<uint64_t>(planes) * groups;
    s.head_splits = 1;
    if (blocks < 512) {
        const uint32_t want = static_cast<uint32_t>((512 + blocks - 1) / blocks);
        s.head_splits = want < rounds ? want : rounds;
    }
    const uint32_t most = 4096 / planes > 0 ? 4096 / planes : 1;
    const dim3 grid(groups < most ? groups : most,
                    (s.segments + s.copies > 0 ? s.segments + s.copies : 1) * s.head_splits, p.batch);
    const size_t lds = size_t(2) * s.steps * lanes * s.seg_pairs * sizeof(f32x2);
    axes_rotate<F32, HALVES, VEC><<<grid, kThreads, lds, stream>>>(p, s);
    return hipGetLastError();
}

template <bool F32, bool HALVES>
hipError_t launch_of(const AxesProblem& p, hipStream_t stream) {
    return p.vectors ? launch<F32, HALVES, true>(p, stream) : launch<F32, HALVES, false>(p, stream);
}

}  // namespace

hipError_t launch_axes(const AxesProblem& p, hipStream_t stream) {
    if (p.f32) return p.halves ? launch_of<true, true>(p, stream) : launch_of<true, false>(p, stream);
    return p.halves ? launch_of<false, true>(p, stream) : launch_of<false, false>(p, stream);
}

}  // namespace ltx3drope
