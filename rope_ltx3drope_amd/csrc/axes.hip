// Rotary positions with several axes: pair i of a head is turned by
//     angle = position[axis(i)][token] * frequency(i)
// whatever the token's positions are, and every head of q and k by the same angles:
//     e' = e cos - o sin,  o' = e sin + o cos         (inverse: by -angle, which is the gradient's way back)
// with (e, o) = (x[2i], x[2i+1]) or, in halves, (x[i], x[i + pairs]).
//
// Angles are formed in 64 bits: a position of 100000 times a frequency near 1 leaves fp32 0.004 of a radian.
// The angle is taken in turns, whose whole number falls away exactly; sine and cosine of the rest are those of
// axes_math.h, within 9.4e-8.
//
// Bound: HBM.  Each channel is read and written once, 16 bytes a lane, and an angle costs about 30 operations and is
// used by all heads that a lane sees.
#include <hip/hip_runtime.h>

#include "axes.h"
#include "axes_math.h"
#include "fastdiv.h"
#include "ltx3drope.h"
#include "stream_store.h"

namespace ltx3drope {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// (cos, sin) of position * turns whole turns.
__device__ __forceinline__ f32x2 cos_sin(double position, double turns) {
    const CosSin v = cos_sin_of_turn(__builtin_amdgcn_fract(position * turns));
    return f32x2{v.c, v.s};
}

__device__ __forceinline__ double position_at(const AxesProblem& p, uint32_t axis, uint32_t b, uint32_t n) {
    const int64_t at = axis * p.position_axis + b * p.position_batch + n * p.position_token;
    if (p.position_type == LTX3DROPE_POSITION_F32) return static_cast<const float*>(p.positions)[at];
    if (p.position_type == LTX3DROPE_POSITION_I32) return static_cast<const int32_t*>(p.positions)[at];
    return static_cast<double>(static_cast<const int64_t*>(p.positions)[at]);
}

// A lane's channels of one head: U pairs of a rotated unit, or V channels that pass through.  V elements an access:
// 16 bytes, two elements, or one.
template <bool F32, bool HALVES, int V>
struct Unit {
    static constexpr int N = axes_unit_accesses(HALVES, V), U = axes_unit_pairs(HALVES, V);
    static constexpr int kElem = F32 ? 4 : 2, kBytes = V * kElem;
    static constexpr int kWords = axes_access_words(F32, V);
    static constexpr uint32_t kRounds = axes_rounds(F32, HALVES, V);
    uint32_t w[N][kWords];

    // byte offset of the second access from the first
    static __device__ __forceinline__ uint32_t second(uint32_t pairs) { return (HALVES ? pairs : 1u) * kElem; }

    static __device__ __forceinline__ void get(uint32_t (&to)[kWords], const char* at) {
        if constexpr (kBytes == 16) {
            const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at));
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = v[j];
        } else if constexpr (kBytes == 8) {
            const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(at));
            to[0] = v[0];
            to[1 % kWords] = v[1];
        } else if constexpr (kBytes == 4) {
            to[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(at));
        } else {
            to[0] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(at));
        }
    }
    // base: the same in every lane
    static __device__ __forceinline__ void put(const uint32_t (&from)[kWords], char* base, uint32_t offset) {
        char* at = base + offset;
        if constexpr (kBytes == 16) {
            stream_store16(stream_u32x4{from[0], from[1 % kWords], from[2 % kWords], from[3 % kWords]}, base, 0x80000000u,
                           offset);
        } else if constexpr (kBytes == 8) {
            __builtin_nontemporal_store(u32x2{from[0], from[1 % kWords]}, reinterpret_cast<u32x2*>(at));
        } else if constexpr (kBytes == 4) {
            __builtin_nontemporal_store(from[0], reinterpret_cast<uint32_t*>(at));
        } else {
            __builtin_nontemporal_store(static_cast<uint16_t>(from[0]), reinterpret_cast<uint16_t*>(at));
        }
    }
    __device__ __forceinline__ void load(const char* at, uint32_t next, bool rotated) {
        get(w[0], at);
        if (N == 2 && rotated) get(w[N - 1], at + next);
    }
    __device__ __forceinline__ void store(char* base, uint32_t offset, uint32_t next, bool rotated) const {
        put(w[0], base, offset);
        if (N == 2 && rotated) put(w[N - 1], base, offset + next);
    }
    // element i of access a
    __device__ __forceinline__ float element(int a, int i) const {
        if constexpr (F32) return __uint_as_float(w[a][i]);
        else return __uint_as_float(i % 2 ? w[a][i / 2] & 0xffff0000u : w[a][i / 2] << 16);
    }
    __device__ __forceinline__ void rotate(const float (&c)[U], const float (&s)[U], uint32_t keep) {
        constexpr bool kApart = N == 2;  // e and o in different accesses
        const Unit was = *this;
        float v[2][U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float e = kApart ? element(0, j) : element(0, 2 * j), o = kApart ? element(N - 1, j) : element(0, 2 * j + 1);
            v[0][j] = fmaf(e, c[j], -(o * s[j]));
            v[1][j] = fmaf(e, s[j], o * c[j]);
        }
        auto at = [&](int a, int i) { return kApart ? v[a][i % U] : v[i % 2][i / 2 % U]; };
#pragma unroll
        for (int a = 0; a < N; ++a)
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (F32) {
                    w[a][i] = __float_as_uint(at(a, i));
                } else {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    const f32x2 two = {at(a, 2 * i), V == 1 ? 0.f : at(a, 2 * i + 1)};
                    w[a][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
                }
            }
        if (keep == 0) return;
        // some pairs stay as they were
#pragma unroll
        for (int a = 0; a < N; ++a)
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                constexpr int kPer = F32 ? 1 : 2;
                uint32_t mask = 0;
#pragma unroll
                for (int h = 0; h < kPer; ++h) {
                    const int pair = (kApart ? kPer * i + h : (kPer * i + h) / 2) % 32;
                    if (keep >> pair & 1) mask |= F32 ? 0xffffffffu : 0xffffu << (16 * h);
                }
                w[a][i] = (was.w[a][i] & mask) | (w[a][i] & ~mask);
            }
    }
};

constexpr float kStays = 2.f;  // in a cosine's place: the pair stays as it is

// One wavefront a workgroup and few rounds a wavefront, in a grid as large as the work: the chip's memory runs fastest
// with short-lived wavefronts that have a few kilobytes on their way (69360 tokens of 32 + 8 heads of 128 in bf16: 259
// to 295 us with workgroups of four wavefronts that went through all heads of some tokens, in three forms; 238 us
// so).  A wavefront takes a token, so that its addresses are scalar.  Its lanes hold a segment of a head (or of the
// channels that pass through), of several heads side by side where that is short, and a round moves those.  The
// segment's angles are formed once, a pair a lane, and handed over in LDS: loads of a frequency and an axis for each
// of a unit's pairs, and of a position that waits for the axis, took longer than the channels (2 x 18360 tokens of
// 4096 in bf16: 634 us so, 462 with the angles handed over, 405 us with none).  axes_shape (axes.h) gives the numbers.
template <bool F32, bool HALVES, int V, bool SOME>
__global__ __launch_bounds__(64) void axes_rotate(AxesProblem p, AxesShape shape) {
    using T = Unit<F32, HALVES, V>;
    constexpr uint32_t U = T::U, kElem = T::kElem, kRounds = T::kRounds, kForms = SOME ? kMostAngles / 64 : U;
    __shared__ double place[SOME ? 64 : 256];               // of the tokens on each axis
    __shared__ __align__(16) f32x2 row[64 * kForms];  // of a segment's pairs, for each token
    const uint32_t lane = threadIdx.x, b = blockIdx.y;
    const uint32_t planes = shape.segments + shape.copies;
    uint32_t rest = fast_div(blockIdx.x, shape.by_planes);
    const uint32_t seg = blockIdx.x - rest * planes;
    uint32_t n, round, last;  // the (first) token, its rounds [round, last)
    uint32_t some = 1;        // tokens
    if (SOME) {
        n = rest * shape.together;
        some = p.tokens - n < shape.together ? p.tokens - n : shape.together;
        round = 0;
        last = shape.rounds;
    } else if (shape.together) {
        n = rest;
        round = 0;
        last = shape.rounds;
    } else if (rest < p.tokens * shape.q_groups) {
        n = fast_div(rest, shape.by_q_groups);
        round = (rest - n * shape.q_groups) * kRounds;
        last = shape.q_rounds;
    } else {
        rest -= p.tokens * shape.q_groups;
        n = fast_div(rest, shape.by_k_groups);
        round = shape.q_rounds + (rest - n * shape.k_groups) * kRounds;
        last = shape.rounds;
    }
    n += p.first_token;
    const uint32_t first = seg * shape.seg_pairs;  // pair
    const uint32_t P = seg >= shape.segments ? 0u
                       : p.pairs - first < shape.seg_pairs ? p.pairs - first : shape.seg_pairs;

    // what the segment's angles need (a token's, or several tokens' side by side)
    uint32_t axis[kForms], whose[kForms], which[kForms];
    double turns[kForms], at = 0.0;
    if (P) {
        if (lane < p.axes * some) {
            const uint32_t t = SOME ? fast_div(lane, shape.by_axes) : 0;
            at = position_at(p, lane - t * p.axes, b, n + t);
        }
#pragma unroll
        for (uint32_t j = 0; j < kForms; ++j) {
            if (SOME && j * 64 >= shape.seg_pairs * some) break;
            whose[j] = SOME ? fast_div(j * 64 + lane, shape.by_pairs) : 0;
            which[j] = j * 64 + lane - whose[j] * shape.seg_pairs;
            const uint32_t i = first + (which[j] < P ? which[j] : 0);
            axis[j] = p.axis[i];
            turns[j] = p.frequency_f32 ? static_cast<const float*>(p.frequencies)[i]
                                       : static_cast<const double*>(p.frequencies)[i];
        }
    }

    // this lane's place in the head, and which of the heads side by side it takes
    const uint32_t all_tail = (p.head_dim - 2 * p.pairs) / V, rot = P / U;
    uint32_t tail = 0, tail0 = 0;  // units that pass through, and the first of them
    if (shape.copies == 0) {
        if (seg + 1 == shape.segments) tail = all_tail;
    } else if (seg >= shape.segments) {
        tail0 = (seg - shape.segments) * 64;
        tail = all_tail - tail0 < 64 ? all_tail - tail0 : 64;
    }
    const uint32_t units = rot + tail, unit = lane % units, slot = lane / units;
    const bool rotated = unit < rot;
    const uint32_t pair = first + unit * U;
    const uint32_t channel = rotated ? (HALVES ? pair : 2 * pair) : 2 * p.pairs + (tail0 + unit - rot) * V;
    const uint32_t next = T::second(p.pairs);
    // the rounds' channels set out
    T x[kRounds];
    bool in[kRounds];
    // f(round, token, whether this lane has a head, the first head's channels, bytes from there: below 2^31)
    auto each = [&](bool out, auto f) {
        uint32_t r = round, t = 0, h = 0, heads = 0;
        int64_t head = 0, step = 0;
        char* at = nullptr;
        bool fresh = true;
#pragma unroll
        for (uint32_t i = 0; i < kRounds; ++i) {
            if (r >= last) {
                if (!SOME || ++t >= some) break;
                r = round;
                fresh = true;
            }
            if (fresh || r == shape.q_rounds) {
                const bool is_q = r < shape.q_rounds;
                h = (is_q ? r : r - shape.q_rounds) * shape.slots;
                heads = is_q ? p.q.heads : p.k.heads;
                int64_t sample, token;
                if (out) {
                    at = is_q ? p.q.out : p.k.out;
                    sample = is_q ? p.q.out_batch : p.k.out_batch;
                    token = is_q ? p.q.out_token : p.k.out_token;
                    head = is_q ? p.q.out_head : p.k.out_head;
                } else {
                    at = const_cast<char*>(is_q ? p.q.in : p.k.in);
                    sample = is_q ? p.q.in_batch : p.k.in_batch;
                    token = is_q ? p.q.in_token : p.k.in_token;
                    head = is_q ? p.q.in_head : p.k.in_head;
                }
                at += (b * sample + (n + t) * token + h * head) * kElem;
                step = shape.slots * head * kElem;
                fresh = false;
            }
            f(i, t, h + slot < heads, at, (slot * static_cast<uint32_t>(head) + channel) * kElem);
            ++r;
            h += shape.slots;
            at += step;
        }
    };
    each(false, [&](uint32_t i, uint32_t, bool there, const char* at, uint32_t offset) {
        in[i] = slot < shape.slots && there;
        if (in[i]) x[i].load(at + offset, next, rotated);
    });

    if (P) {
        if (lane < p.axes * some) place[lane] = at;
        for (uint32_t a = 64 + lane; a < p.axes; a += 64) place[a] = position_at(p, a, b, n);
        __syncthreads();
        const double unit_turns = p.inverse ? -0.15915494309189533577 : 0.15915494309189533577;  // 1 / (2 pi)
#pragma unroll
        for (uint32_t j = 0; j < kForms; ++j) {
            if (SOME && j * 64 >= shape.seg_pairs * some) break;
            if (which[j] < P && whose[j] < some)
                row[j * 64 + lane] = axis[j] < p.axes
                                         ? cos_sin(place[whose[j] * p.axes + axis[j]], turns[j] * unit_turns)
                                         : f32x2{kStays, 0.f};
        }
        __syncthreads();
    }
    float c[U], s[U];
    uint32_t keep = 0;
    auto take = [&](uint32_t t) {
        const f32x2* cs = row + t * shape.seg_pairs + unit * U;
        if constexpr (U % 2 == 0) {
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
        keep = 0;
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) keep |= (c[j] == kStays ? 1u : 0u) << j;
    };
    if (!SOME && rotated) take(0);
    uint32_t taken = ~0u;
    each(true, [&](uint32_t i, uint32_t t, bool, char* at, uint32_t offset) {
        if (SOME && rotated && t != taken) take(t);
        taken = t;
        if (!in[i]) return;
        if (rotated) x[i].rotate(c, s, keep);
        x[i].store(at, offset, next, rotated);
    });
}

template <bool F32, bool HALVES, int V>
hipError_t launch(const AxesProblem& p, hipStream_t stream) {
    const AxesShape s = axes_shape(p);
    const uint32_t most = axes_launch_tokens(s);
    for (uint64_t n = 0; n < p.tokens; n += most) {
        AxesProblem some = p;
        some.first_token = static_cast<uint32_t>(n);
        some.tokens = p.tokens - some.first_token < most ? p.tokens - some.first_token : most;
        const dim3 grid(axes_launch_groups(s, some.tokens), p.batch);
        if (s.together > 1) axes_rotate<F32, HALVES, V, true><<<grid, 64, 0, stream>>>(some, s);
        else axes_rotate<F32, HALVES, V, false><<<grid, 64, 0, stream>>>(some, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool F32, bool HALVES>
hipError_t launch_of(const AxesProblem& p, hipStream_t stream) {
    if (p.vector == 1) return launch<F32, HALVES, 1>(p, stream);
    if (p.vector == 2) return launch<F32, HALVES, 2>(p, stream);
    return launch<F32, HALVES, F32 ? 4 : 8>(p, stream);
}

}  // namespace

hipError_t launch_axes(const AxesProblem& p, hipStream_t stream) {
    if (p.f32) return p.halves ? launch_of<true, true>(p, stream) : launch_of<true, false>(p, stream);
    return p.halves ? launch_of<false, true>(p, stream) : launch_of<false, false>(p, stream);
}

}  // namespace ltx3drope
