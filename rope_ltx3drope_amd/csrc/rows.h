// What the row-wise norms (norm.hip, layer_norm.hip) share: a row of [batch, rows, dim] held in registers by
// T threads, sums over it, the launch shape, and the sums over partial rows of the backward passes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "block.h"

namespace ltx3drope {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
    const __bf16 b = static_cast<__bf16>(v);  // round to nearest even
    return __builtin_bit_cast(uint16_t, b);
}

// A thread's E elements of one row in their stored form.  With vectors, element i*V + j of the
// thread is column (i*T + t)*V + j; without, element i is column i*T + t.
template <bool F32, int E, bool VEC>
struct RowPart {
    static constexpr int V = VEC ? (F32 ? 4 : 8) : 1;
    static constexpr int N = E / V;  // loads
    static constexpr int kWords = F32 ? E : (VEC ? E / 2 : E);
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void* row, uint32_t t, uint32_t T, uint32_t D) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t c = (i * T + t) * V;
            if constexpr (VEC) {
                u32x4 v = {0, 0, 0, 0};
                if (c < D)
                    v = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4*>(static_cast<const char*>(row) + c * (F32 ? 4u : 2u)));
#pragma unroll
                for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
            } else if constexpr (F32) {
                w[i] = c < D ? static_cast<const uint32_t*>(row)[c] : 0u;
            } else {
                w[i] = c < D ? static_cast<const uint16_t*>(row)[c] : 0u;
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0;
    }
    __device__ __forceinline__ void unpack(float (&f)[E]) const {
        if constexpr (F32) {
#pragma unroll
            for (int k = 0; k < E; ++k) f[k] = __uint_as_float(w[k]);
        } else if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                f[2 * k] = __uint_as_float(w[k] << 16);
                f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k) f[k] = bf16_to_f32(w[k]);
        }
    }
};

// Stores a thread's E values, rounded once to the row's type.
template <bool F32, int E, bool VEC>
__device__ __forceinline__ void store_row(void* row, const float (&f)[E], uint32_t t, uint32_t T, uint32_t D) {
    constexpr int V = RowPart<F32, E, VEC>::V;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        const uint32_t c = (i * T + t) * V;
        if (c >= D) continue;
        if constexpr (VEC) {
            u32x4 v;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (F32)
                    v[k] = __float_as_uint(f[i * V + k]);
                else
                    v[k] = f32_to_bf16(f[i * V + 2 * k]) | (uint32_t(f32_to_bf16(f[i * V + 2 * k + 1])) << 16);
            }
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(static_cast<char*>(row) + c * (F32 ? 4u : 2u)));
        } else if constexpr (F32) {
            static_cast<float*>(row)[c] = f[i];
        } else {
            static_cast<uint16_t*>(row)[c] = f32_to_bf16(f[i]);
        }
    }
}

__device__ __forceinline__ float load_param(const void* p, bool f32, size_t i) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// A thread's E parameters of one vector, or `otherwise` where there is no vector or no column.  VEC rows
// with `chunks` (the vectors start on 16 bytes and so does every sample's part) read them 16 bytes at a time.
template <bool F32, int E, bool VEC>
__device__ __forceinline__ void load_params(float (&f)[E], const void* p, size_t first, bool f32, bool chunks,
                                            float otherwise, uint32_t t, uint32_t T, uint32_t D) {
    constexpr int V = RowPart<F32, E, VEC>::V;
#pragma unroll
    for (int k = 0; k < E; ++k) f[k] = otherwise;
    if (p == nullptr) return;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        const uint32_t c = (i * T + t) * V;
        if (c >= D) continue;
        if (VEC && chunks) {
            if (f32) {
#pragma unroll
                for (int h = 0; h < V; h += 4) {
                    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + first + c + h);
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[(i * V + h + k) % E] = __uint_as_float(v[k]);
                }
            } else if constexpr (V == 8) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + first + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[i * V + 2 * k] = __uint_as_float(v[k] << 16);
                    f[i * V + 2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) f[i * V + k] = load_param(p, f32, first + c + k);
        }
    }
}

// The factor that takes the place of (w + offset) * g, or (w + offset) * (1 + g), for one sample.
template <bool F32, int E, bool VEC, class Call>
__device__ __forceinline__ void load_factor(float (&f)[E], const Call& p, const void* w, const void* g, float one,
                                            uint32_t b, uint32_t t, uint32_t T) {
    float other[E];
    load_params<F32, E, VEC>(f, w, 0, p.param_f32, p.chunks, 1.f, t, T, p.dim);
    load_params<F32, E, VEC>(other, g, static_cast<size_t>(b) * p.dim, p.param_f32, p.chunks, 1.f - one, t, T, p.dim);
    const float offset = w ? p.weight_offset : 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) f[k] = (f[k] + offset) * (one + other[k]);
}

// Column of element k of thread t.
template <bool F32, int E, bool VEC>
__device__ __forceinline__ uint32_t column(int k, uint32_t t, uint32_t T) {
    constexpr int V = RowPart<F32, E, VEC>::V;
    return ((k / V) * T + t) * V + k % V;
}

template <int CTRL>
__device__ __forceinline__ float lanes(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// The sum over a wavefront: within each 16 lanes by register moves (pairs, quads, halves of 8, of 16), then
// the four 16s.  No LDS on the way.
__device__ __forceinline__ float wave_sum(float v) {
    v += lanes<0xb1>(v);   // quad_perm 1 0 3 2
    v += lanes<0x4e>(v);   // quad_perm 2 3 0 1
    v += lanes<0x141>(v);  // row_half_mirror
    v += lanes<0x140>(v);  // row_mirror
    const int b = __float_as_int(v);
    return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// The sum of a thread's squares times sq (norm_square_scale), in two chains of additions.  The sums are scaled
// as a whole, unless one of the wavefront's passes fp32's range: scaling every square costs a multiplication
// an element (2 x 34680 rows of 2048 bf16 after a block: 215 us, 213 so, 211 without scaling).
template <int E>
__device__ __forceinline__ float square_sum(const float (&v)[E], float sq) {
    float even = 0.f, odd = 0.f;
#pragma unroll
    for (int k = 0; k < E; k += 2) {
        even = fmaf(v[k], v[k], even);
        odd = fmaf(v[k + 1], v[k + 1], odd);
    }
    const float s = fmaf(odd, sq, even * sq);
    if (__builtin_expect(!__any(!(s < __builtin_inff())), 1)) return s;
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) t = fmaf(v[k] * sq, v[k], t);
    return t;
}

// Sums of K values over the T threads of each row (T a multiple of 64; row g of the workgroup owns
// waves [g*T/64, (g+1)*T/64)).  `lds` holds K floats a wave of the workgroup, and successive calls
// use different parts of it, so that one barrier a call is enough.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, uint32_t t, uint32_t T, uint32_t g) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    const uint32_t W = T / 64;
    if (W == 1) return;
    float* mine = lds + g * W * K;
    if ((t & 63) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) mine[(t / 64) * K + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float s = 0.f;
        for (uint32_t w = 0; w < W; ++w) s += mine[w * K + k];
        v[k] = s;
    }
}

constexpr int kMaxWaves = 16;

__device__ __forceinline__ void store_param(void* p, bool f32, size_t i, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
}

// The joins of partial rows: kCols columns a workgroup, kLanes threads down the parts.
constexpr int kCols = 16, kLanes = 64;

// The sum over the lanes of column `col`, in every thread of lane 0 (in lane order).
__device__ __forceinline__ float lane_sum(float s, float (&lds)[kLanes][kCols + 1], uint32_t col, uint32_t lane) {
    __syncthreads();
    lds[lane][col] = s;
    __syncthreads();
    if (lane < 8) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kLanes / 8; ++i) s += lds[lane * (kLanes / 8) + i][col];
    }
    __syncthreads();
    if (lane < 8) lds[lane][col] = s;
    __syncthreads();
    s = 0.f;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += lds[i][col];
    return s;
}

// Threads a row and rows a workgroup: 8 elements a thread up to 8192 columns (the most that 1024 threads
// then hold), 16 above; rows side by side up to 512 threads, as long as 512 workgroups are left to do.
// Two workgroups of 512 threads a compute unit walk down the rows.  More of them at a time are slower,
// though they hide more: forward, 69360 rows of 2048 bf16, 267 us with 4096 workgroups of 256 threads,
// 222 with 1024, 212 with 512 of 512; a wavefront a row, without barriers, 207 to 216.  Backward, 36720
// rows: 234 us with 512 of 1024 threads, 215 with 1024 of 512, 193 with 512 of 512 (with the vectors read
// 16 bytes at a time and streaming accesses the two are at 204 and 164 us: 5.6 and 5.5 TB/s).
struct Shape {
    bool wide;
    uint32_t T, G;
};

constexpr uint32_t kWorkgroups = 512, kThreads = 512;

inline Shape row_shape(uint32_t batch, uint32_t rows, uint32_t dim) {
    Shape s;
    s.wide = dim > 8192;
    const uint32_t per = s.wide ? 16 : 8;
    s.T = 64 * ((dim + 64 * per - 1) / (64 * per));
    s.G = s.T >= kThreads ? 1 : kThreads / s.T;
    while (s.G > 1 && static_cast<uint64_t>(batch) * ((rows + s.G - 1) / s.G) < kWorkgroups) s.G /= 2;
    return s;
}

inline uint32_t row_parts(uint32_t batch, uint32_t rows, uint32_t G) {
    const uint32_t need = (rows + G - 1) / G;
    const uint32_t most = kWorkgroups / batch;
    return need < most ? need : (most > 0 ? most : 1);
}

static __global__ __launch_bounds__(256) void norm_zero(void* p, size_t n, bool f32) {
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += size_t(gridDim.x) * 256)
        store_param(p, f32, i, 0.f);
}

}  // namespace ltx3drope
