// RMS norms before and after a transformer block, fused with the block's gate, the scaled
// residual and the next norm's scale and shift; and their backward pass.
//
// Per row of width D (rows of sample b), all in fp32:
//     hat(v) = v * rstd(v),  rstd(v) = 1 / sqrt(mean(v^2) + eps)
//     branch = post norm ? hat(y) * (w + off) : y
//     r      = residual_scale * residual + gate_b * branch
//     n      = hat(r) * (nw + off) * (1 + scale_b) + shift_b
// "before" is the case without y: r is the input itself and is not written.
//
// Backward, with v = dn * (nw + off) * (1 + scale_b):
//     dR  = dr + rstd_r * (v - hat(r) * mean(v * hat(r)))         (dr: what reaches r past the norm)
//     dresidual = residual_scale * dR
//     q   = dR * gate_b * (w + off)
//     dy  = rstd_y * (q - hat(y) * mean(q * hat(y)))              (no post norm: q)
// and per sample P1 = sum_rows dn * hat(r), P2 = sum_rows dn, P3 = sum_rows dR * hat(y), from which
//     dscale_b = (nw + off) P1, dshift_b = P2, dnw = sum_b (1 + scale_b) P1,
//     dgate_b = (w + off) P3,   dw = sum_b gate_b P3.
//
// Bound: HBM.  About 6 (forward) and 10 (backward) operations an element and tensor against 2 or 4
// bytes, so each row tensor crosses HBM once: a row stays in registers between its reduction and its
// use.  A workgroup holds G rows side by side, T threads a row, E elements a thread, and walks down
// one sample's rows, so that the per-column factors are read once a workgroup.  The backward's
// per-column sums stay in registers on that walk; each workgroup leaves one partial row and a second
// kernel adds the partials in a fixed order (no atomics: results do not depend on timing).
#include <hip/hip_runtime.h>

#include <utility>

#include "block.h"

namespace ltx3drope {
namespace {

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

// Column of element k of thread t.
template <bool F32, int E, bool VEC>
__device__ __forceinline__ uint32_t column(int k, uint32_t t, uint32_t T) {
    constexpr int V = RowPart<F32, E, VEC>::V;
    return ((k / V) * T + t) * V + k % V;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
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

template <bool F32, int E, bool VEC, bool HAS_Y, bool NEXT>
__global__ __launch_bounds__(1024) void norm_forward(NormForward p) {
    __shared__ float lds[2][2][kMaxWaves];
    const uint32_t T = blockDim.x, t = threadIdx.x, G = blockDim.y, g = threadIdx.y;
    const uint32_t D = p.dim, b = blockIdx.y;
    const bool pf = p.param_f32;
    const float inv_d = 1.0f / static_cast<float>(D);

    // the factor on the branch, the factor and the shift of the next norm
    float fy[HAS_Y ? E : 1], fn[NEXT ? E : 1], sh[NEXT ? E : 1];
#pragma unroll
    for (int k = 0; k < E; ++k) {
        const uint32_t c = column<F32, E, VEC>(k, t, T);
        const bool in = c < D;
        const size_t bc = static_cast<size_t>(b) * D + c;
        if constexpr (HAS_Y) {
            float f = 1.f;
            if (in && p.weight) f = load_param(p.weight, pf, c) + p.weight_offset;
            if (in && p.gate) f *= load_param(p.gate, pf, bc);
            fy[k] = f;
        }
        if constexpr (NEXT) {
            float f = 1.f;
            if (in && p.next_weight) f = load_param(p.next_weight, pf, c) + p.weight_offset;
            if (in && p.next_scale) f *= 1.f + load_param(p.next_scale, pf, bc);
            fn[k] = f;
            sh[k] = in && p.next_shift ? load_param(p.next_shift, pf, bc) : 0.f;
        }
    }

    constexpr size_t es = F32 ? 4 : 2;
    const uint32_t step = gridDim.x * G;
    int phase = 0;
    for (uint32_t s0 = blockIdx.x * G; s0 < p.rows; s0 += step, phase ^= 1) {
        const uint32_t s = s0 + g;
        const bool live = s < p.rows;  // every thread keeps the barriers
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        RowPart<F32, E, VEC> yr, rr;
        if (live) {
            if constexpr (HAS_Y) yr.load(static_cast<const char*>(p.y) + off, t, T, D);
            rr.load(static_cast<const char*>(p.residual) + off, t, T, D);
        } else {
            if constexpr (HAS_Y) yr.clear();
            rr.clear();
        }
        float r[E];
        rr.unpack(r);
        if constexpr (HAS_Y) {
            float y[E];
            yr.unpack(y);
            float rstd = 1.f;
            if (p.post_norm) {
                float ss[1] = {0.f};
#pragma unroll
                for (int k = 0; k < E; ++k) ss[0] = fmaf(y[k], y[k], ss[0]);
                row_sum(ss, lds[phase][0], t, T, g);
                rstd = rsqrtf(fmaf(ss[0], inv_d, p.eps));
            }
#pragma unroll
            for (int k = 0; k < E; ++k) r[k] = fmaf(y[k] * rstd, fy[k], p.residual_scale * r[k]);
            if (live) store_row<F32, E, VEC>(static_cast<char*>(p.r) + off, r, t, T, D);
        }
        if constexpr (NEXT) {
            float ss[1] = {0.f};
#pragma unroll
            for (int k = 0; k < E; ++k) ss[0] = fmaf(r[k], r[k], ss[0]);
            row_sum(ss, lds[phase][1], t, T, g);
            const float rstd = rsqrtf(fmaf(ss[0], inv_d, p.eps));
#pragma unroll
            for (int k = 0; k < E; ++k) r[k] = fmaf(r[k] * rstd, fn[k], sh[k]);
            if (live) store_row<F32, E, VEC>(static_cast<char*>(p.n) + off, r, t, T, D);
        }
    }
}

template <bool F32, int E, bool VEC, bool HAS_Y, bool NEXT>
__global__ __launch_bounds__(1024) void norm_backward(NormBackward p) {
    __shared__ float lds[2][2][3 * kMaxWaves];
    extern __shared__ float cols[];  // (G - 1) * D: the rows' partial sums on their way to row 0
    const uint32_t T = blockDim.x, t = threadIdx.x, G = blockDim.y, g = threadIdx.y;
    const uint32_t D = p.dim, b = blockIdx.y;
    const bool pf = p.param_f32;
    const float inv_d = 1.0f / static_cast<float>(D);

    float fy[HAS_Y ? E : 1], fn[NEXT ? E : 1];
    float p1[NEXT ? E : 1], p2[NEXT ? E : 1], p3[HAS_Y ? E : 1];
#pragma unroll
    for (int k = 0; k < E; ++k) {
        const uint32_t c = column<F32, E, VEC>(k, t, T);
        const bool in = c < D;
        const size_t bc = static_cast<size_t>(b) * D + c;
        if constexpr (HAS_Y) {
            float f = 1.f;
            if (in && p.weight) f = load_param(p.weight, pf, c) + p.weight_offset;
            if (in && p.gate) f *= load_param(p.gate, pf, bc);
            fy[k] = f;
            p3[k] = 0.f;
        }
        if constexpr (NEXT) {
            float f = 1.f;
            if (in && p.next_weight) f = load_param(p.next_weight, pf, c) + p.weight_offset;
            if (in && p.next_scale) f *= 1.f + load_param(p.next_scale, pf, bc);
            fn[k] = f;
            p1[k] = 0.f;
            p2[k] = 0.f;
        }
    }

    constexpr size_t es = F32 ? 4 : 2;
    const uint32_t step = gridDim.x * G;
    int phase = 0;
    for (uint32_t s0 = blockIdx.x * G; s0 < p.rows; s0 += step, phase ^= 1) {
        const uint32_t s = s0 + g;
        const bool live = s < p.rows;
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        RowPart<F32, E, VEC> raw;
        float d[E], y[HAS_Y ? E : 1];
        if (live && p.dr) raw.load(static_cast<const char*>(p.dr) + off, t, T, D);
        else raw.clear();
        raw.unpack(d);
        if constexpr (HAS_Y) {
            if (live && p.y) raw.load(static_cast<const char*>(p.y) + off, t, T, D);
            else raw.clear();
            raw.unpack(y);
        }
        float rstd_y = 1.f;
        if constexpr (NEXT) {
            float r[E], dn[E];
            if (live) raw.load(static_cast<const char*>(p.r) + off, t, T, D);
            else raw.clear();
            raw.unpack(r);
            if (live) raw.load(static_cast<const char*>(p.dn) + off, t, T, D);
            else raw.clear();
            raw.unpack(dn);
            float ss[3] = {0.f, 0.f, 0.f};  // r.r, (dn fn).r, y.y
#pragma unroll
            for (int k = 0; k < E; ++k) {
                ss[0] = fmaf(r[k], r[k], ss[0]);
                ss[1] = fmaf(dn[k] * fn[k], r[k], ss[1]);
                if constexpr (HAS_Y) ss[2] = fmaf(y[k], y[k], ss[2]);
            }
            row_sum(ss, lds[phase][0], t, T, g);
            const float rstd = rsqrtf(fmaf(ss[0], inv_d, p.eps));
            const float proj = ss[1] * rstd * inv_d;  // mean(v * hat(r))
            if constexpr (HAS_Y)
                if (p.post_norm) rstd_y = rsqrtf(fmaf(ss[2], inv_d, p.eps));
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float hat = r[k] * rstd;
                p1[k] = fmaf(dn[k], hat, p1[k]);
                p2[k] += dn[k];
                d[k] = fmaf(rstd, fmaf(-hat, proj, dn[k] * fn[k]), d[k]);
            }
        } else if constexpr (HAS_Y) {
            if (p.post_norm) {
                float ss[1] = {0.f};
#pragma unroll
                for (int k = 0; k < E; ++k) ss[0] = fmaf(y[k], y[k], ss[0]);
                row_sum(ss, lds[phase][0], t, T, g);
                rstd_y = rsqrtf(fmaf(ss[0], inv_d, p.eps));
            }
        }
        if (live) {
            float o[E];
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = p.residual_scale * d[k];
            store_row<F32, E, VEC>(static_cast<char*>(p.dresidual) + off, o, t, T, D);
        }
        if constexpr (HAS_Y) {
            float ss[1] = {0.f};
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float hat = y[k] * rstd_y;
                p3[k] = fmaf(d[k], hat, p3[k]);
                d[k] *= fy[k];
                ss[0] = fmaf(d[k], hat, ss[0]);
                y[k] = hat;
            }
            if (p.post_norm) {
                row_sum(ss, lds[phase][1], t, T, g);
                const float proj = ss[0] * inv_d;
#pragma unroll
                for (int k = 0; k < E; ++k) d[k] = rstd_y * fmaf(-y[k], proj, d[k]);
            }
            if (live) store_row<F32, E, VEC>(static_cast<char*>(p.dy) + off, d, t, T, D);
        }
    }

    // one partial row a workgroup: partial[which][b][part][D]
    if (p.partial == nullptr) return;
    const size_t plane = static_cast<size_t>(p.batch) * gridDim.x * D;
    float* out = p.partial + (static_cast<size_t>(b) * gridDim.x + blockIdx.x) * D;
    auto leave = [&](const float* v, int which) {
        if (G > 1) {
            __syncthreads();
            if (g > 0) {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const uint32_t c = column<F32, E, VEC>(k, t, T);
                    if (c < D) cols[(g - 1) * D + c] = v[k];
                }
            }
            __syncthreads();
        }
        if (g == 0) {
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const uint32_t c = column<F32, E, VEC>(k, t, T);
                if (c >= D) continue;
                float s = v[k];
                for (uint32_t o = 1; o < G; ++o) s += cols[(o - 1) * D + c];
                out[which * plane + c] = s;
            }
        }
    };
    if constexpr (NEXT) {
        leave(p1, 0);
        leave(p2, 1);
    }
    if constexpr (HAS_Y) leave(p3, 2);
}

__device__ __forceinline__ void store_param(void* p, bool f32, size_t i, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
}

// Sums over the partial rows of one sample (gridDim.y samples, kCols columns a workgroup, kLanes
// threads down the parts), then the sample's gradients; the sums over samples are left in
// partial row 0 of each sample for norm_backward_weights.
constexpr int kCols = 32, kLanes = 32;

__global__ __launch_bounds__(kCols* kLanes) void norm_backward_samples(NormBackward p, uint32_t parts) {
    __shared__ float lds[kLanes][kCols + 1];
    const uint32_t col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
    const uint32_t c = blockIdx.x * kCols + col, b = blockIdx.y;
    const size_t plane = static_cast<size_t>(p.batch) * parts * p.dim;
    const size_t base = static_cast<size_t>(b) * parts * p.dim + c;
    float sum[3];
    for (int which = 0; which < 3; ++which) {
        const bool used = which == 2 ? p.has_y : p.next_norm;
        if (!used) continue;  // uniform over the grid
        float s = 0.f;
        if (c < p.dim)
            for (uint32_t i = lane; i < parts; i += kLanes) s += p.partial[which * plane + base + size_t(i) * p.dim];
        __syncthreads();
        lds[lane][col] = s;
        __syncthreads();
        s = 0.f;
        if (lane == 0)
            for (int i = 0; i < kLanes; ++i) s += lds[i][col];
        sum[which] = s;
    }
    if (lane != 0 || c >= p.dim) return;
    const bool pf = p.param_f32;
    const size_t bc = static_cast<size_t>(b) * p.dim + c;
    if (p.next_norm) {
        const float w = p.next_weight ? load_param(p.next_weight, pf, c) + p.weight_offset : 1.f;
        const float f = p.next_scale ? 1.f + load_param(p.next_scale, pf, bc) : 1.f;
        if (p.dnext_scale) store_param(p.dnext_scale, pf, bc, w * sum[0]);
        if (p.dnext_shift) store_param(p.dnext_shift, pf, bc, sum[1]);
        if (p.batch == 1) {
            if (p.dnext_weight) store_param(p.dnext_weight, pf, c, f * sum[0]);
        } else {
            p.partial[base] = f * sum[0];
        }
    }
    if (p.has_y) {
        const float w = p.weight ? load_param(p.weight, pf, c) + p.weight_offset : 1.f;
        const float f = p.gate ? load_param(p.gate, pf, bc) : 1.f;
        if (p.dgate) store_param(p.dgate, pf, bc, w * sum[2]);
        if (p.batch == 1) {
            if (p.dweight) store_param(p.dweight, pf, c, f * sum[2]);
        } else {
            p.partial[2 * plane + base] = f * sum[2];
        }
    }
}

// The weights' gradients: sums over samples of what norm_backward_samples left.
__global__ __launch_bounds__(kCols* kLanes) void norm_backward_weights(NormBackward p, uint32_t parts) {
    __shared__ float lds[kLanes][kCols + 1];
    const uint32_t col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
    const uint32_t c = blockIdx.x * kCols + col;
    const size_t plane = static_cast<size_t>(p.batch) * parts * p.dim;
    for (int which = 0; which < 3; which += 2) {
        void* out = which == 0 ? p.dnext_weight : p.dweight;
        if (out == nullptr) continue;
        float s = 0.f;
        if (c < p.dim)
            for (uint32_t b = lane; b < p.batch; b += kLanes)
                s += p.partial[which * plane + static_cast<size_t>(b) * parts * p.dim + c];
        __syncthreads();
        lds[lane][col] = s;
        __syncthreads();
        if (lane == 0 && c < p.dim) {
            s = 0.f;
            for (int i = 0; i < kLanes; ++i) s += lds[i][col];
            store_param(out, p.param_f32, c, s);
        }
    }
}

template <bool F32, int E, bool VEC>
hipError_t forward_modes(const NormForward& p, dim3 grid, dim3 block, hipStream_t stream) {
    if (!p.has_y)
        norm_forward<F32, E, VEC, false, true><<<grid, block, 0, stream>>>(p);
    else if (p.next_norm)
        norm_forward<F32, E, VEC, true, true><<<grid, block, 0, stream>>>(p);
    else
        norm_forward<F32, E, VEC, true, false><<<grid, block, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool F32, int E, bool VEC>
hipError_t backward_modes(const NormBackward& p, dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
    if (!p.has_y)
        norm_backward<F32, E, VEC, false, true><<<grid, block, lds, stream>>>(p);
    else if (p.next_norm)
        norm_backward<F32, E, VEC, true, true><<<grid, block, lds, stream>>>(p);
    else
        norm_backward<F32, E, VEC, true, false><<<grid, block, lds, stream>>>(p);
    return hipGetLastError();
}

// Threads a row and rows a workgroup for a row width: 8 elements a thread up to 8192 columns (the
// most that 1024 threads then hold), 16 above, and rows side by side up to `threads` threads.
struct Shape {
    bool wide;
    uint32_t T, G;
};

constexpr uint32_t kForwardWorkgroups = 4096, kBackwardWorkgroups = 512;  // 16 and 2 a compute unit

Shape row_shape(uint32_t dim, uint32_t threads) {
    Shape s;
    s.wide = dim > 8192;
    const uint32_t per = s.wide ? 16 : 8;
    s.T = 64 * ((dim + 64 * per - 1) / (64 * per));
    s.G = s.T >= threads ? 1 : threads / s.T;
    return s;
}

uint32_t row_parts(uint32_t batch, uint32_t rows, uint32_t G, uint32_t workgroups) {
    const uint32_t need = (rows + G - 1) / G;
    const uint32_t most = workgroups / batch;
    return need < most ? need : (most > 0 ? most : 1);
}

uint32_t backward_parts(uint32_t batch, uint32_t rows, uint32_t dim) {
    return row_parts(batch, rows, row_shape(dim, 1024).G, kBackwardWorkgroups);
}

__global__ __launch_bounds__(256) void norm_zero(void* p, size_t n, bool f32) {
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += size_t(gridDim.x) * 256)
        store_param(p, f32, i, 0.f);
}

}  // namespace

hipError_t launch_norm_forward(const NormForward& p, bool f32, bool vec, hipStream_t stream) {
    const Shape s = row_shape(p.dim, 256);
    const dim3 block(s.T, s.G), grid(row_parts(p.batch, p.rows, s.G, kForwardWorkgroups), p.batch);
    if (f32) {
        if (s.wide) return vec ? forward_modes<true, 16, true>(p, grid, block, stream) : forward_modes<true, 16, false>(p, grid, block, stream);
        return vec ? forward_modes<true, 8, true>(p, grid, block, stream) : forward_modes<true, 8, false>(p, grid, block, stream);
    }
    if (s.wide) return vec ? forward_modes<false, 16, true>(p, grid, block, stream) : forward_modes<false, 16, false>(p, grid, block, stream);
    return vec ? forward_modes<false, 8, true>(p, grid, block, stream) : forward_modes<false, 8, false>(p, grid, block, stream);
}

size_t norm_backward_workspace(uint32_t batch, uint32_t rows, uint32_t dim) {
    return size_t(3) * batch * backward_parts(batch, rows, dim) * dim * sizeof(float);
}

hipError_t launch_norm_backward(const NormBackward& p, bool f32, bool vec, hipStream_t stream) {
    if (p.batch == 0 || p.rows == 0) {  // no rows: every sum is zero
        const size_t D = p.dim, BD = size_t(p.batch) * p.dim;
        const std::pair<void*, size_t> sums[5] = {{p.dweight, D}, {p.dgate, BD}, {p.dnext_weight, D},
                                                  {p.dnext_scale, BD}, {p.dnext_shift, BD}};
        for (const auto& v : sums)
            if (v.first != nullptr && v.second != 0) norm_zero<<<64, 256, 0, stream>>>(v.first, v.second, p.param_f32);
        return hipGetLastError();
    }
    const Shape s = row_shape(p.dim, 1024);
    const uint32_t parts = backward_parts(p.batch, p.rows, p.dim);
    const dim3 block(s.T, s.G), grid(parts, p.batch);
    const size_t lds = size_t(s.G - 1) * p.dim * sizeof(float);
    hipError_t e;
    if (f32) {
        if (s.wide) e = vec ? backward_modes<true, 16, true>(p, grid, block, lds, stream) : backward_modes<true, 16, false>(p, grid, block, lds, stream);
        else e = vec ? backward_modes<true, 8, true>(p, grid, block, lds, stream) : backward_modes<true, 8, false>(p, grid, block, lds, stream);
    } else {
        if (s.wide) e = vec ? backward_modes<false, 16, true>(p, grid, block, lds, stream) : backward_modes<false, 16, false>(p, grid, block, lds, stream);
        else e = vec ? backward_modes<false, 8, true>(p, grid, block, lds, stream) : backward_modes<false, 8, false>(p, grid, block, lds, stream);
    }
    if (e != hipSuccess || p.partial == nullptr) return e;
    const uint32_t cols = (p.dim + kCols - 1) / kCols;
    norm_backward_samples<<<dim3(cols, p.batch), kCols * kLanes, 0, stream>>>(p, parts);
    e = hipGetLastError();
    if (e != hipSuccess || p.batch == 1 || (!p.dnext_weight && !p.dweight)) return e;
    norm_backward_weights<<<cols, kCols * kLanes, 0, stream>>>(p, parts);
    return hipGetLastError();
}

}  // namespace ltx3drope
