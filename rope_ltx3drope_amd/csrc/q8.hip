// A linear layer in 8-bit integers: rows quantised to one scale a token, and the product with weights
// that carry one scale a channel.
//
//     scale_m = max_k |x_mk| * c,  q_mk = round(x_mk / scale_m)         (fp32, each step rounded once;
//                                                                    c = 1/127 rounded to fp32)
//     y_mn    = (sum_k q_mk w_nk) * scale_m * w_scale_n + bias_n
// The sums are exact: at most 131071 products of at most 2^14 fit 32-bit integers.  A row of zeros
// has scale 0 and zeros; a row whose largest magnitude is not finite keeps that as its scale and gets
// zeros, so that its outputs are NaN and no other row's are.
#include <hip/hip_runtime.h>

#include "block.h"
#include "product.h"

namespace ltx3drope {
namespace {

template <bool F32>
__device__ __forceinline__ float value(const void* row, uint32_t c) {
    if constexpr (F32) return static_cast<const float*>(row)[c];
    else return static_cast<float>(static_cast<const __bf16*>(row)[c]);
}

// The largest of a row's magnitudes, as a bit pattern: magnitudes compare like their bits, and a NaN's
// is above every number's.  T threads a row (a multiple of 64), the rows of a workgroup side by side;
// successive calls use different parts of LDS.
__device__ __forceinline__ uint32_t row_max(uint32_t top, uint32_t* lds, uint32_t t, uint32_t T, uint32_t g) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = __shfl_xor(top, m);
        top = o > top ? o : top;
    }
    const uint32_t W = T / 64;
    if (W == 1) return top;
    if ((t & 63) == 0) lds[g * W + t / 64] = top;
    __syncthreads();
    for (uint32_t w = 0; w < W; ++w) top = lds[g * W + w] > top ? lds[g * W + w] : top;
    return top;
}

__device__ __forceinline__ float scale_of(uint32_t top) { return __uint_as_float(top) * (1.0f / 127.0f); }

// round(x / s) for any scale.
__device__ __forceinline__ int quotient(float x, float s) {
    // a subnormal scale may be far off its value: the quotient is kept within the 8 bits
    const bool plain = s > 0.f && s < __builtin_inff();
    const float v = plain ? rintf(x / s) : 0.f;
    return static_cast<int>(fminf(fmaxf(v, -127.f), 127.f));
}

// The same for 2^-100 < s < 2^100, with r = 1 / s rounded to nearest: x * r is within an ulp of the
// quotient, and one step with the exact remainder gives the rounded quotient itself (Markstein's
// division by a rounded reciprocal).  Adding 1.5 * 2^23 rounds it to an integer whose low byte is the
// number's: six instructions an element, where the general division takes a dozen.
__device__ __forceinline__ uint32_t quotient_byte(float x, float s, float r) {
    const float q0 = x * r;
    const float q = fmaf(fmaf(-q0, s, x), r, q0);
    return __float_as_uint(q + 12582912.f);
}

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400), hi = __builtin_amdgcn_perm(d, c, 0x04000c0c);
    return lo | hi;
}

// Rows of whole 16-byte vectors, NV of them a thread, held in registers between the maximum and the
// quotients.  Bound by the bytes: an element is read once and its byte written once.
template <bool F32, int NV>
__global__ __launch_bounds__(1024) void quantize_vectors(const void* x, int8_t* q, float* scale, uint32_t rows,
                                                         uint32_t dim) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ uint32_t lds[2][16];
    const uint32_t T = blockDim.x, t = threadIdx.x, G = blockDim.y, g = threadIdx.y;
    int phase = 0;
    for (uint32_t r0 = blockIdx.x * G; r0 < rows; r0 += gridDim.x * G, phase ^= 1) {
        const uint32_t r = r0 + g;
        const bool live = r < rows;  // every thread keeps the barriers
        const size_t at = static_cast<size_t>(r) * dim;
        u32x4 v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t c = (i * T + t) * V;
            v[i] = u32x4{0, 0, 0, 0};
            if (live && c < dim)
                v[i] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4*>(static_cast<const char*>(x) + (at + c) * (F32 ? 4 : 2)));
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (F32) {
                    const uint32_t m = v[i][k] & 0x7fffffffu;
                    top = m > top ? m : top;
                } else {
                    const uint32_t lo = v[i][k] << 16 & 0x7fffffffu, hi = v[i][k] & 0x7fff0000u;
                    top = lo > top ? lo : top;
                    top = hi > top ? hi : top;
                }
            }
        top = row_max(top, lds[phase], t, T, g);
        const float s = scale_of(top);
        const bool usual = s > 0x1p-100f && s < 0x1p100f;
        const float rs = 1.0f / s;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint32_t c = (i * T + t) * V;
                if (c >= dim) continue;
                uint32_t out[V / 4];
#pragma unroll
                for (int k = 0; k < V; k += 4) {
                    uint32_t b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f;
                        if constexpr (F32) f = __uint_as_float(v[i][j]);
                        else f = __uint_as_float((k + j) % 2 ? v[i][(k + j) / 2] & 0xffff0000u : v[i][(k + j) / 2] << 16);
                        b[j] = usual ? quotient_byte(f, s, rs) : static_cast<uint32_t>(quotient(f, s));
                    }
                    out[k / 4] = pack_bytes(b[0], b[1], b[2], b[3]);
                }
                __builtin_memcpy(__builtin_assume_aligned(q + at + c, V), out, V);
            }
            if (t == 0) scale[r] = s;
        }
    }
}

// Any row: one workgroup each, which reads it twice, from memory for the largest magnitude and from cache
// for the quotients.
template <bool F32>
__global__ __launch_bounds__(1024) void quantize_rows(const void* x, int8_t* q, float* scale, uint32_t rows,
                                                      uint32_t dim) {
    __shared__ uint32_t lds[2][16];
    int phase = 0;
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x, phase ^= 1) {
        const char* row = static_cast<const char*>(x) + static_cast<size_t>(r) * dim * (F32 ? 4 : 2);
        uint32_t top = 0;
        for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x) {
            const uint32_t m = __float_as_uint(value<F32>(row, c)) & 0x7fffffffu;
            top = m > top ? m : top;
        }
        top = row_max(top, lds[phase], threadIdx.x, blockDim.x, 0);
        const float s = scale_of(top);
        int8_t* out = q + static_cast<size_t>(r) * dim;
        for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x)
            out[c] = static_cast<int8_t>(quotient(value<F32>(row, c), s));
        if (threadIdx.x == 0) scale[r] = s;
    }
}

struct ScaledDone {
    bool f32;
    void* y;
    const float *a_scale, *b_scale, *bias;
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, i32x4 v) const {
        const float sm = a_scale[m];
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = n + i < N ? n + i : N - 1;
            // the integer, its conversion and each product: rounded once each
            o[i] = static_cast<float>(v[i]) * sm * b_scale[c];
            if (bias) o[i] += bias[c];
        }
        if (f32) store4<true>(static_cast<float*>(y) + static_cast<size_t>(m) * N, n, N, o);
        else store4<false>(static_cast<uint16_t*>(y) + static_cast<size_t>(m) * N, n, N, o);
    }
};

bool direct(const Q8Problem& p) { return chunks16(p.a, p.dim, p.dim) && chunks16(p.b, p.dim, p.dim); }

}  // namespace

size_t q8_workspace(const Q8Problem& p) {
    if (p.tokens <= kFewRows) return 0;
    return plan_product<OpI8, false, false>(p.tokens, p.out, p.dim, direct(p), p.dim).partial_bytes;
}

hipError_t launch_q8(const Q8Problem& p, bool f32, hipStream_t stream) {
    Product q{};
    q.a = static_cast<const char*>(p.a);
    q.b[0] = static_cast<const char*>(p.b);
    q.a_pitch = q.b_pitch = p.dim;
    q.M = p.tokens;
    q.N = p.out;
    q.k = p.dim;
    const ScaledDone done{f32, p.y, p.a_scale, p.b_scale, p.bias};
    if (p.tokens <= kFewRows) return launch_few_rows<OpI8, false>(q, done, stream);
    return launch_product<OpI8, false, false, false>(q, direct(p), p.workspace, done, stream);
}

namespace {

template <bool F32>
void quantize(const void* x, int8_t* q, float* scale, uint32_t rows, uint32_t dim, hipStream_t stream) {
    constexpr uint32_t V = F32 ? 4 : 8;
    const bool vectors = dim % V == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % V == 0;
    const uint32_t count = dim / V;
    if (vectors && count <= 4096) {
        // two vectors a thread where 1024 threads hold a row so, else four; at least 256 threads a workgroup
        const uint32_t nv = count <= 2048 ? 2 : 4;
        const uint32_t T = 64 * ((count + 64 * nv - 1) / (64 * nv)), G = T >= 256 ? 1 : 256 / T;
        const uint32_t need = (rows + G - 1) / G;
        const dim3 block(T, G);
        const uint32_t grid = need < 8192 ? need : 8192;
        if (nv == 2) quantize_vectors<F32, 2><<<grid, block, 0, stream>>>(x, q, scale, rows, dim);
        else quantize_vectors<F32, 4><<<grid, block, 0, stream>>>(x, q, scale, rows, dim);
    } else {
        const uint32_t T = dim >= 4096 ? 1024 : 256;
        quantize_rows<F32><<<rows < 16384 ? rows : 16384, T, 0, stream>>>(x, q, scale, rows, dim);
    }
}

}  // namespace

hipError_t launch_q8_quantize(const void* x, void* q, float* scale, uint32_t rows, uint32_t dim, bool f32,
                              hipStream_t stream) {
    if (f32) quantize<true>(x, static_cast<int8_t*>(q), scale, rows, dim, stream);
    else quantize<false>(x, static_cast<int8_t*>(q), scale, rows, dim, stream);
    return hipGetLastError();
}

}  // namespace ltx3drope
