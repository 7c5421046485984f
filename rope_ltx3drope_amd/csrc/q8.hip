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

// One workgroup a row, which it reads twice: from memory for the largest magnitude, from cache for the
// quotients.  NaN counts as larger than any number.
template <bool F32>
__global__ __launch_bounds__(256) void quantize_rows(const void* x, int8_t* q, float* scale, uint32_t rows,
                                                     uint32_t dim) {
    __shared__ uint32_t lds[2][4];
    int phase = 0;
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x, phase ^= 1) {
        const char* row = static_cast<const char*>(x) + static_cast<size_t>(r) * dim * (F32 ? 4 : 2);
        // magnitudes compare like their bit patterns, and a NaN's is above every number's
        uint32_t top = 0;
        for (uint32_t c = threadIdx.x; c < dim; c += 256) {
            const uint32_t m = __float_as_uint(value<F32>(row, c)) & 0x7fffffffu;
            top = m > top ? m : top;
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t o = __shfl_xor(top, m);
            top = o > top ? o : top;
        }
        if ((threadIdx.x & 63) == 0) lds[phase][threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w) top = lds[phase][w] > top ? lds[phase][w] : top;
        const float s = __uint_as_float(top) * (1.0f / 127.0f);
        const bool plain = s > 0.f && s < __builtin_inff();
        int8_t* out = q + static_cast<size_t>(r) * dim;
        for (uint32_t c = threadIdx.x; c < dim; c += 256) {
            // a subnormal scale may be far off its value: the quotient is kept within the 8 bits
            const float v = plain ? rintf(value<F32>(row, c) / s) : 0.f;
            out[c] = static_cast<int8_t>(fminf(fmaxf(v, -127.f), 127.f));
        }
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
    return plan_product<OpI8, false>(p.tokens, p.out, p.dim, direct(p)).partial_bytes;
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

hipError_t launch_q8_quantize(const void* x, void* q, float* scale, uint32_t rows, uint32_t dim, bool f32,
                              hipStream_t stream) {
    const uint32_t grid = rows < 65536 ? rows : 65536;
    if (f32) quantize_rows<true><<<grid, 256, 0, stream>>>(x, static_cast<int8_t*>(q), scale, rows, dim);
    else quantize_rows<false><<<grid, 256, 0, stream>>>(x, static_cast<int8_t*>(q), scale, rows, dim);
    return hipGetLastError();
}

}  // namespace ltx3drope
