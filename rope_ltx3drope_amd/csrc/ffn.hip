// The gated feed-forward block h = act(x Wg^T) * (x Wu^T) and its backward pass.
//
// x [M, D], Wg and Wu [F, D], h [M, F].  Forward: one kernel holds the same rows of both weights
// against a tile of x (product.h, gated), and applies activation and product to the finished sums.
//
// Backward, from the projections g and u that the forward keeps.  They are kept in fp32: in bf16 their
// roundings come on top of those of dg and du and of the gradients themselves (measured: gradients
// within 0.0030 of 64 bits in the 2-norm, 0.0024 with fp32 projections, 0.0017 the output's rounding
// alone).  The round trip through memory is a twentieth of the products' time, where recomputing the
// projections would be a third:
//     dg = dh * u * act'(g),  du = dh * act(g)          in fp32, rounded once for the matrix cores
//     dx = [dg du] [Wg; Wu],  dWg = dg^T x,  dWu = du^T x
// The matrix cores want k innermost on both sides, so one pass writes dg and du both ways round and
// two more turn x and the weights; then dx is one product over k = 2F and dWg, dWu together one over
// k = M.  Rows in the workspace are padded with zeros to whole 16-byte chunks.
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "block.h"
#include "product.h"

namespace ltx3drope {
namespace {

// 1 / (1 + e^-z) by the hardware's exponential and reciprocal, each within about 1 ulp: with the
// product z * log2(e) the relative error is at most about (|z| + 4) * 2^-24, and a sixth of the
// instructions of the exactly rounded division and expf, which an epilogue would feel.
__device__ __forceinline__ float logistic(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// act(g) and act'(g) in fp32.
template <int ACT>
__device__ __forceinline__ float act(float g, float* slope) {
    if constexpr (ACT == 0) {  // silu
        const float s = logistic(g);
        if (slope) *slope = fmaf(g * s, 1.0f - s, s);
        return g * s;
    } else if constexpr (ACT == 1) {  // gelu
        const float c = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
        if (slope) *slope = fmaf(g * 0.39894228040143268f, __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g), c);
        return g * c;
    } else {  // gelu by its tanh formula: (1 + tanh z) / 2 is the logistic function of 2z
        const float z2 = 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
        const float s = logistic(z2);
        if (slope) *slope = fmaf(g * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f * g, g, 1.0f), s);
        return g * s;
    }
}

template <bool F32, int ACT>
struct GatedDone {
    void* h;
    float *g, *u;  // NULL unless kept
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, f32x4 vg, f32x4 vu) const {
        const size_t off = static_cast<size_t>(m) * N * (F32 ? 4 : 2);
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = act<ACT>(vg[i], nullptr) * vu[i];
        store4<F32>(static_cast<char*>(h) + off, n, N, o);
        if (g) {
            store4<true>(g + static_cast<size_t>(m) * N, n, N, vg);
            store4<true>(u + static_cast<size_t>(m) * N, n, N, vu);
        }
    }
};

// Rows [0, split) go to the first matrix, the rest to the second.
template <bool F32>
struct SplitDone {
    void *first, *second;
    uint32_t split;
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, f32x4 v) const {
        char* base = static_cast<char*>(m < split ? first : second);
        store4<F32>(base + static_cast<size_t>(m < split ? m : m - split) * N * (F32 ? 4 : 2), n, N, v);
    }
};

template <bool F32>
__device__ __forceinline__ float get(const void* p, size_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void put(void* p, size_t i, float v) {
    if constexpr (F32) static_cast<float*>(p)[i] = v;
    else static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

// dst[c][r] = src[r][c] for src [rows, cols] into rows of `pitch` elements, of which `width` (at least
// `rows`) are written, zeros past `rows`.  64 x 64 tiles through LDS: both sides in whole lines.
template <bool F32>
__global__ __launch_bounds__(256) void transpose(const void* src, void* dst, uint32_t rows, uint32_t cols,
                                                 uint32_t width, uint64_t pitch) {
    __shared__ float tile[64][65];
    const uint32_t c0 = blockIdx.x * 64, r0 = blockIdx.y * 64, x = threadIdx.x % 64, y = threadIdx.x / 64;
    for (uint32_t i = y; i < 64; i += 4) {
        const uint32_t r = r0 + i, c = c0 + x;
        tile[i][x] = r < rows && c < cols ? get<F32>(src, static_cast<size_t>(r) * cols + c) : 0.f;
    }
    __syncthreads();
    for (uint32_t i = y; i < 64; i += 4) {
        const uint32_t c = c0 + i, r = r0 + x;
        if (c < cols && r < width) put<F32>(dst, c * pitch + r, tile[x][i]);
    }
}

// dg and du, as rows [M][2 * Fp] (dg, then du) and turned [2 * F][Mp] (dg's rows, then du's), with
// zeros in the padding.
template <bool F32, int ACT>
__global__ __launch_bounds__(256) void ffn_slopes(const void* dh, const float* g, const float* u, void* rowsd,
                                                  void* turned, uint32_t M, uint32_t F, uint32_t Fp, uint32_t Mp) {
    __shared__ float tg[64][65], tu[64][65];
    const uint32_t c0 = blockIdx.x * 64, r0 = blockIdx.y * 64, x = threadIdx.x % 64, y = threadIdx.x / 64;
    for (uint32_t i = y; i < 64; i += 4) {
        const uint32_t r = r0 + i, c = c0 + x;
        float dg = 0.f, du = 0.f;
        if (r < M && c < F) {
            const size_t at = static_cast<size_t>(r) * F + c;
            float slope;
            const float a = act<ACT>(g[at], &slope);
            const float d = get<F32>(dh, at);
            dg = d * u[at] * slope;
            du = d * a;
        }
        tg[i][x] = dg;
        tu[i][x] = du;
        if (r < M && c < Fp) {
            put<F32>(rowsd, static_cast<size_t>(r) * 2 * Fp + c, dg);
            put<F32>(rowsd, static_cast<size_t>(r) * 2 * Fp + Fp + c, du);
        }
    }
    __syncthreads();
    for (uint32_t i = y; i < 64; i += 4) {
        const uint32_t c = c0 + i, r = r0 + x;
        if (c < F && r < Mp) {
            put<F32>(turned, static_cast<size_t>(c) * Mp + r, tg[x][i]);
            put<F32>(turned, static_cast<size_t>(F + c) * Mp + r, tu[x][i]);
        }
    }
}

__global__ __launch_bounds__(256) void fill_zero(uint16_t* p, size_t halfs) {
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < halfs; i += size_t(gridDim.x) * 256) p[i] = 0;
}

uint32_t tiles64(uint32_t n) { return (n + 63) / 64; }

template <bool F32>
hipError_t forward(const FfnProblem& p, hipStream_t stream) {
    using Op = typename std::conditional<F32, OpF32, OpBf16>::type;
    const size_t es = F32 ? 4 : 2;
    Product q;
    q.a = static_cast<const char*>(p.x);
    q.b[0] = static_cast<const char*>(p.w_gate);
    q.b[1] = static_cast<const char*>(p.w_up);
    q.a_pitch = q.b_pitch = p.dim * es;
    q.M = p.tokens;
    q.N = p.hidden;
    q.k_bytes = static_cast<uint32_t>(p.dim * es);
    if (p.tokens > kFewRows && !aligned16(q, true)) {
        // rows that no 16-byte chunk divides, or unaligned tensors: padded copies in the workspace
        const size_t pitch = up16(p.dim * es);
        char* at = static_cast<char*>(p.workspace);
        const char* src[3] = {q.a, q.b[0], q.b[1]};
        const char* dst[3];
        const uint32_t rows[3] = {p.tokens, p.hidden, p.hidden};
        for (int i = 0; i < 3; ++i) {
            launch_pad_rows<typename std::conditional<F32, uint32_t, uint16_t>::type>(src[i], at, rows[i], p.dim * es,
                                                                                      stream);
            dst[i] = at;
            at += rows[i] * pitch;
        }
        q.a = dst[0];
        q.b[0] = dst[1];
        q.b[1] = dst[2];
        q.a_pitch = q.b_pitch = pitch;
        q.k_bytes = static_cast<uint32_t>(pitch);
    }
    switch (p.activation) {
        case 0: return launch_product<Op, true>(q, GatedDone<F32, 0>{p.h, p.g, p.u}, stream);
        case 1: return launch_product<Op, true>(q, GatedDone<F32, 1>{p.h, p.g, p.u}, stream);
        default: return launch_product<Op, true>(q, GatedDone<F32, 2>{p.h, p.g, p.u}, stream);
    }
}

struct BackwardLayout {
    size_t Fp, Mp;                        // padded widths, elements
    size_t rows, turned, x_t, w_t, bytes;  // offsets and total
};

BackwardLayout backward_layout(const FfnBackwardProblem& p, size_t es) {
    BackwardLayout l;
    l.Fp = up16(p.hidden * es) / es;
    l.Mp = up16(p.tokens * es) / es;
    l.rows = 0;
    l.turned = l.rows + up16(size_t(p.tokens) * 2 * l.Fp * es);
    l.x_t = l.turned + up16(size_t(2) * p.hidden * l.Mp * es);
    l.w_t = l.x_t + up16(size_t(p.dim) * l.Mp * es);
    l.bytes = l.w_t + up16(size_t(p.dim) * 2 * l.Fp * es);
    return l;
}

template <bool F32>
hipError_t backward(const FfnBackwardProblem& p, hipStream_t stream) {
    using Op = typename std::conditional<F32, OpF32, OpBf16>::type;
    const size_t es = F32 ? 4 : 2;
    if (p.tokens == 0 || p.hidden == 0) {  // empty sums
        const size_t dx = size_t(p.tokens) * p.dim * es / 2, dw = size_t(p.hidden) * p.dim * es / 2;
        const std::pair<void*, size_t> outs[3] = {{p.dx, dx}, {p.dw_gate, dw}, {p.dw_up, dw}};
        for (const auto& o : outs)
            if (o.first && o.second) fill_zero<<<1024, 256, 0, stream>>>(static_cast<uint16_t*>(o.first), o.second);
        return hipGetLastError();
    }
    const BackwardLayout l = backward_layout(p, es);
    char* ws = static_cast<char*>(p.workspace);
    const uint32_t Fp = static_cast<uint32_t>(l.Fp), Mp = static_cast<uint32_t>(l.Mp);
    const dim3 grid(tiles64(Fp), tiles64(Mp));
    void *rows = ws + l.rows, *turned = ws + l.turned;
    switch (p.activation) {
        case 0: ffn_slopes<F32, 0><<<grid, 256, 0, stream>>>(p.dh, p.g, p.u, rows, turned, p.tokens, p.hidden, Fp, Mp); break;
        case 1: ffn_slopes<F32, 1><<<grid, 256, 0, stream>>>(p.dh, p.g, p.u, rows, turned, p.tokens, p.hidden, Fp, Mp); break;
        default: ffn_slopes<F32, 2><<<grid, 256, 0, stream>>>(p.dh, p.g, p.u, rows, turned, p.tokens, p.hidden, Fp, Mp);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.dx) {
        char* w_t = ws + l.w_t;
        const dim3 wg(tiles64(p.dim), tiles64(Fp));
        transpose<F32><<<wg, 256, 0, stream>>>(p.w_gate, w_t, p.hidden, p.dim, Fp, 2 * l.Fp);
        transpose<F32><<<wg, 256, 0, stream>>>(p.w_up, w_t + l.Fp * es, p.hidden, p.dim, Fp, 2 * l.Fp);
        Product q{};
        q.a = static_cast<const char*>(rows);
        q.b[0] = w_t;
        q.a_pitch = q.b_pitch = 2 * l.Fp * es;
        q.M = p.tokens;
        q.N = p.dim;
        q.k_bytes = static_cast<uint32_t>(2 * l.Fp * es);
        e = launch_product<Op, false>(q, SplitDone<F32>{p.dx, p.dx, p.tokens}, stream);
        if (e != hipSuccess) return e;
    }
    if (p.dw_gate) {
        char* x_t = ws + l.x_t;
        transpose<F32><<<dim3(tiles64(p.dim), tiles64(Mp)), 256, 0, stream>>>(p.x, x_t, p.tokens, p.dim, Mp, l.Mp);
        Product q{};
        q.a = static_cast<const char*>(turned);
        q.b[0] = x_t;
        q.a_pitch = q.b_pitch = l.Mp * es;
        q.M = 2 * p.hidden;
        q.N = p.dim;
        q.k_bytes = static_cast<uint32_t>(l.Mp * es);
        e = launch_product<Op, false>(q, SplitDone<F32>{p.dw_gate, p.dw_up, p.hidden}, stream);
    }
    return e;
}

}  // namespace

size_t ffn_workspace(const FfnProblem& p, bool f32) {
    const size_t es = f32 ? 4 : 2;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.w_gate) |
                           reinterpret_cast<uintptr_t>(p.w_up) | (p.dim * es);
    if (p.tokens <= kFewRows || bits % 16 == 0) return 0;
    return (size_t(p.tokens) + 2 * size_t(p.hidden)) * up16(p.dim * es);
}

size_t ffn_backward_workspace(const FfnBackwardProblem& p, bool f32) { return backward_layout(p, f32 ? 4 : 2).bytes; }

hipError_t launch_ffn(const FfnProblem& p, bool f32, hipStream_t stream) {
    return f32 ? forward<true>(p, stream) : forward<false>(p, stream);
}

hipError_t launch_ffn_backward(const FfnBackwardProblem& p, bool f32, hipStream_t stream) {
    return f32 ? backward<true>(p, stream) : backward<false>(p, stream);
}

}  // namespace ltx3drope
