// The gated feed-forward block h = act(x Wg^T) * (x Wu^T) and its backward pass.
//
// x [M, D], Wg and Wu [F, D], h [M, F].  Forward: one kernel holds the same rows of both weights
// against a tile of x (product.h, gated), and applies activation and product to the finished sums.
//
// Backward, from the projections g and u that the forward keeps.  They are kept in fp32: in bf16 their
// roundings come on top of those of dg and du and of the gradients themselves (measured: gradients
// within 0.0030 of 64 bits in the 2-norm, 0.0023 to 0.0024 with fp32 projections, 0.0017 the output's rounding
// alone).  The round trip through memory costs a ninth of a training step (4096 tokens, 2048 -> 8192
// bf16: 90 of 791 us; half of that in bf16), where recomputing the projections would cost 220 us:
//     dg = dh * u * act'(g),  du = dh * act(g)          in fp32, rounded once for the matrix cores
//     dx = [dg du] [Wg; Wu],  dWg = dg^T x,  dWu = du^T x
// dg and du lie side by side, [M][2 Fp], so that dx is one product over k = 2F and dWg, dWu together
// one over k = M.  Where an operand has k outermost (the weights for dx, both operands for dW), LDS
// holds rows of k and the reads from it turn them (product.h): nothing is transposed in memory.
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

// act(g) and act'(g) in fp32; kind is the same for a whole launch.
__device__ __forceinline__ float act(int kind, float g, float* slope) {
    if (kind == 0) {  // silu
        const float s = logistic(g);
        if (slope) *slope = fmaf(g * s, 1.0f - s, s);
        return g * s;
    }
    if (kind == 1) {
        // gelu, by the complement: 1 + erf would cancel on the negative side (0 from -5.5 on).  It costs up
        // to 4 % of a forward call (4096 tokens, 2048 -> 8192 bf16: 241 us, 232 with 1 + erf).
        const float c = 0.5f * erfcf(g * -0.70710678118654752f);
        if (slope) *slope = fmaf(g * 0.39894228040143268f, __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g), c);
        return g * c;
    }
    // gelu by its tanh formula: (1 + tanh z) / 2 is the logistic function of 2z
    const float z2 = 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
    const float s = logistic(z2);
    if (slope) {
        // s or 1 - s is 0 long before g^2 passes 2^100: held there, so that 0 is not multiplied by infinity
        const float g2 = fminf(g * g, 0x1p100f);
        *slope = fmaf(g * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f, g2, 1.0f), s);
    }
    return g * s;
}

template <bool F32>
struct GatedDone {
    int kind;
    void* h;
    float *g, *u;  // NULL unless kept
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, f32x4 vg, f32x4 vu) const {
        const size_t off = static_cast<size_t>(m) * N * (F32 ? 4 : 2);
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = act(kind, vg[i], nullptr) * vu[i];
        store4<F32>(static_cast<char*>(h) + off, n, N, o);
        if (g) {
            store4<true>(g + static_cast<size_t>(m) * N, n, N, vg);
            store4<true>(u + static_cast<size_t>(m) * N, n, N, vu);
        }
    }
};

template <bool F32>
struct RowsDone {
    void* out;
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, f32x4 v) const {
        store4<F32>(static_cast<char*>(out) + static_cast<size_t>(m) * N * (F32 ? 4 : 2), n, N, v);
    }
};

// Output rows 0 .. rows - 1 are the first matrix's, those from `second_at` on the second's; between and
// behind them lies padding.
template <bool F32>
struct SplitDone {
    void *first, *second;
    uint32_t rows, second_at;
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, f32x4 v) const {
        const bool other = m >= second_at;
        const uint32_t r = other ? m - second_at : m;
        if (r >= rows) return;
        store4<F32>(static_cast<char*>(other ? second : first) + static_cast<size_t>(r) * N * (F32 ? 4 : 2), n, N, v);
    }
};

template <bool F32>
__device__ __forceinline__ float get(const void* p, size_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}
// Eight floats of any alignment that nobody reads again.
__device__ __forceinline__ void load8(float (&v)[8], const float* p) {
    typedef float any_f32x4 __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x4 q = __builtin_nontemporal_load(reinterpret_cast<const any_f32x4*>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * i + k] = q[k];
    }
}

// dg and du as rows [M][2 * Fp]: dg, zeros up to Fp, du, zeros.  Eight columns a thread; bound by the
// bytes (10 read and 4 written an element in bf16).
template <bool F32>
__global__ __launch_bounds__(256) void ffn_slopes(const void* dh, const float* g, const float* u, void* out, uint32_t M,
                                                  uint32_t F, uint32_t Fp, int kind) {
    const uint32_t per_row = Fp / 8;
    const size_t total = static_cast<size_t>(M) * per_row;
    for (size_t t = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; t < total; t += size_t(gridDim.x) * 256) {
        const uint32_t r = static_cast<uint32_t>(t / per_row), c = static_cast<uint32_t>(t % per_row) * 8;
        const size_t at = static_cast<size_t>(r) * F + c;
        float vg[8] = {}, vu[8] = {}, d[8] = {};
        if (c + 8 <= F) {
            load8(vg, g + at);
            load8(vu, u + at);
            if constexpr (F32) {
                load8(d, static_cast<const float*>(dh) + at);
            } else {
                typedef __bf16 any_bf16x8 __attribute__((ext_vector_type(8), aligned(2)));
                const bf16x8 h = __builtin_nontemporal_load(
                    reinterpret_cast<const any_bf16x8*>(static_cast<const __bf16*>(dh) + at));
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = static_cast<float>(h[i]);
            }
        } else {
            for (int i = 0; i < 8; ++i)
                if (c + i < F) {
                    vg[i] = g[at + i];
                    vu[i] = u[at + i];
                    d[i] = get<F32>(dh, at + i);
                }
        }
        float dg[8], du[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float slope;
            const float a = act(kind, vg[i], &slope);
            const bool in = c + i < F;
            dg[i] = in ? d[i] * vu[i] * slope : 0.f;
            du[i] = in ? d[i] * a : 0.f;
        }
        char* row = static_cast<char*>(out) + (static_cast<size_t>(r) * 2 * Fp + c) * (F32 ? 4 : 2);
        auto put = [](char* to, const float(&v)[8]) {
            if constexpr (F32) {
                __builtin_memcpy(__builtin_assume_aligned(to, 16), v, 32);
            } else {
                bf16x8 h;
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = static_cast<__bf16>(v[i]);
                __builtin_memcpy(__builtin_assume_aligned(to, 16), &h, 16);
            }
        };
        put(row, dg);
        put(row + static_cast<size_t>(Fp) * (F32 ? 4 : 2), du);
    }
}

__global__ __launch_bounds__(256) void fill_zero(uint16_t* p, size_t halfs) {
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < halfs; i += size_t(gridDim.x) * 256) p[i] = 0;
}

template <bool F32>
using OpOf = typename std::conditional<F32, OpF32, OpBf16>::type;

template <bool F32>
bool forward_direct(const FfnProblem& p) {
    const size_t row = p.dim * (F32 ? 4 : 2);
    return chunks16(p.x, row, row) && chunks16(p.w_gate, row, row) && chunks16(p.w_up, row, row);
}

template <bool F32>
size_t forward_workspace(const FfnProblem& p) {
    if (p.tokens <= kFewRows) return 0;
    return plan_product<OpOf<F32>, true, false>(p.tokens, p.hidden, p.dim, forward_direct<F32>(p), p.dim * (F32 ? 4 : 2))
        .partial_bytes;
}

template <bool F32>
hipError_t forward(const FfnProblem& p, hipStream_t stream) {
    Product q{};
    q.a = static_cast<const char*>(p.x);
    q.b[0] = static_cast<const char*>(p.w_gate);
    q.b[1] = static_cast<const char*>(p.w_up);
    q.a_pitch = q.b_pitch = p.dim * (F32 ? 4 : 2);
    q.M = p.tokens;
    q.N = p.hidden;
    q.k = p.dim;
    const GatedDone<F32> done{p.activation, p.h, p.g, p.u};
    if (p.tokens <= kFewRows) return launch_few_rows<OpOf<F32>, true>(q, done, stream);
    return launch_product<OpOf<F32>, true, false, false>(q, forward_direct<F32>(p), p.workspace, done, stream);
}

// The backward's workspace: the slopes' rows, then what the products that are split over k need.
struct BackwardLayout {
    uint32_t Fp;  // hidden, padded to whole steps of k
    bool dx_direct, dw_direct;
    size_t slopes, bytes;
};

template <bool F32>
BackwardLayout backward_layout(const FfnBackwardProblem& p) {
    const size_t es = F32 ? 4 : 2, row = p.dim * es;
    const uint32_t step = kRowBytes / es;
    BackwardLayout l;
    l.Fp = (p.hidden + step - 1) / step * step;
    l.dx_direct = chunks16(p.w_gate, row, row) && chunks16(p.w_up, row, row);
    l.dw_direct = chunks16(p.x, row, row);
    l.slopes = size_t(p.tokens) * 2 * l.Fp * es;  // whole 128-byte steps
    const size_t a = p.dx ? plan_product<OpOf<F32>, false, true>(p.tokens, p.dim, 2 * l.Fp, l.dx_direct, row).partial_bytes : 0;
    const size_t b = p.dw_gate ? plan_product<OpOf<F32>, false, true>(2 * l.Fp, p.dim, p.tokens, l.dw_direct, row).partial_bytes : 0;
    l.bytes = l.slopes + (a > b ? a : b);
    return l;
}

template <bool F32>
hipError_t backward(const FfnBackwardProblem& p, hipStream_t stream) {
    const size_t es = F32 ? 4 : 2;
    if (p.tokens == 0 || p.hidden == 0) {  // empty sums
        const size_t dx = size_t(p.tokens) * p.dim * es / 2, dw = size_t(p.hidden) * p.dim * es / 2;
        const std::pair<void*, size_t> outs[3] = {{p.dx, dx}, {p.dw_gate, dw}, {p.dw_up, dw}};
        for (const auto& o : outs)
            if (o.first && o.second) fill_zero<<<1024, 256, 0, stream>>>(static_cast<uint16_t*>(o.first), o.second);
        return hipGetLastError();
    }
    const BackwardLayout l = backward_layout<F32>(p);
    char* slopes = static_cast<char*>(p.workspace);
    char* partial = slopes + l.slopes;
    const size_t groups = (size_t(p.tokens) * (l.Fp / 8) + 255) / 256;
    ffn_slopes<F32><<<static_cast<uint32_t>(groups < 16384 ? groups : 16384), 256, 0, stream>>>(
        p.dh, p.g, p.u, slopes, p.tokens, p.hidden, l.Fp, p.activation);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.dx) {
        Product q{};
        q.a = slopes;
        q.b[0] = static_cast<const char*>(p.w_gate);
        q.b[1] = static_cast<const char*>(p.w_up);
        q.a_pitch = 2 * l.Fp * es;
        q.b_pitch = p.dim * es;
        q.M = p.tokens;
        q.N = p.dim;
        q.k = 2 * l.Fp;
        q.k_second = l.Fp;
        q.k_rows = p.hidden;
        e = launch_product<OpOf<F32>, false, false, true>(q, l.dx_direct, partial, RowsDone<F32>{p.dx}, stream);
    }
    if (e == hipSuccess && p.dw_gate) {
        Product q{};
        q.a = slopes;
        q.b[0] = static_cast<const char*>(p.x);
        q.a_pitch = 2 * l.Fp * es;
        q.b_pitch = p.dim * es;
        q.M = 2 * l.Fp;
        q.N = p.dim;
        q.k = p.tokens;
        e = launch_product<OpOf<F32>, false, true, true>(
            q, l.dw_direct, partial, SplitDone<F32>{p.dw_gate, p.dw_up, p.hidden, l.Fp}, stream);
    }
    return e;
}

}  // namespace

size_t ffn_workspace(const FfnProblem& p, bool f32) {
    return f32 ? forward_workspace<true>(p) : forward_workspace<false>(p);
}

size_t ffn_backward_workspace(const FfnBackwardProblem& p, bool f32) {
    return f32 ? backward_layout<true>(p).bytes : backward_layout<false>(p).bytes;
}

hipError_t launch_ffn(const FfnProblem& p, bool f32, hipStream_t stream) {
    return f32 ? forward<true>(p, stream) : forward<false>(p, stream);
}

hipError_t launch_ffn_backward(const FfnBackwardProblem& p, bool f32, hipStream_t stream) {
    return f32 ? backward<true>(p, stream) : backward<false>(p, stream);
}

}  // namespace ltx3drope
