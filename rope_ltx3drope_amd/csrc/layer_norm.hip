// Layer norms before and after a transformer block, fused with the block's gate, the residual and the
// norm's own weight, bias and per-sample scale and shift; and their backward pass.
//
// Per row of width D (rows of sample b), in fp32 but for the mean:
//     r      = residual + gate_b * y                     (before a block: r is the input itself)
//     hat(r) = (r - mean(r)) * rstd,  rstd = 1 / sqrt(mean((r - mean(r))^2) + eps)
//     n      = (hat(r) * w + bias) * (1 + scale_b) + shift_b
//
// Backward, with v = dn * w * (1 + scale_b):
//     dR = dr + rstd * (v - mean(v) - hat(r) * mean(v * hat(r)))     (dr: what reaches r past the norm)
//     dresidual = dR,  dy = gate_b * dR
// and per sample P1 = sum_rows dn * hat(r), P2 = sum_rows dn, P3 = sum_rows dR * y, from which
//     dscale_b = w P1 + bias P2, dshift_b = P2, dw = sum_b (1 + scale_b) P1,
//     dbias = sum_b (1 + scale_b) P2, dgate_b = P3.
//
// The mean is taken first and the squares around it: their difference would lose what a row with a large
// mean has left.  The mean is formed in 64 bits (the sum of up to 2^14 equal numbers is exact there) and taken
// off as two fp32 numbers: rounded to one it would be off by 2^-24 of itself, which may be many times the
// row's spread.  A row of one value is zeros with a variance of zero, whatever the value.  It costs no time: a
// sum in fp32 and a second one of what its rounding left took 228 us a call where this takes 201 to 209 (2 x 34680 x
// 2048 bf16 after a block).
//
// Bound: HBM.  Layout, walk over the rows and partial sums are those of rows.h and norm.hip.  That call moves 5.4 to
// 5.65 TB/s (the RMS norm there takes 210 to 222 us and a plain kernel of two streams in and two out 192); its
// backward, 2 x 18360, 167 us (5.4 TB/s), 7 of them to join the vectors' gradients; before a block, fp32 rows of 2053 off
// the 16 bytes, 3 x 1021, 15 us (3.4 TB/s, 4-byte loads); one row of 4096 for each of four samples: the kernel 3.8 us.
#include <hip/hip_runtime.h>

#include <utility>

#include "block.h"
#include "rows.h"

namespace ltx3drope {
namespace {

// A row's mean as the sum of two fp32 numbers.
struct Mean {
    float hi, lo;
};

template <int CTRL>
__device__ __forceinline__ double lanes64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// The mean of a row's elements, E a thread with zeros past the row's end, in the order of row_sum, whose rules
// for `lds` (a number a wavefront) hold.  inv_d: 1 / D; the quotient is corrected by its exact remainder, so
// that the mean of equal numbers is that number.
template <int E>
__device__ __forceinline__ Mean row_mean(const float (&r)[E], double* lds, double d, double inv_d, uint32_t t, uint32_t T,
                                         uint32_t g) {
    double even = 0.0, odd = 0.0;
#pragma unroll
    for (int k = 0; k < E; k += 2) {
        even += r[k];
        odd += r[k + 1];
    }
    double v = even + odd;
    v += lanes64<0xb1>(v);   // quad_perm 1 0 3 2
    v += lanes64<0x4e>(v);   // quad_perm 2 3 0 1
    v += lanes64<0x141>(v);  // row_half_mirror
    v += lanes64<0x140>(v);  // row_mirror
    auto lane = [&](int l) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), l);
        const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), l);
        return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
    };
    double sum = (lane(0) + lane(16)) + (lane(32) + lane(48));
    const uint32_t W = T / 64;
    if (W > 1) {
        double* mine = lds + g * W;
        if ((t & 63) == 0) mine[t / 64] = sum;
        __syncthreads();
        sum = 0.0;
        for (uint32_t w = 0; w < W; ++w) sum += mine[w];
    }
    const double about = sum * inv_d, mean = fma(fma(-about, d, sum), inv_d, about);
    const float hi = static_cast<float>(mean);
    return Mean{hi, static_cast<float>(mean - hi)};
}

// r less its mean, with zeros past the row's end (where r is zero).
template <bool F32, int E, bool VEC>
__device__ __forceinline__ void subtract(float (&r)[E], Mean mean, uint32_t t, uint32_t T, uint32_t D) {
    constexpr int V = RowPart<F32, E, VEC>::V;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
        const bool in = (i * T + t) * V < D;
        const float hi = in ? mean.hi : 0.f, lo = in ? mean.lo : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) r[i * V + j] = (r[i * V + j] - hi) - lo;
    }
}

// The norm's factor w * (1 + scale_b) and, if asked for, its term bias * (1 + scale_b) + shift_b.
template <bool F32, int E, bool VEC, class Call>
__device__ __forceinline__ void load_factor(float (&f)[E], float* term, const Call& p, const void* shift, uint32_t b,
                                            uint32_t t, uint32_t T) {
    const size_t first = static_cast<size_t>(b) * p.dim;
    float s[E];
    load_params<F32, E, VEC>(f, p.weight, 0, p.param_f32, p.chunks, 1.f, t, T, p.dim);
    load_params<F32, E, VEC>(s, p.scale, first, p.param_f32, p.chunks, 0.f, t, T, p.dim);
#pragma unroll
    for (int k = 0; k < E; ++k) f[k] *= 1.f + s[k];
    if (term == nullptr) return;
    float bias[E], sh[E];
    load_params<F32, E, VEC>(bias, p.bias, 0, p.param_f32, p.chunks, 0.f, t, T, p.dim);
    load_params<F32, E, VEC>(sh, shift, first, p.param_f32, p.chunks, 0.f, t, T, p.dim);
#pragma unroll
    for (int k = 0; k < E; ++k) term[k] = fmaf(bias[k], 1.f + s[k], sh[k]);
}

template <bool F32, int E, bool VEC, bool AFTER>
__global__ __launch_bounds__(1024) void layer_norm_forward(LayerNormForward p) {
    __shared__ double lds_sum[2][kMaxWaves];
    __shared__ float lds[2][kMaxWaves];
    const uint32_t T = blockDim.x, t = threadIdx.x, G = blockDim.y, g = threadIdx.y;
    const uint32_t D = p.dim, b = blockIdx.y;
    const float sq = p.square_scale, inv_d = 1.0f / static_cast<float>(D), inv_sq = inv_d / sq;  // sq: a power of two
    const double d64 = D, inv_d64 = 1.0 / d64;

    constexpr size_t es = F32 ? 4 : 2;
    const uint32_t step = gridDim.x * G;
    RowPart<F32, E, VEC> yr, rr;
    auto load = [&](uint32_t s) {
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        if (s < p.rows) {
            if constexpr (AFTER) yr.load(static_cast<const char*>(p.y) + off, t, T, D);
            rr.load(static_cast<const char*>(p.residual) + off, t, T, D);
        } else {
            if constexpr (AFTER) yr.clear();
            rr.clear();
        }
    };
    load(blockIdx.x * G + g);
    float fy[AFTER ? E : 1], fn[E], sh[E];
    if constexpr (AFTER)
        load_params<F32, E, VEC>(fy, p.gate, static_cast<size_t>(b) * D, p.param_f32, p.chunks, 1.f, t, T, D);
    load_factor<F32, E, VEC>(fn, sh, p, p.shift, b, t, T);
    int phase = 0;
    for (uint32_t s0 = blockIdx.x * G; s0 < p.rows; s0 += step, phase ^= 1) {
        const uint32_t s = s0 + g;
        const bool live = s < p.rows;  // every thread keeps the barriers
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        float r[E];
        rr.unpack(r);
        if constexpr (AFTER) {
            float y[E];
            yr.unpack(y);
#pragma unroll
            for (int k = 0; k < E; ++k) r[k] = fmaf(y[k], fy[k], r[k]);
        }
        load(s + step);  // the next row travels while this one is summed
        if constexpr (AFTER)
            if (live) store_row<F32, E, VEC>(static_cast<char*>(p.r) + off, r, t, T, D);
        subtract<F32, E, VEC>(r, row_mean(r, lds_sum[phase], d64, inv_d64, t, T, g), t, T, D);
        float ss[1] = {square_sum(r, sq)};
        row_sum(ss, lds[phase], t, T, g);
        const float rstd = rsqrtf(ss[0] * inv_sq + p.eps);
#pragma unroll
        for (int k = 0; k < E; ++k) r[k] = fmaf(r[k] * rstd, fn[k], sh[k]);
        if (live) store_row<F32, E, VEC>(static_cast<char*>(p.n) + off, r, t, T, D);
    }
}

template <bool F32, int E, bool VEC, bool AFTER>
__global__ __launch_bounds__(1024) void layer_norm_backward(LayerNormBackward p) {
    __shared__ double lds_sum[2][kMaxWaves];
    __shared__ float lds[2][3 * kMaxWaves];
    extern __shared__ float cols[];  // (G - 1) * D: the rows' partial sums on their way to row 0
    const uint32_t T = blockDim.x, t = threadIdx.x, G = blockDim.y, g = threadIdx.y;
    const uint32_t D = p.dim, b = blockIdx.y;
    const float sq = p.square_scale, inv_d = 1.0f / static_cast<float>(D), inv_sq = inv_d / sq;
    const double d64 = D, inv_d64 = 1.0 / d64;

    float fy[AFTER ? E : 1], fn[E];
    float p1[E] = {}, p2[E] = {}, p3[AFTER ? E : 1] = {};
    if constexpr (AFTER)
        load_params<F32, E, VEC>(fy, p.gate, static_cast<size_t>(b) * D, p.param_f32, p.chunks, 1.f, t, T, D);
    load_factor<F32, E, VEC>(fn, nullptr, p, nullptr, b, t, T);

    constexpr size_t es = F32 ? 4 : 2;
    const uint32_t step = gridDim.x * G;
    int phase = 0;
    for (uint32_t s0 = blockIdx.x * G; s0 < p.rows; s0 += step, phase ^= 1) {
        const uint32_t s = s0 + g;
        const bool live = s < p.rows;
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        float d[E], r[E], dn[E];
        RowPart<F32, E, VEC> raw_d, raw_y, raw_r, raw_n;
        auto get = [&](RowPart<F32, E, VEC>& to, const void* from) {
            if (live && from) to.load(static_cast<const char*>(from) + off, t, T, D);
            else to.clear();
        };
        get(raw_r, p.r);
        get(raw_n, p.dn);
        get(raw_d, p.dr);
        if constexpr (AFTER) get(raw_y, p.y);
        raw_r.unpack(r);
        raw_n.unpack(dn);
        subtract<F32, E, VEC>(r, row_mean(r, lds_sum[phase], d64, inv_d64, t, T, g), t, T, D);
        float ss[3] = {square_sum(r, sq), 0.f, 0.f};  // ..., v, v.(r - mean)
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float v = dn[k] * fn[k];
            ss[1] += v;
            ss[2] = fmaf(v, r[k], ss[2]);
        }
        row_sum(ss, lds[phase], t, T, g);
        const float rstd = rsqrtf(ss[0] * inv_sq + p.eps);
        const float mean_v = ss[1] * inv_d;
        const float proj = ss[2] * rstd * inv_d;  // mean(v * hat(r))
        raw_d.unpack(d);
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float hat = r[k] * rstd;
            p1[k] = fmaf(dn[k], hat, p1[k]);
            p2[k] += dn[k];
            d[k] = fmaf(rstd, fmaf(-hat, proj, fmaf(dn[k], fn[k], -mean_v)), d[k]);
        }
        if (live) store_row<F32, E, VEC>(static_cast<char*>(p.dresidual) + off, d, t, T, D);
        if constexpr (AFTER) {
            float y[E];
            raw_y.unpack(y);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                p3[k] = fmaf(d[k], y[k], p3[k]);
                d[k] *= fy[k];
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
    leave(p1, 0);
    leave(p2, 1);
    if constexpr (AFTER)
        if (p.dgate) leave(p3, 2);
}

// Sums over the partial rows and from them the gradients: blockIdx.z = 0 the norm's (P1 and P2), 1 the
// gate's (P3); kCols columns a workgroup, kLanes threads down the parts.  A workgroup goes through all
// samples, and adds up the weight's and the bias's gradients on the way, where they are few (gridDim.y
// = 1); else each has its own workgroup and leaves its part in partial row 0 for
// layer_norm_backward_weights.
__global__ __launch_bounds__(kCols* kLanes) void layer_norm_backward_join(LayerNormBackward p, uint32_t parts) {
    __shared__ float lds[kLanes][kCols + 1];
    const bool gate = blockIdx.z == 1;
    const uint32_t col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
    const uint32_t c = blockIdx.x * kCols + col;
    const bool all = gridDim.y == 1, pf = p.param_f32, mine = lane == 0 && c < p.dim;
    const size_t plane = static_cast<size_t>(p.batch) * parts * p.dim;
    const float w = mine && !gate && p.weight ? load_param(p.weight, pf, c) : 1.f;
    const float bias = mine && !gate && p.bias ? load_param(p.bias, pf, c) : 0.f;
    float dw = 0.f, dbias = 0.f;
    for (uint32_t b = blockIdx.y; b < (all ? p.batch : blockIdx.y + 1); ++b) {
        float* part = p.partial + static_cast<size_t>(b) * parts * p.dim + c;
        float s1 = 0.f, s2 = 0.f;
        if (c < p.dim) {
            if (gate) {
#pragma unroll 4
                for (uint32_t i = lane; i < parts; i += kLanes) s1 += part[2 * plane + static_cast<size_t>(i) * p.dim];
            } else {
#pragma unroll 4
                for (uint32_t i = lane; i < parts; i += kLanes) {
                    s1 += part[static_cast<size_t>(i) * p.dim];
                    s2 += part[plane + static_cast<size_t>(i) * p.dim];
                }
            }
        }
        s1 = lane_sum(s1, lds, col, lane);
        if (!gate) s2 = lane_sum(s2, lds, col, lane);
        if (!mine) continue;
        const size_t bc = static_cast<size_t>(b) * p.dim + c;
        if (gate) {
            store_param(p.dgate, pf, bc, s1);
            continue;
        }
        const float f = 1.f + (p.scale ? load_param(p.scale, pf, bc) : 0.f);
        if (p.dshift) store_param(p.dshift, pf, bc, s2);
        if (p.dscale) store_param(p.dscale, pf, bc, fmaf(w, s1, bias * s2));
        if (all) {
            dw = fmaf(f, s1, dw);
            dbias = fmaf(f, s2, dbias);
        } else {
            part[0] = f * s1;
            part[plane] = f * s2;
        }
    }
    if (!all || gate || !mine) return;
    if (p.dweight) store_param(p.dweight, pf, c, dw);
    if (p.dbias) store_param(p.dbias, pf, c, dbias);
}

// The weight's (blockIdx.z = 0) and the bias's (1) gradients: sums over the samples of what
// layer_norm_backward_join left.
__global__ __launch_bounds__(kCols* kLanes) void layer_norm_backward_weights(LayerNormBackward p, uint32_t parts) {
    __shared__ float lds[kLanes][kCols + 1];
    const uint32_t col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
    const uint32_t c = blockIdx.x * kCols + col;
    void* out = blockIdx.z == 0 ? p.dweight : p.dbias;
    if (out == nullptr) return;
    float s = 0.f;
    if (c < p.dim)
        for (uint32_t b = lane; b < p.batch; b += kLanes)
            s += p.partial[(static_cast<size_t>(blockIdx.z) * p.batch + b) * parts * p.dim + c];
    s = lane_sum(s, lds, col, lane);
    if (lane == 0 && c < p.dim) store_param(out, p.param_f32, c, s);
}

template <bool F32, int E>
hipError_t forward_of(const LayerNormForward& p, bool vec, dim3 grid, dim3 block, hipStream_t stream) {
    if (vec) {
        if (p.after) layer_norm_forward<F32, E, true, true><<<grid, block, 0, stream>>>(p);
        else layer_norm_forward<F32, E, true, false><<<grid, block, 0, stream>>>(p);
    } else {
        if (p.after) layer_norm_forward<F32, E, false, true><<<grid, block, 0, stream>>>(p);
        else layer_norm_forward<F32, E, false, false><<<grid, block, 0, stream>>>(p);
    }
    return hipGetLastError();
}

template <bool F32, int E>
hipError_t backward_of(const LayerNormBackward& p, bool vec, dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
    if (vec) {
        if (p.after) layer_norm_backward<F32, E, true, true><<<grid, block, lds, stream>>>(p);
        else layer_norm_backward<F32, E, true, false><<<grid, block, lds, stream>>>(p);
    } else {
        if (p.after) layer_norm_backward<F32, E, false, true><<<grid, block, lds, stream>>>(p);
        else layer_norm_backward<F32, E, false, false><<<grid, block, lds, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm_forward(const LayerNormForward& p, bool f32, bool vec, hipStream_t stream) {
    const Shape s = row_shape(p.batch, p.rows, p.dim);
    const dim3 block(s.T, s.G), grid(row_parts(p.batch, p.rows, s.G), p.batch);
    if (f32)
        return s.wide ? forward_of<true, 16>(p, vec, grid, block, stream) : forward_of<true, 8>(p, vec, grid, block, stream);
    return s.wide ? forward_of<false, 16>(p, vec, grid, block, stream) : forward_of<false, 8>(p, vec, grid, block, stream);
}

hipError_t launch_layer_norm_backward(const LayerNormBackward& p, bool f32, bool vec, hipStream_t stream) {
    if (p.batch == 0 || p.rows == 0) {  // no rows: every sum is zero
        const size_t D = p.dim, BD = size_t(p.batch) * p.dim;
        const std::pair<void*, size_t> sums[5] = {{p.dweight, D}, {p.dbias, D}, {p.dgate, BD}, {p.dscale, BD},
                                                  {p.dshift, BD}};
        for (const auto& v : sums)
            if (v.first != nullptr && v.second != 0) norm_zero<<<64, 256, 0, stream>>>(v.first, v.second, p.param_f32);
        return hipGetLastError();
    }
    const Shape s = row_shape(p.batch, p.rows, p.dim);
    const uint32_t parts = row_parts(p.batch, p.rows, s.G);
    const dim3 block(s.T, s.G), grid(parts, p.batch);
    const size_t lds = size_t(s.G - 1) * p.dim * sizeof(float);
    hipError_t e;
    if (f32)
        e = s.wide ? backward_of<true, 16>(p, vec, grid, block, lds, stream) : backward_of<true, 8>(p, vec, grid, block, lds, stream);
    else
        e = s.wide ? backward_of<false, 16>(p, vec, grid, block, lds, stream) : backward_of<false, 8>(p, vec, grid, block, lds, stream);
    if (e != hipSuccess || p.partial == nullptr) return e;
    const uint32_t cols = (p.dim + kCols - 1) / kCols;
    const bool few = p.batch <= 4;
    layer_norm_backward_join<<<dim3(cols, few ? 1 : p.batch, p.dgate ? 2 : 1), kCols * kLanes, 0, stream>>>(p, parts);
    e = hipGetLastError();
    if (e != hipSuccess || few || (!p.dweight && !p.dbias)) return e;
    layer_norm_backward_weights<<<dim3(cols, 1, 2), kCols * kLanes, 0, stream>>>(p, parts);
    return hipGetLastError();
}

}  // namespace ltx3drope
