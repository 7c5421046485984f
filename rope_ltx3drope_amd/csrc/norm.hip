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
//
// Above 8192 columns a row takes 16 elements a thread of 1024, which have 128 registers each: most backward
// kernels, and the forward ones off 16 bytes, then keep up to 93 values a thread in scratch memory.  12288
// columns in bf16, after a block: forward, 2 x 5780 rows, 194 us = 5.9 TB/s without scratch; backward,
// 2 x 2890 rows, 513 us = 1.7 TB/s with 248 bytes of it a thread.
#include <hip/hip_runtime.h>

#include <utility>

#include "block.h"
#include "rows.h"

namespace ltx3drope {
namespace {

template <bool F32, int E, bool VEC, bool HAS_Y, bool NEXT>
__global__ __launch_bounds__(1024) void norm_forward(NormForward p) {
    __shared__ float lds[2][2][kMaxWaves];
    const uint32_t T = blockDim.x, t = threadIdx.x, G = blockDim.y, g = threadIdx.y;
    const uint32_t D = p.dim, b = blockIdx.y;
    const float sq = p.square_scale, inv_sq = 1.0f / static_cast<float>(D) / sq;  // sq: a power of two

    constexpr size_t es = F32 ? 4 : 2;
    const uint32_t step = gridDim.x * G;
    RowPart<F32, E, VEC> yr, rr;
    auto load = [&](uint32_t s) {
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        if (s < p.rows) {
            if constexpr (HAS_Y) yr.load(static_cast<const char*>(p.y) + off, t, T, D);
            rr.load(static_cast<const char*>(p.residual) + off, t, T, D);
        } else {
            if constexpr (HAS_Y) yr.clear();
            rr.clear();
        }
    };
    load(blockIdx.x * G + g);
    // the factor on the branch, the factor and the shift of the next norm
    float fy[HAS_Y ? E : 1], fn[NEXT ? E : 1], sh[NEXT ? E : 1];
    if constexpr (HAS_Y) load_factor<F32, E, VEC>(fy, p, p.weight, p.gate, 0.f, b, t, T);
    if constexpr (NEXT) {
        load_factor<F32, E, VEC>(fn, p, p.next_weight, p.next_scale, 1.f, b, t, T);
        load_params<F32, E, VEC>(sh, p.next_shift, static_cast<size_t>(b) * D, p.param_f32, p.chunks, 0.f, t, T, D);
    }
    int phase = 0;
    for (uint32_t s0 = blockIdx.x * G; s0 < p.rows; s0 += step, phase ^= 1) {
        const uint32_t s = s0 + g;
        const bool live = s < p.rows;  // every thread keeps the barriers
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        float r[E], y[HAS_Y ? E : 1];
        rr.unpack(r);
        if constexpr (HAS_Y) yr.unpack(y);
        load(s + step);  // the next row travels while this one is summed
        if constexpr (HAS_Y) {
            float rstd = 1.f;
            if (p.post_norm) {
                float ss[1] = {square_sum(y, sq)};
                row_sum(ss, lds[phase][0], t, T, g);
                rstd = rsqrtf(fmaf(ss[0], inv_sq, p.eps));
            }
#pragma unroll
            for (int k = 0; k < E; ++k) r[k] = fmaf(y[k] * rstd, fy[k], p.residual_scale * r[k]);
            if (live) store_row<F32, E, VEC>(static_cast<char*>(p.r) + off, r, t, T, D);
        }
        if constexpr (NEXT) {
            float ss[1] = {square_sum(r, sq)};
            row_sum(ss, lds[phase][1], t, T, g);
            const float rstd = rsqrtf(fmaf(ss[0], inv_sq, p.eps));
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
    const float inv_d = 1.0f / static_cast<float>(D);
    const float sq = p.square_scale, inv_sq = inv_d / sq;  // sq: a power of two

    float fy[HAS_Y ? E : 1], fn[NEXT ? E : 1];
    float p1[NEXT ? E : 1] = {}, p2[NEXT ? E : 1] = {}, p3[HAS_Y ? E : 1] = {};
    if constexpr (HAS_Y) load_factor<F32, E, VEC>(fy, p, p.weight, p.gate, 0.f, b, t, T);
    if constexpr (NEXT) load_factor<F32, E, VEC>(fn, p, p.next_weight, p.next_scale, 1.f, b, t, T);

    constexpr size_t es = F32 ? 4 : 2;
    const uint32_t step = gridDim.x * G;
    int phase = 0;
    for (uint32_t s0 = blockIdx.x * G; s0 < p.rows; s0 += step, phase ^= 1) {
        const uint32_t s = s0 + g;
        const bool live = s < p.rows;
        const size_t off = (static_cast<size_t>(b) * p.rows + s) * D * es;
        float d[E], y[HAS_Y ? E : 1], r[NEXT ? E : 1], dn[NEXT ? E : 1];
        auto get = [&](auto& to, const void* from) {
            RowPart<F32, E, VEC> raw;
            if (live && from) raw.load(static_cast<const char*>(from) + off, t, T, D);
            else raw.clear();
            raw.unpack(to);
        };
        get(d, p.dr);
        if constexpr (HAS_Y) get(y, p.y);
        if constexpr (NEXT) {
            get(r, p.r);
            get(dn, p.dn);
        }
        float rstd_y = 1.f;
        if constexpr (NEXT) {
            float ss[3] = {square_sum(r, sq), 0.f, 0.f};  // r.r sq, (dn fn).r, y.y sq
            if constexpr (HAS_Y) ss[2] = square_sum(y, sq);
#pragma unroll
            for (int k = 0; k < E; ++k) ss[1] = fmaf(dn[k] * fn[k], r[k], ss[1]);
            row_sum(ss, lds[phase][0], t, T, g);
            const float rstd = rsqrtf(fmaf(ss[0], inv_sq, p.eps));
            const float proj = ss[1] * rstd * inv_d;  // mean(v * hat(r))
            if constexpr (HAS_Y)
                if (p.post_norm) rstd_y = rsqrtf(fmaf(ss[2], inv_sq, p.eps));
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float hat = r[k] * rstd;
                p1[k] = fmaf(dn[k], hat, p1[k]);
                p2[k] += dn[k];
                d[k] = fmaf(rstd, fmaf(-hat, proj, dn[k] * fn[k]), d[k]);
            }
        } else if constexpr (HAS_Y) {
            if (p.post_norm) {
                float ss[1] = {square_sum(y, sq)};
                row_sum(ss, lds[phase][0], t, T, g);
                rstd_y = rsqrtf(fmaf(ss[0], inv_sq, p.eps));
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

// Sums over the partial rows, one of the three sums (blockIdx.z) and kCols columns a workgroup, kLanes
// threads down the parts, and from them the gradients.  A workgroup goes through all samples, and adds up
// the weight's gradient on the way, where they are few (gridDim.y = 1); else each has its own workgroup
// and leaves its part in partial row 0 for norm_backward_weights.
__global__ __launch_bounds__(kCols* kLanes) void norm_backward_join(NormBackward p, uint32_t parts) {
    __shared__ float lds[kLanes][kCols + 1];
    const uint32_t which = blockIdx.z;
    if (!(which == 2 ? p.has_y : p.next_norm)) return;
    const uint32_t col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
    const uint32_t c = blockIdx.x * kCols + col;
    const bool all = gridDim.y == 1, pf = p.param_f32;
    const void* weight = which == 2 ? p.weight : p.next_weight;
    const void* factor = which == 2 ? p.gate : p.next_scale;
    void* dfactor = which == 2 ? p.dgate : p.dnext_scale;
    void* dweight = which == 2 ? p.dweight : p.dnext_weight;
    float total = 0.f;
    for (uint32_t b = blockIdx.y; b < (all ? p.batch : blockIdx.y + 1); ++b) {
        float* part = p.partial + (static_cast<size_t>(which) * p.batch + b) * parts * p.dim + c;
        float s = 0.f;
        if (c < p.dim) {
#pragma unroll 4
            for (uint32_t i = lane; i < parts; i += kLanes) s += part[static_cast<size_t>(i) * p.dim];
        }
        s = lane_sum(s, lds, col, lane);
        if (lane != 0 || c >= p.dim) continue;
        const size_t bc = static_cast<size_t>(b) * p.dim + c;
        if (which == 1) {
            if (p.dnext_shift) store_param(p.dnext_shift, pf, bc, s);
            continue;
        }
        const float w = weight ? load_param(weight, pf, c) + p.weight_offset : 1.f;
        const float f = (which == 2 ? 0.f : 1.f) + (factor ? load_param(factor, pf, bc) : (which == 2 ? 1.f : 0.f));
        if (dfactor) store_param(dfactor, pf, bc, w * s);
        if (all) total = fmaf(f, s, total);
        else part[0] = f * s;
    }
    if (all && which != 1 && dweight && lane == 0 && c < p.dim) store_param(dweight, pf, c, total);
}

// The weights' gradients: sums over the samples of what norm_backward_join left.
__global__ __launch_bounds__(kCols* kLanes) void norm_backward_weights(NormBackward p, uint32_t parts) {
    __shared__ float lds[kLanes][kCols + 1];
    const uint32_t col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
    const uint32_t c = blockIdx.x * kCols + col, which = blockIdx.z * 2;
    void* out = which == 0 ? p.dnext_weight : p.dweight;
    if (out == nullptr) return;
    float s = 0.f;
    if (c < p.dim)
        for (uint32_t b = lane; b < p.batch; b += kLanes)
            s += p.partial[(static_cast<size_t>(which) * p.batch + b) * parts * p.dim + c];
    s = lane_sum(s, lds, col, lane);
    if (lane == 0 && c < p.dim) store_param(out, p.param_f32, c, s);
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

}  // namespace

hipError_t launch_norm_forward(const NormForward& p, bool f32, bool vec, hipStream_t stream) {
    const Shape s = row_shape(p.batch, p.rows, p.dim);
    const dim3 block(s.T, s.G), grid(row_parts(p.batch, p.rows, s.G), p.batch);
    if (f32) {
        if (s.wide) return vec ? forward_modes<true, 16, true>(p, grid, block, stream) : forward_modes<true, 16, false>(p, grid, block, stream);
        return vec ? forward_modes<true, 8, true>(p, grid, block, stream) : forward_modes<true, 8, false>(p, grid, block, stream);
    }
    if (s.wide) return vec ? forward_modes<false, 16, true>(p, grid, block, stream) : forward_modes<false, 16, false>(p, grid, block, stream);
    return vec ? forward_modes<false, 8, true>(p, grid, block, stream) : forward_modes<false, 8, false>(p, grid, block, stream);
}

size_t norm_backward_workspace(uint32_t batch, uint32_t rows, uint32_t dim) {
    return size_t(3) * batch * row_parts(batch, rows, row_shape(batch, rows, dim).G) * dim * sizeof(float);
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
    const Shape s = row_shape(p.batch, p.rows, p.dim);
    const uint32_t parts = row_parts(p.batch, p.rows, s.G);
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
    const bool few = p.batch <= 4;
    norm_backward_join<<<dim3(cols, few ? 1 : p.batch, 3), kCols * kLanes, 0, stream>>>(p, parts);
    e = hipGetLastError();
    if (e != hipSuccess || few || (!p.dnext_weight && !p.dweight)) return e;
    norm_backward_weights<<<dim3(cols, 1, 2), kCols * kLanes, 0, stream>>>(p, parts);
    return hipGetLastError();
}

}  // namespace ltx3drope
