// A linear layer in 8-bit floating point (e4m3) with a scale for each block of 128 numbers: the quantisers and
// the product.
//
//     scale = max |x| / 448 over a block,  q = e4m3(x / scale)                  (fp32, each step rounded once)
//     y_mn  = sum_kb a_scale[m][kb] b_scale[n][kb] (sum_{k in kb} a_mk b_nk) + bias_n
// A block is 128 of a row (activations, gradients), or 128 x 128 (weights: then b_scale has one row for 128
// rows of b).  A block of zeros has scale 0 and zeros; one whose largest magnitude is not finite keeps that
// as its scale and gets zeros, so that its products are NaN.
#include <hip/hip_runtime.h>

#include "block.h"
#include "product.h"

namespace ltx3drope {
namespace {

// ---- the quantisers --------------------------------------------------------------------------------

constexpr float kTop = 448.f;  // the largest e4m3 number
constexpr uint32_t kBlock = 128;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// A block's scale and its rounded reciprocal, for the quotients.
struct Divisor {
    float s, r;
    bool usual;
    __device__ __forceinline__ explicit Divisor(uint32_t top) {
        s = __uint_as_float(top) / kTop;
        // subnormal numbers on the way cost the remainder below its exactness
        usual = s > 0x1p-80f && s < 0x1p100f;
        r = 1.0f / s;
    }
    // x / s rounded to fp32, within e4m3's range.  Usually x * r is within an ulp of the quotient, and one step
    // with the exact remainder gives the rounded quotient (Markstein's division by a rounded reciprocal); its
    // size is at most 448 (1 + 2^-24), which rounds to 448.  That step loses the sign of -0.
    __device__ __forceinline__ float quotient(float x) const {
        if (usual) {
            const float q0 = x * r;
            return __builtin_copysignf(fmaf(fmaf(-q0, s, x), r, q0), x);
        }
        const bool plain = s > 0.f && s < __builtin_inff();
        return plain ? fminf(fmaxf(x / s, -kTop), kTop) : 0.f;
    }
    // four numbers as e4m3, rounded to nearest even
    __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) const {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(a), quotient(b), 0, false);
        return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(quotient(c), quotient(d), v, true));
    }
};

// 8 numbers of a row from column c on, zeros from `end` on.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(float (&f)[8], const char* row, uint32_t c, uint32_t end) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
        if (c >= end) return;  // rows are whole vectors of 8
        if constexpr (F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + c * 4u + h * 16));
#pragma unroll
                for (int k = 0; k < 4; ++k) f[4 * h + k] = __uint_as_float(v[k]);
            }
        } else {
            const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + c * 2u));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[2 * k] = __uint_as_float(v[k] << 16);
                f[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            f[i] = 0.f;
            if (c + i < end) {
                if constexpr (F32) f[i] = reinterpret_cast<const float*>(row)[c + i];
                else f[i] = static_cast<float>(reinterpret_cast<const __bf16*>(row)[c + i]);
            }
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* row, uint32_t c, uint32_t end, uint32_t lo, uint32_t hi) {
    if constexpr (VEC) {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        if (c < end) *reinterpret_cast<u32x2*>(row + c) = u32x2{lo, hi};
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (c + i < end) row[c + i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i % 4)));
    }
}

// The largest over 16 neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    auto lanes = [](uint32_t x, auto ctrl) {
        return static_cast<uint32_t>(
            __builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    v = larger(v, lanes(v, std::integral_constant<int, 0xb1>{}));   // quad_perm 1 0 3 2
    v = larger(v, lanes(v, std::integral_constant<int, 0x4e>{}));   // quad_perm 2 3 0 1
    v = larger(v, lanes(v, std::integral_constant<int, 0x141>{}));  // row_half_mirror
    return larger(v, lanes(v, std::integral_constant<int, 0x140>{}));  // row_mirror
}

// Rows alone: 16 lanes a block, 8 numbers a lane; a number is read once and its byte written once.
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void f8_rows_of(const char* x, uint8_t* q, float* scale, uint64_t blocks,
                                                  uint32_t per_row, uint32_t dim) {
    const uint32_t lane = threadIdx.x & 15;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 16 + threadIdx.x / 16; i < blocks;
         i += static_cast<uint64_t>(gridDim.x) * 16) {
        const uint64_t r = i / per_row;
        const uint32_t c = static_cast<uint32_t>(i - r * per_row) * kBlock + lane * 8;
        float f[8];
        load8<F32, VEC>(f, x + r * dim * (F32 ? 4 : 2), c, dim);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = larger(top, magnitude(f[k]));
        const Divisor d(max16(top));
        store8<VEC>(q + r * dim, c, dim, d.four(f[0], f[1], f[2], f[3]), d.four(f[4], f[5], f[6], f[7]));
        if (lane == 0) scale[i] = d.s;
    }
}

// Tiles of 128 x 128: a workgroup of 256 threads holds one in registers, 8 columns and every 16th row a thread.
// BLOCKS: one scale for the tile; otherwise one a row and, turned, one a column.  TURNED: also x^T, whose
// bytes cross LDS (a column's 128 are one line of the turned matrix).
template <bool F32, bool VEC, bool BLOCKS, bool TURNED>
__global__ __launch_bounds__(256) void f8_tiles_of(F8Quantize p) {
    constexpr uint32_t kPitch = kBlock + 16;  // 16-byte pieces of neighbouring columns in different banks
    __shared__ uint32_t tops[4][kBlock];
    __shared__ __align__(16) uint8_t turned[TURNED ? kBlock * kPitch : 16];
    const uint32_t tid = threadIdx.x, lane = tid & 15, line = tid / 16, wave = tid / 64;
    const uint32_t tiles_c = (p.dim + kBlock - 1) / kBlock, tiles_r = (p.rows + kBlock - 1) / kBlock;
    const uint32_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;
    const uint32_t r0 = tr * kBlock, c = tc * kBlock + lane * 8;
    const char* x = static_cast<const char*>(p.x);
    uint8_t* q = static_cast<uint8_t*>(p.q);
    float f[8][8];
    uint32_t row_top[8], col_top[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = r0 + i * 16 + line;
        if (r < p.rows) {
            load8<F32, VEC>(f[i], x + static_cast<size_t>(r) * p.dim * (F32 ? 4 : 2), c, p.dim);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        row_top[i] = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t m = magnitude(f[i][k]);
            row_top[i] = larger(row_top[i], m);
            col_top[k] = larger(col_top[k], m);
        }
    }
    if constexpr (BLOCKS || TURNED) {
        // columns over the four lines of a wavefront, then over the wavefronts
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            col_top[k] = larger(col_top[k], __shfl_xor(col_top[k], 16));
            col_top[k] = larger(col_top[k], __shfl_xor(col_top[k], 32));
            if ((tid & 63) < 16) tops[wave][lane * 8 + k] = col_top[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w) col_top[k] = larger(col_top[k], tops[w][lane * 8 + k]);
    }
    uint32_t block_top = 0;
    if constexpr (BLOCKS) {
#pragma unroll
        for (int k = 0; k < 8; ++k) block_top = larger(block_top, col_top[k]);
        block_top = max16(block_top);
    }
    const Divisor whole(block_top);
    if (BLOCKS && tid == 0) {
        p.scale[static_cast<size_t>(tr) * tiles_c + tc] = whole.s;
        if (TURNED) p.scale_turned[static_cast<size_t>(tc) * tiles_r + tr] = whole.s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = r0 + i * 16 + line;
        const Divisor d(BLOCKS ? block_top : max16(row_top[i]));
        if (r < p.rows) {
            store8<VEC>(q + static_cast<size_t>(r) * p.dim, c, p.dim, d.four(f[i][0], f[i][1], f[i][2], f[i][3]),
                        d.four(f[i][4], f[i][5], f[i][6], f[i][7]));
            if (!BLOCKS && lane == 0) p.scale[static_cast<size_t>(r) * tiles_c + tc] = d.s;
        }
    }
    if constexpr (TURNED) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const Divisor d(BLOCKS ? block_top : col_top[k]);
            const uint32_t lo = d.four(f[0][k], f[1][k], f[2][k], f[3][k]);
            const uint32_t hi = d.four(f[4][k], f[5][k], f[6][k], f[7][k]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                turned[(lane * 8 + k) * kPitch + i * 16 + line] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i % 4)));
            if (!BLOCKS && line == 0 && c + k < p.dim) p.scale_turned[static_cast<size_t>(c + k) * tiles_r + tr] = d.s;
        }
        __syncthreads();
        // 8 threads a column, 16 rows each
        uint8_t* out = static_cast<uint8_t*>(p.q_turned);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t col = i * 32 + tid / 8, row = (tid % 8) * 16, cc = tc * kBlock + col;
            if (cc >= p.dim || r0 + row >= p.rows) continue;
            const u32x4 v = *reinterpret_cast<const u32x4*>(turned + col * kPitch + row);
            uint8_t* to = out + cc * p.turned_pitch + r0 + row;
            if (p.turned_chunks) {
                *reinterpret_cast<u32x4*>(to) = v;  // the pitch has room for whole pieces
            } else {
                for (uint32_t j = 0; j < 16; ++j)
                    if (r0 + row + j < p.rows) to[j] = static_cast<uint8_t>(v[j / 4] >> (8 * (j % 4)));
            }
        }
    }
}

// ---- the product -----------------------------------------------------------------------------------

struct OpF8 {
    using Acc = f32x4;
    using Sum = float;
    static constexpr int kElem = 1;
};

// The scales of one product: a's [M][blocks], b's [N][blocks] or one row for 128 rows of b.
struct F8Scales {
    const float *a, *b;
    uint32_t blocks;
};

// One block of k of 16 rows as the matrix cores take it, and the sums of such blocks of 16 rows of B by 16 of A.
// Lane l holds, of row l % 16, the 16-byte pieces l / 16 of both halves of the block.
//
// Eight: the 8-bit instruction, 16 x 16 x 128 in 32 cycles, twice bf16's rate.  It adds the products of each 8
// neighbours of k with what 2^-13 of the largest of them (by its exponents) leaves, and these sums in fp32
// (measured: beside 448 * 448 a product of 2^2 among the same 8 is lost, one of 2^-6 elsewhere is not).  Next to
// a result in bf16 that is little: on normal data it comes to 3e-5 of the result, and bf16's own rounding
// to 1.7e-3.  A result in fp32 is not made so:
// Sixteen: e4m3 is exact in bf16, whose instructions have exact products and fp32 sums.
struct Eight {
    u32x4 v[2];
    __device__ __forceinline__ explicit Eight(const u32x4 (&pieces)[2]) : v{pieces[0], pieces[1]} {}
    __device__ __forceinline__ static f32x4 product(const Eight& b, const Eight& a) {
        typedef int i32x8 __attribute__((ext_vector_type(8)));
        auto all = [](const Eight& x) {
            return i32x8{static_cast<int>(x.v[0][0]), static_cast<int>(x.v[0][1]), static_cast<int>(x.v[0][2]),
                         static_cast<int>(x.v[0][3]), static_cast<int>(x.v[1][0]), static_cast<int>(x.v[1][1]),
                         static_cast<int>(x.v[1][2]), static_cast<int>(x.v[1][3])};
        };
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(all(b), all(a), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0,
                                                                0, 0);
    }
};
struct Sixteen {
    u32x4 v[4];
    __device__ __forceinline__ explicit Sixteen(const u32x4 (&pieces)[2]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = pieces[i / 4][i % 4];
            v[i / 2][i % 2 * 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
            v[i / 2][i % 2 * 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true));
        }
    }
    __device__ __forceinline__ static f32x4 product(const Sixteen& b, const Sixteen& a) {
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) OpBf16::mac(c, b.v[i], a.v[i]);
        return c;
    }
};

// Four bytes a lane from the buffer to LDS, lane l's to lds + 4 * l; as lds_copy16.
__device__ __forceinline__ void lds_copy4(u32x4 buffer, char* lds, uint32_t voffset, uint32_t soffset) {
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(at), "v"(voffset),
                 "s"(buffer), "s"(soffset));
}

// BM x BN tiles, WM x WN wavefronts; a step is one block of k, whose operands and scales come to LDS together.
// B_ROWS: b has a scale a row.  DIRECT: operands whose rows start on 16 bytes are copied without passing
// through registers.
template <class Units, int BM, int BN, int WM, int WN, int RING, bool B_ROWS, bool DIRECT, class Done>
__global__ __launch_bounds__(WM* WN * 64) void f8_tiles(Product p, F8Scales scales, Done done) {
    constexpr int NW = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    using SA = Side<OpF8, BM, false>;
    using SB = Side<OpF8, BN, false>;
    constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;       // 1 KB copies a wavefront makes of each operand
    constexpr uint32_t RA = BM / NW, RB = BN / NW;          // rows whose scales a wavefront copies
    constexpr int kAtB = BM * kRowBytes, kAtScales = kAtB + BN * kRowBytes;
    constexpr int kSlot = kAtScales + (B_ROWS ? 2 : 1) * NW * 256;
    static_assert(CA * 8 * NW == BM && CB * 8 * NW == BN && RA <= 64 && RB <= 64, "copies split evenly");
    static_assert(FN * 16 <= 128, "a wavefront's rows of b lie in one block of 128");
    __shared__ __align__(1024) char lds[RING * kSlot];

    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave / WN, wn = wave % WN;
    const uint32_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN, tiles = tiles_m * tiles_n;
    const uint32_t tile = blockIdx.x % tiles, split = blockIdx.x / tiles;
    uint32_t tm, tn;
    tile_of(tile, tiles_m, tiles_n, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BN;
    const uint32_t all_steps = scales.blocks;
    const uint32_t first = split * all_steps / p.splits, last = (split + 1) * all_steps / p.splits;

    uint32_t line_a[CA], byte_a[CA], line_b[CB], byte_b[CB];
#pragma unroll
    for (int i = 0; i < CA; ++i) SA::place((i * NW + wave) * 64 + lane, line_a[i], byte_a[i]);
#pragma unroll
    for (int i = 0; i < CB; ++i) SB::place((i * NW + wave) * 64 + lane, line_b[i], byte_b[i]);
    // scales of rows past the end are those of the last row (their sums are dropped)
    const uint32_t scale_m = m0 + wave * RA + lane % RA, scale_n = n0 + wave * RB + lane % RB;
    const float* sa = scales.a + static_cast<size_t>(scale_m < p.M ? scale_m : p.M - 1) * scales.blocks;
    const float* sb = scales.b + static_cast<size_t>(scale_n < p.N ? scale_n : p.N - 1) * (B_ROWS ? scales.blocks : 0);

    u32x4 ra, rb, rsa, rsb;
    uint32_t va[CA], vb[CB], vsa = 0, vsb = 0;
    if constexpr (DIRECT) {
        // whole dwords: the up to three bytes past a row's end are cleared with the rest of its piece
        auto rsrc = [&](const char* base, uint64_t pitch, uint32_t row0, uint32_t rows, uint32_t R) {
            return buffer_of(base + row0 * pitch, pitch, rows - row0 < R ? rows - row0 : R, (p.k + 3) & ~3u);
        };
        auto scale_rsrc = [&](const float* base, uint32_t row0, uint32_t rows, uint32_t R) {
            return buffer_of(reinterpret_cast<const char*>(base + static_cast<size_t>(row0) * scales.blocks),
                             scales.blocks * 4u, rows - row0 < R ? rows - row0 : R, scales.blocks * 4);
        };
        ra = rsrc(p.a, p.a_pitch, m0, p.M, BM);
        rb = rsrc(p.b[0], p.b_pitch, n0, p.N, BN);
        rsa = scale_rsrc(scales.a, m0, p.M, BM);
        vsa = (wave * RA + lane % RA) * scales.blocks * 4;
        if constexpr (B_ROWS) {
            rsb = scale_rsrc(scales.b, n0, p.N, BN);
            vsb = (wave * RB + lane % RB) * scales.blocks * 4;
        }
#pragma unroll
        for (int i = 0; i < CA; ++i)
            va[i] = m0 + line_a[i] < p.M ? static_cast<uint32_t>(line_a[i] * p.a_pitch) + byte_a[i] : kOutOfRange;
#pragma unroll
        for (int i = 0; i < CB; ++i)
            vb[i] = n0 + line_b[i] < p.N ? static_cast<uint32_t>(line_b[i] * p.b_pitch) + byte_b[i] : kOutOfRange;
    }
    // a step past this workgroup's last one brings zeros without touching memory
    const uint32_t k_end = last * kRowBytes < p.k ? last * kRowBytes : p.k;
    constexpr int kCopies = CA + CB + 1 + B_ROWS;
    auto copy = [&](uint32_t step, uint32_t slot) {
        char* to = lds + slot * kSlot + wave * 1024;
        const uint32_t k = step * kRowBytes;
#pragma unroll
        for (int i = 0; i < CA; ++i) lds_copy16(ra, to + i * NW * 1024, k + byte_a[i] >= k_end ? kOutOfRange : va[i], k);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            lds_copy16(rb, to + kAtB + i * NW * 1024, k + byte_b[i] >= k_end ? kOutOfRange : vb[i], k);
        char* s = lds + slot * kSlot + kAtScales + wave * 256;
        lds_copy4(rsa, s, step < last ? vsa : kOutOfRange, step * 4);
        if constexpr (B_ROWS) lds_copy4(rsb, s + NW * 256, step < last ? vsb : kOutOfRange, step * 4);
    };
    struct Held {
        u32x4 v[DIRECT ? 1 : CA + CB];
        float sa, sb;
    };
    auto hold = [&](Held& to, uint32_t step) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < CA; ++i) {
                const uint32_t m = m0 + line_a[i] < p.M ? m0 + line_a[i] : p.M - 1;
                to.v[i] = load_chunk<OpF8, false, false>(p.a + m * p.a_pitch, step * kRowBytes + byte_a[i], p.k);
            }
#pragma unroll
            for (int i = 0; i < CB; ++i) {
                const uint32_t n = n0 + line_b[i] < p.N ? n0 + line_b[i] : p.N - 1;
                to.v[CA + i] = load_chunk<OpF8, false, false>(p.b[0] + n * p.b_pitch, step * kRowBytes + byte_b[i], p.k);
            }
            to.sa = sa[step];
            if constexpr (B_ROWS) to.sb = sb[step];
        }
    };
    auto put_held = [&](const Held& from, uint32_t slot) {
        if constexpr (!DIRECT) {
            char* at = lds + slot * kSlot + wave * 1024 + lane * 16;
#pragma unroll
            for (int i = 0; i < CA; ++i) *reinterpret_cast<u32x4*>(at + i * NW * 1024) = from.v[i];
#pragma unroll
            for (int i = 0; i < CB; ++i) *reinterpret_cast<u32x4*>(at + kAtB + i * NW * 1024) = from.v[CA + i];
            float* s = reinterpret_cast<float*>(lds + slot * kSlot + kAtScales + wave * 256) + lane;
            s[0] = from.sa;
            if constexpr (B_ROWS) s[NW * 64] = from.sb;
        }
    };
    // Copies bring whole 16-byte pieces: what a row's last piece holds past k is cleared, a row a thread.
    auto clear_tail = [&](uint32_t slot) {
        const uint32_t rem = (p.k & (kRowBytes - 1)), piece = rem / 16;
        for (uint32_t r = tid; r < BM + BN; r += NW * 64) {
            const uint32_t line = r < BM ? r : r - BM;
            char* at = lds + slot * kSlot + (r < BM ? 0 : kAtB) + line * kRowBytes + ((piece ^ SA::swizzle(line)) << 4);
            u32x4 v = *reinterpret_cast<u32x4*>(at);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t keep = rem % 16 > 4u * w ? rem % 16 - 4u * w : 0u;  // bytes of this word
                if (keep < 4) v[w] &= (1u << (8 * keep)) - 1;
            }
            *reinterpret_cast<u32x4*>(at) = v;
        }
        wait_for_lds_and_meet();
    };

    f32x4 acc[FM][FN] = {};
    // the scale of b's block of 128 rows: lane l holds that of step `from` + l
    const uint32_t strip = (n0 + wn * FN * 16) / 128;
    const float* sb_strip = scales.b + static_cast<size_t>(strip) * scales.blocks;
    float sb_lanes = 0.f;
    const uint32_t rows_b = (p.N + 127) / 128;
    auto multiply = [&](uint32_t step, uint32_t slot) {
        float sbw = 1.f;
        if constexpr (!B_ROWS) {
            const uint32_t i = (step - first) & 63;
            if (i == 0) sb_lanes = strip < rows_b && step + lane < last ? sb_strip[step + lane] : 0.f;
            sbw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sb_lanes), static_cast<int>(i)));
        }
        const char* at = lds + slot * kSlot;
        const float* s = reinterpret_cast<const float*>(at + kAtScales);
        auto read = [&](const char* block) {
            u32x4 v[2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) v[kk] = *reinterpret_cast<const u32x4*>(block + SB::lane_base(lane, kk));
            return Units(v);
        };
        f32x4 sbn[B_ROWS ? FN : 1];
        auto b_block = [&](int j) { return read(at + kAtB + (wn * FN + j) * 16 * kRowBytes); };
        const Units fb[4] = {b_block(0), b_block(1 % FN), b_block(2 % FN), b_block(3 % FN)};
        static_assert(FN <= 4, "a wavefront holds up to 64 rows of b");
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (B_ROWS) {
                const uint32_t r = (wn * FN + j) * 16 + (lane >> 4) * 4;
                sbn[j] = *reinterpret_cast<const f32x4*>(s + NW * 64 + r / RB * 64 + r % RB);
            }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const uint32_t row = (wm * FM + i) * 16;
            const Units fa = read(at + row * kRowBytes);
            const uint32_t r = row + (lane & 15);
            const float sm = s[r / RA * 64 + r % RA] * sbw;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const f32x4 part = Units::product(fb[j], fa);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = B_ROWS ? sm * sbn[B_ROWS ? j : 0][e] : sm;
                    acc[i][j][e] = fmaf(part[e], f, acc[i][j][e]);
                }
            }
        }
    };
    const bool tail = DIRECT && p.k % 16 != 0 && last == all_steps;

    if constexpr (DIRECT) {
        for (int i = 0; i < RING - 1; ++i) copy(first + i, i);
        uint32_t slot = 0, free = RING - 1;
        for (uint32_t s = first; s < last; ++s) {
            wait_and_meet<(RING - 2) * kCopies>();
            copy(s + RING - 1, free);
            free = slot;
            if (tail && s + 1 == last) clear_tail(slot);
            multiply(s, slot);
            slot = slot + 1 == RING ? 0 : slot + 1;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives its workgroup
    } else {
        Held even, odd;
        auto turn = [&](uint32_t s, Held& next, Held& after) {
            const uint32_t slot = (s - first) & 1;
            wait_for_lds_and_meet();
            if (s + 2 < last) hold(after, s + 2);
            multiply(s, slot);
            if (s + 1 < last) put_held(next, slot ^ 1);
        };
        hold(even, first);
        if (first + 1 < last) hold(odd, first + 1);
        put_held(even, 0);
        for (uint32_t s = first; s < last; s += 2) {
            turn(s, odd, even);
            if (s + 1 < last) turn(s + 1, even, odd);
        }
    }

    if (p.splits > 1) {
        f32x4* out = reinterpret_cast<f32x4*>(p.partial) +
                     (static_cast<size_t>(split) * tiles + tile) * (FM * FN * NW * 64) + tid;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) out[(i * FN + j) * NW * 64] = acc[i][j];
        return;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t m = m0 + (wm * FM + i) * 16 + (lane & 15);
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t n = n0 + (wn * FN + j) * 16 + (lane >> 4) * 4;
            if (n < p.N) done(m, n, p.N, acc[i][j]);
        }
    }
}

// Up to 16 rows of A: B is read once, straight into registers, 16 of its rows a workgroup, and the wavefronts
// of a workgroup take blocks of k in turn.  Their sums meet in LDS.  Bound by the bytes of B, beside which the
// bf16 units cost nothing.
template <bool B_ROWS, bool ALIGNED, class Done>
__global__ __launch_bounds__(512) void f8_few(Product p, F8Scales scales, Done done) {
    constexpr uint32_t NW = 8, U = 2;  // U blocks in flight
    __shared__ f32x4 lds[NW][64];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 16, r = lane & 15, piece = (lane >> 4) * 16;
    const uint32_t n = n0 + r < p.N ? n0 + r : p.N - 1;  // rows past the end repeat the last one
    const uint32_t m = r < p.M ? r : p.M - 1;
    const char *rb = p.b[0] + n * p.b_pitch, *ra = p.a + m * p.a_pitch;
    const float* sa = scales.a + static_cast<size_t>(m) * scales.blocks;
    const uint32_t nn = n0 + (lane >> 4) * 4;
    const float* sb[B_ROWS ? 4 : 1];
#pragma unroll
    for (uint32_t e = 0; e < (B_ROWS ? 4 : 1); ++e) {
        const uint32_t c = nn + e < p.N ? nn + e : p.N - 1;
        sb[e] = scales.b + static_cast<size_t>(B_ROWS ? c : n0 / 128) * scales.blocks;
    }
    f32x4 acc = {};
    for (uint32_t kb0 = wave; kb0 < scales.blocks; kb0 += NW * U) {
        u32x4 b[U][2], a[U][2];
        float s[U][B_ROWS ? 4 : 1];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t kb = kb0 + u * NW, k = kb * kBlock + piece;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b[u][h] = load_chunk<OpF8, ALIGNED, false>(rb, k + h * 64, p.k);
                a[u][h] = load_chunk<OpF8, ALIGNED, false>(ra, k + h * 64, p.k);
            }
            const uint32_t at = kb < scales.blocks ? kb : scales.blocks - 1;
#pragma unroll
            for (uint32_t e = 0; e < (B_ROWS ? 4 : 1); ++e) s[u][e] = kb < scales.blocks ? sa[at] * sb[e][at] : 0.f;
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (kb0 + u * NW >= scales.blocks) break;
            const f32x4 part = Sixteen::product(Sixteen(b[u]), Sixteen(a[u]));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(part[e], s[u][B_ROWS ? e : 0], acc[e]);
        }
    }
    lds[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    f32x4 sum = {};
    for (uint32_t w = 0; w < NW; ++w) sum += lds[w][lane];
    if (r < p.M && nn < p.N) done(r, nn, p.N, sum);
}

struct BiasDone {
    bool f32;
    void* y;
    const float* bias;
    __device__ __forceinline__ void operator()(uint32_t m, uint32_t n, uint32_t N, f32x4 v) const {
        if (bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += bias[n + i < N ? n + i : N - 1];
        }
        if (f32) store4<true>(static_cast<float*>(y) + static_cast<size_t>(m) * N, n, N, v);
        else store4<false>(static_cast<uint16_t*>(y) + static_cast<size_t>(m) * N, n, N, v);
    }
};

// Whether rows start on 16 bytes (their ends are cleared, or not loaded).
bool pieces16(const void* p, uint64_t pitch) { return ((reinterpret_cast<uintptr_t>(p) | pitch) & 15) == 0; }
bool direct(const F8Problem& p) { return pieces16(p.a, p.a_pitch) && pieces16(p.b, p.b_pitch); }

template <class Units, int BM, int BN, int WM, int WN, int RING, bool B_ROWS, bool DIRECT>
hipError_t launch_f8_tiles(const Product& p, const F8Scales& s, const Plan& plan, const BiasDone& done, hipStream_t stream) {
    constexpr int threads = WM * WN * 64;
    f8_tiles<Units, BM, BN, WM, WN, RING, B_ROWS, DIRECT><<<plan.tiles * p.splits, threads, 0, stream>>>(p, s, done);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    product_join<OpF8, BM, BN, WM, WN, false><<<plan.tiles * (BM / WM / 16), threads, 0, stream>>>(p, done);
    return hipGetLastError();
}

template <bool B_ROWS>
hipError_t launch_f8_few(const F8Problem& f, const Product& p, const F8Scales& s, const BiasDone& done, hipStream_t stream) {
    const uint32_t groups = (p.N + 15) / 16;
    if (direct(f) && p.k % 16 == 0) f8_few<B_ROWS, true><<<groups, 512, 0, stream>>>(p, s, done);
    else f8_few<B_ROWS, false><<<groups, 512, 0, stream>>>(p, s, done);
    return hipGetLastError();
}

template <class Units, bool B_ROWS>
hipError_t launch_f8_of(const F8Problem& f, Product p, const F8Scales& s, const BiasDone& done, hipStream_t stream) {
    const Plan plan = plan_product<OpF8, false, false>(p.M, p.N, p.k, direct(f), p.b_pitch);
    p.splits = plan.splits;
    p.partial = static_cast<float*>(f.workspace);
    if (plan.bn == 256) return launch_f8_tiles<Units, 256, 256, 2, 4, 2, B_ROWS, true>(p, s, plan, done, stream);
    if (plan.bn == 128) return launch_f8_tiles<Units, 256, 128, 4, 2, 2, B_ROWS, true>(p, s, plan, done, stream);
    if (plan.bm == 128)
        return direct(f) ? launch_f8_tiles<Units, 128, 64, 2, 2, 2, B_ROWS, true>(p, s, plan, done, stream)
                         : launch_f8_tiles<Units, 128, 64, 2, 2, 2, B_ROWS, false>(p, s, plan, done, stream);
    return direct(f) ? launch_f8_tiles<Units, 64, 64, 2, 2, 3, B_ROWS, true>(p, s, plan, done, stream)
                     : launch_f8_tiles<Units, 64, 64, 2, 2, 2, B_ROWS, false>(p, s, plan, done, stream);
}

}  // namespace

size_t f8_workspace(const F8Problem& p) {
    if (p.tokens <= kFewRows) return 0;
    return plan_product<OpF8, false, false>(p.tokens, p.out, p.dim, direct(p), p.b_pitch).partial_bytes;
}

hipError_t launch_f8(const F8Problem& f, bool f32, hipStream_t stream) {
    Product p{};
    p.a = static_cast<const char*>(f.a);
    p.b[0] = static_cast<const char*>(f.b);
    p.a_pitch = f.a_pitch;
    p.b_pitch = f.b_pitch;
    p.M = f.tokens;
    p.N = f.out;
    p.k = f.dim;
    const F8Scales s{f.a_scale, f.b_scale, (f.dim + kBlock - 1) / kBlock};
    const BiasDone done{f32, f.y, f.bias};
    if (f.tokens <= kFewRows)
        return f.b_rows ? launch_f8_few<true>(f, p, s, done, stream) : launch_f8_few<false>(f, p, s, done, stream);
    if (f32)
        return f.b_rows ? launch_f8_of<Sixteen, true>(f, p, s, done, stream)
                        : launch_f8_of<Sixteen, false>(f, p, s, done, stream);
    return f.b_rows ? launch_f8_of<Eight, true>(f, p, s, done, stream) : launch_f8_of<Eight, false>(f, p, s, done, stream);
}

namespace {

template <bool F32, bool VEC>
hipError_t quantize(const F8Quantize& p, hipStream_t stream) {
    const uint32_t tiles = ((p.rows + kBlock - 1) / kBlock) * ((p.dim + kBlock - 1) / kBlock);
    if (p.blocks) {
        if (p.q_turned) f8_tiles_of<F32, VEC, true, true><<<tiles, 256, 0, stream>>>(p);
        else f8_tiles_of<F32, VEC, true, false><<<tiles, 256, 0, stream>>>(p);
    } else if (p.q_turned) {
        f8_tiles_of<F32, VEC, false, true><<<tiles, 256, 0, stream>>>(p);
    } else {
        const uint32_t per_row = (p.dim + kBlock - 1) / kBlock;
        const uint64_t blocks = static_cast<uint64_t>(p.rows) * per_row, need = (blocks + 15) / 16;
        f8_rows_of<F32, VEC><<<static_cast<uint32_t>(need < 8192 ? need : 8192), 256, 0, stream>>>(
            static_cast<const char*>(p.x), static_cast<uint8_t*>(p.q), p.scale, blocks, per_row, p.dim);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize(const F8Quantize& p, bool f32, hipStream_t stream) {
    const bool vec = p.dim % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0;
    if (f32) return vec ? quantize<true, true>(p, stream) : quantize<true, false>(p, stream);
    return vec ? quantize<false, true>(p, stream) : quantize<false, false>(p, stream);
}

}  // namespace ltx3drope
