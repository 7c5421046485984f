// Matrix products C[m][n] = sum_k A[m][k] * B[n][k] on the matrix cores (device code; both operands
// row-major with k innermost), with a functor for what happens to a finished tile.
//
// The products treat a row of k as bytes: a 16-byte chunk holds 8 bf16, 16 int8 or 4 fp32 numbers,
// and one step of a wavefront multiplies 16 rows of A by 16 rows of B over 4 chunks.  Lane l holds
// chunk l / 16 of row l % 16 of either operand.  The order of k inside a step is the same on both
// sides, so any order gives the same sum of products.  B goes in as the instruction's first operand
// and A as its second: the result then holds, in lane l, row m = l % 16 of A against the four
// consecutive rows n = 4 * (l / 16) .. + 3 of B, and an output row is written four numbers at a time.
//
// "Gated" products multiply A by two matrices at once (the gate's and the up projection's weights):
// every wavefront holds the same rows n of both, and the functor gets both sums.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ltx3drope {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct OpBf16 {
    using Acc = f32x4;
    static constexpr int kElem = 2;
    static __device__ __forceinline__ void mac(Acc& c, u32x4 b, u32x4 a) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0,
                                                    0, 0);
    }
};
struct OpI8 {
    using Acc = i32x4;
    static constexpr int kElem = 1;
    static __device__ __forceinline__ void mac(Acc& c, u32x4 b, u32x4 a) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0,
                                                  0);
    }
};
struct OpF32 {
    using Acc = f32x4;
    static constexpr int kElem = 4;
    static __device__ __forceinline__ void mac(Acc& c, u32x4 b, u32x4 a) {
        const f32x4 fb = __builtin_bit_cast(f32x4, b), fa = __builtin_bit_cast(f32x4, a);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[j], c, 0, 0, 0);
    }
};

// One product.  Sizes are 32-bit; the host keeps a tile's rows (at most 256 of them) within 2^31 bytes.
struct Product {
    const char* a;
    const char* b[2];  // [1] only for gated products
    uint64_t a_pitch, b_pitch;  // bytes from row to row
    uint32_t M, N;              // rows of A, rows of each B
    uint32_t k_bytes;           // bytes of k in a row
};

constexpr int kRowBytes = 128;  // bytes of k that a tile holds of each row at a time
constexpr uint32_t kOutOfRange = 0x80000000u;

// Tile (tm, tn) of workgroup `id`.  Workgroups go to the 8 XCDs in turn: each XCD gets one contiguous
// run of tiles, and a run walks down groups of 8 tile rows, so that the tiles that one XCD's L2 serves
// at a time share their rows of A and B.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t total = tiles_m * tiles_n, q = total / 8, r = total % 8, x = id % 8, i = id / 8;
    const uint32_t t = x < r ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
    const uint32_t width = 8 * tiles_n, first = t / width * 8;
    const uint32_t rows = tiles_m - first < 8 ? tiles_m - first : 8;
    tm = first + (t % width) % rows;
    tn = (t % width) / rows;
}

__device__ __forceinline__ void lds_copy16(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voffset, uint32_t soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voffset, soffset, 0, 0);
}

// All outstanding loads into LDS have landed, this wavefront's LDS reads are done, and so are every
// other wavefront's.
__device__ __forceinline__ void wait_all_and_meet() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Position of chunk c of tile row r inside the row's 128 bytes: spread so that the lanes of one LDS
// read fall into different banks.
__device__ __forceinline__ uint32_t swizzle(uint32_t r) { return (r >> 1) & 7; }

// BM x BN tiles, WM x WN wavefronts, each with (BM / WM) x (BN / WN) of the tile in registers.
// A row's next 128 bytes travel from memory to the other half of the LDS while this half is multiplied.
// k_bytes and the pitches are multiples of 16 and the pointers 16-byte aligned (host's duty).
template <class Op, int BM, int BN, int WM, int WN, bool GATED, class Done>
__global__ __launch_bounds__(WM* WN * 64) void product_tiles(Product p, Done done) {
    constexpr int NW = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int kStage = (BM + BN) * kRowBytes;
    constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;  // copies a wavefront makes of each operand
    static_assert(CA * 8 * NW == BM && CB * 8 * NW == BN, "tile rows split evenly over the wavefronts");
    static_assert(!GATED || (CB % 2 == 0 && FN % 2 == 0), "both halves of B in every wavefront");
    __shared__ __align__(1024) char lds[2 * kStage];

    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave / WN, wn = wave % WN;
    constexpr int BNB = GATED ? BN / 2 : BN;  // rows of each B in a tile
    uint32_t tm, tn;
    tile_of(blockIdx.x, (p.M + BM - 1) / BM, (p.N + BNB - 1) / BNB, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BNB;
    const uint32_t rows_a = p.M - m0 < BM ? p.M - m0 : BM, rows_b = p.N - n0 < BNB ? p.N - n0 : BNB;

    auto resource = [&](const char* base, uint32_t row, uint64_t pitch, uint32_t rows) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base + row * pitch), 0,
                                                 static_cast<int>((rows - 1) * pitch + p.k_bytes), 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t ra = resource(p.a, m0, p.a_pitch, rows_a);
    const __amdgpu_buffer_rsrc_t rb0 = resource(p.b[0], n0, p.b_pitch, rows_b);
    const __amdgpu_buffer_rsrc_t rb1 = GATED ? resource(p.b[1], n0, p.b_pitch, rows_b) : rb0;

    // copy i of this wavefront fills rows 8 * (i * NW + wave) .. + 7 of the tile; lane l brings the
    // 16 bytes that belong at slot l % 8 of row l / 8.  Rows that do not exist are out of range: zeros.
    uint32_t va[CA], vb[CB];
    uint32_t chunk;
    {
        const uint32_t r8 = lane >> 3;
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const uint32_t r = (i * NW + wave) * 8 + r8, c = (lane & 7) ^ swizzle(r);
            va[i] = r < rows_a ? static_cast<uint32_t>(r * p.a_pitch) + c * 16 : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            const uint32_t r = ((GATED ? i % (CB / 2) : i) * NW + wave) * 8 + r8;
            const uint32_t c = (lane & 7) ^ swizzle(r);
            vb[i] = r < rows_b ? static_cast<uint32_t>(r * p.b_pitch) + c * 16 : kOutOfRange;
        }
        // NW is even: every copy of a lane has the same chunk
        chunk = ((lane & 7) ^ swizzle(wave * 8 + r8)) * 16;
    }
    static_assert(NW % 2 == 0, "one chunk a lane");

    const uint32_t steps = (p.k_bytes + kRowBytes - 1) / kRowBytes;
    auto fetch = [&](uint32_t step) {
        char* at = lds + (step & 1) * kStage;
        const uint32_t k = step * kRowBytes;
        const bool past = k + chunk >= p.k_bytes;  // only in the last step
#pragma unroll
        for (int i = 0; i < CA; ++i)
            lds_copy16(ra, at + (i * NW + wave) * 1024, past ? kOutOfRange : va[i], k);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            lds_copy16(GATED && i >= CB / 2 ? rb1 : rb0, at + BM * kRowBytes + (i * NW + wave) * 1024,
                       past ? kOutOfRange : vb[i], k);
    };

    using Acc = typename Op::Acc;
    Acc acc[FM][FN] = {};
    // this lane's place in a 16-row block; the blocks start at multiples of 16 rows
    const uint32_t row = (lane & 15) * kRowBytes, sw = swizzle(lane & 15);
    const uint32_t pos[2] = {row + (((lane >> 4) ^ sw) << 4), row + (((4 + (lane >> 4)) ^ sw) << 4)};
    const uint32_t a_at = wm * (BM / WM) * kRowBytes;
    // gated: half of the wavefront's blocks are rows of the gate, half the same rows of the other
    auto b_block = [&](int j) {
        if constexpr (GATED) return (j < FN / 2 ? 0 : BN / 2) + wn * (BN / WN / 2) + (j % (FN / 2)) * 16;
        else return wn * (BN / WN) + j * 16;
    };

    fetch(0);
    for (uint32_t s = 0; s < steps; ++s) {
        wait_all_and_meet();
        if (s + 1 < steps) fetch(s + 1);
        const char* at = lds + (s & 1) * kStage;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            u32x4 a[FM], b[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[j] = *reinterpret_cast<const u32x4*>(at + BM * kRowBytes + b_block(j) * kRowBytes + pos[kk]);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                a[i] = *reinterpret_cast<const u32x4*>(at + a_at + i * 16 * kRowBytes + pos[kk]);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) Op::mac(acc[i][j], b[j], a[i]);
        }
    }

#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t m = m0 + wm * (BM / WM) + i * 16 + (lane & 15);
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < (GATED ? FN / 2 : FN); ++j) {
            const uint32_t n = n0 + (GATED ? wn * (BN / WN / 2) : wn * (BN / WN)) + j * 16 + (lane >> 4) * 4;
            if (n >= p.N) continue;
            if constexpr (GATED) done(m, n, p.N, acc[i][j], acc[i][j + FN / 2]);
            else done(m, n, p.N, acc[i][j]);
        }
    }
}

// 16 bytes of a row from byte k on; what lies past `end` is zero.  Without alignment the last chunk is
// read one element at a time.
template <class Op, bool ALIGNED>
__device__ __forceinline__ u32x4 load_chunk(const char* row, uint32_t k, uint32_t end) {
    u32x4 v = {0, 0, 0, 0};
    if constexpr (ALIGNED) {
        if (k < end) v = *reinterpret_cast<const u32x4*>(row + k);
    } else {
        if (k + 16 <= end) {
            __builtin_memcpy(&v, row + k, 16);
        } else if (k < end) {
            for (uint32_t i = 0; i < end - k; i += Op::kElem) {
                uint32_t e = 0;
                __builtin_memcpy(&e, row + k + i, Op::kElem);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (i / 4 == static_cast<uint32_t>(w)) v[w] |= e << (8 * (i % 4));
            }
        }
    }
    return v;
}

// Few rows of A (at most 16 * MF): B is read once, straight into registers, 16 of its rows a workgroup,
// and the wavefronts of a workgroup share out k.  Their sums meet in LDS.  Bound by the bytes of B.
template <class Op, int MF, int NW, bool GATED, bool ALIGNED, class Done>
__global__ __launch_bounds__(NW * 64) void product_rows(Product p, Done done) {
    constexpr int NB = GATED ? 2 : 1;
    using Acc = typename Op::Acc;
    __shared__ Acc lds[NW][NB * MF][64];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 16, r = lane & 15;
    const uint32_t n = n0 + r < p.N ? n0 + r : p.N - 1;  // rows past the end repeat the last one
    const char* rb[NB];
#pragma unroll
    for (int q = 0; q < NB; ++q) rb[q] = p.b[q] + n * p.b_pitch;
    const char* ra[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const uint32_t m = i * 16 + r < p.M ? i * 16 + r : p.M - 1;
        ra[i] = p.a + m * p.a_pitch;
    }
    Acc acc[NB][MF] = {};
    const uint32_t kl = (lane >> 4) * 16;
    constexpr int U = MF > 1 ? 2 : 4;  // steps of k in flight; 128 bytes or more of a row at a time
    for (uint32_t k0 = wave * 64 * U; k0 < p.k_bytes; k0 += NW * 64 * U) {
        u32x4 b[U][NB], a[U][MF];
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const uint32_t k = k0 + s * 64 + kl;
#pragma unroll
            for (int q = 0; q < NB; ++q) b[s][q] = load_chunk<Op, ALIGNED>(rb[q], k, p.k_bytes);
#pragma unroll
            for (int i = 0; i < MF; ++i) a[s][i] = load_chunk<Op, ALIGNED>(ra[i], k, p.k_bytes);
        }
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int q = 0; q < NB; ++q)
#pragma unroll
                for (int i = 0; i < MF; ++i) Op::mac(acc[q][i], b[s][q], a[s][i]);
    }
#pragma unroll
    for (int q = 0; q < NB; ++q)
#pragma unroll
        for (int i = 0; i < MF; ++i) lds[wave][q * MF + i][lane] = acc[q][i];
    __syncthreads();
    for (uint32_t i = wave; i < MF; i += NW) {
        Acc sum[NB] = {};
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int q = 0; q < NB; ++q) sum[q] += lds[w][q * MF + i][lane];
        const uint32_t m = i * 16 + r, nn = n0 + (lane >> 4) * 4;
        if (m < p.M && nn < p.N) {
            if constexpr (GATED) done(m, nn, p.N, sum[0], sum[1]);
            else done(m, nn, p.N, sum[0]);
        }
    }
}

// Four consecutive outputs from column n on, those below N, in fp32 or rounded once to bf16.
template <bool F32>
__device__ __forceinline__ void store4(void* row, uint32_t n, uint32_t N, f32x4 v) {
    if constexpr (F32) {
        float* o = static_cast<float*>(row) + n;
        if (n + 4 <= N) {
            __builtin_memcpy(o, &v, 16);
        } else {
            for (int i = 0; i < 4; ++i)
                if (n + i < N) o[i] = v[i];
        }
    } else {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        const bf16x4 b = __builtin_convertvector(v, bf16x4);
        __bf16* o = static_cast<__bf16*>(row) + n;
        if (n + 4 <= N) {
            __builtin_memcpy(o, &b, 8);
        } else {
            for (int i = 0; i < 4; ++i)
                if (n + i < N) o[i] = b[i];
        }
    }
}

// Copies rows of `bytes` bytes into rows of `pitch` bytes (a multiple of 16) with zeros behind: operands
// whose rows are not whole 16-byte chunks, or that do not start on one.
template <typename T>
__global__ __launch_bounds__(256) void pad_rows(const T* src, T* dst, uint32_t rows, uint32_t width,
                                                uint32_t pitch) {
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (uint32_t c = threadIdx.x; c < pitch; c += 256)
            dst[static_cast<size_t>(r) * pitch + c] = c < width ? src[static_cast<size_t>(r) * width + c] : T(0);
}

inline size_t up16(size_t n) { return (n + 15) / 16 * 16; }

template <typename T>
inline void launch_pad_rows(const void* src, void* dst, uint32_t rows, size_t bytes, hipStream_t stream) {
    pad_rows<T><<<rows < 8192 ? rows : 8192, 256, 0, stream>>>(
        static_cast<const T*>(src), static_cast<T*>(dst), rows, static_cast<uint32_t>(bytes / sizeof(T)),
        static_cast<uint32_t>(up16(bytes) / sizeof(T)));
}

// The tile product's grid.
template <int BM, int BN>
inline uint32_t tile_count(uint32_t M, uint32_t N) {
    return ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
}

inline bool aligned16(const Product& p, bool gated) {
    uintptr_t bits = reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.b[0]) | p.a_pitch | p.b_pitch |
                     p.k_bytes;
    if (gated) bits |= reinterpret_cast<uintptr_t>(p.b[1]);
    return bits % 16 == 0;
}

constexpr uint32_t kFewRows = 64;  // most rows of A that product_rows takes

template <class Op, bool GATED, class Done>
hipError_t launch_product(const Product& p, const Done& done, hipStream_t stream) {
    const bool al = aligned16(p, GATED);
    const uint32_t groups = (p.N + 15) / 16;
    if (p.M <= kFewRows) {
        if (p.M <= 16) {
            if (al) product_rows<Op, 1, 8, GATED, true, Done><<<groups, 512, 0, stream>>>(p, done);
            else product_rows<Op, 1, 8, GATED, false, Done><<<groups, 512, 0, stream>>>(p, done);
        } else {
            if (al) product_rows<Op, 4, 8, GATED, true, Done><<<groups, 512, 0, stream>>>(p, done);
            else product_rows<Op, 4, 8, GATED, false, Done><<<groups, 512, 0, stream>>>(p, done);
        }
        return hipGetLastError();
    }
    if (!al) return hipErrorInvalidValue;  // the caller lays such operands out first
    const uint32_t big = tile_count<256, GATED ? 128 : 256>(p.M, p.N);
    if (big >= 192)
        product_tiles<Op, 256, 256, 2, 4, GATED, Done><<<big, 512, 0, stream>>>(p, done);
    else
        product_tiles<Op, 128, 128, 2, 2, GATED, Done>
            <<<tile_count<128, GATED ? 64 : 128>(p.M, p.N), 256, 0, stream>>>(p, done);
    return hipGetLastError();
}

}  // namespace ltx3drope
