// Matrix products C[m][n] = sum_k A[m][k] * B[n][k] with a functor for what happens to finished sums:
// product_tiles on the matrix cores for many rows of A, product_rows for up to 16, product_tokens for up
// to 8.  Kernels, and the rules that choose among them.
//
// The matrix cores' products treat a row of k as bytes: a 16-byte chunk holds 8 bf16, 16 int8 or 4 fp32 numbers,
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
#include <type_traits>

namespace ltx3drope {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct OpBf16 {
    using Acc = f32x4;
    using Sum = float;
    static constexpr int kElem = 2, kTokens = 4;  // most rows of A for product_tokens
    static __device__ __forceinline__ void mac(Acc& c, u32x4 b, u32x4 a) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0,
                                                    0, 0);
    }
    // the eight products of a chunk
    static __device__ __forceinline__ float dot(u32x4 a, u32x4 b, float s) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t x = a[j], y = b[j];  // a cast of a[j] itself takes element 0
            s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), __builtin_bit_cast(bf16x2, y), s, false);
        }
        return s;
    }
};
struct OpI8 {
    using Acc = i32x4;
    using Sum = int;
    static constexpr int kElem = 1, kTokens = 1;
    static __device__ __forceinline__ void mac(Acc& c, u32x4 b, u32x4 a) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0,
                                                  0);
    }
    static __device__ __forceinline__ int dot(u32x4 a, u32x4 b, int s) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s = __builtin_amdgcn_sdot4(static_cast<int>(a[j]), static_cast<int>(b[j]), s, false);
        return s;
    }
};
struct OpF32 {
    using Acc = f32x4;
    using Sum = float;
    static constexpr int kElem = 4, kTokens = 8;
    static __device__ __forceinline__ void mac(Acc& c, u32x4 b, u32x4 a) {
        const f32x4 fb = __builtin_bit_cast(f32x4, b), fa = __builtin_bit_cast(f32x4, a);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[j], c, 0, 0, 0);
    }
    static __device__ __forceinline__ float dot(u32x4 a, u32x4 b, float s) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(__uint_as_float(a[j]), __uint_as_float(b[j]), s);
        return s;
    }
};

// One product, C[m][n] = sum_k A[m][k] * B[n][k].  An operand is stored with k innermost (rows of the
// output's index, the k of one after the other) or with k outermost (rows of k, the output's index along
// them).  Sizes are 32-bit; the host keeps what a tile addresses (256 rows of an operand with k
// innermost, 64 of one with k outermost) within 2^31 bytes.
struct Product {
    const char* a;
    const char* b[2];           // [1]: the second matrix of a gated product, or B's rows of k from k_second on
    uint64_t a_pitch, b_pitch;  // bytes from row to row
    uint32_t M, N;              // output sizes (N: of each B)
    uint32_t k;                 // length of the sums
    uint32_t k_second;          // k outermost: where b[1] takes over (a multiple of a step), or 0 for never
    uint32_t k_rows;            // ... and the rows of k that b[0] and b[1] hold each (zeros from there on)
    float* partial;             // splits > 1: [splits][tiles][BM * BN] sums
    uint32_t splits;
};

constexpr int kRowBytes = 128;  // bytes of k that a tile holds of each row at a time
constexpr uint32_t kOutOfRange = 0x80000000u;

// Tile (tm, tn) of workgroup `id` of tiles_m * tiles_n.  Workgroups go to the 8 XCDs in turn: each XCD
// gets one contiguous run of tiles, and a run walks down groups of 8 tile rows, so that the tiles that
// one XCD's L2 serves at a time share their rows of A and B.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t total = tiles_m * tiles_n, q = total / 8, r = total % 8, x = id % 8, i = id / 8;
    const uint32_t t = x < r ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
    const uint32_t width = 8 * tiles_n, first = t / width * 8;
    const uint32_t rows = tiles_m - first < 8 ? tiles_m - first : 8;
    tm = first + (t % width) % rows;
    tn = (t % width) / rows;
}

// A raw buffer descriptor of `lines` lines of `bytes` bytes, `pitch` apart (the same in every lane): what
// lies past its end reads as zero.
__device__ __forceinline__ u32x4 buffer_of(const char* base, uint64_t pitch, uint32_t lines, uint32_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    auto uniform = [](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); };
    return u32x4{uniform(static_cast<uint32_t>(at)), uniform(static_cast<uint32_t>(at >> 32)),
                 uniform(lines == 0 ? 0u : static_cast<uint32_t>((lines - 1) * pitch + bytes)), 0x00020000u};
}

// Sends 16 bytes a lane from the buffer to LDS, lane l's to lds + 16 * l.  The instruction is written out
// because the compiler, which cannot tell which LDS bytes a builtin copy fills, waits for all copies
// before every turning read of another slot (16384 x 2048, k 4096 outermost on both sides: 308 us with
// the builtin, 252 so).  It leaves no register behind but m0, which nothing else in these kernels uses;
// its arrival is awaited by wait_and_meet.
__device__ __forceinline__ void lds_copy16(u32x4 buffer, char* lds, uint32_t voffset, uint32_t soffset) {
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(at), "v"(voffset),
                 "s"(buffer), "s"(soffset));
}

// All but this wavefront's N newest copies have landed, its LDS reads and writes are done, and so are
// every other wavefront's.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// v without its first d bytes, moved down, zeros behind.
__device__ __forceinline__ u32x4 drop_bytes(u32x4 v, uint32_t d) {
    const uint32_t n = d < 16 ? d : 16;
    uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
    const uint32_t bits = (n & 7) * 8;
    if (n >= 8) {
        lo = hi;
        hi = 0;
    }
    lo = bits ? lo >> bits | hi << (64 - bits) : lo;
    hi >>= bits;
    if (n == 16) lo = 0;
    return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                 static_cast<uint32_t>(hi >> 32)};
}

// This wavefront's LDS reads and writes are done, and so are every other wavefront's; loads on their way
// into registers stay there.
__device__ __forceinline__ void wait_for_lds_and_meet() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes of a row from byte k on; what lies past `end` is zero.  Without alignment a chunk that reaches
// past the end is read from the row's last 16 bytes, so that every lane makes one load; only rows
// shorter than that are read one element at a time.  STREAM: nobody reads these bytes again soon.
template <class Op, bool ALIGNED, bool STREAM>
__device__ __forceinline__ u32x4 load_chunk(const char* row, uint32_t k, uint32_t end) {
    u32x4 v = {0, 0, 0, 0};
    if constexpr (ALIGNED) {
        const u32x4* at = reinterpret_cast<const u32x4*>(row + k);
        if (k < end) v = STREAM ? __builtin_nontemporal_load(at) : *at;
    } else if (end >= 16) {
        typedef u32x4 any_u32x4 __attribute__((aligned(1)));
        const uint32_t at = k + 16 <= end ? k : end - 16;
        v = *reinterpret_cast<const any_u32x4*>(row + at);
        if (k != at) v = drop_bytes(v, k - at);
    } else {
        for (uint32_t i = 0; k + i < end; i += Op::kElem) {
            uint32_t e = 0;
            __builtin_memcpy(&e, row + k + i, Op::kElem);
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (i / 4 == static_cast<uint32_t>(w)) v[w] |= e << (8 * (i % 4));
        }
    }
    return v;
}

// One operand's part of a tile: R rows of the output's index against 128 bytes of k, in LDS.
//
// k innermost: tile row r is 128 bytes, eight 16-byte chunks; chunk c lies at slot c ^ (r / 2 % 8).
// k outermost: LDS rows are rows of k, R elements each, in units of 16 elements; unit u of row k lies at
// unit u ^ spread(k).  Both keep the lanes of one LDS read in different banks.
template <class Op, int R, bool K_OUTER>
struct Side {
    static constexpr int kStepK = kRowBytes / Op::kElem;  // k of a step
    static constexpr int kBytes = R * kRowBytes;          // LDS bytes of a step
    static constexpr int kLdsRow = K_OUTER ? R * Op::kElem : kRowBytes;
    static constexpr int kUnit = 16 * Op::kElem;

    static __device__ __forceinline__ uint32_t swizzle(uint32_t r) { return (r >> 1) & 7; }
    static __device__ __forceinline__ uint32_t spread(uint32_t k) {
        return (Op::kElem == 4 ? (k >> 2) & 3 : (k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
    }

    // What 16-byte place `at` of the LDS image holds: row `line` (of the output's index or of k) of the
    // tile, 16 bytes from byte `byte` of the line on.
    static __device__ __forceinline__ void place(uint32_t at, uint32_t& line, uint32_t& byte) {
        line = at * 16 / kLdsRow;
        const uint32_t slot = at % (kLdsRow / 16);
        if constexpr (K_OUTER) {
            constexpr uint32_t c = kUnit / 16;
            byte = (((slot / c) ^ spread(line)) * c + slot % c) * 16;
        } else {
            byte = (slot ^ swizzle(line)) * 16;
        }
    }

    // This lane's 16 bytes of block `blk` (16 rows of the output's index), half step kk.
    // base: block_base(lane, blk) for k outermost, lane_base(lane) otherwise.
    static __device__ __forceinline__ uint32_t lane_base(uint32_t lane, int kk) {
        return (lane & 15) * kRowBytes + (((kk * 4 + (lane >> 4)) ^ swizzle(lane & 15)) << 4);
    }
    static __device__ __forceinline__ uint32_t block_base(uint32_t lane, uint32_t blk) {
        const uint32_t q = lane >> 4;
        if constexpr (Op::kElem == 4) {
            return q * 4 * kLdsRow + ((blk ^ q) * kUnit) + (lane & 15) * 4;  // k = 16 kk + 4 q + j
        } else {
            const uint32_t k = q * 8 + (lane & 15) / 4;  // 4 lanes bring 16 numbers of one k
            return k * kLdsRow + ((blk ^ spread(k)) * kUnit) + (lane & 3) * 8;
        }
    }
    static __device__ __forceinline__ u32x4 outer_frag(const char* lds, uint32_t base, int kk) {
        if constexpr (Op::kElem == 4) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(lds + base + (kk * 16 + j) * kLdsRow);
            return v;
        } else {
            // each read turns 4 rows of k by 16 numbers: lane l gets number l % 16 of all four
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
            u32x2 h[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                h[j] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (__attribute__((address_space(3))) s16x4*)(lds + base + (kk * 32 + j * 4) * kLdsRow)));
            return u32x4{h[0][0], h[0][1], h[1][0], h[1][1]};
        }
    }
};

// BM x BN tiles, WM x WN wavefronts, each with (BM / WM) x (BN / WN) of the tile in registers.
// DIRECT: 16-byte aligned operands go from memory to LDS without passing through registers; otherwise
// they pass through them (any alignment).  A_OUTER, B_OUTER: k outermost.
template <class Op, int BM, int BN, int WM, int WN, bool PIPELINED, bool GATED, bool A_OUTER, bool B_OUTER, bool DIRECT,
          class Done>
__global__ __launch_bounds__(WM* WN * 64) void product_tiles(Product p, Done done) {
    constexpr int NW = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int BNB = GATED ? BN / 2 : BN;  // rows of each B in a tile
    using SA = Side<Op, BM, A_OUTER>;
    using SB = Side<Op, BNB, B_OUTER>;
    // LDS: rings of kSlotsA steps of A and kSlotsB of B (256 x 256: 3 and 2, all 160 KB).  The copies have a
    // step's time to land at the least; with the third slot A's have two, and half as many bytes again
    // are on their way at any time, which is what the copies' rate goes by (8192 x 8192 x 8192 in bf16:
    // 887 us with two slots each, 848 so; copies alone 743, and 587 with two whole steps on their way).
    constexpr int kRing = DIRECT && BM == 64 ? 3 : 2;  // not PIPELINED: slots of either
    constexpr int kSlotsA = PIPELINED ? 3 : kRing, kSlotsB = PIPELINED ? 2 : kRing, kStepK = SA::kStepK;
    constexpr int kBytesB = BN * kRowBytes, kAtB = kSlotsA * SA::kBytes;
    constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;  // 1 KB copies a wavefront makes of each operand
    static_assert(CA * 8 * NW == BM && CB * 8 * NW == BN, "a tile's copies split evenly over the wavefronts");
    static_assert(!GATED || (CB % 2 == 0 && FN % 2 == 0 && !B_OUTER), "both halves of B in every wavefront");
    __shared__ __align__(1024) char lds[kAtB + kSlotsB * kBytesB];

    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave / WN, wn = wave % WN;
    const uint32_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BNB - 1) / BNB, tiles = tiles_m * tiles_n;
    const uint32_t tile = blockIdx.x % tiles, split = blockIdx.x / tiles;
    uint32_t tm, tn;
    tile_of(tile, tiles_m, tiles_n, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BNB;
    const uint32_t all_steps = (p.k + kStepK - 1) / kStepK;
    const uint32_t first = split * all_steps / p.splits, last = (split + 1) * all_steps / p.splits;

    // ---- from memory to LDS: copy i of this wavefront fills KB i * NW + wave of an operand's image
    uint32_t line_a[CA], byte_a[CA], line_b[CB], byte_b[CB];
#pragma unroll
    for (int i = 0; i < CA; ++i) SA::place((i * NW + wave) * 64 + lane, line_a[i], byte_a[i]);
#pragma unroll
    for (int i = 0; i < CB; ++i)
        SB::place(((GATED ? i % (CB / 2) : i) * NW + wave) * 64 + lane, line_b[i], byte_b[i]);

    // the descriptor of an operand for one step, and this lane's byte in it (or out of range: zeros)
    auto inner_rsrc = [&](const char* base, uint64_t pitch, uint32_t row0, uint32_t rows, uint32_t R) {
        const uint32_t n = rows - row0 < R ? rows - row0 : R;
        return buffer_of(base + row0 * pitch, pitch, n, p.k * Op::kElem);
    };
    u32x4 ra, rb0, rb1;
    uint32_t va[CA], vb[CB];
    if constexpr (DIRECT) {
        if constexpr (!A_OUTER) ra = inner_rsrc(p.a, p.a_pitch, m0, p.M, BM);
        if constexpr (!B_OUTER) {
            rb0 = inner_rsrc(p.b[0], p.b_pitch, n0, p.N, BNB);
            rb1 = GATED ? inner_rsrc(p.b[1], p.b_pitch, n0, p.N, BNB) : rb0;
        }
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const bool in = A_OUTER ? m0 * Op::kElem + byte_a[i] < p.M * Op::kElem : m0 + line_a[i] < p.M;
            va[i] = in ? static_cast<uint32_t>(line_a[i] * p.a_pitch) + byte_a[i] : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            const bool in = B_OUTER ? n0 * Op::kElem + byte_b[i] < p.N * Op::kElem : n0 + line_b[i] < p.N;
            vb[i] = in ? static_cast<uint32_t>(line_b[i] * p.b_pitch) + byte_b[i] : kOutOfRange;
        }
    }
    // for k outermost: which matrix a step belongs to, its first row of k, and how many of a step's rows exist
    auto b_segment = [&](uint32_t step, uint32_t& k0, uint32_t& rows) {
        const uint32_t k = step * kStepK;
        const bool second = p.k_second != 0 && k >= p.k_second;
        k0 = second ? k - p.k_second : k;
        const uint32_t have = p.k_second != 0 ? p.k_rows : p.k;
        rows = k0 < have ? (have - k0 < kStepK ? have - k0 : kStepK) : 0;
        return second ? p.b[1] : p.b[0];
    };
    // a step past this workgroup's last one brings zeros without touching memory
    const uint32_t k_end = last * kRowBytes < p.k * Op::kElem ? last * kRowBytes : p.k * Op::kElem;
    auto aim_a = [&](uint32_t step) {
        const uint32_t k = step * kRowBytes;
        if constexpr (A_OUTER) {
            const uint32_t k0 = step * kStepK;
            const uint32_t rows = step >= last ? 0 : (p.k - k0 < kStepK ? p.k - k0 : kStepK);
            ra = buffer_of(p.a + k0 * p.a_pitch + m0 * Op::kElem, p.a_pitch, rows, (p.M - m0) * Op::kElem);
        }
        return k;
    };
    auto copy_a = [&](uint32_t k, uint32_t slot, int i) {
        const bool past = !A_OUTER && k + byte_a[i] >= k_end;
        lds_copy16(ra, lds + slot * SA::kBytes + (i * NW + wave) * 1024, past ? kOutOfRange : va[i], A_OUTER ? 0 : k);
    };
    auto fetch_a = [&](uint32_t step, uint32_t slot) {
        const uint32_t k = aim_a(step);
#pragma unroll
        for (int i = 0; i < CA; ++i) copy_a(k, slot, i);
    };
    auto aim_b = [&](uint32_t step) {
        const uint32_t k = step * kRowBytes;
        if constexpr (B_OUTER) {
            uint32_t k0, rows;
            const char* base = b_segment(step, k0, rows);
            rb0 = buffer_of(base + k0 * p.b_pitch + n0 * Op::kElem, p.b_pitch, step >= last ? 0 : rows,
                            (p.N - n0) * Op::kElem);
        }
        return k;
    };
    auto copy_b = [&](uint32_t k, uint32_t slot, int i) {
        const bool past = !B_OUTER && k + byte_b[i] >= k_end;
        lds_copy16(GATED && i >= CB / 2 ? rb1 : rb0, lds + kAtB + slot * kBytesB + (i * NW + wave) * 1024,
                   past ? kOutOfRange : vb[i], B_OUTER ? 0 : k);
    };
    auto fetch_b = [&](uint32_t step, uint32_t slot) {
        const uint32_t k = aim_b(step);
#pragma unroll
        for (int i = 0; i < CB; ++i) copy_b(k, slot, i);
    };
    struct Held {
        u32x4 v[DIRECT ? 1 : CA + CB];
    };
    // rows past the output's end repeat the last one (their sums are dropped); rows of k past the end are zero
    auto hold = [&](Held& to, uint32_t step) {
        if constexpr (!DIRECT) {
            const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < CA; ++i) {
                if constexpr (A_OUTER) {
                    const uint32_t k = step * kStepK + line_a[i], last_k = p.k - 1;
                    to.v[i] = load_chunk<Op, false, false>(p.a + (k < last_k ? k : last_k) * p.a_pitch,
                                                           m0 * Op::kElem + byte_a[i], p.M * Op::kElem);
                    if (k > last_k) to.v[i] = zero;
                } else {
                    const uint32_t m = m0 + line_a[i] < p.M ? m0 + line_a[i] : p.M - 1;
                    to.v[i] = load_chunk<Op, false, false>(p.a + m * p.a_pitch, step * kRowBytes + byte_a[i],
                                                           p.k * Op::kElem);
                }
            }
#pragma unroll
            for (int i = 0; i < CB; ++i) {
                u32x4& h = to.v[CA + i];
                if constexpr (B_OUTER) {
                    uint32_t k0, rows;
                    const char* base = b_segment(step, k0, rows);
                    const uint32_t row = rows == 0 ? 0 : k0 + (line_b[i] < rows ? line_b[i] : rows - 1);
                    h = load_chunk<Op, false, false>(base + row * p.b_pitch, n0 * Op::kElem + byte_b[i],
                                                     p.N * Op::kElem);
                    if (line_b[i] >= rows) h = zero;
                } else {
                    const uint32_t n = n0 + line_b[i] < p.N ? n0 + line_b[i] : p.N - 1;
                    h = load_chunk<Op, false, false>(p.b[GATED && i >= CB / 2] + n * p.b_pitch,
                                                     step * kRowBytes + byte_b[i], p.k * Op::kElem);
                }
            }
        }
    };
    auto put_held = [&](const Held& from, uint32_t slot) {
        if constexpr (!DIRECT) {
            char* at = lds + wave * 1024 + lane * 16;
#pragma unroll
            for (int i = 0; i < CA; ++i) *reinterpret_cast<u32x4*>(at + slot * SA::kBytes + i * NW * 1024) = from.v[i];
#pragma unroll
            for (int i = 0; i < CB; ++i)
                *reinterpret_cast<u32x4*>(at + kAtB + slot * kBytesB + i * NW * 1024) = from.v[CA + i];
        }
    };

    // ---- from LDS to the matrix cores
    using Acc = typename Op::Acc;
    Acc acc[FM][FN] = {};
    // the wavefront's block j of B; gated: half are rows of the first matrix, half the same rows of the other
    auto b_block = [&](int j) -> uint32_t {
        if constexpr (GATED) return (j < FN / 2 ? 0 : BN / 32) + wn * (FN / 2) + j % (FN / 2);
        else return wn * FN + j;
    };
    uint32_t base_a[A_OUTER ? FM : 2], base_b[B_OUTER ? FN : 2];
    if constexpr (A_OUTER) {
#pragma unroll
        for (int i = 0; i < FM; ++i) base_a[i] = SA::block_base(lane, wm * FM + i);
    } else {
        for (int kk = 0; kk < 2; ++kk) base_a[kk] = wm * FM * 16 * kRowBytes + SA::lane_base(lane, kk);
    }
    if constexpr (B_OUTER) {
#pragma unroll
        for (int j = 0; j < FN; ++j) base_b[j] = kAtB + SB::block_base(lane, b_block(j));
    } else {
        for (int kk = 0; kk < 2; ++kk) base_b[kk] = kAtB + SB::lane_base(lane, kk);
    }
    u32x4 fa[2][FM], fb[2][FN];
    // operand block n of a half step: B's blocks, then A's
    auto read_one = [&](const char* at_a, const char* at_b, int kk, int n) {
        if (n < FN) {
            if constexpr (B_OUTER) fb[kk][n] = SB::outer_frag(at_b, base_b[n], kk);
            else fb[kk][n] = *reinterpret_cast<const u32x4*>(at_b + base_b[kk] + b_block(n) * 16 * kRowBytes);
        } else {
            if constexpr (A_OUTER) fa[kk][n - FN] = SA::outer_frag(at_a, base_a[n - FN], kk);
            else fa[kk][n - FN] = *reinterpret_cast<const u32x4*>(at_a + base_a[kk] + (n - FN) * 16 * kRowBytes);
        }
    };
    auto read = [&](uint32_t slot_a, uint32_t slot_b, int kk) {
#pragma unroll
        for (int n = 0; n < FN + FM; ++n) read_one(lds + slot_a * SA::kBytes, lds + slot_b * kBytesB, kk, n);
    };
    auto multiply = [&](int kk) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) Op::mac(acc[i][j], fb[kk][j], fa[kk][i]);
    };
    // One row of blocks is multiplied while some of the operands of half step kk of the given slots are
    // read; `between` says what else goes there.  Pinned in this order: left alone, the compiler puts all
    // reads (and copies) first, and the matrix cores wait for them.
    auto multiply_and_read = [&](int kk, uint32_t slot_a, uint32_t slot_b, auto between) {
        const char *at_a = lds + slot_a * SA::kBytes, *at_b = lds + slot_b * kBytesB;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int n = i * (FN + FM) / FM; n < (i + 1) * (FN + FM) / FM; ++n) read_one(at_a, at_b, kk ^ 1, n);
            between(i);
#pragma unroll
            for (int j = 0; j < FN; ++j) Op::mac(acc[i][j], fb[kk][j], fa[kk][i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if constexpr (PIPELINED) {
        // Half a step is multiplied while the next half step's operands are read from LDS.  The step
        // after this one has to be in LDS, and this one's slots are free, once every wavefront has read
        // its second half: they meet between the two multiplications, with operands for the second in
        // registers, and the copies for the freed slots set out.
        fetch_b(first, 0);
        fetch_a(first, 0);
        fetch_a(first + 1, 1);
        fetch_b(first + 1, 1);
        fetch_a(first + 2, 2);
        wait_and_meet<2 * CA + CB>();
        read(0, 0, 0);
        uint32_t sa = 0, sb = 0;  // the step's slots
        for (uint32_t s = first; s + 1 < last; ++s) {
            const uint32_t next = sa == 2 ? 0 : sa + 1;
            __builtin_amdgcn_s_setprio(1);  // whoever still multiplies goes first
            multiply_and_read(0, sa, sb, [](int) {});
            __builtin_amdgcn_s_setprio(0);
            wait_and_meet<CA>();  // all but A's copies for the step after the next
            const uint32_t kb = aim_b(s + 2), ka = aim_a(s + 3);
            multiply_and_read(1, next, sb ^ 1, [&](int i) {
#pragma unroll
                for (int c = i * (CA + CB) / FM; c < (i + 1) * (CA + CB) / FM; ++c) {
                    if (c < CB) copy_b(kb, sb, c);
                    else copy_a(ka, sa, c - CB);
                }
            });
            sa = next;
            sb ^= 1;
        }
        read(sa, sb, 1);
        multiply(0);
        multiply(1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives its workgroup
    } else if constexpr (DIRECT) {
        // several workgroups share a compute unit and fill each other's waits
        for (int i = 0; i < kRing - 1; ++i) {
            fetch_a(first + i, i);
            fetch_b(first + i, i);
        }
        uint32_t slot = 0, free = kRing - 1;
        for (uint32_t s = first; s < last; ++s) {
            wait_and_meet<(kRing - 2) * (CA + CB)>();
            fetch_a(s + kRing - 1, free);
            fetch_b(s + kRing - 1, free);
            free = slot;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                read(slot, slot, kk);
                multiply(kk);
            }
            slot = slot + 1 == kRing ? 0 : slot + 1;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy outlives its workgroup
    } else {
        // two steps ahead in registers: a load has two steps' time to arrive
        Held even, odd;
        auto turn = [&](uint32_t s, Held& next, Held& after) {
            const uint32_t slot = (s - first) & 1;
            wait_for_lds_and_meet();
            if (s + 2 < last) hold(after, s + 2);
            read(slot, slot, 0);
            read(slot, slot, 1);
            multiply(0);
            multiply(1);
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
        Acc* out = reinterpret_cast<Acc*>(p.partial) +
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
        for (int j = 0; j < (GATED ? FN / 2 : FN); ++j) {
            const uint32_t n = n0 + b_block(j) * 16 + (lane >> 4) * 4;
            if (n >= p.N) continue;
            if constexpr (GATED) done(m, n, p.N, acc[i][j], acc[i][j + FN / 2]);
            else done(m, n, p.N, acc[i][j]);
        }
    }
}

// The parts of a product whose sums were split over k, added in order of k.  One workgroup a tile and
// block of 16 rows, the lanes as in product_tiles.
template <class Op, int BM, int BN, int WM, int WN, bool GATED, class Done>
__global__ __launch_bounds__(WM* WN * 64) void product_join(Product p, Done done) {
    constexpr int NW = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int BNB = GATED ? BN / 2 : BN;
    using Acc = typename Op::Acc;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave / WN, wn = wave % WN;
    const uint32_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BNB - 1) / BNB, tiles = tiles_m * tiles_n;
    const uint32_t tile = blockIdx.x / FM, i = blockIdx.x % FM;
    uint32_t tm, tn;
    tile_of(tile, tiles_m, tiles_n, tm, tn);
    const uint32_t m = tm * BM + (wm * FM + i) * 16 + (lane & 15);
    if (m >= p.M) return;
    const Acc* in = reinterpret_cast<const Acc*>(p.partial) + static_cast<size_t>(tile) * (FM * FN * NW * 64) + tid;
    const size_t step = static_cast<size_t>(tiles) * (FM * FN * NW * 64);
    Acc sum[FN] = {};
    for (uint32_t s = 0; s < p.splits; ++s)
#pragma unroll
        for (int j = 0; j < FN; ++j) sum[j] += in[s * step + (i * FN + j) * NW * 64];
#pragma unroll
    for (int j = 0; j < (GATED ? FN / 2 : FN); ++j) {
        const uint32_t n = tn * BNB + (GATED ? wn * (FN / 2) + j : wn * FN + j) * 16 + (lane >> 4) * 4;
        if (n >= p.N) continue;
        if constexpr (GATED) done(m, n, p.N, sum[j], sum[j + FN / 2]);
        else done(m, n, p.N, sum[j]);
    }
}

// The sum over a wavefront, in every lane.
template <class T>
__device__ __forceinline__ T lanes_sum(T v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// A few rows of A (bf16 1 to 4, fp32 1 to 8, int8 one: Op::kTokens): a wavefront takes one row of B (of
// each B; two for more than one row of A, so that they share its loads), its lanes along k, some KB of it
// at a time, and multiplies it by every row of A in registers.  Bound by the bytes of B, which it reads
// in whole kilobytes.  2 x 10240 rows of 4096 bf16: 26 us for one row of A (6.4 TB/s), 35 for four; the
// matrix cores' layout, 16 rows of B a load (product_rows), takes 37 and 40, and 41 against 50 for eight.
// fp32: 50, 57 for four and 74 for eight, against 88 for nine there.  int8, 4096 rows of 10240: 10 us,
// and there 11 for two and 13 for eight.  The four wavefronts of a workgroup put their sums side by side for
// `done`.
template <class Op, int MT, bool GATED, bool ALIGNED, class Done>
__global__ __launch_bounds__(256) void product_tokens(Product p, Done done) {
    constexpr int NB = GATED ? 2 : 1, KV = MT > 4 ? 2 : 4, RW = MT > 1 ? 2 : 1;  // rows of B a wavefront
    using Sum = typename Op::Sum;
    __shared__ Sum lds[NB][MT][4 * RW];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 4 * RW;
    const uint32_t k_bytes = p.k * Op::kElem;
    const char* rb[NB][RW];
#pragma unroll
    for (int q = 0; q < NB; ++q)
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            const uint32_t n = n0 + wave * RW + w;
            rb[q][w] = p.b[q] + (n < p.N ? n : p.N - 1) * p.b_pitch;
        }
    Sum sum[NB][RW][MT] = {};
    for (uint32_t k0 = 0; k0 < k_bytes; k0 += KV * 1024) {
        u32x4 b[NB][RW][KV];
#pragma unroll
        for (int q = 0; q < NB; ++q)
#pragma unroll
            for (int w = 0; w < RW; ++w)
#pragma unroll
                for (int i = 0; i < KV; ++i)
                    b[q][w][i] = load_chunk<Op, ALIGNED, true>(rb[q][w], k0 + i * 1024 + lane * 16, k_bytes);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const char* ra = p.a + (m < static_cast<int>(p.M) ? m : 0) * p.a_pitch;
#pragma unroll
            for (int i = 0; i < KV; ++i) {
                const u32x4 a = load_chunk<Op, ALIGNED, false>(ra, k0 + i * 1024 + lane * 16, k_bytes);
#pragma unroll
                for (int q = 0; q < NB; ++q)
#pragma unroll
                    for (int w = 0; w < RW; ++w) sum[q][w][m] = Op::dot(a, b[q][w][i], sum[q][w][m]);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < NB; ++q)
#pragma unroll
        for (int w = 0; w < RW; ++w)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const Sum s = lanes_sum(sum[q][w][m]);
                if (lane == 0) lds[q][m][wave * RW + w] = s;
            }
    __syncthreads();
    const uint32_t m = threadIdx.x % MT, four = threadIdx.x / MT, n = n0 + four * 4;
    if (four < RW && m < p.M && n < p.N) {
        typename Op::Acc v[NB];
#pragma unroll
        for (int q = 0; q < NB; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[q][i] = lds[q][m][four * 4 + i];
        if constexpr (GATED) done(m, n, p.N, v[0], v[1]);
        else done(m, n, p.N, v[0]);
    }
}

// Up to 16 rows of A, where product_tokens is not better: B is read once, straight into registers, 16 of its rows a workgroup, and the
// wavefronts of a workgroup share out k.  Their sums meet in LDS.  Bound by the bytes of B.
template <class Op, bool GATED, bool ALIGNED, class Done>
__global__ __launch_bounds__(512) void product_rows(Product p, Done done) {
    constexpr int NB = GATED ? 2 : 1, NW = 8, U = 4;  // U steps of k in flight: 256 bytes of a row at a time
    using Acc = typename Op::Acc;
    __shared__ Acc lds[NW][NB][64];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * 16, r = lane & 15;
    const uint32_t n = n0 + r < p.N ? n0 + r : p.N - 1;  // rows past the end repeat the last one
    const char* rb[NB];
#pragma unroll
    for (int q = 0; q < NB; ++q) rb[q] = p.b[q] + n * p.b_pitch;
    const char* ra = p.a + (r < p.M ? r : p.M - 1) * p.a_pitch;
    const uint32_t k_bytes = p.k * Op::kElem, kl = (lane >> 4) * 16;
    Acc acc[NB] = {};
    for (uint32_t k0 = wave * 64 * U; k0 < k_bytes; k0 += NW * 64 * U) {
        u32x4 b[U][NB], a[U];
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const uint32_t k = k0 + s * 64 + kl;
#pragma unroll
            for (int q = 0; q < NB; ++q) b[s][q] = load_chunk<Op, ALIGNED, false>(rb[q], k, k_bytes);
            a[s] = load_chunk<Op, ALIGNED, false>(ra, k, k_bytes);
        }
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int q = 0; q < NB; ++q) Op::mac(acc[q], b[s][q], a[s]);
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) lds[wave][q][lane] = acc[q];
    __syncthreads();
    if (wave != 0) return;
    Acc sum[NB] = {};
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int q = 0; q < NB; ++q) sum[q] += lds[w][q][lane];
    const uint32_t nn = n0 + (lane >> 4) * 4;
    if (r < p.M && nn < p.N) {
        if constexpr (GATED) done(r, nn, p.N, sum[0], sum[1]);
        else done(r, nn, p.N, sum[0]);
    }
}

// Four consecutive outputs from column n on, those below N, in fp32 or rounded once to bf16.
template <bool F32>
__device__ __forceinline__ void store4(void* row, uint32_t n, uint32_t N, f32x4 v) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    using Elem = typename std::conditional<F32, float, __bf16>::type;
    using Four = typename std::conditional<F32, f32x4, bf16x4>::type;
    typedef Four AnyFour __attribute__((aligned(F32 ? 4 : 2)));
    const Four b = __builtin_convertvector(v, Four);
    Elem* o = static_cast<Elem*>(row) + n;
    if (n + 4 <= N) {
        *reinterpret_cast<AnyFour*>(o) = b;
    } else {
        for (int i = 0; i < 4; ++i)
            if (n + i < N) o[i] = b[i];
    }
}

constexpr uint32_t kFewRows = 16;  // most rows of A that the kernels without tiles take
// Most outputs that product_tokens takes for one row of A: 64 threads each, and a launch holds fewer than
// 2^32.  product_rows has 32 an output.
constexpr uint32_t kTokenOutputs = uint32_t(1) << 25;

// How a product runs: its tile (gated: bn / 2 columns of either B), and over how many workgroups its sums
// are split.
struct Plan {
    uint32_t bm, bn, tiles, splits;
    size_t partial_bytes;
};

// Microseconds that a tile's workgroup takes: a step of k while the chip is nearly empty (`alone`), its
// share of a step on a full compute unit (`full`; `outer` times that with k outermost, `torn` times
// where rows of k do not start on 128-byte lines), and a tile's start and end (`ends`).
struct TileCost {
    uint32_t bm, bn;
    float alone, full, outer, torn, ends;
};

// Fitted to products timed on the card, in us, k innermost unless stated:
//     bf16 (int8 alike, k twice as long)  256x256  256x128  128x128  128x64  64x64
//     4096 x 16384, k 2048                    239      298      297      -      -
//     4096 x  2048, k 4096                     88       62       68     88    100
//     2048 x  2048, k 4096                     89       52       46     41     51
//     the same, k outermost on both sides       -       60       54     43     57
//      512 x  8704, k 1536                      -       25       27     26     28
//      512 x  4352, k 1536                     38       24       21     18     16
//      128 x  4096, k 4096                      -       48       42     36     26 (15 split in four)
//      509 x  8662, k 1544: rows off the lines  44       29       29     35     36
//     4096 x  4096, k 4104: the same           114      138      155    215    275
//     fp32 4096 x 4096, k 2048                  -        -      500      -    507
// so 128 x 128 is never the best by much, and is left out.  The wide tiles and the smallest keep a
// third step of A on its way (product_tiles, PIPELINED); 128 x 64, three of which share a compute unit,
// is faster without: 2048 x 2048 with k outermost 43 us against 45.
template <class Op>
inline constexpr TileCost kTileCosts[4] = {
    {256, 256, 1.6f, 1.6f, 1.0f, 1.1f, 7.0f},
    {256, 128, 0.62f, 0.86f, 1.12f, 1.2f, 4.0f},
    {128, 64, 0.46f, 0.275f, 1.05f, 1.42f, 1.2f},
    {64, 64, 0.32f, 0.17f, 1.12f, 1.5f, 0.8f},
};
template <>
inline constexpr TileCost kTileCosts<OpF32>[4] = {
    {0, 0, 0, 0, 0, 0, 0},
    {0, 0, 0, 0, 0, 0, 0},
    {128, 64, 1.05f, 0.98f, 1.0f, 1.0f, 1.2f},
    {64, 64, 0.6f, 0.49f, 1.0f, 1.0f, 0.8f},
};

// The tile and split with the least time by these costs.  pitch: bytes from row to row of B.  Splitting
// adds the sums' way through memory and a launch; every part keeps 4 steps of k.  Operands that go through
// registers (!direct) take 2.2 times as long a step on a nearly empty chip.
template <class Op, bool GATED, bool OUTER>
inline Plan plan_product(uint32_t M, uint32_t N, uint32_t k, bool direct, uint64_t pitch) {
    const uint32_t units = 256;
    const uint32_t steps = (k * Op::kElem + kRowBytes - 1) / kRowBytes;
    Plan best{};
    float least = 0.f;
    for (const TileCost& c : kTileCosts<Op>) {
        if (c.bm == 0 || (c.bm == 256 && !direct)) continue;
        const uint32_t bn = GATED ? c.bn / 2 : c.bn;
        const uint32_t tiles = ((M + c.bm - 1) / c.bm) * ((N + bn - 1) / bn);
        const float full = c.full * (OUTER ? c.outer : pitch % 128 != 0 ? c.torn : 1.f);
        for (uint32_t splits = 1; splits <= 16; splits += splits < 4 ? 1 : 2) {
            if (splits > 1 && (steps / splits < 4 || tiles >= 2 * units)) break;
            const float depth = static_cast<float>((steps + splits - 1) / splits);
            const float rounds = static_cast<float>((tiles * splits + units - 1) / units);
            const float one = depth * c.alone * (direct ? 1.f : 2.2f) + c.ends, many = rounds * (depth * full + c.ends);
            float us = one > many ? one : many;
            const size_t bytes = splits > 1 ? size_t(splits) * tiles * c.bm * c.bn * 4 : 0;
            if (splits > 1) us += 2.f + static_cast<float>(bytes) * 2 / 5e6f;
            if (best.tiles == 0 || us < least) {
                best = Plan{c.bm, c.bn, tiles, splits, bytes};
                least = us;
            }
        }
    }
    return best;
}

// Whether an operand can go to LDS directly.
inline bool chunks16(const void* p, uint64_t pitch, uint64_t row_bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | pitch | row_bytes) & 15) == 0;
}

template <class Op, int BM, int BN, int WM, int WN, bool PIPELINED, bool GATED, bool A_OUTER, bool B_OUTER,
          bool DIRECT, class Done>
inline hipError_t launch_tiles(const Product& p, const Plan& plan, const Done& done, hipStream_t stream) {
    constexpr int threads = WM * WN * 64;
    product_tiles<Op, BM, BN, WM, WN, PIPELINED, GATED, A_OUTER, B_OUTER, DIRECT, Done>
        <<<plan.tiles * p.splits, threads, 0, stream>>>(p, done);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    product_join<Op, BM, BN, WM, WN, GATED, Done><<<plan.tiles * (BM / WM / 16), threads, 0, stream>>>(p, done);
    return hipGetLastError();
}

// Tiles of 64 with k innermost: whole steps with three slots for both operands (not PIPELINED) keep more of
// B on its way, half steps (PIPELINED) keep the matrix cores busier.  32 x 20480, k 4096 in bf16 (B from
// memory): 38 us and 50; 64 rows 45 and 53; 128 rows 60 and 59; 512 x 4352, k 1536: 17 and 16.  int8
// 128 x 10240, k 4096: 14 and 17; fp32 301 x 5568, k 1104: 42 and 44.  Five or eight slots are slower than three.
constexpr uint32_t kStreamedRows = 128;

template <class Op, bool GATED, bool A_OUTER, bool B_OUTER, class Done>
hipError_t launch_product(Product p, bool direct, void* workspace, const Done& done, hipStream_t stream) {
    const Plan plan = plan_product<Op, GATED, A_OUTER || B_OUTER>(p.M, p.N, p.k, direct, p.b_pitch);
    p.splits = plan.splits;
    p.partial = static_cast<float*>(workspace);
    if constexpr (Op::kElem != 4) {
        if (plan.bn == 256)
            return launch_tiles<Op, 256, 256, 2, 4, true, GATED, A_OUTER, B_OUTER, true>(p, plan, done, stream);
        if (plan.bn == 128)
            return launch_tiles<Op, 256, 128, 4, 2, true, GATED, A_OUTER, B_OUTER, true>(p, plan, done, stream);
    }
    if (plan.bm == 128)
        return direct ? launch_tiles<Op, 128, 64, 2, 2, false, GATED, A_OUTER, B_OUTER, true>(p, plan, done, stream)
                      : launch_tiles<Op, 128, 64, 2, 2, false, GATED, A_OUTER, B_OUTER, false>(p, plan, done, stream);
    if constexpr (!A_OUTER && !B_OUTER) {
        if (direct && (Op::kElem != 2 || p.M <= kStreamedRows))
            return launch_tiles<Op, 64, 64, 2, 2, false, GATED, A_OUTER, B_OUTER, true>(p, plan, done, stream);
    }
    constexpr bool halves = Op::kElem == 2 || A_OUTER || B_OUTER;
    return direct ? launch_tiles<Op, 64, 64, 2, 2, halves, GATED, A_OUTER, B_OUTER, true>(p, plan, done, stream)
                  : launch_tiles<Op, 64, 64, 2, 2, false, GATED, A_OUTER, B_OUTER, false>(p, plan, done, stream);
}

template <class Op, bool GATED, class Done>
hipError_t launch_few_rows(const Product& p, const Done& done, hipStream_t stream) {
    const uint64_t bytes = uint64_t(p.k) * Op::kElem;
    const bool al = chunks16(p.a, p.a_pitch, bytes) && chunks16(p.b[0], p.b_pitch, bytes) &&
                    (!GATED || chunks16(p.b[1], p.b_pitch, bytes));
    if (p.M == 1 && p.N <= kTokenOutputs) {
        const uint32_t groups = (p.N + 3) / 4;
        if (al) product_tokens<Op, 1, GATED, true, Done><<<groups, 256, 0, stream>>>(p, done);
        else product_tokens<Op, 1, GATED, false, Done><<<groups, 256, 0, stream>>>(p, done);
    } else if (p.M > 1 && p.M <= Op::kTokens) {
        if constexpr (Op::kTokens > 1) {
            const uint32_t groups = (p.N + 7) / 8;
            if (Op::kTokens == 4 || p.M <= 4) {
                if (al) product_tokens<Op, 4, GATED, true, Done><<<groups, 256, 0, stream>>>(p, done);
                else product_tokens<Op, 4, GATED, false, Done><<<groups, 256, 0, stream>>>(p, done);
            } else if constexpr (Op::kTokens == 8) {
                if (al) product_tokens<Op, 8, GATED, true, Done><<<groups, 256, 0, stream>>>(p, done);
                else product_tokens<Op, 8, GATED, false, Done><<<groups, 256, 0, stream>>>(p, done);
            }
        }
    } else if (const uint32_t tiles = (p.N + (GATED ? 31 : 63)) / (GATED ? 32 : 64);
               Op::kElem == 2 && al && tiles >= 256) {
        // A tile a compute unit or more: copies to LDS carry the weights faster than registers.  2 x 10240
        // rows of 4096 bf16: 38 us for 5 to 16 rows, product_rows 41 to 47; 2 x 16384 of 1024: 12 and 13 to
        // 15.  fp32 is the other way: 139 and 96 for 16 rows; int8 gives no tile a compute unit at
        // usual sizes, and splits need a workspace.
        Product q = p;
        q.splits = 1;
        return launch_tiles<Op, 64, 64, 2, 2, false, GATED, false, false, true>(q, Plan{64, 64, tiles, 1, 0}, done,
                                                                                stream);
    } else {
        const uint32_t groups = (p.N + 15) / 16;
        if (al) product_rows<Op, GATED, true, Done><<<groups, 512, 0, stream>>>(p, done);
        else product_rows<Op, GATED, false, Done><<<groups, 512, 0, stream>>>(p, done);
    }
    return hipGetLastError();
}

}  // namespace ltx3drope
