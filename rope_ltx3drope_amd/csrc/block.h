// The transformer-block operators: what the host side (block_api.cpp) hands to the kernel launchers
// (norm.hip, layer_norm.hip, ffn.hip, q8.hip, f8.hip).  Sizes fit in 32 bits unless they are size_t; offsets into tensors are formed in 64.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ltx3drope {

// Row tensors are [batch, rows, dim]; weights [dim]; gate, next_scale and next_shift [batch, dim].
// Vectors that a call leaves out are NULL.  Without per-sample vectors the host folds the batch into
// the rows (batch = 1).
struct NormForward {
    const void *y, *residual, *weight, *gate, *next_weight, *next_scale, *next_shift;
    void *r, *n;
    uint32_t batch, rows, dim;
    float eps, weight_offset, residual_scale;
    float square_scale;  // norm_square_scale(eps)
    bool has_y, post_norm, next_norm, param_f32;
    bool chunks;  // the vectors, and each sample's part of them, start on 16 bytes
};

struct NormBackward {
    const void *dr, *dn, *y, *r, *weight, *gate, *next_weight, *next_scale;
    void *dresidual, *dy, *dweight, *dgate, *dnext_weight, *dnext_scale, *dnext_shift;
    float* partial;  // [3][batch][parts][dim], NULL when no vector's gradient is asked for
    uint32_t batch, rows, dim;
    float eps, weight_offset, residual_scale;
    float square_scale;
    bool has_y, post_norm, next_norm, param_f32, chunks;
};

constexpr int64_t kNormMaxDim = 16384;    // 1024 threads of 16 elements hold one row

// A row's squares are added up times this power of two: 1 / kNormMaxDim, so that their sum stays in fp32's
// range wherever their mean does.  It is exact but where a scaled square falls below 2^-126; those are off
// by 2^-150 each, 2^-136 in the mean, which is less than fp32 resolves beside an eps of 2^-110 or more.
// Below that the squares are added up as they are.
inline float norm_square_scale(float eps) { return eps >= 0x1p-110f ? 0x1p-14f : 1.f; }
static_assert(kNormMaxDim == 1 << 14, "norm_square_scale takes a row's length out of its sum");
constexpr int64_t kNormMaxBatch = 65535;  // one grid row a sample

// vec: every row pointer is 16-byte aligned and a row is whole 16-byte vectors.
hipError_t launch_norm_forward(const NormForward& p, bool f32, bool vec, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackward& p, bool f32, bool vec, hipStream_t stream);
size_t norm_backward_workspace(uint32_t batch, uint32_t rows, uint32_t dim);

// The layer norms (layer_norm.hip), in the same shapes: r is the norm's input, gate, scale and shift are
// [batch, dim], weight and bias [dim].
struct LayerNormForward {
    const void *y, *residual, *gate, *weight, *bias, *scale, *shift;
    void *r, *n;
    uint32_t batch, rows, dim;
    float eps, square_scale;
    bool after, param_f32, chunks;
};

struct LayerNormBackward {
    const void *dr, *dn, *y, *r, *gate, *weight, *bias, *scale;
    void *dresidual, *dy, *dgate, *dweight, *dbias, *dscale, *dshift;
    float* partial;  // [3][batch][parts][dim], NULL when no vector's gradient is asked for
    uint32_t batch, rows, dim;
    float eps, square_scale;
    bool after, param_f32, chunks;
};

// The backward's workspace is norm_backward_workspace's.
hipError_t launch_layer_norm_forward(const LayerNormForward& p, bool f32, bool vec, hipStream_t stream);
hipError_t launch_layer_norm_backward(const LayerNormBackward& p, bool f32, bool vec, hipStream_t stream);

// The gated feed-forward block (ffn.hip).  x [tokens, dim], weights [hidden, dim], h, g, u and dh
// [tokens, hidden], g and u in fp32.  activation: LTX3DROPE_ACT_*.
struct FfnProblem {
    const void *x, *w_gate, *w_up;
    void* h;
    float *g, *u;  // both or neither
    void* workspace;
    uint32_t tokens, dim, hidden;
    int activation;
};
struct FfnBackwardProblem {
    const void *dh, *x, *w_gate, *w_up;
    const float *g, *u;
    void *dx, *dw_gate, *dw_up;  // dx may be NULL; the weights' both or neither
    void* workspace;
    uint32_t tokens, dim, hidden;
    int activation;
};
constexpr int64_t kFfnMaxSize = int64_t(1) << 21;  // a tile of 256 rows of 2 * hidden fp32 stays within 2^31 bytes
constexpr int64_t kMaxTiles = int64_t(1) << 23;    // 64 x 32 output tiles of a launch of 256 threads each
size_t ffn_workspace(const FfnProblem& p, bool f32);
size_t ffn_backward_workspace(const FfnBackwardProblem& p, bool f32);
hipError_t launch_ffn(const FfnProblem& p, bool f32, hipStream_t stream);
hipError_t launch_ffn_backward(const FfnBackwardProblem& p, bool f32, hipStream_t stream);

// The 8-bit linear layer (q8.hip): a [tokens, dim] and b [out, dim] int8, y [tokens, out].
struct Q8Problem {
    const void *a, *b;
    const float *a_scale, *b_scale, *bias;  // [tokens], [out], [out] or NULL
    void* y;
    void* workspace;
    uint32_t tokens, dim, out;
};
constexpr int64_t kQ8MaxDim = 131071;  // (2^31 - 1) / 2^14: the sums stay within 32-bit integers
size_t q8_workspace(const Q8Problem& p);
hipError_t launch_q8(const Q8Problem& p, bool f32, hipStream_t stream);
hipError_t launch_q8_quantize(const void* x, void* q, float* scale, uint32_t rows, uint32_t dim, bool f32,
                              hipStream_t stream);

// The linear layer in 8-bit floating point (f8.hip): a [tokens, dim] and b [out, dim] e4m3, their rows a_pitch and
// b_pitch bytes apart, y [tokens, out]; a scale for 128 of k: a_scale [tokens, blocks], b_scale [out, blocks]
// (b_rows) or [out / 128, blocks], with strides in numbers.
struct F8Problem {
    const void *a, *b;
    const float *a_scale, *b_scale, *bias;
    void* y;
    void* workspace;
    uint64_t a_pitch, b_pitch, a_scale_block, b_scale_block;
    uint32_t a_scale_row, b_scale_row;
    uint32_t tokens, dim, out;
    bool b_rows;
};
constexpr int64_t kF8MaxDim = int64_t(1) << 21;
constexpr int64_t kF8MaxPitch = int64_t(1) << 22;     // 256 rows of this many bytes and ...
constexpr int64_t kF8MaxScaleRow = int64_t(1) << 20;  // ... of this many scales stay within 2^31
size_t f8_workspace(const F8Problem& p);
hipError_t launch_f8(const F8Problem& p, bool f32, hipStream_t stream);

// x [rows, dim] to e4m3 with scales for 128 of a row or (blocks) 128 x 128; q_turned [dim, rows], its rows
// turned_pitch bytes apart, may be NULL.
struct F8Quantize {
    const void* x;
    void *q, *q_turned;
    float *scale, *scale_turned;
    uint64_t turned_pitch;
    uint64_t scale_row, scale_block, turned_row, turned_block;  // strides in numbers
    uint32_t rows, dim;
    bool blocks;
    bool turned_chunks;  // q_turned starts on 16 bytes and so does each of its rows, with room for whole pieces
};
hipError_t launch_f8_quantize(const F8Quantize& p, bool f32, hipStream_t stream);

}  // namespace ltx3drope
