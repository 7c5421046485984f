// The transformer-block operators: what the host side (block_api.cpp) hands to the kernel launchers
// (norm.hip, ffn.hip, q8.hip).  Sizes fit in 32 bits unless they are size_t; offsets into tensors are formed in 64.
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

}  // namespace ltx3drope
