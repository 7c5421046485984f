// The transformer-block operators: what the host side (block_api.cpp) hands to the kernel launchers
// (norm.hip).  Sizes fit in 32 bits unless they are size_t; offsets into tensors are formed in 64.
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
    bool has_y, post_norm, next_norm, param_f32;
};

struct NormBackward {
    const void *dr, *dn, *y, *r, *weight, *gate, *next_weight, *next_scale;
    void *dresidual, *dy, *dweight, *dgate, *dnext_weight, *dnext_scale, *dnext_shift;
    float* partial;  // [3][batch][parts][dim], NULL when no vector's gradient is asked for
    uint32_t batch, rows, dim;
    float eps, weight_offset, residual_scale;
    bool has_y, post_norm, next_norm, param_f32;
};

constexpr int64_t kNormMaxDim = 16384;    // 1024 threads of 16 elements hold one row
constexpr int64_t kNormMaxBatch = 65535;  // one grid row a sample

// vec: every row pointer is 16-byte aligned and a row is whole 16-byte vectors.
hipError_t launch_norm_forward(const NormForward& p, bool f32, bool vec, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackward& p, bool f32, bool vec, hipStream_t stream);
size_t norm_backward_workspace(uint32_t batch, uint32_t rows, uint32_t dim);

}  // namespace ltx3drope
