// C ABI of the transformer-block operators: argument checks and dispatch.
#include <cmath>
#include <cstring>

#include "block.h"
#include "internal.h"
#include "spans.h"

namespace ltx3drope {
namespace {

bool flag(int32_t v) { return v == 0 || v == 1; }

size_t elem(int dtype) { return dtype == LTX3DROPE_DTYPE_F32 ? 4 : 2; }

// The sizes and types that the norms share: OK, or the reason of a refusal.
template <class Call>
int check_rows(const Call& c, bool per_sample) {
    if ((c.dtype != LTX3DROPE_DTYPE_F32 && c.dtype != LTX3DROPE_DTYPE_BF16) ||
        (c.param_dtype != LTX3DROPE_DTYPE_F32 && c.param_dtype != c.dtype))
        return LTX3DROPE_REASON_DTYPE;
    if (c.dim <= 0 || c.batch < 0 || c.rows < 0) return LTX3DROPE_REASON_NONPOSITIVE_DIM;
    const int64_t lim = int64_t(1) << 31;
    if (c.dim > kNormMaxDim || c.batch >= lim || c.rows >= lim || (c.rows != 0 && c.batch > (lim - 1) / c.rows) ||
        (per_sample && c.batch > kNormMaxBatch))
        return LTX3DROPE_REASON_TOO_LARGE;
    return LTX3DROPE_REASON_OK;
}

// The scalars that both directions of the norm share: a status, and for E_UNSUPPORTED the reason.
template <class Call>
int check_norm(const Call& c, bool per_sample, int* why) {
    if (!flag(c.after) || !flag(c.post_norm) || !flag(c.next_norm) || c.reserved != 0 || !std::isfinite(c.eps) ||
        c.eps <= 0.f || !std::isfinite(c.weight_offset) || !std::isfinite(c.residual_scale))
        return LTX3DROPE_E_INVALID;
    if (!c.after && (c.post_norm || !c.next_norm || c.residual_scale != 1.f || c.y || c.weight || c.gate))
        return LTX3DROPE_E_INVALID;
    *why = check_rows(c, per_sample);
    return *why == LTX3DROPE_REASON_OK ? LTX3DROPE_OK : LTX3DROPE_E_UNSUPPORTED;
}

bool norm_per_sample(const ltx3drope_norm_backward_t& c) {
    return c.gate || c.next_scale || c.dgate || c.dnext_scale || c.dnext_shift;
}

size_t norm_workspace(const ltx3drope_norm_backward_t& c) {
    if (!c.dweight && !c.dgate && !c.dnext_weight && !c.dnext_scale && !c.dnext_shift) return 0;
    if (c.batch == 0 || c.rows == 0) return 0;
    const bool per_sample = norm_per_sample(c);
    return norm_backward_workspace(static_cast<uint32_t>(per_sample ? c.batch : 1),
                                   static_cast<uint32_t>(per_sample ? c.rows : c.batch * c.rows),
                                   static_cast<uint32_t>(c.dim));
}

// The layer norms' scalars, both directions.
template <class Call>
int check_layer_norm(const Call& c, bool per_sample, int* why) {
    if (!flag(c.after) || c.reserved != 0 || !std::isfinite(c.eps) || c.eps <= 0.f) return LTX3DROPE_E_INVALID;
    if (!c.after && (c.y || c.gate)) return LTX3DROPE_E_INVALID;
    *why = check_rows(c, per_sample);
    return *why == LTX3DROPE_REASON_OK ? LTX3DROPE_OK : LTX3DROPE_E_UNSUPPORTED;
}

bool layer_norm_per_sample(const ltx3drope_layer_norm_backward_t& c) {
    return c.gate || c.scale || c.dgate || c.dscale || c.dshift;
}

size_t layer_norm_workspace(const ltx3drope_layer_norm_backward_t& c) {
    if (!c.dgate && !c.dweight && !c.dbias && !c.dscale && !c.dshift) return 0;
    if (c.batch == 0 || c.rows == 0) return 0;
    const bool per_sample = layer_norm_per_sample(c);
    return norm_backward_workspace(static_cast<uint32_t>(per_sample ? c.batch : 1),
                                   static_cast<uint32_t>(per_sample ? c.rows : c.batch * c.rows),
                                   static_cast<uint32_t>(c.dim));
}

// A product's launch: 64 x 32 tiles (the smallest) of 256 threads stay below 2^32 threads.  The kernels
// without tiles take 64 threads an output up to 2^25 outputs a token and 32 above, of fewer than 2^26.
bool too_many_tiles(int64_t M, int64_t N) { return (M / 64 + 1) * (N / 32 + 1) > kMaxTiles; }

// The feed-forward block's scalars, both directions.
template <class Call>
int check_ffn(const Call& c, int* why) {
    if (c.activation < LTX3DROPE_ACT_SILU || c.activation > LTX3DROPE_ACT_GELU_TANH) return LTX3DROPE_E_INVALID;
    if (c.dtype != LTX3DROPE_DTYPE_F32 && c.dtype != LTX3DROPE_DTYPE_BF16) {
        *why = LTX3DROPE_REASON_DTYPE;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    if (c.dim <= 0 || c.tokens < 0 || c.hidden < 0) {
        *why = LTX3DROPE_REASON_NONPOSITIVE_DIM;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    if (c.tokens >= kFfnMaxSize || c.dim >= kFfnMaxSize || c.hidden >= kFfnMaxSize / 2 ||
        too_many_tiles(c.tokens, c.hidden) || too_many_tiles(c.tokens, c.dim) || too_many_tiles(2 * c.hidden, c.dim)) {
        *why = LTX3DROPE_REASON_TOO_LARGE;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    return LTX3DROPE_OK;
}

FfnProblem ffn_problem(const ltx3drope_gated_ffn_t& c) {
    FfnProblem p;
    p.x = c.x;
    p.w_gate = c.w_gate;
    p.w_up = c.w_up;
    p.h = c.h;
    p.g = c.g;
    p.u = c.u;
    p.workspace = c.workspace;
    p.tokens = static_cast<uint32_t>(c.tokens);
    p.dim = static_cast<uint32_t>(c.dim);
    p.hidden = static_cast<uint32_t>(c.hidden);
    p.activation = c.activation;
    return p;
}

FfnBackwardProblem ffn_problem(const ltx3drope_gated_ffn_backward_t& c) {
    FfnBackwardProblem p;
    p.dh = c.dh;
    p.x = c.x;
    p.w_gate = c.w_gate;
    p.w_up = c.w_up;
    p.g = c.g;
    p.u = c.u;
    p.dx = c.dx;
    p.dw_gate = c.dw_gate;
    p.dw_up = c.dw_up;
    p.workspace = c.workspace;
    p.tokens = static_cast<uint32_t>(c.tokens);
    p.dim = static_cast<uint32_t>(c.dim);
    p.hidden = static_cast<uint32_t>(c.hidden);
    p.activation = c.activation;
    return p;
}

int check_q8(const ltx3drope_q8_matmul_t& c, int* why) {
    if (c.reserved != 0) return LTX3DROPE_E_INVALID;
    if (c.dtype != LTX3DROPE_DTYPE_F32 && c.dtype != LTX3DROPE_DTYPE_BF16) {
        *why = LTX3DROPE_REASON_DTYPE;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    if (c.dim <= 0 || c.tokens < 0 || c.out < 0) {
        *why = LTX3DROPE_REASON_NONPOSITIVE_DIM;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    const int64_t lim = int64_t(1) << 26;
    if (c.dim > kQ8MaxDim || c.tokens >= lim || c.out >= lim || too_many_tiles(c.tokens, c.out)) {
        *why = LTX3DROPE_REASON_TOO_LARGE;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    return LTX3DROPE_OK;
}

Q8Problem q8_problem(const ltx3drope_q8_matmul_t& c) {
    Q8Problem p;
    p.a = c.a;
    p.b = c.b;
    p.a_scale = c.a_scale;
    p.b_scale = c.b_scale;
    p.bias = c.bias;
    p.y = c.y;
    p.workspace = c.workspace;
    p.tokens = static_cast<uint32_t>(c.tokens);
    p.dim = static_cast<uint32_t>(c.dim);
    p.out = static_cast<uint32_t>(c.out);
    return p;
}

// Bytes that rows x blocks scales with these strides (row, block) reach over; the callers' limits keep it below
// 2^61.
constexpr int64_t kF8MaxScaleBlock = int64_t(1) << 31;
size_t scale_bytes(size_t rows, size_t blocks, const int64_t (&strides)[2]) {
    return ((rows - 1) * static_cast<size_t>(strides[0]) + (blocks - 1) * static_cast<size_t>(strides[1]) + 1) * 4;
}

// Whether no two of rows x blocks scales share a place.
bool distinct_scales(int64_t rows, int64_t blocks, const int64_t (&s)[2]) {
    if (rows > 1 && blocks > 1)
        return s[0] > 0 && s[1] > 0 && (s[0] > (blocks - 1) * s[1] || s[1] > (rows - 1) * s[0]);
    return (rows <= 1 || s[0] > 0) && (blocks <= 1 || s[1] > 0);
}

int check_f8(const ltx3drope_f8_matmul_t& c, int* why) {
    if (!flag(c.b_rows)) return LTX3DROPE_E_INVALID;
    if (c.dtype != LTX3DROPE_DTYPE_F32 && c.dtype != LTX3DROPE_DTYPE_BF16) {
        *why = LTX3DROPE_REASON_DTYPE;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    if (c.dim <= 0 || c.tokens < 0 || c.out < 0) {
        *why = LTX3DROPE_REASON_NONPOSITIVE_DIM;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    if (c.a_pitch < c.dim || c.b_pitch < c.dim) return LTX3DROPE_E_INVALID;
    for (const int64_t(*v)[2] : {&c.a_scale_strides, &c.b_scale_strides})
        if ((*v)[0] < 0 || (*v)[1] < 0) return LTX3DROPE_E_INVALID;
    const int64_t lim = int64_t(1) << 26;
    if (c.dim >= kF8MaxDim || c.a_pitch >= kF8MaxPitch || c.b_pitch >= kF8MaxPitch || c.tokens >= lim || c.out >= lim ||
        c.a_scale_strides[0] >= kF8MaxScaleRow || c.b_scale_strides[0] >= kF8MaxScaleRow ||
        c.a_scale_strides[1] >= kF8MaxScaleBlock || c.b_scale_strides[1] >= kF8MaxScaleBlock ||
        too_many_tiles(c.tokens, c.out)) {
        *why = LTX3DROPE_REASON_TOO_LARGE;
        return LTX3DROPE_E_UNSUPPORTED;
    }
    return LTX3DROPE_OK;
}

F8Problem f8_problem(const ltx3drope_f8_matmul_t& c) {
    F8Problem p;
    p.a = c.a;
    p.b = c.b;
    p.a_scale = c.a_scale;
    p.b_scale = c.b_scale;
    p.bias = c.bias;
    p.y = c.y;
    p.workspace = c.workspace;
    p.a_pitch = static_cast<uint64_t>(c.a_pitch);
    p.b_pitch = static_cast<uint64_t>(c.b_pitch);
    p.a_scale_row = static_cast<uint32_t>(c.a_scale_strides[0]);
    p.a_scale_block = static_cast<uint64_t>(c.a_scale_strides[1]);
    p.b_scale_row = static_cast<uint32_t>(c.b_scale_strides[0]);
    p.b_scale_block = static_cast<uint64_t>(c.b_scale_strides[1]);
    p.tokens = static_cast<uint32_t>(c.tokens);
    p.dim = static_cast<uint32_t>(c.dim);
    p.out = static_cast<uint32_t>(c.out);
    p.b_rows = c.b_rows != 0;
    return p;
}

}  // namespace
}  // namespace ltx3drope

using namespace ltx3drope;

extern "C" {

int ltx3drope_norm(const ltx3drope_norm_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_norm_t& c = *call;
    const bool per_sample = c.gate || c.next_scale || c.next_shift;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_norm(c, per_sample, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if ((!c.after && c.r) || (!c.next_norm && (c.n || c.next_weight || c.next_scale || c.next_shift)))
        return LTX3DROPE_E_INVALID;
    if (c.batch == 0 || c.rows == 0) return LTX3DROPE_OK;
    if (!c.residual || (c.after && (!c.y || !c.r)) || (c.next_norm && !c.n))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t es = elem(c.dtype), ps = elem(c.param_dtype);
    const size_t row = static_cast<size_t>(c.batch * c.rows) * static_cast<size_t>(c.dim) * es;
    const size_t vec = static_cast<size_t>(c.dim) * ps, vecs = vec * static_cast<size_t>(c.batch);
    Spans t;
    t.add(c.residual, row, es, Role::RowIn);
    t.add(c.y, row, es, Role::RowIn);
    t.add(c.r, row, es, Role::RowOut);
    t.add(c.n, row, es, Role::RowOut);
    t.add(c.weight, vec, ps, Role::Param);
    t.add(c.next_weight, vec, ps, Role::Param);
    t.add(c.gate, vecs, ps, Role::Param);
    t.add(c.next_scale, vecs, ps, Role::Param);
    t.add(c.next_shift, vecs, ps, Role::Param);
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    NormForward p;
    p.y = c.y;
    p.residual = c.residual;
    p.weight = c.weight;
    p.gate = c.gate;
    p.next_weight = c.next_weight;
    p.next_scale = c.next_scale;
    p.next_shift = c.next_shift;
    p.r = c.r;
    p.n = c.n;
    p.batch = static_cast<uint32_t>(per_sample ? c.batch : 1);
    p.rows = static_cast<uint32_t>(per_sample ? c.rows : c.batch * c.rows);
    p.dim = static_cast<uint32_t>(c.dim);
    p.eps = c.eps;
    p.weight_offset = c.weight_offset;
    p.residual_scale = c.residual_scale;
    p.square_scale = norm_square_scale(c.eps);
    p.has_y = c.after != 0;
    p.post_norm = c.post_norm != 0;
    p.next_norm = c.next_norm != 0;
    p.param_f32 = c.param_dtype == LTX3DROPE_DTYPE_F32;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32;
    const bool vectors = aligned16(t, {Role::RowIn, Role::RowOut}) && (static_cast<size_t>(c.dim) * es) % 16 == 0;
    p.chunks = aligned16(t, {Role::Param}) && vec % 16 == 0;
    DeviceGuard guard(device);
    if (launch_norm_forward(p, f32, vectors, static_cast<hipStream_t>(stream)) != hipSuccess) return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int64_t ltx3drope_norm_backward_workspace(const ltx3drope_norm_backward_t* call) {
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_norm(*call, norm_per_sample(*call), &why);
    return st == LTX3DROPE_OK ? static_cast<int64_t>(norm_workspace(*call)) : st;
}

int ltx3drope_norm_backward(const ltx3drope_norm_backward_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_norm_backward_t& c = *call;
    const bool per_sample = norm_per_sample(c);
    int why = LTX3DROPE_REASON_OK;
    const int st = check_norm(c, per_sample, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    const bool need_y = c.after && (c.post_norm || c.gate || c.weight);
    if ((!c.after && (c.dy || c.dweight || c.dgate)) || (c.dweight && !c.weight) || (c.dgate && !c.gate) ||
        (c.dnext_weight && !c.next_weight) || (c.dnext_scale && !c.next_scale) ||
        (!c.next_norm && (c.dn || c.next_weight || c.next_scale || c.dnext_shift)))
        return LTX3DROPE_E_INVALID;
    const size_t ws = norm_workspace(c);
    if (c.workspace_bytes < 0 || static_cast<size_t>(c.workspace_bytes) < ws) return LTX3DROPE_E_INVALID;
    const bool empty = c.batch == 0 || c.rows == 0;
    if (!empty && (!c.dresidual || (c.after && !c.dy) || (need_y && !c.y) || (c.next_norm && (!c.dn || !c.r)) ||
                   (ws != 0 && !c.workspace)))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t es = elem(c.dtype), ps = elem(c.param_dtype);
    const size_t row = static_cast<size_t>(c.batch * c.rows) * static_cast<size_t>(c.dim) * es;
    const size_t vec = static_cast<size_t>(c.dim) * ps, vecs = vec * static_cast<size_t>(c.batch);
    Spans t;
    t.add(c.dr, row, es, Role::RowIn);
    t.add(c.dn, row, es, Role::RowIn);
    if (need_y) t.add(c.y, row, es, Role::RowIn);
    if (c.next_norm) t.add(c.r, row, es, Role::RowIn);
    t.add(c.dresidual, row, es, Role::RowOut);
    t.add(c.dy, row, es, Role::RowOut);
    if (!empty) {
        t.add(c.weight, vec, ps, Role::Param);
        t.add(c.next_weight, vec, ps, Role::Param);
        t.add(c.gate, vecs, ps, Role::Param);
        t.add(c.next_scale, vecs, ps, Role::Param);
    }
    t.add(c.dweight, vec, ps, Role::ParamOut);
    t.add(c.dnext_weight, vec, ps, Role::ParamOut);
    t.add(c.dgate, vecs, ps, Role::ParamOut);
    t.add(c.dnext_scale, vecs, ps, Role::ParamOut);
    t.add(c.dnext_shift, vecs, ps, Role::ParamOut);
    if (ws != 0) t.add(c.workspace, ws, 16, Role::Scratch);
    if (t.n == 0) return LTX3DROPE_OK;  // an empty call without a vector's gradient
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    NormBackward p;
    p.dr = c.dr;
    p.dn = c.dn;
    p.y = need_y ? c.y : nullptr;
    p.r = c.r;
    p.weight = c.weight;
    p.gate = c.gate;
    p.next_weight = c.next_weight;
    p.next_scale = c.next_scale;
    p.dresidual = c.dresidual;
    p.dy = c.dy;
    p.dweight = c.dweight;
    p.dgate = c.dgate;
    p.dnext_weight = c.dnext_weight;
    p.dnext_scale = c.dnext_scale;
    p.dnext_shift = c.dnext_shift;
    p.partial = ws != 0 ? static_cast<float*>(c.workspace) : nullptr;
    p.batch = static_cast<uint32_t>(per_sample ? c.batch : 1);
    p.rows = static_cast<uint32_t>(per_sample ? c.rows : c.batch * c.rows);
    p.dim = static_cast<uint32_t>(c.dim);
    p.eps = c.eps;
    p.weight_offset = c.weight_offset;
    p.residual_scale = c.residual_scale;
    p.square_scale = norm_square_scale(c.eps);
    p.has_y = c.after != 0;
    p.post_norm = c.post_norm != 0;
    p.next_norm = c.next_norm != 0;
    p.param_f32 = c.param_dtype == LTX3DROPE_DTYPE_F32;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32;
    const bool vectors = aligned16(t, {Role::RowIn, Role::RowOut}) && (static_cast<size_t>(c.dim) * es) % 16 == 0;
    p.chunks = aligned16(t, {Role::Param}) && vec % 16 == 0;
    DeviceGuard guard(device);
    if (launch_norm_backward(p, f32, vectors, static_cast<hipStream_t>(stream)) != hipSuccess) return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int ltx3drope_layer_norm(const ltx3drope_layer_norm_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_layer_norm_t& c = *call;
    const bool per_sample = c.gate || c.scale || c.shift;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_layer_norm(c, per_sample, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if (!c.after && c.r) return LTX3DROPE_E_INVALID;
    if (c.batch == 0 || c.rows == 0) return LTX3DROPE_OK;
    if (!c.residual || !c.n || (c.after && (!c.y || !c.r))) return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t es = elem(c.dtype), ps = elem(c.param_dtype);
    const size_t row = static_cast<size_t>(c.batch * c.rows) * static_cast<size_t>(c.dim) * es;
    const size_t vec = static_cast<size_t>(c.dim) * ps, vecs = vec * static_cast<size_t>(c.batch);
    Spans t;
    t.add(c.residual, row, es, Role::RowIn);
    t.add(c.y, row, es, Role::RowIn);
    t.add(c.r, row, es, Role::RowOut);
    t.add(c.n, row, es, Role::RowOut);
    t.add(c.weight, vec, ps, Role::Param);
    t.add(c.bias, vec, ps, Role::Param);
    t.add(c.gate, vecs, ps, Role::Param);
    t.add(c.scale, vecs, ps, Role::Param);
    t.add(c.shift, vecs, ps, Role::Param);
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    LayerNormForward p;
    p.y = c.y;
    p.residual = c.residual;
    p.gate = c.gate;
    p.weight = c.weight;
    p.bias = c.bias;
    p.scale = c.scale;
    p.shift = c.shift;
    p.r = c.r;
    p.n = c.n;
    p.batch = static_cast<uint32_t>(per_sample ? c.batch : 1);
    p.rows = static_cast<uint32_t>(per_sample ? c.rows : c.batch * c.rows);
    p.dim = static_cast<uint32_t>(c.dim);
    p.eps = c.eps;
    p.square_scale = norm_square_scale(c.eps);
    p.after = c.after != 0;
    p.param_f32 = c.param_dtype == LTX3DROPE_DTYPE_F32;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32;
    const bool vectors = aligned16(t, {Role::RowIn, Role::RowOut}) && (static_cast<size_t>(c.dim) * es) % 16 == 0;
    p.chunks = aligned16(t, {Role::Param}) && vec % 16 == 0;
    DeviceGuard guard(device);
    if (launch_layer_norm_forward(p, f32, vectors, static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int64_t ltx3drope_layer_norm_backward_workspace(const ltx3drope_layer_norm_backward_t* call) {
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_layer_norm(*call, layer_norm_per_sample(*call), &why);
    return st == LTX3DROPE_OK ? static_cast<int64_t>(layer_norm_workspace(*call)) : st;
}

int ltx3drope_layer_norm_backward(const ltx3drope_layer_norm_backward_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_layer_norm_backward_t& c = *call;
    const bool per_sample = layer_norm_per_sample(c);
    int why = LTX3DROPE_REASON_OK;
    const int st = check_layer_norm(c, per_sample, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if ((!c.after && (c.dy || c.dgate)) || (c.dgate && !c.gate) || (c.dweight && !c.weight) || (c.dscale && !c.scale))
        return LTX3DROPE_E_INVALID;
    const size_t ws = layer_norm_workspace(c);
    if (c.workspace_bytes < 0 || static_cast<size_t>(c.workspace_bytes) < ws) return LTX3DROPE_E_INVALID;
    const bool empty = c.batch == 0 || c.rows == 0, need_y = c.dgate != nullptr;
    if (!empty && (!c.dresidual || !c.dn || !c.r || (c.after && !c.dy) || (need_y && !c.y) || (ws != 0 && !c.workspace)))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t es = elem(c.dtype), ps = elem(c.param_dtype);
    const size_t row = static_cast<size_t>(c.batch * c.rows) * static_cast<size_t>(c.dim) * es;
    const size_t vec = static_cast<size_t>(c.dim) * ps, vecs = vec * static_cast<size_t>(c.batch);
    Spans t;
    t.add(c.dr, row, es, Role::RowIn);
    t.add(c.dn, row, es, Role::RowIn);
    if (need_y) t.add(c.y, row, es, Role::RowIn);
    t.add(c.r, row, es, Role::RowIn);
    t.add(c.dresidual, row, es, Role::RowOut);
    t.add(c.dy, row, es, Role::RowOut);
    if (!empty) {
        t.add(c.weight, vec, ps, Role::Param);
        t.add(c.bias, vec, ps, Role::Param);
        t.add(c.gate, vecs, ps, Role::Param);
        t.add(c.scale, vecs, ps, Role::Param);
    }
    t.add(c.dweight, vec, ps, Role::ParamOut);
    t.add(c.dbias, vec, ps, Role::ParamOut);
    t.add(c.dgate, vecs, ps, Role::ParamOut);
    t.add(c.dscale, vecs, ps, Role::ParamOut);
    t.add(c.dshift, vecs, ps, Role::ParamOut);
    if (ws != 0) t.add(c.workspace, ws, 16, Role::Scratch);
    if (t.n == 0) return LTX3DROPE_OK;  // an empty call without a vector's gradient
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    LayerNormBackward p;
    p.dr = c.dr;
    p.dn = c.dn;
    p.y = need_y ? c.y : nullptr;
    p.r = c.r;
    p.gate = c.gate;
    p.weight = c.weight;
    p.bias = c.bias;
    p.scale = c.scale;
    p.dresidual = c.dresidual;
    p.dy = c.dy;
    p.dgate = c.dgate;
    p.dweight = c.dweight;
    p.dbias = c.dbias;
    p.dscale = c.dscale;
    p.dshift = c.dshift;
    p.partial = ws != 0 ? static_cast<float*>(c.workspace) : nullptr;
    p.batch = static_cast<uint32_t>(per_sample ? c.batch : 1);
    p.rows = static_cast<uint32_t>(per_sample ? c.rows : c.batch * c.rows);
    p.dim = static_cast<uint32_t>(c.dim);
    p.eps = c.eps;
    p.square_scale = norm_square_scale(c.eps);
    p.after = c.after != 0;
    p.param_f32 = c.param_dtype == LTX3DROPE_DTYPE_F32;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32;
    const bool vectors = aligned16(t, {Role::RowIn, Role::RowOut}) && (static_cast<size_t>(c.dim) * es) % 16 == 0;
    p.chunks = aligned16(t, {Role::Param}) && vec % 16 == 0;
    DeviceGuard guard(device);
    if (launch_layer_norm_backward(p, f32, vectors, static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int64_t ltx3drope_gated_ffn_workspace(const ltx3drope_gated_ffn_t* call) {
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_ffn(*call, &why);
    if (st != LTX3DROPE_OK) return st;
    if (call->tokens == 0 || call->hidden == 0) return 0;
    return static_cast<int64_t>(ffn_workspace(ffn_problem(*call), call->dtype == LTX3DROPE_DTYPE_F32));
}

int ltx3drope_gated_ffn(const ltx3drope_gated_ffn_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_gated_ffn_t& c = *call;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_ffn(c, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if ((c.g == nullptr) != (c.u == nullptr)) return LTX3DROPE_E_INVALID;
    if (c.tokens == 0 || c.hidden == 0) return LTX3DROPE_OK;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32;
    const FfnProblem p = ffn_problem(c);
    const size_t ws = ffn_workspace(p, f32);
    if (c.workspace_bytes < 0 || static_cast<size_t>(c.workspace_bytes) < ws) return LTX3DROPE_E_INVALID;
    if (!c.x || !c.w_gate || !c.w_up || !c.h || (ws != 0 && !c.workspace))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t es = elem(c.dtype), M = p.tokens, D = p.dim, F = p.hidden;
    Spans t;
    t.add(c.x, M * D * es, es, Role::Param);
    t.add(c.w_gate, F * D * es, es, Role::Param);
    t.add(c.w_up, F * D * es, es, Role::Param);
    t.add(c.h, M * F * es, es, Role::ParamOut);
    for (const void* o : {c.g, c.u}) t.add(o, M * F * 4, 4, Role::ParamOut);
    if (ws != 0) t.add(c.workspace, ws, 16, Role::Scratch);
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    DeviceGuard guard(device);
    if (launch_ffn(p, f32, static_cast<hipStream_t>(stream)) != hipSuccess) return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int64_t ltx3drope_gated_ffn_backward_workspace(const ltx3drope_gated_ffn_backward_t* call) {
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_ffn(*call, &why);
    if (st != LTX3DROPE_OK) return st;
    if (call->tokens == 0 || call->hidden == 0) return 0;
    return static_cast<int64_t>(ffn_backward_workspace(ffn_problem(*call), call->dtype == LTX3DROPE_DTYPE_F32));
}

int ltx3drope_gated_ffn_backward(const ltx3drope_gated_ffn_backward_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_gated_ffn_backward_t& c = *call;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_ffn(c, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if ((c.dw_gate == nullptr) != (c.dw_up == nullptr)) return LTX3DROPE_E_INVALID;
    if (c.dx == nullptr && c.dw_gate == nullptr) return LTX3DROPE_OK;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32, empty = c.tokens == 0 || c.hidden == 0;
    const FfnBackwardProblem p = ffn_problem(c);
    const size_t ws = empty ? 0 : ffn_backward_workspace(p, f32);
    if (c.workspace_bytes < 0 || static_cast<size_t>(c.workspace_bytes) < ws) return LTX3DROPE_E_INVALID;
    const size_t es = elem(c.dtype), M = p.tokens, D = p.dim, F = p.hidden;
    if (!empty && (!c.dh || !c.g || !c.u || (c.dw_gate && !c.x) || (c.dx && (!c.w_gate || !c.w_up)) || !c.workspace))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    Spans t;
    if (!empty) {
        t.add(c.dh, M * F * es, es, Role::Param);
        for (const void* i : {c.g, c.u}) t.add(i, M * F * 4, 4, Role::Param);
        if (c.dw_gate) t.add(c.x, M * D * es, es, Role::Param);
        if (c.dx)
            for (const void* i : {c.w_gate, c.w_up}) t.add(i, F * D * es, es, Role::Param);
        t.add(c.workspace, ws, 16, Role::Scratch);
    }
    t.add(c.dx, M * D * es, es, Role::ParamOut);
    t.add(c.dw_gate, F * D * es, es, Role::ParamOut);
    t.add(c.dw_up, F * D * es, es, Role::ParamOut);
    if (t.n == 0) return LTX3DROPE_OK;
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    DeviceGuard guard(device);
    if (launch_ffn_backward(p, f32, static_cast<hipStream_t>(stream)) != hipSuccess) return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int ltx3drope_q8_quantize(int dtype, int64_t rows, int64_t dim, const void* x, void* q, float* scale, void* stream,
                          int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (dtype != LTX3DROPE_DTYPE_F32 && dtype != LTX3DROPE_DTYPE_BF16) return refuse(LTX3DROPE_REASON_DTYPE, reason);
    if (dim <= 0 || rows < 0) return refuse(LTX3DROPE_REASON_NONPOSITIVE_DIM, reason);
    const int64_t lim = int64_t(1) << 31;
    if (dim >= lim || rows >= lim || (rows != 0 && dim > ((int64_t(1) << 48) - 1) / rows))
        return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
    if (rows == 0) return LTX3DROPE_OK;
    if (!x || !q || !scale) return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t n = static_cast<size_t>(rows) * static_cast<size_t>(dim), es = elem(dtype);
    Spans t;
    t.add(x, n * es, es, Role::Param);
    t.add(q, n, 1, Role::ParamOut);
    t.add(scale, static_cast<size_t>(rows) * 4, 4, Role::ParamOut);
    int device = -1;
    const int why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    DeviceGuard guard(device);
    if (launch_q8_quantize(x, q, scale, static_cast<uint32_t>(rows), static_cast<uint32_t>(dim),
                           dtype == LTX3DROPE_DTYPE_F32, static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int64_t ltx3drope_q8_matmul_workspace(const ltx3drope_q8_matmul_t* call) {
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_q8(*call, &why);
    if (st != LTX3DROPE_OK) return st;
    if (call->tokens == 0 || call->out == 0) return 0;
    return static_cast<int64_t>(q8_workspace(q8_problem(*call)));
}

int ltx3drope_q8_matmul(const ltx3drope_q8_matmul_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_q8_matmul_t& c = *call;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_q8(c, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if (c.tokens == 0 || c.out == 0) return LTX3DROPE_OK;
    const Q8Problem p = q8_problem(c);
    const size_t ws = q8_workspace(p);
    if (c.workspace_bytes < 0 || static_cast<size_t>(c.workspace_bytes) < ws) return LTX3DROPE_E_INVALID;
    if (!c.a || !c.b || !c.a_scale || !c.b_scale || !c.y || (ws != 0 && !c.workspace))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t M = p.tokens, K = p.dim, N = p.out, es = elem(c.dtype);
    Spans t;
    t.add(c.a, M * K, 1, Role::Param);
    t.add(c.b, N * K, 1, Role::Param);
    t.add(c.a_scale, M * 4, 4, Role::Param);
    t.add(c.b_scale, N * 4, 4, Role::Param);
    t.add(c.bias, N * 4, 4, Role::Param);
    t.add(c.y, M * N * es, es, Role::ParamOut);
    if (ws != 0) t.add(c.workspace, ws, 16, Role::Scratch);
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    DeviceGuard guard(device);
    if (launch_q8(p, c.dtype == LTX3DROPE_DTYPE_F32, static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int ltx3drope_f8_quantize(const ltx3drope_f8_quantize_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_f8_quantize_t& c = *call;
    if (!flag(c.blocks) || (c.q_turned == nullptr) != (c.scale_turned == nullptr) ||
        (c.q_turned && c.turned_pitch < c.rows))
        return LTX3DROPE_E_INVALID;
    if (c.dtype != LTX3DROPE_DTYPE_F32 && c.dtype != LTX3DROPE_DTYPE_BF16) return refuse(LTX3DROPE_REASON_DTYPE, reason);
    if (c.dim <= 0 || c.rows < 0) return refuse(LTX3DROPE_REASON_NONPOSITIVE_DIM, reason);
    const int64_t lim = int64_t(1) << 31;
    if (c.dim >= lim || c.rows >= lim || (c.q_turned && c.turned_pitch >= 2 * lim))
        return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
    const int64_t tiles_r = (c.rows + 127) / 128, tiles_c = (c.dim + 127) / 128;
    const int64_t scale_rows = c.blocks ? tiles_r : c.rows, turned_rows = c.blocks ? tiles_c : c.dim;
    if (tiles_r * tiles_c >= int64_t(1) << 24) return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
    for (const int64_t(*v)[2] : {&c.scale_strides, &c.scale_turned_strides})
        for (int64_t n : *v) {
            if (n < 0) return LTX3DROPE_E_INVALID;
            if (n >= kF8MaxScaleBlock) return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
        }
    if (scale_rows * c.scale_strides[0] >= int64_t(1) << 58 || turned_rows * c.scale_turned_strides[0] >= int64_t(1) << 58)
        return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
    if (c.rows == 0) return LTX3DROPE_OK;
    if (!c.x || !c.q || !c.scale) return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t n = static_cast<size_t>(c.rows) * static_cast<size_t>(c.dim), es = elem(c.dtype);
    Spans t;
    t.add(c.x, n * es, es, Role::Param);
    t.add(c.q, n, 1, Role::ParamOut);
    t.add(c.scale, scale_bytes(scale_rows, tiles_c, c.scale_strides), 4, Role::ParamOut);
    t.add(c.q_turned, static_cast<size_t>(c.dim) * static_cast<size_t>(c.turned_pitch), 1, Role::ParamOut);
    t.add(c.scale_turned, scale_bytes(turned_rows, tiles_r, c.scale_turned_strides), 4, Role::ParamOut);
    if (!distinct_scales(scale_rows, tiles_c, c.scale_strides) ||
        (c.q_turned && !distinct_scales(turned_rows, tiles_r, c.scale_turned_strides)))
        return refuse(LTX3DROPE_REASON_OVERLAP, reason);
    int device = -1;
    const int why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    F8Quantize p;
    p.x = c.x;
    p.q = c.q;
    p.q_turned = c.q_turned;
    p.scale = c.scale;
    p.scale_turned = c.scale_turned;
    p.turned_pitch = static_cast<uint64_t>(c.turned_pitch);
    p.scale_row = static_cast<uint64_t>(c.scale_strides[0]);
    p.scale_block = static_cast<uint64_t>(c.scale_strides[1]);
    p.turned_row = static_cast<uint64_t>(c.scale_turned_strides[0]);
    p.turned_block = static_cast<uint64_t>(c.scale_turned_strides[1]);
    p.rows = static_cast<uint32_t>(c.rows);
    p.dim = static_cast<uint32_t>(c.dim);
    p.blocks = c.blocks != 0;
    p.turned_chunks = ((reinterpret_cast<uintptr_t>(c.q_turned) | p.turned_pitch) & 15) == 0;
    DeviceGuard guard(device);
    if (launch_f8_quantize(p, c.dtype == LTX3DROPE_DTYPE_F32, static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int64_t ltx3drope_f8_matmul_workspace(const ltx3drope_f8_matmul_t* call) {
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_f8(*call, &why);
    if (st != LTX3DROPE_OK) return st;
    if (call->tokens == 0 || call->out == 0) return 0;
    return static_cast<int64_t>(f8_workspace(f8_problem(*call)));
}

int ltx3drope_f8_matmul(const ltx3drope_f8_matmul_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_f8_matmul_t& c = *call;
    int why = LTX3DROPE_REASON_OK;
    const int st = check_f8(c, &why);
    if (st == LTX3DROPE_E_UNSUPPORTED) return refuse(why, reason);
    if (st != LTX3DROPE_OK) return st;
    if (c.tokens == 0 || c.out == 0) return LTX3DROPE_OK;
    const F8Problem p = f8_problem(c);
    const size_t ws = f8_workspace(p);
    if (c.workspace_bytes < 0 || static_cast<size_t>(c.workspace_bytes) < ws) return LTX3DROPE_E_INVALID;
    if (!c.a || !c.b || !c.a_scale || !c.b_scale || !c.y || (ws != 0 && !c.workspace))
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    const size_t M = p.tokens, K = p.dim, N = p.out, es = elem(c.dtype), blocks = (K + 127) / 128;
    Spans t;
    t.add(c.a, (M - 1) * p.a_pitch + K, 1, Role::Param);
    t.add(c.b, (N - 1) * p.b_pitch + K, 1, Role::Param);
    t.add(c.a_scale, scale_bytes(M, blocks, c.a_scale_strides), 4, Role::Param);
    t.add(c.b_scale, scale_bytes(p.b_rows ? N : (N + 127) / 128, blocks, c.b_scale_strides), 4, Role::Param);
    t.add(c.bias, N * 4, 4, Role::Param);
    t.add(c.y, M * N * es, es, Role::ParamOut);
    if (ws != 0) t.add(c.workspace, ws, 16, Role::Scratch);
    int device = -1;
    why = check_spans(t, &device);
    if (why != LTX3DROPE_REASON_OK) return refuse(why, reason);
    DeviceGuard guard(device);
    if (launch_f8(p, c.dtype == LTX3DROPE_DTYPE_F32, static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

}  // extern "C"
