// C ABI of the rotary positions with several axes: argument checks and dispatch.
#include <algorithm>
#include <cmath>

#include "axes.h"
#include "internal.h"
#include "spans.h"

namespace ltx3drope {
namespace {

struct Dim {
    int64_t size, stride;
};

// A tensor [batch, tokens, heads, head_dim] as the checks see it: its dimensions of more than one element,
// the largest stride first, and its span in elements.
struct Strided {
    const void* p;
    Dim dims[3];
    int n = 0;
    int64_t width, span;
    bool out;
};

constexpr int64_t kMaxSpan = int64_t(1) << 60;

// False: the tensor spans kMaxSpan bytes or more.
bool describe(Strided* t, const void* p, const int64_t (&strides)[3], int64_t batch, int64_t tokens, int64_t heads,
              int64_t width, int64_t es, bool out) {
    t->p = p;
    t->out = out;
    t->width = t->span = width;
    const int64_t sizes[3] = {batch, tokens, heads};
    for (int i = 0; i < 3; ++i) {
        if (sizes[i] <= 1) continue;
        int64_t reach;
        if (__builtin_mul_overflow(sizes[i] - 1, strides[i], &reach) || reach >= kMaxSpan / es) return false;
        t->span += reach;
        t->dims[t->n++] = Dim{sizes[i], strides[i]};
    }
    std::sort(t->dims, t->dims + t->n, [](const Dim& a, const Dim& b) { return a.stride > b.stride; });
    return t->span < kMaxSpan / es;
}

// Whether no two indexes of the tensor meet in one element (every stride passes what lies inside it).
bool distinct(const Strided& t) {
    int64_t inside = t.width;
    for (int i = t.n - 1; i >= 0; --i) {
        if (t.dims[i].stride < inside) return false;
        inside += (t.dims[i].size - 1) * t.dims[i].stride;
    }
    return true;
}

// Whether two tensors share no element: their ranges are apart, or they lie side by side in every period of the
// outer dimensions that they have in common.
bool apart(const Strided& x, const Strided& y, int64_t es) {
    const Strided &a = x.p <= y.p ? x : y, &b = x.p <= y.p ? y : x;
    const int64_t bytes = static_cast<const char*>(b.p) - static_cast<const char*>(a.p);
    if (bytes >= a.span * es) return true;
    if (bytes % es) return false;
    const int64_t delta = bytes / es;
    int64_t span_a = a.span, span_b = b.span;
    for (int j = 0; j < a.n && j < b.n; ++j) {
        if (a.dims[j].size != b.dims[j].size || a.dims[j].stride != b.dims[j].stride) return false;
        span_a -= (a.dims[j].size - 1) * a.dims[j].stride;
        span_b -= (b.dims[j].size - 1) * b.dims[j].stride;
        if (delta < span_a) continue;
        int64_t inside = delta + span_b;  // of both, in one period of dimension j
        bool fits = true;
        for (int i = j; i >= 0 && fits; --i) {
            fits = a.dims[i].stride >= inside;
            inside += (a.dims[i].size - 1) * a.dims[i].stride;
        }
        if (fits) return true;
    }
    return false;
}

bool same(const Strided& a, const Strided& b) {
    if (a.p != b.p || a.n != b.n) return false;
    for (int i = 0; i < a.n; ++i)
        if (a.dims[i].size != b.dims[i].size || a.dims[i].stride != b.dims[i].stride) return false;
    return true;
}

// A stride that no index passes has any value: the launcher reckons with 0.
int64_t step(int64_t size, int64_t stride) { return size > 1 ? stride : 0; }

AxesTensor tensor(const void* in, void* out, const int64_t (&si)[3], const int64_t (&so)[3], const ltx3drope_axes_t& c,
                  int64_t heads) {
    return AxesTensor{static_cast<const char*>(in), static_cast<char*>(out), step(c.batch, si[0]), step(c.tokens, si[1]),
                      step(heads, si[2]), step(c.batch, so[0]), step(c.tokens, so[1]), step(heads, so[2]),
                      static_cast<uint32_t>(heads)};
}

}  // namespace
}  // namespace ltx3drope

using namespace ltx3drope;

extern "C" {

int ltx3drope_axes_apply(const ltx3drope_axes_t* call, void* stream, int* reason) {
    if (reason) *reason = LTX3DROPE_REASON_OK;
    if (call == nullptr) return LTX3DROPE_E_INVALID;
    const ltx3drope_axes_t& c = *call;
    if ((c.pairing != LTX3DROPE_PAIRING_ADJACENT && c.pairing != LTX3DROPE_PAIRING_HALVES) ||
        (c.inverse != 0 && c.inverse != 1) || c.position_type < LTX3DROPE_POSITION_I64 ||
        c.position_type > LTX3DROPE_POSITION_F32 || c.frequency_type < LTX3DROPE_FREQUENCY_F64 ||
        c.frequency_type > LTX3DROPE_FREQUENCY_F32 || c.axes < 1 || c.axes > 255)
        return LTX3DROPE_E_INVALID;
    for (const int64_t(*s)[3] : {&c.q_strides, &c.k_strides, &c.q_out_strides, &c.k_out_strides, &c.position_strides})
        for (int64_t v : *s)
            if (v < 0) return LTX3DROPE_E_INVALID;
    if (c.k_heads == 0 && (c.k || c.k_out)) return LTX3DROPE_E_INVALID;
    if (c.dtype != LTX3DROPE_DTYPE_F32 && c.dtype != LTX3DROPE_DTYPE_BF16) return refuse(LTX3DROPE_REASON_DTYPE, reason);
    if (c.head_dim <= 0 || c.pairs <= 0 || c.batch < 0 || c.tokens < 0 || c.q_heads < 0 || c.k_heads < 0)
        return refuse(LTX3DROPE_REASON_NONPOSITIVE_DIM, reason);
    if (c.pairs > c.head_dim / 2) return refuse(LTX3DROPE_REASON_SPLIT_SUM, reason);
    if (c.batch > kAxesMaxBatch || c.q_heads > kAxesMaxHeads || c.k_heads > kAxesMaxHeads ||
        c.head_dim > kAxesMaxWidth || c.tokens >= int64_t(1) << 31)
        return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
    if (c.batch == 0 || c.tokens == 0 || c.q_heads + c.k_heads == 0) return LTX3DROPE_OK;
    const bool f32 = c.dtype == LTX3DROPE_DTYPE_F32;
    const int64_t es = f32 ? 4 : 2, ps = c.position_type == LTX3DROPE_POSITION_I64 ? 8 : 4;
    const int64_t fs = c.frequency_type == LTX3DROPE_FREQUENCY_F64 ? 8 : 4;
    Strided t[4], at;
    int n = 0;
    bool fits = true;
    if (c.q_heads) {
        fits = describe(&t[n++], c.q, c.q_strides, c.batch, c.tokens, c.q_heads, c.head_dim, es, false) &&
               describe(&t[n++], c.q_out, c.q_out_strides, c.batch, c.tokens, c.q_heads, c.head_dim, es, true);
    }
    if (fits && c.k_heads) {
        fits = describe(&t[n++], c.k, c.k_strides, c.batch, c.tokens, c.k_heads, c.head_dim, es, false) &&
               describe(&t[n++], c.k_out, c.k_out_strides, c.batch, c.tokens, c.k_heads, c.head_dim, es, true);
    }
    if (!fits || !describe(&at, c.positions, c.position_strides, c.axes, c.batch, c.tokens, 1, ps, false))
        return refuse(LTX3DROPE_REASON_TOO_LARGE, reason);
    if ((c.q_heads && (!c.q || !c.q_out)) || (c.k_heads && (!c.k || !c.k_out)) || !c.positions || !c.frequencies ||
        !c.axis)
        return refuse(LTX3DROPE_REASON_NULLPTR, reason);
    Spans all;
    for (int i = 0; i < n; ++i)
        all.add(t[i].p, static_cast<size_t>(t[i].span * es), static_cast<size_t>(es), t[i].out ? Role::RowOut : Role::RowIn);
    const int tensors = all.n;
    all.add(c.positions, static_cast<size_t>(at.span * ps), static_cast<size_t>(ps), Role::Param);
    all.add(c.frequencies, static_cast<size_t>(c.pairs * fs), static_cast<size_t>(fs), Role::Param);
    all.add(c.axis, static_cast<size_t>(c.pairs), 1, Role::Param);
    if (const int why = check_alignment(all)) return refuse(why, reason);
    for (int i = 0; i < n; ++i) {
        if (!t[i].out) continue;
        if (!distinct(t[i])) return refuse(LTX3DROPE_REASON_OVERLAP, reason);
        for (int j = 0; j < n; ++j)
            if (j != i && !(j + 1 == i && same(t[i], t[j])) && !apart(t[i], t[j], es))
                return refuse(LTX3DROPE_REASON_OVERLAP, reason);
        for (int j = tensors; j < all.n; ++j)
            if (ranges_overlap(all.s[i].p, all.s[i].bytes, all.s[j].p, all.s[j].bytes))
                return refuse(LTX3DROPE_REASON_OVERLAP, reason);
    }
    int device = -1;
    if (const int why = check_memory(all, &device)) return refuse(why, reason);

    AxesProblem p;
    p.q = tensor(c.q, c.q_out, c.q_strides, c.q_out_strides, c, c.q_heads);
    p.k = tensor(c.k, c.k_out, c.k_strides, c.k_out_strides, c, c.k_heads);
    p.positions = c.positions;
    p.position_axis = step(c.axes, c.position_strides[0]);
    p.position_batch = step(c.batch, c.position_strides[1]);
    p.position_token = step(c.tokens, c.position_strides[2]);
    p.frequencies = c.frequencies;
    p.axis = c.axis;
    p.batch = static_cast<uint32_t>(c.batch);
    p.tokens = static_cast<uint32_t>(c.tokens);
    p.head_dim = static_cast<uint32_t>(c.head_dim);
    p.pairs = static_cast<uint32_t>(c.pairs);
    p.axes = static_cast<uint32_t>(c.axes);
    p.f32 = f32;
    p.halves = c.pairing == LTX3DROPE_PAIRING_HALVES;
    p.inverse = c.inverse != 0;
    p.frequency_f32 = c.frequency_type == LTX3DROPE_FREQUENCY_F32;
    p.position_type = c.position_type;
    p.vector = 1;
    for (uint32_t v : {f32 ? 4u : 8u, 2u}) {
        const int64_t bytes = v * es;
        bool fit = axes_vector_widths(v, p.halves, p.head_dim, p.pairs);
        for (int i = 0; i < n && fit; ++i) {
            fit = reinterpret_cast<uintptr_t>(t[i].p) % bytes == 0;
            for (int j = 0; j < t[i].n; ++j) fit = fit && t[i].dims[j].stride * es % bytes == 0;
        }
        if (fit) {
            p.vector = v;
            break;
        }
    }
    DeviceGuard guard(device);
    if (launch_axes(p, static_cast<hipStream_t>(stream)) != hipSuccess) return LTX3DROPE_E_HIP;
    count_launch();
    return LTX3DROPE_OK;
}

int ltx3drope_axes_frequencies(int axes, const int64_t* widths, double base, int joint, double* frequencies,
                               uint8_t* axis) {
    if (axes < 1 || axes > 255 || !widths || !frequencies || !axis || !std::isfinite(base) || base <= 0.0 ||
        (joint != 0 && joint != 1))
        return LTX3DROPE_E_INVALID;
    int64_t total = 0;
    for (int a = 0; a < axes; ++a) {
        if (widths[a] <= 0 || widths[a] % 2 || widths[a] > kAxesMaxWidth) return LTX3DROPE_E_INVALID;
        total += widths[a];
    }
    int64_t j = 0;
    for (int a = 0; a < axes; ++a)
        for (int64_t i = 0; i < widths[a] / 2; ++i, ++j) {
            const double of = static_cast<double>(joint ? total : widths[a]);
            frequencies[j] = std::pow(base, -2.0 * static_cast<double>(joint ? j : i) / of);
            axis[j] = static_cast<uint8_t>(a);
        }
    return LTX3DROPE_OK;
}

}  // extern "C"
