// The checks that the entry points' tensors share: alignment, overlaps and device memory.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "internal.h"

namespace ltx3drope {

enum class Role { Param, RowIn, RowOut, ParamOut, Scratch };

struct Span {
    const void* p;
    size_t bytes, align;
    Role role;
};

// The tensors of one call, collected for the checks that they share.
struct Spans {
    Span s[24];
    int n = 0;
    void add(const void* p, size_t bytes, size_t align, Role role) {
        if (p != nullptr && bytes != 0) s[n++] = Span{p, bytes, align, role};
    }
};

inline bool is_output(Role r) { return r == Role::RowOut || r == Role::ParamOut || r == Role::Scratch; }

// The device-memory rules; *device receives the tensors' device.
inline int check_memory(const Spans& t, int* device) {
    // Tensors of one allocation (an allocator's blocks, a model's buffers) are asked for once: a range
    // inside one that this call has found is device memory of the same GPU.
    constexpr int kAllocations = 4;
    uintptr_t from[kAllocations], to[kAllocations];
    int known = 0, on = -1;
    for (int i = 0; i < t.n; ++i) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(t.s[i].p);
        bool inside = false;
        for (int j = 0; j < known; ++j) inside = inside || (p >= from[j] && p < to[j] && t.s[i].bytes <= to[j] - p);
        if (inside) continue;
        DeviceRange a;
        if (!device_range(t.s[i].p, &a)) return LTX3DROPE_REASON_NOT_DEVICE_PTR;
        if (on < 0) on = a.device;
        const int r = check_range(a, t.s[i].p, t.s[i].bytes, on);
        if (r != LTX3DROPE_REASON_OK) return r;
        if (known < kAllocations) {
            from[known] = a.base;
            to[known++] = a.base + a.size;
        }
    }
    if (on < 0) return LTX3DROPE_REASON_NOT_DEVICE_PTR;
    *device = on;
    return LTX3DROPE_REASON_OK;
}

inline int check_alignment(const Spans& t) {
    for (int i = 0; i < t.n; ++i)
        if (reinterpret_cast<uintptr_t>(t.s[i].p) % t.s[i].align) return LTX3DROPE_REASON_ALIGN;
    return LTX3DROPE_REASON_OK;
}

// ALIGN, OVERLAP, then the device-memory rules; *device receives the tensors' device.
inline int check_spans(const Spans& t, int* device) {
    if (const int why = check_alignment(t)) return why;
    for (int i = 0; i < t.n; ++i) {
        if (!is_output(t.s[i].role)) continue;
        for (int j = 0; j < t.n; ++j) {
            if (j == i || !ranges_overlap(t.s[i].p, t.s[i].bytes, t.s[j].p, t.s[j].bytes)) continue;
            const bool own_row = t.s[i].role == Role::RowOut && t.s[j].role == Role::RowIn && t.s[i].p == t.s[j].p;
            if (!own_row) return LTX3DROPE_REASON_OVERLAP;
        }
    }
    return check_memory(t, device);
}

inline int refuse(int why, int* reason) {
    if (reason) *reason = why;
    count_rejected();
    return LTX3DROPE_E_UNSUPPORTED;
}

inline bool aligned16(const Spans& t, std::initializer_list<Role> roles) {
    for (int i = 0; i < t.n; ++i)
        for (Role r : roles)
            if (t.s[i].role == r && reinterpret_cast<uintptr_t>(t.s[i].p) % 16) return false;
    return true;
}

}  // namespace ltx3drope
