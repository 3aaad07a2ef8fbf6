// kda_spans.h -- host-side checks of which buffers of a call lie on one another.
#pragma once

#include "kda_internal.h"

namespace kda {

// A buffer of a call; no pointer or no bytes: not used.
struct Span {
    const void *at;
    size_t bytes;
};
inline bool meet(const Span &a, const Span &b) {
    return a.at != nullptr && b.at != nullptr && a.bytes > 0 && b.bytes > 0 && overlaps(a.at, a.bytes, b.at, b.bytes);
}
// Whether any of `out` lies on another of them or on any of `in`.
template <size_t N, size_t M>
bool any_meet(const Span (&out)[N], const Span (&in)[M]) {
    for (size_t i = 0; i < N; ++i) {
        for (size_t j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return true;
        for (const Span &x : in)
            if (meet(out[i], x)) return true;
    }
    return false;
}
inline Span rows_span(const void *at, int64_t rows, int64_t ld, int64_t width, size_t es) {
    return {at, rows > 0 ? (size_t(rows - 1) * size_t(ld) + size_t(width)) * es : 0};
}
inline bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace kda
