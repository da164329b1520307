// Host-side checks shared by the C ABI's files.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace host {

// Workgroups of a launch: fewer than 2^32 threads.
constexpr int64_t kMaxWorkgroups = (1 << 24) - 1;   // of 256 threads

struct Span {
    uintptr_t lo, hi;      // [lo, hi)
    uintptr_t stride, width;   // bytes from row to row, bytes of a row (0: contiguous)
};
inline Span span(const void* p, int64_t bytes) {
    const uintptr_t a = (uintptr_t)p;
    return Span{a, a + (uintptr_t)(p && bytes > 0 ? bytes : 0), 0, 0};
}
// rows of `width` elements, `stride` apart
inline Span rows_span(const void* p, int64_t rows, int64_t stride, int64_t width, int64_t es) {
    Span s = span(p, rows > 0 ? ((rows - 1) * stride + width) * es : 0);
    s.stride = (uintptr_t)(stride * es);
    s.width = (uintptr_t)(width * es);
    return s;
}
inline bool overlaps(const Span& a, const Span& b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}
// Like overlaps, but two sets of rows with one stride may lie side by side
// within the same wider rows.
inline bool overlaps_rows(const Span& a, const Span& b) {
    if (!overlaps(a, b)) return false;
    if (a.stride == 0 || a.stride != b.stride) return true;
    const Span &f = a.lo <= b.lo ? a : b, &g = a.lo <= b.lo ? b : a;
    const uintptr_t d = (g.lo - f.lo) % f.stride;
    return !(d >= f.width && d + g.width <= f.stride);
}
inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}
inline bool dtype_ok(int t) { return t == KDA_BF16 || t == KDA_F32; }
inline int64_t elem_size(int t) { return t == KDA_BF16 ? 2 : 4; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace host
}  // namespace kda
