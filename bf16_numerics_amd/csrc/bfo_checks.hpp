// bfo_checks.hpp -- host-side argument checks shared by the C ABI's sources.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace bfo {

inline bool alignedTo(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The byte range [lo, hi) an array argument covers; a null pointer covers
// nothing.
struct Span {
    uintptr_t lo, hi;
};

inline Span span(const void *p, uint64_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p);
    if (!p) return {0, 0};
    return {x, bytes > UINTPTR_MAX - x ? UINTPTR_MAX : x + uintptr_t(bytes)};
}

inline bool overlap(const Span &a, const Span &b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// True when two of the arrays of one call share a byte: the kernels read and
// write them as distinct (restrict) buffers.
inline bool anyOverlap(std::initializer_list<Span> spans) {
    for (const Span *a = spans.begin(); a != spans.end(); ++a)
        for (const Span *b = a + 1; b != spans.end(); ++b)
            if (overlap(*a, *b)) return true;
    return false;
}

// A row-major matrix argument: rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *p;
    uint64_t rows, width, stride;

    Span whole() const { return p && rows ? span(p, (rows - 1) * stride + width) : Span{0, 0}; }
};

// True when a byte of one matrix is a byte of the other.  Matrices with the
// same stride may lie side by side in the columns of one wider buffer.
inline bool overlap(const Rows &a, const Rows &b) {
    const Span x = a.whole(), y = b.whole();
    if (!overlap(x, y)) return false;
    if (a.stride != b.stride || a.rows < 2 || b.rows < 2) return true;
    const uint64_t gap = (y.lo >= x.lo ? y.lo - x.lo : a.stride - (x.lo - y.lo) % a.stride) % a.stride;
    return !(gap >= a.width && a.stride - gap >= b.width);
}

}  // namespace bfo
