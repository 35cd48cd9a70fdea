// bfo_args.hpp -- how the host sides of the training-loop operators check
// matrices and arrays.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/bf16opt.h"
#include "bfo_checks.hpp"
#include "bfo_internal.hpp"

namespace bfo {

constexpr uint64_t kMaxRows = uint64_t(1) << 31;
constexpr uint64_t kMaxBytes = uint64_t(1) << 62;  // of one matrix

inline bool knownType(int dtype) { return dtype == BFO_BF16 || dtype == BFO_F32; }
inline uint64_t sizeOf(int dtype) { return dtype == BFO_BF16 ? 2 : 4; }

inline int done(hipError_t e) { return e == hipSuccess ? BFO_OK : recordHipFailure(e); }

// A matrix of `cols` used columns of `size` bytes; the status its sizes and
// pointer earn.
inline int matrixOf(const void *p, uint64_t stride, uint64_t rows, uint64_t cols, uint64_t size, Rows &out) {
    out = Rows{p, rows, cols * size, stride * size};
    if (rows > kMaxRows || stride > kMaxBytes / size) return BFO_ERANGE;
    if (rows && !p) return BFO_EINVAL;
    if (rows > 1) {
        if (stride < cols) return BFO_EINVAL;
        if (stride * size > kMaxBytes / rows) return BFO_ERANGE;
    }
    return alignedTo(p, size) ? BFO_OK : BFO_EMISALIGNED;
}

inline int matrix(const void *p, uint64_t stride, uint64_t rows, uint64_t cols, int dtype, Rows &out) {
    return matrixOf(p, stride, rows, cols, sizeOf(dtype), out);
}
// A matrix that may be NULL, which has no rows then.
inline int optionalMatrix(const void *p, uint64_t stride, uint64_t rows, uint64_t cols, uint64_t size, Rows &out) {
    if (p) return matrixOf(p, stride, rows, cols, size, out);
    out = Rows{nullptr, 0, 0, 0};
    return BFO_OK;
}

// One array argument with the way it is used.
struct Use {
    Span at;
    bool written;
};
inline Use reads(const void *p, uint64_t bytes) { return {span(p, bytes), false}; }
inline Use writes(const void *p, uint64_t bytes) { return {span(p, bytes), true}; }

// True when a written array shares a byte with another array of the call.
template <int N>
bool conflict(const Use (&use)[N]) {
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j)
            if ((use[i].written || use[j].written) && overlap(use[i].at, use[j].at)) return true;
    return false;
}
// The same between matrices and plain arrays.
template <int N>
bool conflict(const Rows &m, bool written, const Use (&use)[N]) {
    for (int i = 0; i < N; ++i)
        if ((written || use[i].written) && overlap(m.whole(), use[i].at)) return true;
    return false;
}

// True when a written matrix shares a byte with another one of the call; but
// where both are marked `inPlace`, a written one may be the same matrix as one
// that is read.  (Only matrices of one type may be marked: the kernels read a
// value before they write it, not the bytes of other columns around it.)
struct MatrixUse {
    Rows at;
    bool written, inPlace;
};
template <int N>
bool conflict(const MatrixUse (&use)[N]) {
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j) {
            const MatrixUse &a = use[i], &b = use[j];
            if (!(a.written || b.written) || !overlap(a.at, b.at)) continue;
            const bool same = a.at.p == b.at.p && (a.at.stride == b.at.stride || a.at.rows < 2);
            if (!(same && a.written != b.written && a.inPlace && b.inPlace)) return true;
        }
    return false;
}
template <int N, int M>
bool conflict(const MatrixUse (&matrices)[N], const Use (&use)[M]) {
    for (const MatrixUse &m : matrices)
        if (conflict(m.at, m.written, use)) return true;
    return conflict(use);
}

inline bool allAligned(std::initializer_list<const void *> ps, uintptr_t a) {
    for (const void *p : ps)
        if (!alignedTo(p, a)) return false;
    return true;
}

}  // namespace bfo
