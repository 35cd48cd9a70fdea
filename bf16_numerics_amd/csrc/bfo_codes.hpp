// bfo_codes.hpp -- what the operators between a block's matrix products share:
// ways to load and store a row's chunks, and 8-bit codes with scales.
//
// Codes: values of a row in groups of kGroup columns (or the whole row), each
// code an 8-bit integer or an e4m3 float, each value code * scale.
//
// scale = max(amax / top, 2^-126), amax the group's largest absolute value and
// top what the code type holds at most (127, 448), so that the largest value
// takes the whole range and a group of zeros has a scale to divide by; the
// code is value / scale rounded to nearest even.  A value is off by at most
// half a step: scale / 2 for integers, 2^-4 of itself for e4m3 (or
// scale * 2^-10 below scale * 2^-6).  For normally distributed values integers
// of a group of 128 are about four times as exact; e4m3 keeps small values
// beside large ones.  Absolute values are compared as bit patterns, in which a
// NaN is above infinity: a group that holds either gets a scale that is not
// finite and all its values read back as NaN.
#pragma once

#include <type_traits>

#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

// Words moved down by `bytes`, less than there are, zeros behind them.  (Written
// out: of a choice between two words in a loop the compiler makes one of their
// addresses, and puts them into LDS.)
template <int kWords>
__device__ __forceinline__ void moveDown(uint32_t (&w)[kWords], int bytes) {
    static_assert(kWords == 1 || kWords == 2 || kWords == 4, "4, 8 or 16 bytes");
    const bool eight = bytes & 8, four = bytes & 4;
    uint32_t a = w[0], b = 0u, c = 0u, d = 0u;
    if constexpr (kWords > 1) b = w[1];
    if constexpr (kWords > 2) {
        c = w[2], d = w[3];
        a = eight ? c : a, b = eight ? d : b, c = eight ? 0u : c, d = eight ? 0u : d;
    }
    if constexpr (kWords > 1) a = four ? b : a, b = four ? c : b, c = four ? d : c, d = four ? 0u : d;
    w[0] = __builtin_amdgcn_alignbyte(b, a, bytes & 3);
    if constexpr (kWords > 1) w[1] = __builtin_amdgcn_alignbyte(c, b, bytes & 3);
    if constexpr (kWords > 2) {
        w[2] = __builtin_amdgcn_alignbyte(d, c, bytes & 3);
        w[3] = __builtin_amdgcn_alignbyte(0u, d, bytes & 3);
    }
}

// How a row's chunks are loaded: kEven, widths of whole chunks; kEvenStream, those
// nontemporally; kRagged, any other width from a chunk on; kNarrow, less than a
// chunk, value by value.  But for the last, no load waits for a branch: of a row
// that ends inside the chunk, or before it, its last whole one is asked for, and
// settle puts it in place where the values are used.  (Behind a branch the compiler
// waits for every load before it: backward of 16384 x 1600 bf16 from codes 41.5 us
// against 34.2; of 8192 x 5003, whose ends were read value by value, 152 against 80.
// Nontemporal stores would gain ragged rows 1 to 3%.)
enum Loads { kNarrow, kRagged, kEven, kEvenStream };
constexpr bool inParts(Loads loads) { return loads == kNarrow || loads == kRagged; }
template <Loads kLoads, typename T, int E>
__device__ __forceinline__ void loadChunk(Chunk<T, E> &w, const T *row, int c, int C, bool live) {
    if constexpr (kLoads == kNarrow) w.loadRow(row, c, C, live);
    else w.template load<kLoads == kEvenStream>(row + min(c, C - E));
}
template <Loads kLoads, typename T, int E>
__device__ __forceinline__ void settle(Chunk<T, E> &w, int c, int C, bool live) {
    if constexpr (kLoads == kRagged) moveDown(w.w, min(max(c - (C - E), 0), E - 1) * int(sizeof(T)));
    if (kLoads != kNarrow && (!live || c >= C)) w.zero();
}
// The row to load from.
__device__ __forceinline__ uint64_t loadedRow(uint64_t row, uint64_t rows) { return min(row, rows - 1); }
template <Loads kLoads, typename T, int E>
__device__ __forceinline__ void storeChunk(Chunk<T, E> w, T *row, int c, int C) {
    if constexpr (inParts(kLoads)) {
        w.storeRow(row, c, C);
    } else if (c < C) {
        // The compiler stores values that it has just rounded to bf16 without the hint.
        if constexpr (kLoads == kEvenStream) w.forget();
        w.template store<kLoads == kEvenStream>(row + c);
    }
}
template <Loads kLoads, typename T, int E>
__device__ __forceinline__ void storeChunk(T *row, int c, int C, const float (&v)[E]) {
    if constexpr (inParts(kLoads)) storeRow(row, c, 0, C, v);
    else storeChunk<kLoads>(Chunk<T, E>(v), row, c, C);
}
template <Loads kValue>
using Constant = std::integral_constant<Loads, kValue>;

// f with the way to load rows of a call that moves `bytes`.
template <typename T, typename F>
void byLoads(uint32_t cols, uint64_t bytes, F f) {
    constexpr uint32_t E = 16 / sizeof(T);
    if (cols < E) f(Constant<kNarrow>{});
    else if (cols % E) f(Constant<kRagged>{});
    else if (streams(bytes)) f(Constant<kEvenStream>{});
    else f(Constant<kEven>{});
}

constexpr int kGroup = int(BFO_GROUP);

// Words that may start at any byte.
typedef uint32_t Bytes4 __attribute__((aligned(1)));
typedef uint32_t Bytes8 __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ uint32_t absBits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The value that the lane kBy on in a row of 16 has (in the shape that the compiler
// makes one instruction of with the maximum that it goes into).
template <int kBy>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), kRowRotate + kBy, 0xF, 0xF, true));
}
// The largest of the values of the kLanes lanes (16 or 32 from a multiple of it
// on, or the wavefront), in all of them.
template <int kLanes>
__device__ __forceinline__ uint32_t laneMax(uint32_t v) {
    static_assert(kLanes == 16 || kLanes == 32 || kLanes == 64, "one DPP row, two or the wavefront");
    if constexpr (kLanes == 64) {
        return waveExtreme<true>(v);
    } else {
        v = max(v, rotated<8>(v));
        v = max(v, rotated<4>(v));
        v = max(v, rotated<2>(v));
        v = max(v, rotated<1>(v));
        if constexpr (kLanes == 32) {
            const auto both = __builtin_amdgcn_permlane16_swap(v, v, false, false);
            v = max(uint32_t(both[0]), uint32_t(both[1]));
        }
        return v;
    }
}

// The scale of values up to `amax` (its bits) and its reciprocal.
struct CodeScale {
    float scale, inverse;
};
template <int kType>
__device__ __forceinline__ CodeScale codeScale(uint32_t amax) {
    constexpr float kTopInverse = kType == BFO_I8 ? 1.0f / 127.0f : 1.0f / 448.0f, kSmallest = 0x1p-126f;
    float s = __uint_as_float(amax) * kTopInverse;
    s = s < kSmallest ? kSmallest : s;  // a NaN stays
    // The hardware's reciprocal is a step off at most, from where one of Newton's steps
    // rounds it as a division would.  (Of an infinity it makes a NaN, which the codes of
    // such a group may be.)
    const float r = __builtin_amdgcn_rcpf(s);
    return {s, fmaf(fmaf(-s, r, 1.0f), r, r)};
}

// The codes of N values, four to a word.
template <int kType, int N>
__device__ __forceinline__ void encode(const float (&v)[N], float inverse, uint32_t (&w)[N / 4]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if constexpr (kType == BFO_I8) {
            // Added to 1.5 * 2^23, a number is rounded to an integer in the sum's low bits.
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(v[i + e] * inverse + 12582912.0f);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
            w[i / 4] = lo | hi;
        } else {
            int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[i] * inverse, v[i + 1] * inverse, 0, false);
            r = __builtin_amdgcn_cvt_pk_fp8_f32(v[i + 2] * inverse, v[i + 3] * inverse, r, true);
            w[i / 4] = uint32_t(r);
        }
    }
}

// The values that N codes stand for.
template <int kType, int N>
__device__ __forceinline__ void decode(const uint32_t (&w)[N / 4], float scale, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if constexpr (kType == BFO_I8) {
            const uint32_t u = w[i / 4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i + e] = float(int8_t(u >> (8 * e))) * scale;
        } else {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[i / 4]), false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[i / 4]), true);
            v[i] = lo[0] * scale, v[i + 1] = lo[1] * scale;
            v[i + 2] = hi[0] * scale, v[i + 3] = hi[1] * scale;
        }
    }
}

template <int N>
__device__ __forceinline__ void getCodes(const uint8_t *p, uint32_t (&w)[N / 4]) {
    if constexpr (N == 8) {
        const Bytes8 q = *reinterpret_cast<const Bytes8 *>(p);
        w[0] = q.x, w[1] = q.y;
    } else {
        w[0] = *reinterpret_cast<const Bytes4 *>(p);
    }
}
// N codes of a row, from column c on, as loadChunk and settle load values.
template <Loads kLoads, int N>
__device__ __forceinline__ void loadCodes(const uint8_t *row, int c, int C, bool live, uint32_t (&w)[N / 4]) {
    if constexpr (kLoads == kNarrow) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (live && c + i < C) w[i / 4] |= uint32_t(row[c + i]) << (8 * (i % 4));
    } else {
        getCodes<N>(row + min(c, C - N), w);
    }
}
template <Loads kLoads, int N>
__device__ __forceinline__ void settleCodes(uint32_t (&w)[N / 4], int c, int C, bool live) {
    if constexpr (kLoads == kRagged) moveDown(w, min(max(c - (C - N), 0), N - 1));
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = live && c < C ? w[i] : 0u;
}
template <Loads kLoads, bool kNontemporal, int N>
__device__ __forceinline__ void storeCodes(uint8_t *base, int c, int cols, const uint32_t (&w)[N / 4]) {
    if (inParts(kLoads) ? c + N <= cols : c < cols) {
        if constexpr (N == 8) {
            const Bytes8 q{w[0], w[1]};
            Bytes8 *p = reinterpret_cast<Bytes8 *>(base + c);
            if constexpr (kNontemporal) __builtin_nontemporal_store(q, p);
            else *p = q;
        } else {
            Bytes4 *p = reinterpret_cast<Bytes4 *>(base + c);
            if constexpr (kNontemporal) __builtin_nontemporal_store(Bytes4(w[0]), p);
            else *p = w[0];
        }
    } else if (inParts(kLoads) && c < cols) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < cols) base[c + i] = uint8_t(w[i / 4] >> (8 * (i % 4)));
    }
}

}  // namespace
}  // namespace bfo
