// bfo_device.hpp -- device helpers of the training-loop operators' kernels:
// 16-byte chunks of bf16 or fp32 values, and wavefront reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfo {

// The storage type of bf16 values (their bit patterns).
using bf16_t = uint16_t;

// Words that may start at any 2-byte boundary: gfx950 loads and stores of up
// to 16 bytes need no alignment, so rows of odd widths take the same
// instructions as aligned ones.
typedef uint32_t Words1 __attribute__((aligned(2)));
typedef uint32_t Words2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ float toFloat(bf16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ float toFloat(float v) { return v; }

// bf16 by round to nearest even (one v_cvt_pk_bf16_f32 for two values).
__device__ __forceinline__ uint32_t packBf16(float lo, float hi) {
    typedef __bf16 Bf16x2 __attribute__((ext_vector_type(2)));
    const Bf16x2 v = {__bf16(lo), __bf16(hi)};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void storeOne(bf16_t *p, float v) { *p = bf16_t(packBf16(v, 0.0f)); }
__device__ __forceinline__ void storeOne(float *p, float v) { *p = v; }

// N consecutive values of type T in registers, as they lie in memory (8, 16
// or 32 bytes).
template <typename T, int N>
struct Chunk {
    static constexpr int kWords = N * int(sizeof(T)) / 4;
    uint32_t w[kWords];

    Chunk() = default;
    // N values, rounded to T.
    __device__ __forceinline__ explicit Chunk(const float *v) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : packBf16(v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    }
    // Makes the compiler forget what it knows of the values, so that they stay
    // packed from one use to the next.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    template <bool kNontemporal = false>
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kWords == 2) {
            const Words2 *q = reinterpret_cast<const Words2 *>(p);
            const Words2 v = kNontemporal ? __builtin_nontemporal_load(q) : *q;
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const Words4 *q = reinterpret_cast<const Words4 *>(p) + i / 4;
                const Words4 v = kNontemporal ? __builtin_nontemporal_load(q) : *q;
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
            }
        }
    }
    // Adds the other chunk's values, rounding to T.
    __device__ __forceinline__ void add(const Chunk &o) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint((*this)[i] + o[i]);
            else w[i] = packBf16((*this)[2 * i] + o[2 * i], (*this)[2 * i + 1] + o[2 * i + 1]);
        }
    }
    template <bool kNontemporal = false>
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const Words4 v{w[i], w[i + 1], w[i + 2], w[i + 3]};
            if constexpr (kNontemporal) __builtin_nontemporal_store(v, reinterpret_cast<Words4 *>(p) + i / 4);
            else *(reinterpret_cast<Words4 *>(p) + i / 4) = v;
        }
    }
    // Stores the columns [c, c + N) of those from `base` on that lie in [0, cols).
    __device__ __forceinline__ void storeRow(T *base, int c, int cols) const {
        if (c + N <= cols) {
            store(base + c);
        } else if (c < cols) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c + i < cols) storeOne(base + c + i, (*this)[i]);
        }
    }
    // Columns [c, c + N) of those from `base` on, of which [0, cols) are there;
    // 0 for the others, and for all if not `live`.  The zeros come first, so that
    // no load waits for another one's lanes.  Here and below a `base` that is the
    // same in all lanes keeps the addresses at one scalar and one lane offset.
    __device__ __forceinline__ void loadRow(const T *base, int c, int cols, bool live = true) {
        zero();
        if (live && c + N <= cols) load(base + c);
        else if (live && c < cols) loadPart(base, c, 0, cols);
    }
    // The same with [lo, hi) there and -inf elsewhere.
    template <bool kNontemporal = false>
    __device__ __forceinline__ void loadScores(const T *base, int c, int lo, int hi) {
        constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : 0xFF80u;
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? kNone : kNone | kNone << 16;
        if (c >= lo && c + N <= hi) load<kNontemporal>(base + c);
        else if (c + N > lo && c < hi) loadPart(base, c, lo, hi);
    }
    // Value by value, those of [lo, hi) only.
    __device__ __forceinline__ void loadPart(const T *base, int c, int lo, int hi) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (c + i >= lo && c + i < hi) {
                if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(base[c + i]);
                else if (i & 1) w[i >> 1] = (w[i >> 1] & 0x0000FFFFu) | uint32_t(base[c + i]) << 16;
                else w[i >> 1] = (w[i >> 1] & 0xFFFF0000u) | base[c + i];
            }
        }
    }
};

// Stores N values, rounded to T, at those of the columns [c, c + N) from
// `base` on that lie in [lo, hi).
template <typename T, int N>
__device__ __forceinline__ void storeRow(T *base, int c, int lo, int hi, const float (&v)[N]) {
    if (c >= lo && c + N <= hi) {
        Chunk<T, N>(v).store(base + c);
    } else if (c + N > lo && c < hi) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i >= lo && c + i < hi) storeOne(base + c + i, v[i]);
    }
}

// Reductions over 16 lanes or the whole wavefront through DPP: rotations
// within rows of 16 (every lane of a row ends with the same bits), then rows
// added to their successors, so that lane 63 holds the total.  About a tenth
// of the latency of exchanges through the LDS crossbar.
template <int kCtrl, int kRowMask = 0xF>
__device__ __forceinline__ float dpp(float old, float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(old), __float_as_uint(v), kCtrl, kRowMask, 0xF,
                                                       false));
}
constexpr int kRowRotate = 0x120, kRowBroadcast15 = 0x142, kRowBroadcast31 = 0x143;
__device__ __forceinline__ float lastLane(float v) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
template <int kLanes>
__device__ __forceinline__ float laneSum(float v) {
    static_assert(kLanes == 16 || kLanes == 32 || kLanes == 64, "one DPP row, two or the wavefront");
    v += dpp<kRowRotate + 8>(0.0f, v);
    v += dpp<kRowRotate + 4>(0.0f, v);
    v += dpp<kRowRotate + 2>(0.0f, v);
    v += dpp<kRowRotate + 1>(0.0f, v);
    if constexpr (kLanes == 32) {
        const auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(both[0]) + __uint_as_float(both[1]);
    }
    if constexpr (kLanes == 64) {
        v += dpp<kRowBroadcast15, 0xA>(0.0f, v);
        v += dpp<kRowBroadcast31, 0xC>(0.0f, v);
        v = lastLane(v);
    }
    return v;
}
// The wavefront's largest number (a NaN is passed over).
__device__ __forceinline__ float waveMax(float v) {
    v = fmaxf(v, dpp<kRowRotate + 8>(v, v));
    v = fmaxf(v, dpp<kRowRotate + 4>(v, v));
    v = fmaxf(v, dpp<kRowRotate + 2>(v, v));
    v = fmaxf(v, dpp<kRowRotate + 1>(v, v));
    v = fmaxf(v, dpp<kRowBroadcast15, 0xA>(v, v));
    v = fmaxf(v, dpp<kRowBroadcast31, 0xC>(v, v));
    return lastLane(v);
}

// The wavefront's smallest or largest value.
template <bool kMax>
__device__ __forceinline__ uint32_t waveExtreme(uint32_t v) {
    auto with = [&](uint32_t o) { v = kMax ? max(v, o) : min(v, o); };
    with(__builtin_amdgcn_update_dpp(v, v, kRowRotate + 8, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(v, v, kRowRotate + 4, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(v, v, kRowRotate + 2, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(v, v, kRowRotate + 1, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(v, v, kRowBroadcast15, 0xA, 0xF, false));
    with(__builtin_amdgcn_update_dpp(v, v, kRowBroadcast31, 0xC, 0xF, false));
    return __builtin_amdgcn_readlane(v, 63);
}

// 2^x and the larger of numbers (a NaN is passed over), one instruction each.
__device__ __forceinline__ float exp2Fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kLowest = -3.402823466e+38f;

}  // namespace bfo
