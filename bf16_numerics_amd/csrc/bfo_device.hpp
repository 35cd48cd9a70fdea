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

    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
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
    // The first n < N values; the others 0.
    __device__ __forceinline__ void loadPart(const T *p, int n) {
        zero();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i < n) {
                if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(p[i]);
                else w[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
            }
        }
    }
    // Columns [c, c + N) of a row of `cols`, 0 beyond it.
    template <bool kNontemporal = false>
    __device__ __forceinline__ void loadRow(const T *row, uint32_t c, uint32_t cols) {
        if (c + N <= cols) load<kNontemporal>(row + c);
        else if (c < cols) loadPart(row + c, int(cols - c));
        else zero();
    }
};

// Stores N values at columns [c, c + N) of a row of `cols`, rounded to T.
template <bool kNontemporal = false, typename T, int N>
__device__ __forceinline__ void storeRow(T *row, uint32_t c, uint32_t cols, const float (&v)[N]) {
    if (c + N <= cols) {
        uint32_t w[N * sizeof(T) / 4];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
            else if (i % 2 == 0) w[i / 2] = packBf16(v[i], v[i + 1]);
        }
#pragma unroll
        for (int i = 0; i < int(N * sizeof(T) / 4); i += 4) {
            const Words4 q = {w[i], w[i + 1], w[i + 2], w[i + 3]};
            Words4 *p = reinterpret_cast<Words4 *>(row + c) + i / 4;
            if constexpr (kNontemporal) __builtin_nontemporal_store(q, p);
            else *p = q;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + uint32_t(i) < cols) storeOne(row + c + i, v[i]);
    }
}

// Sum over aligned groups of kLanes lanes, the same bits in every lane of a
// group.
template <int kLanes>
__device__ __forceinline__ float laneSum(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// 2^x and the larger of numbers (a NaN is passed over), one instruction each.
__device__ __forceinline__ float exp2Fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowest = -3.402823466e+38f;

}  // namespace bfo
