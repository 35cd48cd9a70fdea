// bfo_rows.hpp -- what the norms over rows share: sums over the lanes that hold
// a row, sums over the rows for the parameters' gradients, and the choice of a
// kernel by types and width.
#pragma once

#include <type_traits>

#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

// Sums of kCount values each over the kLanes lanes that share a row.  Rows
// wider than a wavefront go through LDS, `red` holding the wavefronts' sums;
// alternating between two such arrays, one barrier a call is enough.
template <int kLanes, int kBlock, int kCount>
__device__ __forceinline__ void rowSums(float (&v)[kCount], float (&red)[kBlock / 64][kCount]) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] = laneSum<(kLanes < 64 ? kLanes : 64)>(v[i]);
    if constexpr (kLanes > 64) {
        constexpr int kWaves = kLanes / 64;
        const int wave = int(threadIdx.x >> 6), first = wave / kWaves * kWaves;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < kCount; ++i) red[wave][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            v[i] = red[first][i];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v[i] += red[first + w][i];
        }
    }
}

// The calling lane's row group within its workgroup: a scalar where a
// wavefront has one row.
template <int kLanes>
__device__ __forceinline__ uint32_t rowGroup() {
    const uint32_t group = threadIdx.x / kLanes;
    if constexpr (kLanes >= 64) return uint32_t(__builtin_amdgcn_readfirstlane(int(group)));
    else return group;
}

template <typename W>
__device__ __forceinline__ void storeParam(W *out, float v, bool add) {
    storeOne(out, add ? toFloat(*out) + v : v);
}

// Column slabs of a launch that sums over all rows by columns.  Workgroups go to the
// XCDs in turn: the slabs that share a row's 128-byte lines are given to one XCD,
// whose L2 then reads them once.
constexpr uint32_t kXcds = 8;
template <typename T, int kSlabCols>
struct Slabs {
    static constexpr uint32_t kShare = 128 / (kSlabCols * sizeof(T));  // slabs of a line
    static __host__ __device__ uint32_t workgroups(uint32_t cols) {
        const uint32_t lines = (cols + kSlabCols * kShare - 1) / (kSlabCols * kShare);
        return (lines + kXcds - 1) / kXcds * kXcds * kShare;
    }
    static __device__ uint32_t firstColumn(uint32_t workgroup) {
        const uint32_t line = workgroup / (kXcds * kShare) * kXcds + workgroup % kXcds;
        return (line * kShare + workgroup / kXcds % kShare) * kSlabCols;
    }
};

// Sums of the partials' `count` rows, `stride` floats apart, of dweight's columns and
// behind them dbias's: 32 columns per workgroup; 32 groups of lanes add every 32nd
// row each, then the groups' sums are added in order.
constexpr int kParamCols = 32, kParamGroups = 32;
template <typename W>
__global__ __launch_bounds__(kParamCols *kParamGroups) void paramSumKernel(const float *__restrict__ partials,
                                                                           uint32_t count, uint32_t stride,
                                                                           uint32_t cols, W *dweight, W *dbias,
                                                                           int add) {
    __shared__ float sums[kParamGroups][kParamCols + 1];
    const uint32_t lane = threadIdx.x % kParamCols, group = threadIdx.x / kParamCols;
    const uint32_t c = blockIdx.x * kParamCols + lane;
    W *out = blockIdx.y ? dbias : dweight;
    const float *in = partials + uint64_t(blockIdx.y) * cols + c;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 16
        for (uint32_t r = group; r < count; r += kParamGroups) s += in[uint64_t(r) * stride];
    }
    sums[group][lane] = s;
    __syncthreads();
    if (group == 0 && c < cols) {
        float t = 0.0f;
#pragma unroll
        for (int g = 0; g < kParamGroups; ++g) t += sums[g][lane];
        storeParam(out + c, t, add != 0);
    }
}

uint32_t gridFor(uint64_t rows, int perBlock, uint32_t most) {
    const uint64_t n = (rows + perBlock - 1) / perBlock;
    return uint32_t(n < most ? n : most);
}

template <typename F>
auto byWidth(uint32_t cols, F f) {
    if (cols <= 128) return f(std::integral_constant<int, 0>{});
    if (cols <= 512) return f(std::integral_constant<int, 1>{});
    if (cols <= 1024) return f(std::integral_constant<int, 2>{});
    if (cols <= 2048) return f(std::integral_constant<int, 3>{});
    if (cols <= 4096) return f(std::integral_constant<int, 4>{});
    if (cols <= 8192) return f(std::integral_constant<int, 5>{});
    return f(std::integral_constant<int, 6>{});
}

template <typename F>
hipError_t byTypes(int dtype, int paramDtype, F f) {
    if (dtype == BFO_BF16) {
        if (paramDtype == BFO_BF16) f(bf16_t(0), bf16_t(0));
        else f(bf16_t(0), float(0));
    } else {
        if (paramDtype == BFO_BF16) f(float(0), bf16_t(0));
        else f(float(0), float(0));
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace bfo
