// bfo_rmsnorm.hip -- gfx950 kernels of root-mean-square norm with the
// residual's addition and 8-bit codes, forward and backward.
//
// A row is held in registers by a group of lanes, 16 bytes of it per lane and
// chunk, so it is read once: the sum, its square, the result and the codes of a
// group of columns (whose lanes are neighbours of one wavefront) come from the
// same registers.
#include "bfo_codes.hpp"
#include "bfo_rows.hpp"

namespace bfo {
namespace {

// The largest of one value each of the kLanes lanes that share a row, as rowSums.
template <int kLanes, int kBlock>
__device__ __forceinline__ uint32_t rowMax(uint32_t v, uint32_t (&red)[kBlock / 64]) {
    v = laneMax<(kLanes < 64 ? kLanes : 64)>(v);
    if constexpr (kLanes > 64) {
        constexpr int kWaves = kLanes / 64;
        const int wave = int(threadIdx.x >> 6), first = wave / kWaves * kWaves;
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = red[first];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v = max(v, red[first + w]);
    }
    return v;
}

// Columns of a row in codes, with one scale for each group (or `whole` row).
template <int kType, int kLanes, int kChunks, int kBlock, int E>
__device__ __forceinline__ void writeCodes(const RmsNormForward &a, uint64_t row, const float (&v)[kChunks][E],
                                           uint32_t (&red)[kBlock / 64]) {
    constexpr int kWidth = kLanes * E, kGroupLanes = kGroup / E;
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const bool live = row < a.rows;
    uint8_t *codes = static_cast<uint8_t *>(a.codes.p) + row * a.codes.stride;
    if (a.group == 0) {
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) amax = max(amax, absBits(v[k][e]));
        const CodeScale s = codeScale<kType>(rowMax<kLanes, kBlock>(amax, red));
        if (live && lane == 0) a.scales[row] = s.scale;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            uint32_t w[E / 4];
            encode<kType, E>(v[k], s.inverse, w);
            if (live) storeCodes<E>(codes + kWidth * k, c, C - kWidth * k, w);
        }
        return;
    }
    const uint32_t groups = (a.cols + kGroup - 1) / kGroup;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) amax = max(amax, absBits(v[k][e]));
        const CodeScale s = codeScale<kType>(laneMax<kGroupLanes>(amax));
        uint32_t w[E / 4];
        encode<kType, E>(v[k], s.inverse, w);
        const int left = C - kWidth * k - c;
        if (live && left > 0) {
            storeCodes<E>(codes + kWidth * k, c, C - kWidth * k, w);
            if (lane % kGroupLanes == 0) a.scales[row * groups + uint32_t(kWidth * k + c) / kGroup] = s.scale;
        }
    }
}

// kLanes lanes own a row, kChunks 16-byte chunks each; kBlock / kLanes rows
// per workgroup at a time.
template <typename T, typename W, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void rmsForwardKernel(RmsNormForward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int kWidth = kLanes * E;  // columns from chunk to chunk
    __shared__ float red[2][kBlock / 64][1];
    __shared__ uint32_t most[2][kBlock / 64];
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const float inv = 1.0f / float(C);
    Chunk<W, E> w[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) w[k].loadRow(static_cast<const W *>(a.weight) + kWidth * k, c, C - kWidth * k);
    int turn = 0;
    for (uint64_t base = uint64_t(blockIdx.x) * kRows; base < a.rows; base += uint64_t(gridDim.x) * kRows) {
        const uint64_t row = base + rowGroup<kLanes>();
        const bool live = row < a.rows;
        const T *x = static_cast<const T *>(a.x.p) + row * a.x.stride;
        Chunk<T, E> raw[kChunks], more[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) raw[k].loadRow(x + kWidth * k, c, C - kWidth * k, live);
        if (a.residual.p) {
            const T *r = static_cast<const T *>(a.residual.p) + row * a.residual.stride;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) more[k].loadRow(r + kWidth * k, c, C - kWidth * k, live);
#pragma unroll
            for (int k = 0; k < kChunks; ++k) raw[k].add(more[k]);
            if (a.total.p && live) {
                T *t = static_cast<T *>(a.total.p) + row * a.total.stride;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) raw[k].storeRow(t + kWidth * k, c, C - kWidth * k);
            }
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] = fmaf(raw[k][e], raw[k][e], s[0]);
        rowSums<kLanes, kBlock>(s, red[turn]);
        const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
        float v[kChunks][E];
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] = raw[k][e] * rstd;
        if (lane == 0 && live && a.rstd) a.rstd[row] = rstd;
        if (a.codes.p && !a.codesOfOut) {
            if (a.codeType == BFO_I8) writeCodes<BFO_I8, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
            else writeCodes<BFO_E4M3, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            w[k].forget();
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] *= w[k][e];
        }
        if (a.codes.p && a.codesOfOut) {
            if (a.codeType == BFO_I8) writeCodes<BFO_I8, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
            else writeCodes<BFO_E4M3, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
        }
        turn ^= 1;
        if (a.out.p && live) {
            T *out = static_cast<T *>(a.out.p) + row * a.out.stride;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) storeRow(out + kWidth * k, c, 0, C - kWidth * k, v[k]);
        }
    }
}

// The normalised values of a row: kept as the row itself, or as codes.
template <typename T, int E, bool kCoded>
struct Normalised;
template <typename T, int E>
struct Normalised<T, E, false> {
    Chunk<T, E> raw;
    __device__ __forceinline__ void load(const RmsNormBackward &a, uint64_t row, int first, int c, bool live) {
        raw.loadRow(static_cast<const T *>(a.x.p) + row * a.x.stride + first, c, int(a.cols) - first, live);
    }
    __device__ __forceinline__ void values(const RmsNormBackward &, float rstd, float (&v)[E]) const {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = raw[e] * rstd;
    }
};
template <typename T, int E>
struct Normalised<T, E, true> {
    uint32_t w[E / 4];
    float scale;
    __device__ __forceinline__ void load(const RmsNormBackward &a, uint64_t row, int first, int c, bool live) {
        const int C = int(a.cols);
        loadCodes<E>(static_cast<const uint8_t *>(a.codes.p) + row * a.codes.stride + first, c, C - first, live, w);
        const uint32_t groups = a.group ? (a.cols + kGroup - 1) / kGroup : 1;
        const uint32_t group = a.group ? uint32_t(first + c) / kGroup : 0;
        scale = live && first + c < C ? a.scales[row * groups + group] : 0.0f;
    }
    __device__ __forceinline__ void values(const RmsNormBackward &a, float, float (&v)[E]) const {
        if (a.codeType == BFO_I8) decode<BFO_I8, E>(w, scale, v);
        else decode<BFO_E4M3, E>(w, scale, v);
    }
};

// Stage 1: dx of the workgroup's rows, and its sums of dout * xhat per column,
// which stay in registers over the rows, are added over the row groups through
// LDS and end as one row of the partials.
template <typename T, typename W, bool kCoded, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void rmsBackwardKernel(RmsNormBackward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int kWidth = kLanes * E;
    __shared__ float red[2][kBlock / 64][1];
    __shared__ float sums[kRows > 1 ? kChunks * E * kLanes : 1];
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const uint32_t sub = rowGroup<kLanes>();
    const float inv = 1.0f / float(C);
    const bool addDx = (a.accumulate & BFO_ACCUMULATE_DX) != 0;
    Chunk<W, E> w[kChunks];
    float dw[kChunks][E];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        w[k].loadRow(static_cast<const W *>(a.weight) + kWidth * k, c, C - kWidth * k);
#pragma unroll
        for (int e = 0; e < E; ++e) dw[k][e] = 0.0f;
    }
    int turn = 0;
    for (uint64_t base = uint64_t(blockIdx.x) * kRows; base < a.rows; base += uint64_t(gridDim.x) * kRows) {
        const uint64_t row = base + sub;
        const bool live = row < a.rows;
        const T *g = static_cast<const T *>(a.dout.p) + row * a.dout.stride;
        const float rstd = live ? a.rstd[row] : 0.0f;
        Normalised<T, E, kCoded> kept[kChunks];
        Chunk<T, E> gr[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            kept[k].load(a, row, kWidth * k, c, live);
            gr[k].loadRow(g + kWidth * k, c, C - kWidth * k, live);
        }
        float xhat[kChunks][E], s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            w[k].forget();
            kept[k].values(a, rstd, xhat[k]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s[0] = fmaf(gr[k][e] * w[k][e], xhat[k][e], s[0]);
                dw[k][e] = fmaf(gr[k][e], xhat[k][e], dw[k][e]);
            }
        }
        rowSums<kLanes, kBlock>(s, red[turn]);
        turn ^= 1;
        if (!live) continue;
        const float mean = s[0] * inv;
        T *dx = static_cast<T *>(a.dx.p) + row * a.dx.stride;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            w[k].forget();
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = fmaf(-xhat[k][e], mean, gr[k][e] * w[k][e]) * rstd;
            if (addDx) {
                Chunk<T, E> old;
                old.loadRow(dx + kWidth * k, c, C - kWidth * k);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] += old[e];
            }
            storeRow(dx + kWidth * k, c, 0, C - kWidth * k, y);
            if (a.out.p) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = xhat[k][e] * w[k][e];
                storeRow(static_cast<T *>(a.out.p) + row * a.out.stride + kWidth * k, c, 0, C - kWidth * k, y);
            }
        }
    }
    if constexpr (kRows > 1) {
        // The groups add in turn: group 0 first, then 1, ...
        __syncthreads();
        for (int r = 0; r < kRows; ++r) {
            if (int(sub) == r) {
#pragma unroll
                for (int i = 0; i < kChunks * E; ++i) {
                    float *p = &sums[i * kLanes + lane], &d = dw[i / E][i % E];
                    if (r > 0) d += *p;
                    if (r < kRows - 1) *p = d;
                }
            }
            __syncthreads();
        }
        if (int(sub) != kRows - 1) return;
    }
    float *part = a.partials + uint64_t(blockIdx.x) * C;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) storeRow(part + kWidth * k, c, 0, C - kWidth * k, dw[k]);
}

// How a row of up to kCols columns is spread, as layer norm's rows are: kLanes
// lanes hold it in kChunks 16-byte chunks each, in workgroups of kBlock lanes.
template <int kWidth, typename T>
struct ForwardShape {
    static constexpr int kCols = kWidth == 0 ? 128 : 256 << kWidth;
    static constexpr int kLanes = kWidth == 0 ? 8 * int(sizeof(T)) : kWidth == 1 ? 64 : 16 << kWidth;
    static constexpr int kChunks = kCols / kLanes / (16 / int(sizeof(T)));
    static constexpr int kBlock = kLanes < 256 ? 256 : kLanes;
};
template <int kWidth, typename T>
struct BackwardShape {
    static constexpr int kCols = kWidth == 0 ? 128 : 256 << kWidth;
    static constexpr int kLanes = kWidth == 0 ? 8 * int(sizeof(T)) : kWidth < 6 ? 32 << kWidth : 1024;
    static constexpr int kChunks = kCols / kLanes / (16 / int(sizeof(T)));
    static constexpr int kBlock = kWidth == 0 ? 256 : kLanes < 512 ? 512 : kLanes;
    static constexpr int kRows = kBlock / kLanes;
};

}  // namespace

uint32_t rmsBackwardBlocks(uint64_t rows, uint32_t cols) {
    const int perBlock = byWidth(cols, [](auto width) { return BackwardShape<decltype(width)::value, bf16_t>::kRows; });
    return gridFor(rows, perBlock, cols <= 4096 ? 512 : 256);
}

uint64_t rmsWorkspaceBound(uint64_t rows, uint32_t cols) {
    const uint64_t own = rmsWorkspaceBytes(rows, cols), narrower = cols > 4096 ? rmsWorkspaceBytes(rows, 4096) : 0;
    return own > narrower ? own : narrower;
}

hipError_t launchRmsNormForward(const RmsNormForward &a, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
        byWidth(a.cols, [&](auto width) {
            using S = ForwardShape<decltype(width)::value, decltype(t)>;
            const uint32_t most = 256 * 16 * 256 / S::kBlock;
            hipLaunchKernelGGL((rmsForwardKernel<decltype(t), decltype(w), S::kLanes, S::kChunks, S::kBlock>),
                               dim3(gridFor(a.rows, S::kBlock / S::kLanes, most)), dim3(S::kBlock), 0, stream, a);
        });
    });
}

hipError_t launchRmsNormBackward(const RmsNormBackward &a, hipStream_t stream) {
    const uint32_t blocks = rmsBackwardBlocks(a.rows, a.cols);
    return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        if (blocks)
            byWidth(a.cols, [&](auto width) {
                using S = BackwardShape<decltype(width)::value, T>;
                if (a.codes.p)
                    hipLaunchKernelGGL((rmsBackwardKernel<T, W, true, S::kLanes, S::kChunks, S::kBlock>), dim3(blocks),
                                       dim3(S::kBlock), 0, stream, a);
                else
                    hipLaunchKernelGGL((rmsBackwardKernel<T, W, false, S::kLanes, S::kChunks, S::kBlock>),
                                       dim3(blocks), dim3(S::kBlock), 0, stream, a);
            });
        hipLaunchKernelGGL((paramSumKernel<W>), dim3((a.cols + kParamCols - 1) / kParamCols),
                           dim3(kParamCols * kParamGroups), 0, stream, a.partials, blocks, a.cols, a.cols,
                           static_cast<W *>(a.dweight), static_cast<W *>(nullptr),
                           a.accumulate & BFO_ACCUMULATE_PARAMS);
    });
}

}  // namespace bfo
