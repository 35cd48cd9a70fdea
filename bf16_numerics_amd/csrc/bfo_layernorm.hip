// bfo_layernorm.hip -- gfx950 kernels of layer norm, forward and backward.
//
// A row is held in registers by a group of lanes (16, one wavefront, or a
// workgroup of 256 or 512), 16 bytes of it per lane and chunk, so it is read
// once: the mean, then the sum of squared differences from it, then the
// result come from the same registers.
#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

constexpr uint32_t kMaxGrid = 1u << 21;

// Sum over the kLanes lanes that share a row.  Rows wider than a wavefront go
// through LDS: `red` holds two slots per wavefront and alternates, so one
// barrier per sum is enough.
template <int kLanes>
__device__ __forceinline__ float rowSum(float v, float *red) {
    v = laneSum<(kLanes < 64 ? kLanes : 64)>(v);
    if constexpr (kLanes > 64) {
        constexpr int kWaves = kLanes / 64;
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += red[i];
    }
    return v;
}

// kLanes lanes own a row, kChunks 16-byte chunks each; kBlock / kLanes rows
// per workgroup.
template <typename T, typename W, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void lnForwardKernel(LayerNormForward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    __shared__ float red[2][kBlock / 64];
    const uint32_t lane = threadIdx.x % kLanes, C = a.cols;
    const float inv = 1.0f / float(C);
    for (uint64_t row = uint64_t(blockIdx.x) * kRows + threadIdx.x / kLanes; row < a.rows;
         row += uint64_t(gridDim.x) * kRows) {
        const T *x = static_cast<const T *>(a.x.p) + row * a.x.stride;
        Chunk<T, E> v[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) v[k].loadRow(x, (lane + kLanes * k) * E, C);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) s += v[k][e];
        const float mean = rowSum<kLanes>(s, red[0]) * inv;
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const uint32_t c = (lane + kLanes * k) * E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = c + uint32_t(e) < C ? v[k][e] - mean : 0.0f;
                q = fmaf(d, d, q);
            }
        }
        const float rstd = 1.0f / sqrtf(rowSum<kLanes>(q, red[1]) * inv + a.eps);
        T *out = static_cast<T *>(a.out.p) + row * a.out.stride;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const uint32_t c = (lane + kLanes * k) * E;
            Chunk<W, E> w, b;
            w.loadRow(static_cast<const W *>(a.weight), c, C);
            if (a.bias) b.loadRow(static_cast<const W *>(a.bias), c, C);
            else b.zero();
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = fmaf((v[k][e] - mean) * rstd, w[e], b[e]);
            storeRow(out, c, C, y);
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Stage 1: dx of the workgroup's rows, and its sums of dout * xhat and dout
// per column, which stay in registers over the rows, are added over the
// groups of lanes through LDS and end as one row of the partials.
template <typename T, typename W, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void lnBackwardKernel(LayerNormBackward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int kSlots = kChunks * E;
    __shared__ float red[4][kBlock / 64];
    __shared__ float sums[kRows > 1 ? 2 * kSlots * kLanes : 1];
    const uint32_t lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes, C = a.cols;
    const float inv = 1.0f / float(C);
    const bool addDx = (a.accumulate & BFO_ACCUMULATE_DX) != 0;
    Chunk<W, E> w[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) w[k].loadRow(static_cast<const W *>(a.weight), (lane + kLanes * k) * E, C);
    float dw[kSlots], db[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) dw[i] = db[i] = 0.0f;
    int turn = 0;
    for (uint64_t row = uint64_t(blockIdx.x) * kRows + sub; row < a.rows; row += uint64_t(gridDim.x) * kRows) {
        const T *x = static_cast<const T *>(a.x.p) + row * a.x.stride;
        const T *g = static_cast<const T *>(a.dout.p) + row * a.dout.stride;
        const float mean = a.mean[row], rstd = a.rstd[row];
        Chunk<T, E> xv[kChunks], gv[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            xv[k].loadRow(x, (lane + kLanes * k) * E, C);
            gv[k].loadRow(g, (lane + kLanes * k) * E, C);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xhat = (xv[k][e] - mean) * rstd, h = gv[k][e] * w[k][e];
                s1 += h;
                s2 = fmaf(h, xhat, s2);
                dw[k * E + e] = fmaf(gv[k][e], xhat, dw[k * E + e]);
                db[k * E + e] += gv[k][e];
            }
        const float c1 = rowSum<kLanes>(s1, red[turn]) * inv;
        const float c2 = rowSum<kLanes>(s2, red[turn + 1]) * inv;
        turn ^= 2;
        T *dx = static_cast<T *>(a.dx.p) + row * a.dx.stride;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const uint32_t c = (lane + kLanes * k) * E;
            Chunk<T, E> old;
            if (addDx) old.loadRow(dx, c, C);
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xhat = (xv[k][e] - mean) * rstd, h = gv[k][e] * w[k][e];
                const float d = rstd * (h - c1 - xhat * c2);
                y[e] = addDx ? old[e] + d : d;
            }
            storeRow(dx, c, C, y);
        }
    }
    float *part = a.partials + uint64_t(blockIdx.x) * 2 * C;
    if constexpr (kRows > 1) {
        // The groups add in turn: group 0 first, then 1, ...
        for (int r = 0; r < kRows; ++r) {
            if (int(sub) == r) {
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
                    float *p = &sums[i * kLanes + lane], *q = p + kSlots * kLanes;
                    if (r > 0) dw[i] += *p, db[i] += *q;
                    if (r < kRows - 1) *p = dw[i], *q = db[i];
                }
            }
            __syncthreads();
        }
        if (int(sub) != kRows - 1) return;
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        float vw[E], vb[E];
#pragma unroll
        for (int e = 0; e < E; ++e) vw[e] = dw[k * E + e], vb[e] = db[k * E + e];
        storeRow(part, (lane + kLanes * k) * E, C, vw);
        storeRow(part + C, (lane + kLanes * k) * E, C, vb);
    }
}

// Stage 2: 32 columns per workgroup; 32 groups of lanes add every 32nd partial
// row each, then the groups' sums are added in order.
constexpr int kParamCols = 32, kParamGroups = 32;
template <typename W>
__global__ __launch_bounds__(kParamCols *kParamGroups) void lnParamKernel(const float *__restrict__ partials,
                                                                          uint32_t count, uint32_t cols,
                                                                          W *dweight, W *dbias, int add) {
    __shared__ float sums[kParamGroups][kParamCols + 1];
    const uint32_t lane = threadIdx.x % kParamCols, group = threadIdx.x / kParamCols;
    const uint32_t c = blockIdx.x * kParamCols + lane;
    W *out = blockIdx.y ? dbias : dweight;
    const float *in = partials + uint64_t(blockIdx.y) * cols + c;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (uint32_t r = group; r < count; r += kParamGroups) s += in[uint64_t(r) * 2 * cols];
    }
    sums[group][lane] = s;
    __syncthreads();
    if (group == 0 && c < cols) {
        float t = 0.0f;
#pragma unroll
        for (int g = 0; g < kParamGroups; ++g) t += sums[g][lane];
        if (add) t += toFloat(out[c]);
        storeOne(out + c, t);
    }
}

uint32_t gridFor(uint64_t rows, int perBlock, uint32_t most) {
    const uint64_t n = (rows + perBlock - 1) / perBlock;
    return uint32_t(n < most ? n : most);
}

// The widest row of each shape: kLanes lanes x kBytes bytes of it per lane
// (kBytes / 16 chunks), in workgroups of kBlock.  fp32 rows take twice the
// chunks of bf16 rows up to 2,048 columns and twice the lanes above.
template <typename F>
void byWidth(uint32_t cols, F f) {
    if (cols <= 128) f(std::integral_constant<int, 0>{});
    else if (cols <= 512) f(std::integral_constant<int, 1>{});
    else if (cols <= 1024) f(std::integral_constant<int, 2>{});
    else if (cols <= 2048) f(std::integral_constant<int, 3>{});
    else if (cols <= 4096) f(std::integral_constant<int, 4>{});
    else if (cols <= 8192) f(std::integral_constant<int, 5>{});
    else f(std::integral_constant<int, 6>{});
}
template <int kWidth, typename T>
struct Shape {
    static constexpr bool f32 = sizeof(T) == 4;
    static constexpr int kLanes = kWidth == 0 ? 16 : kWidth <= 3 ? 64 : f32 ? 512 : 256;
    static constexpr int kCols = kWidth == 0 ? 128 : 256 << kWidth;
    static constexpr int kChunks = kCols / kLanes / (16 / int(sizeof(T)));
    static constexpr int kBlock = kLanes < 256 ? 256 : kLanes;
    static constexpr int kRows = kBlock / kLanes;
};
// Rows per workgroup of each width, the same for both types.
constexpr uint32_t rowsPerBlock(uint32_t cols) { return cols <= 128 ? 16 : cols <= 2048 ? 4 : 1; }

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

constexpr uint32_t kBackwardBlocks = 512;

}  // namespace

uint32_t lnBackwardBlocks(uint64_t rows, uint32_t cols) {
    return gridFor(rows, int(rowsPerBlock(cols)), kBackwardBlocks);
}

hipError_t launchLayerNormForward(const LayerNormForward &a, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
        byWidth(a.cols, [&](auto width) {
            using T = decltype(t);
            using S = Shape<decltype(width)::value, T>;
            hipLaunchKernelGGL((lnForwardKernel<T, decltype(w), S::kLanes, S::kChunks, S::kBlock>),
                               dim3(gridFor(a.rows, S::kRows, kMaxGrid)), dim3(S::kBlock), 0, stream, a);
        });
    });
}

hipError_t launchLayerNormBackward(const LayerNormBackward &a, hipStream_t stream) {
    const uint32_t blocks = lnBackwardBlocks(a.rows, a.cols);
    return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        if (blocks)
            byWidth(a.cols, [&](auto width) {
                using S = Shape<decltype(width)::value, T>;
                static_assert(S::kRows == int(rowsPerBlock(S::kCols)), "the partition is the same for both types");
                hipLaunchKernelGGL((lnBackwardKernel<T, W, S::kLanes, S::kChunks, S::kBlock>), dim3(blocks),
                                   dim3(S::kBlock), 0, stream, a);
            });
        hipLaunchKernelGGL((lnParamKernel<W>), dim3((a.cols + kParamCols - 1) / kParamCols, a.dbias ? 2 : 1),
                           dim3(kParamCols * kParamGroups), 0, stream, a.partials, blocks, a.cols,
                           static_cast<W *>(a.dweight), static_cast<W *>(a.dbias),
                           a.accumulate & BFO_ACCUMULATE_PARAMS);
    });
}

}  // namespace bfo
