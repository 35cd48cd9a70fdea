// bfo_rmsnorm.hip -- gfx950 kernels of root-mean-square norm with the
// residual's addition and 8-bit codes, forward and backward.
//
//   t = x + residual, rounded; rstd = 1 / sqrt(sum(t^2) / cols + eps)
//   xhat = t * rstd;  out = xhat * weight
//   dx = rstd * (h - xhat * sum(h * xhat) / cols), h = weight * dout
//   dweight = sum over the rows of dout * xhat
//
// A row is held in registers by a group of lanes, 16 bytes of it per lane and
// chunk, so it is read once: the sum, its square, the result and the codes of a
// group of columns (whose lanes are neighbours of one wavefront) come from the
// same registers.  Bound by memory: 8192 x 4096 bf16 with residual, total, out and
// codes (303 MB) 49.3 us, 6.1 TB/s; backward from codes with out again (236 MB)
// 42.7 us, of which the first launch, at 6.2 TB/s with its partial sums, 39.  Of the
// steps there: forward 58.3 in plain loads and stores, 49.8 nontemporal; backward
// 47.6, 42.8 nontemporal.
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
template <int kType, Loads kLoads, int kLanes, int kChunks, int kBlock, int E>
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
            if (live) storeCodes<kLoads, false, E>(codes + kWidth * k, c, C - kWidth * k, w);
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
            storeCodes<kLoads, false, E>(codes + kWidth * k, c, C - kWidth * k, w);
            if (lane % kGroupLanes == 0) a.scales[row * groups + uint32_t(kWidth * k + c) / kGroup] = s.scale;
        }
    }
}

// E weights from column c on, 0 behind the last.
template <int E>
__device__ __forceinline__ void loadWeights(const void *weight, int type, int c, int C, float (&w)[E]) {
    if (type == BFO_BF16) {
        Chunk<bf16_t, E> q;
        q.loadRow(static_cast<const bf16_t *>(weight), c, C);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = q[e];
    } else {
        Chunk<float, E> q;
        q.loadRow(static_cast<const float *>(weight), c, C);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = q[e];
    }
}

// kLanes lanes own a row, kChunks 16-byte chunks each; kBlock / kLanes rows
// per workgroup at a time.
template <typename T, Loads kLoads, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void rmsForwardKernel(RmsNormForward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int kWidth = kLanes * E;  // columns from chunk to chunk
    __shared__ float red[2][kBlock / 64][1];
    __shared__ uint32_t most[2][kBlock / 64];
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const float inv = 1.0f / float(C);
    float w[kChunks][E];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) loadWeights(a.weight, a.paramDtype, kWidth * k + c, C, w[k]);
    int turn = 0;
    for (uint64_t base = uint64_t(blockIdx.x) * kRows; base < a.rows; base += uint64_t(gridDim.x) * kRows) {
        const uint64_t row = base + rowGroup<kLanes>(), from = loadedRow(row, a.rows);
        const bool live = row < a.rows;
        Chunk<T, E> raw[kChunks];
        const T *x = static_cast<const T *>(a.x.p) + from * a.x.stride;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) loadChunk<kLoads>(raw[k], x, kWidth * k + c, C, live);
        if (a.residual.p) {
            Chunk<T, E> more[kChunks];
            const T *r = static_cast<const T *>(a.residual.p) + from * a.residual.stride;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) loadChunk<kLoads>(more[k], r, kWidth * k + c, C, live);
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                raw[k].add(more[k]);
                settle<kLoads>(raw[k], kWidth * k + c, C, live);
            }
            if (a.total.p && live) {
                T *t = static_cast<T *>(a.total.p) + row * a.total.stride;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) storeChunk<kLoads>(raw[k], t, kWidth * k + c, C);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kChunks; ++k) settle<kLoads>(raw[k], kWidth * k + c, C, live);
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
            if (a.codeType == BFO_I8) writeCodes<BFO_I8, kLoads, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
            else writeCodes<BFO_E4M3, kLoads, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] *= w[k][e];
        if (a.codes.p && a.codesOfOut) {
            if (a.codeType == BFO_I8) writeCodes<BFO_I8, kLoads, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
            else writeCodes<BFO_E4M3, kLoads, kLanes, kChunks, kBlock>(a, row, v, most[turn]);
        }
        turn ^= 1;
        if (a.out.p && live) {
            T *out = static_cast<T *>(a.out.p) + row * a.out.stride;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) storeChunk<kLoads>(out, kWidth * k + c, C, v[k]);
        }
    }
}

// The normalised values of N columns: kept as the row itself, or as codes.
template <typename T, int N, bool kCoded, Loads kLoads>
struct Normalised;
template <typename T, int N, Loads kLoads>
struct Normalised<T, N, false, kLoads> {
    Chunk<T, N> raw;
    __device__ __forceinline__ void load(const RmsNormBackward &a, uint64_t row, int c, bool live) {
        loadChunk<kLoads>(raw, static_cast<const T *>(a.x.p) + row * a.x.stride, c, int(a.cols), live);
    }
    __device__ __forceinline__ void values(const RmsNormBackward &a, float rstd, int c, bool live, float (&v)[N]) {
        settle<kLoads>(raw, c, int(a.cols), live);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = raw[e] * rstd;
    }
};
template <typename T, int N, Loads kLoads>
struct Normalised<T, N, true, kLoads> {
    uint32_t w[N / 4];
    float scale;
    __device__ __forceinline__ void load(const RmsNormBackward &a, uint64_t row, int c, bool live) {
        const int C = int(a.cols);
        loadCodes<kLoads, N>(static_cast<const uint8_t *>(a.codes.p) + row * a.codes.stride, c, C, live, w);
        const uint32_t groups = a.group ? (a.cols + kGroup - 1) / kGroup : 1;
        scale = a.scales[row * groups + (a.group ? uint32_t(min(c, C - 1)) / kGroup : 0)];
    }
    __device__ __forceinline__ void values(const RmsNormBackward &a, float, int c, bool live, float (&v)[N]) {
        const bool there = live && c < int(a.cols);
        settleCodes<kLoads, N>(w, c, int(a.cols), live);
        scale = there ? scale : 0.0f;  // of another row or group it may be no number
        if (a.codeType == BFO_I8) decode<BFO_I8, N>(w, scale, v);
        else decode<BFO_E4M3, N>(w, scale, v);
    }
};

// dx of the rows first, first + step, ... of a workgroup's kBlock / kLanes row
// groups; with kSums, each lane's sums of dout * xhat per column.
template <typename T, bool kCoded, Loads kLoads, int kLanes, int kChunks, int kBlock, bool kSums, int kSlots, int E>
__device__ __forceinline__ void rowGradients(const RmsNormBackward &a, uint64_t first, uint64_t step,
                                             float (&red)[2][kBlock / 64][1], float (&dw)[kSlots][E]) {
    constexpr int kWidth = kLanes * E;
    const int c = int(threadIdx.x % kLanes) * E, C = int(a.cols);
    const uint32_t sub = rowGroup<kLanes>();
    const float inv = 1.0f / float(C);
    const bool addDx = (a.accumulate & BFO_ACCUMULATE_DX) != 0;
    float w[kChunks][E];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) loadWeights(a.weight, a.paramDtype, kWidth * k + c, C, w[k]);
    int turn = 0;
    for (uint64_t base = first; base < a.rows; base += step) {
        const uint64_t row = base + sub, from = loadedRow(row, a.rows);
        const bool live = row < a.rows;
        const float rstd = a.rstd[from];
        const T *g = static_cast<const T *>(a.dout.p) + from * a.dout.stride;
        Normalised<T, E, kCoded, kLoads> kept[kChunks];
        Chunk<T, E> gr[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            kept[k].load(a, from, kWidth * k + c, live);
            loadChunk<kLoads>(gr[k], g, kWidth * k + c, C, live);
        }
        float xhat[kChunks][E], h[kChunks][E], s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            kept[k].values(a, live ? rstd : 0.0f, kWidth * k + c, live, xhat[k]);
            settle<kLoads>(gr[k], kWidth * k + c, C, live);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[k][e] = gr[k][e] * w[k][e];
                s[0] = fmaf(h[k][e], xhat[k][e], s[0]);
                if constexpr (kSums) dw[k][e] = fmaf(gr[k][e], xhat[k][e], dw[k][e]);
            }
        }
        rowSums<kLanes, kBlock>(s, red[turn]);
        turn ^= 1;
        if (!live) continue;
        const float mean = s[0] * inv;
        T *dx = static_cast<T *>(a.dx.p) + row * a.dx.stride;
        T *out = static_cast<T *>(a.out.p) + row * a.out.stride;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = fmaf(-xhat[k][e], mean, h[k][e]) * rstd;
            if (addDx) {
                Chunk<T, E> old;
                old.loadRow(dx, kWidth * k + c, C);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] += old[e];
            }
            storeChunk<kLoads>(dx, kWidth * k + c, C, y);
            if (a.out.p) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = xhat[k][e] * w[k][e];
                storeChunk<kLoads>(out, kWidth * k + c, C, y);
            }
        }
    }
}

// Stage 1: dx of the workgroup's rows, and its sums of dout * xhat per column,
// which stay in registers over the rows, are added over the row groups through
// LDS and end as one row of the partials.
template <typename T, bool kCoded, Loads kLoads, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock, 4) void rmsBackwardKernel(RmsNormBackward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int kWidth = kLanes * E;
    __shared__ float red[2][kBlock / 64][1];
    __shared__ float sums[kRows > 1 ? kChunks * E * kLanes : 1];
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const uint32_t sub = rowGroup<kLanes>();
    float dw[kChunks][E];
#pragma unroll
    for (int i = 0; i < kChunks * E; ++i) dw[i / E][i % E] = 0.0f;
    rowGradients<T, kCoded, kLoads, kLanes, kChunks, kBlock, true>(a, uint64_t(blockIdx.x) * kRows,
                                                                   uint64_t(gridDim.x) * kRows, red, dw);
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
    for (int k = 0; k < kChunks; ++k) storeRow(part, kWidth * k + c, 0, C, dw[k]);
}

// Few rows, in one launch and without partials: rstd is given, so dweight needs
// nothing of dx.  The first workgroups sum kSlabCols columns each over all rows (4
// columns a lane), the others form dx; both read dout and the kept rows, which the
// caches hold.
template <typename T, bool kCoded, Loads kLoads, int kLanes, int kChunks, int kBlock, int kSlabCols>
__global__ __launch_bounds__(kBlock) void rmsBackwardFewKernel(RmsNormBackward a, uint32_t slabs) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int N = 4, kRowLanes = kSlabCols / N, kGroups = kBlock / kRowLanes, kAtOnce = 4;
    constexpr int kParts = kBlock / kSlabCols;  // lanes that add one column's sums
    __shared__ float red[2][kBlock / 64][1];
    __shared__ float sums[kGroups][kSlabCols + 1];
    if (blockIdx.x >= slabs) {
        float none[1][E];
        rowGradients<T, kCoded, kLoads, kLanes, kChunks, kBlock, false>(a, uint64_t(blockIdx.x - slabs) * kRows,
                                                                      uint64_t(gridDim.x - slabs) * kRows, red, none);
        return;
    }
    const int c0 = int(Slabs<T, kSlabCols>::firstColumn(blockIdx.x)), C = int(a.cols);
    if (c0 >= C) return;
    const int c = c0 + int(threadIdx.x % kRowLanes) * N;
    const uint32_t group = threadIdx.x / kRowLanes;
    float dw[N] = {};
    for (uint64_t base = group; base < a.rows; base += kGroups * kAtOnce) {
        Normalised<T, N, kCoded, kLoads> kept[kAtOnce];
        Chunk<T, N> gr[kAtOnce];
        float rstd[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint64_t row = base + kGroups * i, from = loadedRow(row, a.rows);
            kept[i].load(a, from, c, row < a.rows);
            loadChunk<kLoads>(gr[i], static_cast<const T *>(a.dout.p) + from * a.dout.stride, c, C, row < a.rows);
            rstd[i] = a.rstd[from];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const bool live = base + kGroups * i < a.rows;
            float xhat[N];
            kept[i].values(a, live ? rstd[i] : 0.0f, c, live, xhat);
            settle<kLoads>(gr[i], c, C, live);
#pragma unroll
            for (int e = 0; e < N; ++e) dw[e] = fmaf(gr[i][e], xhat[e], dw[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sums[group][c - c0 + e] = dw[e];
    __syncthreads();
    const int column = int(threadIdx.x) / kParts, part = int(threadIdx.x) % kParts;
    float t = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups / kParts; ++g) t += sums[part * (kGroups / kParts) + g][column];
#pragma unroll
    for (int d = 1; d < kParts; d *= 2) t += __shfl_xor(t, d, 64);
    if (part == 0 && c0 + column < C) {
        const bool add = (a.accumulate & BFO_ACCUMULATE_PARAMS) != 0;
        if (a.paramDtype == BFO_BF16) storeParam(static_cast<bf16_t *>(a.dweight) + c0 + column, t, add);
        else storeParam(static_cast<float *>(a.dweight) + c0 + column, t, add);
    }
}

// How a row of up to kCols columns is spread: kLanes lanes hold it in kChunks
// 16-byte chunks each, in workgroups of kBlock lanes.  Forward, 8192 x 4096 bf16: four
// chunks a lane 60 us, two 58, one 58 (plain loads and stores).  Backward, bf16 from
// codes, one / two / four chunks a lane: 8192 x 4096 42.5 / 42.7 / 49.6 us, 16384 x 1600
// 35.3 / 34.2 / 41.6, 4096 x 8192 49.4 / 45.4 / 48.8 (one in 256 workgroups of 1,024
// lanes); fp32 two chunks 40.8 and four 43.4 at 4096 x 4096.
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
    static constexpr int kWide = 8 * int(sizeof(T)) << kWidth;  // two chunks a lane
    static constexpr int kLanes = kWidth == 0 ? 8 * int(sizeof(T)) : kWide < 64 ? 64 : kWide > 1024 ? 1024 : kWide;
    static constexpr int kChunks = kCols / kLanes / (16 / int(sizeof(T)));
    static constexpr int kBlock = kWidth == 0 ? 256 : kLanes < 512 ? 512 : kLanes;
    static constexpr int kRows = kBlock / kLanes;
};

// Up to here one launch for all gradients takes no longer than rows and partials, as
// called from Python on inputs that no cache holds, from bf16 codes: 2,048 rows of
// 2,048 columns 11.5 us against 13.0 (4,096 rows 19.1 and 13.1), 1,024 of 4,096 10.6
// and 13.1 (2,048: 16.0 and 13.5), 512 of 8,192 10.6 and 13.6 (1,024: 16.2 and 15.8), 256
// of 16,384 12.4 and 14.2 (512: 18.3 and 16.9); fp32 rows 2,048 of 1,600 12.0 and 12.8,
// of 2,048 14.0 and 13.0.  A column workgroup walks all rows by itself.
uint64_t fewRows(uint32_t cols) { return cols <= 2048 ? 2048 : cols <= 4096 ? 1024 : cols <= 8192 ? 512 : 256; }
template <int kCols, typename F>
void bySlab(uint64_t rows, F f) {
    if constexpr (kCols > 4096) f(std::integral_constant<int, 32>{});
    else if constexpr (kCols > 2048) f(std::integral_constant<int, 16>{});
    else if (rows <= 512) f(std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 8>{});
}

template <typename F>
void byType(int dtype, F f) {
    dtype == BFO_BF16 ? f(bf16_t(0)) : f(float(0));
}

}  // namespace

// Workgroups of stage 1: two a CU, or one where a row takes 1,024 lanes.  8192 x 4096
// bf16 in 512 / 768 / 1,024: 42.7 / 45.6 / 54.7 us (256 of twice the lanes 43.6).
uint32_t rmsBackwardBlocks(uint64_t rows, uint32_t cols) {
    if (rows <= fewRows(cols)) return 0;
    const int perBlock = byWidth(cols, [](auto width) { return BackwardShape<decltype(width)::value, bf16_t>::kRows; });
    return gridFor(rows, perBlock, cols <= 8192 ? 512 : 256);
}

// Up to 8,192 columns the size grows with both: more columns mean no fewer
// workgroups, from no more rows on.  Above, there are half as many workgroups.
uint64_t rmsWorkspaceBound(uint64_t rows, uint32_t cols) {
    const uint64_t own = rmsWorkspaceBytes(rows, cols), narrower = cols > 8192 ? rmsWorkspaceBytes(rows, 8192) : 0;
    return own > narrower ? own : narrower;
}

hipError_t launchRmsNormForward(const RmsNormForward &a, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    byType(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int matrices = 1 + (a.residual.p ? 1 : 0) + (a.total.p ? 1 : 0) + (a.out.p ? 1 : 0);
        byLoads<T>(a.cols, a.rows * a.cols * (matrices * sizeof(T) + (a.codes.p ? 1 : 0)), [&](auto loads) {
            byWidth(a.cols, [&](auto width) {
                using S = ForwardShape<decltype(width)::value, T>;
                // At most 16 workgroups of 256 lanes a CU, which keep their weights over
                // their rows.
                const uint32_t most = 256 * 16 * 256 / S::kBlock;
                if constexpr (decltype(loads)::value != kNarrow || decltype(width)::value == 0)
                    hipLaunchKernelGGL((rmsForwardKernel<T, decltype(loads)::value, S::kLanes, S::kChunks, S::kBlock>),
                                       dim3(gridFor(a.rows, S::kBlock / S::kLanes, most)), dim3(S::kBlock), 0, stream,
                                       a);
            });
        });
    });
    return hipGetLastError();
}

hipError_t launchRmsNormBackward(const RmsNormBackward &a, hipStream_t stream) {
    const uint32_t blocks = rmsBackwardBlocks(a.rows, a.cols);
    if (a.rows)
        byType(a.dtype, [&](auto t) {
            using T = decltype(t);
            auto wide = [&](auto coded) {
                byWidth(a.cols, [&](auto width) {
                    using S = BackwardShape<decltype(width)::value, T>;
                    if (blocks) {
                        const int matrices = 2 + (a.x.p ? 1 : 0) + (a.out.p ? 1 : 0);
                        byLoads<T>(a.cols, a.rows * a.cols * (matrices * sizeof(T) + (a.x.p ? 0 : 1)), [&](auto loads) {
                            if constexpr (decltype(loads)::value != kNarrow || decltype(width)::value == 0)
                                hipLaunchKernelGGL((rmsBackwardKernel<T, decltype(coded)::value, decltype(loads)::value,
                                                                      S::kLanes, S::kChunks, S::kBlock>),
                                                   dim3(blocks), dim3(S::kBlock), 0, stream, a);
                        });
                    } else {
                        bySlab<S::kCols>(a.rows, [&](auto columns) {
                            constexpr int kSlabCols = decltype(columns)::value;
                            const uint32_t slabs = Slabs<T, kSlabCols>::workgroups(a.cols);
                            auto with = [&](auto loads) {
                                hipLaunchKernelGGL((rmsBackwardFewKernel<T, decltype(coded)::value,
                                                                         decltype(loads)::value, S::kLanes, S::kChunks,
                                                                         S::kBlock, kSlabCols>),
                                                   dim3(slabs + gridFor(a.rows, S::kRows, 1024)), dim3(S::kBlock), 0,
                                                   stream, a, slabs);
                            };
                            if constexpr (decltype(width)::value == 0)
                                if (a.cols < 16 / sizeof(T)) return with(Constant<kNarrow>{});
                            with(Constant<kRagged>{});
                        });
                    }
                });
            };
            a.codes.p ? wide(std::true_type{}) : wide(std::false_type{});
        });
    if (blocks || !a.rows) byType(a.paramDtype, [&](auto w) {
        using W = decltype(w);
        hipLaunchKernelGGL((paramSumKernel<W>), dim3((a.cols + kParamCols - 1) / kParamCols),
                           dim3(kParamCols * kParamGroups), 0, stream, a.partials, blocks, a.cols, a.cols,
                           static_cast<W *>(a.dweight), static_cast<W *>(nullptr),
                           a.accumulate & BFO_ACCUMULATE_PARAMS);
    });
    return hipGetLastError();
}

}  // namespace bfo
