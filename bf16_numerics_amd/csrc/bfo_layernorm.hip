// bfo_layernorm.hip -- gfx950 kernels of layer norm, forward and backward.
//
// A row is held in registers by a group of lanes (16 lanes up to a workgroup),
// 16 bytes of it per lane and chunk, so it is read once: the mean, then the
// sum of squared differences from it, then the result come from the same
// registers.
#include "bfo_device.hpp"
#include "bfo_ops.hpp"
#include "bfo_rows.hpp"

namespace bfo {
namespace {

// kLanes lanes own a row, kChunks 16-byte chunks each; kBlock / kLanes rows
// per workgroup at a time.
template <typename T, typename W, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void lnForwardKernel(LayerNormForward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    __shared__ float red[2][kBlock / 64][1];
    constexpr int kWidth = kLanes * E;  // columns from chunk to chunk
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const float inv = 1.0f / float(C);
    Chunk<W, E> w[kChunks], b[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        w[k].loadRow(static_cast<const W *>(a.weight) + kWidth * k, c, C - kWidth * k);
        b[k].loadRow(static_cast<const W *>(a.bias) + kWidth * k, c, C - kWidth * k, a.bias != nullptr);
    }
    for (uint64_t base = uint64_t(blockIdx.x) * kRows; base < a.rows; base += uint64_t(gridDim.x) * kRows) {
        const uint64_t row = base + rowGroup<kLanes>();
        const T *x = static_cast<const T *>(a.x.p) + row * a.x.stride;
        Chunk<T, E> raw[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) raw[k].loadRow(x + kWidth * k, c, C - kWidth * k, row < a.rows);
        float v[kChunks][E], s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[k][e] = raw[k][e];
                s[0] += v[k][e];
            }
        rowSums<kLanes, kBlock>(s, red[0]);
        const float mean = s[0] * inv;
        float q[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const int left = C - kWidth * k - c;  // columns of the chunk that are there
            float t = q[0];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[k][e] -= mean;
                t = fmaf(v[k][e], v[k][e], t);
            }
            if (left >= E) {
                q[0] = t;
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) q[0] = e < left ? fmaf(v[k][e], v[k][e], q[0]) : q[0];
            }
        }
        rowSums<kLanes, kBlock>(q, red[1]);
        const float rstd = 1.0f / sqrtf(q[0] * inv + a.eps);
        if (row < a.rows) {
            T *out = static_cast<T *>(a.out.p) + row * a.out.stride;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                w[k].forget();
                b[k].forget();
                float y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = fmaf(v[k][e] * rstd, w[k][e], b[k][e]);
                storeRow(out + kWidth * k, c, 0, C - kWidth * k, y);
            }
            if (lane == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
    }
}

// dx of the rows first, first + step, ... of a workgroup's kBlock / kLanes row
// groups; with kSums, each lane's sums of dout * xhat and dout per column.
template <typename T, typename W, int kLanes, int kChunks, int kBlock, bool kSums, int kSlots>
__device__ __forceinline__ void rowGradients(const LayerNormBackward &a, uint64_t first, uint64_t step,
                                             float (&red)[2][kBlock / 64][2], float (&dw)[kSlots],
                                             float (&db)[kSlots]) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kWidth = kLanes * E;  // columns from chunk to chunk
    const int c = int(threadIdx.x % kLanes) * E, C = int(a.cols);
    const uint32_t sub = rowGroup<kLanes>();
    const float inv = 1.0f / float(C);
    const bool addDx = (a.accumulate & BFO_ACCUMULATE_DX) != 0;
    Chunk<W, E> w[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) w[k].loadRow(static_cast<const W *>(a.weight) + kWidth * k, c, C - kWidth * k);
    int turn = 0;
    for (uint64_t base = first; base < a.rows; base += step) {
        const uint64_t row = base + sub;
        const bool live = row < a.rows;
        const T *x = static_cast<const T *>(a.x.p) + row * a.x.stride;
        const T *g = static_cast<const T *>(a.dout.p) + row * a.dout.stride;
        const float mean = live ? a.mean[row] : 0.0f, rstd = live ? a.rstd[row] : 0.0f;
        Chunk<T, E> xr[kChunks], gr[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            xr[k].loadRow(x + kWidth * k, c, C - kWidth * k, live);
            gr[k].loadRow(g + kWidth * k, c, C - kWidth * k, live);
        }
        float xhat[kChunks * E], h[kChunks * E], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            if constexpr (kChunks * E > 8) w[k].forget();  // two registers a value are too many
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = k * E + e;
                xhat[j] = (xr[k][e] - mean) * rstd;
                h[j] = gr[k][e] * w[k][e];
                s[0] += h[j];
                s[1] = fmaf(h[j], xhat[j], s[1]);
                if constexpr (kSums) {
                    dw[j] = fmaf(gr[k][e], xhat[j], dw[j]);
                    db[j] += gr[k][e];
                }
            }
        }
        rowSums<kLanes, kBlock>(s, red[turn]);
        turn ^= 1;
        if (!live) continue;
        // dx = rstd * (h - mean(h) - xhat * mean(h * xhat))
        const float c1 = s[0] * inv * rstd, c2 = s[1] * inv * rstd;
        T *dx = static_cast<T *>(a.dx.p) + row * a.dx.stride;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = fmaf(h[k * E + e], rstd, -fmaf(xhat[k * E + e], c2, c1));
            if (addDx) {
                Chunk<T, E> old;
                old.loadRow(dx + kWidth * k, c, C - kWidth * k);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] += old[e];
            }
            storeRow(dx + kWidth * k, c, 0, C - kWidth * k, y);
        }
    }
}

// Stage 1: dx of the workgroup's rows, and its sums per column, which stay in
// registers over the rows, are added over the row groups through LDS and end
// as one row of the partials.
template <typename T, typename W, int kLanes, int kChunks, int kBlock>
__global__ __launch_bounds__(kBlock) void lnBackwardKernel(LayerNormBackward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int kRows = kBlock / kLanes;
    constexpr int kSlots = kChunks * E;
    constexpr int kWidth = kLanes * E;
    __shared__ float red[2][kBlock / 64][2];
    __shared__ float sums[kRows > 1 ? 2 * kSlots * kLanes : 1];
    const int lane = int(threadIdx.x % kLanes), c = lane * E, C = int(a.cols);
    const uint32_t sub = rowGroup<kLanes>();
    float dw[kSlots], db[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) dw[i] = db[i] = 0.0f;
    rowGradients<T, W, kLanes, kChunks, kBlock, true>(a, uint64_t(blockIdx.x) * kRows, uint64_t(gridDim.x) * kRows, red,
                                                      dw, db);
    float *part = a.partials + uint64_t(blockIdx.x) * 2 * C;
    if constexpr (kRows > 1) {
        // The groups add in turn: group 0 first, then 1, ...
        __syncthreads();
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
        storeRow(part + kWidth * k, c, 0, C - kWidth * k, vw);
        storeRow(part + C + kWidth * k, c, 0, C - kWidth * k, vb);
    }
}

// Few rows, in one launch and without partials: mean and rstd are given, so
// dweight and dbias need nothing of dx.  The first workgroups sum kSlabCols
// columns each over all rows (4 columns a lane), the others form dx; both read x
// and dout, which the caches hold.
template <typename T, typename W, int kLanes, int kChunks, int kBlock, int kSlabCols>
__global__ __launch_bounds__(kBlock) void lnBackwardFewKernel(LayerNormBackward a, uint32_t slabs) {
    constexpr int kRows = kBlock / kLanes;
    constexpr int N = 4, kRowLanes = kSlabCols / N, kGroups = kBlock / kRowLanes, kAtOnce = 4;
    constexpr int kParts = kBlock / (2 * kSlabCols);  // lanes that add one column's sums
    __shared__ float red[2][kBlock / 64][2];
    __shared__ float sums[kGroups][2 * kSlabCols + 1];
    if (blockIdx.x >= slabs) {
        float none[1];
        rowGradients<T, W, kLanes, kChunks, kBlock, false>(a, uint64_t(blockIdx.x - slabs) * kRows,
                                                           uint64_t(gridDim.x - slabs) * kRows, red, none, none);
        return;
    }
    const int c0 = int(Slabs<T, kSlabCols>::firstColumn(blockIdx.x)), left = int(a.cols) - c0;
    if (left <= 0) return;
    const int c = int(threadIdx.x % kRowLanes) * N;
    const uint32_t group = threadIdx.x / kRowLanes;
    float dw[N] = {}, db[N] = {};
    for (uint64_t base = group; base < a.rows; base += kGroups * kAtOnce) {
        Chunk<T, N> xr[kAtOnce], gr[kAtOnce];
        float mean[kAtOnce], rstd[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint64_t row = base + kGroups * i;
            const bool live = row < a.rows;
            xr[i].loadRow(static_cast<const T *>(a.x.p) + row * a.x.stride + c0, c, left, live);
            gr[i].loadRow(static_cast<const T *>(a.dout.p) + row * a.dout.stride + c0, c, left, live);
            mean[i] = live ? a.mean[row] : 0.0f;
            rstd[i] = live ? a.rstd[row] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                dw[e] = fmaf(gr[i][e], (xr[i][e] - mean[i]) * rstd[i], dw[e]);
                db[e] += gr[i][e];
            }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        sums[group][c + e] = dw[e];
        sums[group][kSlabCols + c + e] = db[e];
    }
    __syncthreads();
    const int column = int(threadIdx.x) / kParts, part = int(threadIdx.x) % kParts;
    float t = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups / kParts; ++g) t += sums[part * (kGroups / kParts) + g][column];
#pragma unroll
    for (int d = 1; d < kParts; d *= 2) t += __shfl_xor(t, d, 64);
    const int at = column % kSlabCols;
    if (part == 0 && at < left) {
        W *out = static_cast<W *>(column < kSlabCols ? a.dweight : a.dbias);
        if (out) storeParam(out + c0 + at, t, (a.accumulate & BFO_ACCUMULATE_PARAMS) != 0);
    }
}

// How a row of up to kCols columns is spread: kLanes lanes hold it in kChunks
// 16-byte chunks each, in workgroups of kBlock lanes.  A lane that holds little
// leaves registers for more wavefronts, whose loads hide one another's latency
// better than prefetching a row ahead did; a row spread over more wavefronts
// meets more barriers.  Forward, 16384 x 1600 bf16: 23 us with two chunks in two
// wavefronts, 26 with one chunk in four, 30 with four in one; backward: 36 us
// with one chunk in four wavefronts, 48 with four in one, 52 with four in one and
// the next row prefetched.
template <int kWidth, typename T>
struct ForwardShape {
    static constexpr int kCols = kWidth == 0 ? 128 : 256 << kWidth;
    static constexpr int kLanes = kWidth == 0 ? 16 : kWidth == 1 ? 64 : 16 << kWidth;
    static constexpr int kChunks = kCols / kLanes / (16 / int(sizeof(T)));
    static constexpr int kBlock = kLanes < 256 ? 256 : kLanes;
};
template <int kWidth, typename T>
struct BackwardShape {
    static constexpr int kCols = kWidth == 0 ? 128 : 256 << kWidth;
    static constexpr int kLanes = kWidth == 0 ? 16 : kWidth < 6 ? 32 << kWidth : 1024;
    static constexpr int kChunks = kCols / kLanes / (16 / int(sizeof(T)));
    static constexpr int kBlock = kWidth == 0 ? 256 : kLanes < 512 ? 512 : kLanes;
    static constexpr int kRows = kBlock / kLanes;
};

// Up to here one launch for all gradients takes no longer than rows and partials,
// as called from Python on inputs that no cache holds: 2,048 rows of 1,600 bf16
// 12.4 us against 13.9 for 2,049 (fp32 15.2 and 15.7), of 801 11.3 and 13.9 (fp32
// 13.4 and 13.7, where the kernels alone take 11.5 and 10.4); kernels alone, 1,024
// of 4,096 9.3 against 16.1 (fp32 14.0 and 16.3), 512 of 8,192 10.1 against 12, one
// row of 1,600 2.9 against 5.0.  Twice as many are slower: a column workgroup walks
// all rows by itself.  The limit goes by columns, as the workspace's size does,
// which knows no type.
uint64_t fewRows(uint32_t cols) { return cols <= 2048 ? 2048 : cols <= 4096 ? 1024 : 512; }
// Workgroups of narrow slabs walk more rows at a time, and are more: 1,024 rows of 1,600 bf16 6.3 us with 16 columns,
// 5.7 with 8, but 256 rows 3.2 and 3.6; 512 rows of 4,096 6.4 with 32, 5.4 with 16;
// 512 rows of 8,192 10.1 with 32, 13.4 with 16.  The slabs of a line on one XCD: 16
// columns, 1,024 x 768 6.2 -> 4.6 us, 1,024 x 1,600 7.6 -> 6.3.
template <int kCols, typename F>
void bySlab(uint64_t rows, F f) {
    if constexpr (kCols > 4096) f(std::integral_constant<int, 32>{});
    else if constexpr (kCols > 2048) f(std::integral_constant<int, 16>{});
    else if (rows <= 512) f(std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 8>{});
}

}  // namespace

// Workgroups of stage 1: two a CU, or one where a row takes 1,024 lanes and a
// CU has registers for one workgroup (4096 x 8192 bf16: 50 us against 55 with
// 512, whose partials are twice as many).
uint32_t lnBackwardBlocks(uint64_t rows, uint32_t cols) {
    if (rows <= fewRows(cols)) return 0;
    const int perBlock = byWidth(cols, [](auto width) {
        constexpr int kWidth = decltype(width)::value;
        static_assert(BackwardShape<kWidth, bf16_t>::kRows == BackwardShape<kWidth, float>::kRows,
                      "the partition is the same for both types");
        return BackwardShape<kWidth, float>::kRows;
    });
    return gridFor(rows, perBlock, cols <= 4096 ? 512 : 256);
}

// Up to 4,096 columns the size grows with both: more columns mean no fewer
// workgroups, from no more rows on.  Above, there are half as many workgroups.
uint64_t lnWorkspaceBound(uint64_t rows, uint32_t cols) {
    const uint64_t own = lnWorkspaceBytes(rows, cols), narrower = cols > 4096 ? lnWorkspaceBytes(rows, 4096) : 0;
    return own > narrower ? own : narrower;
}

hipError_t launchLayerNormForward(const LayerNormForward &a, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
        byWidth(a.cols, [&](auto width) {
            using S = ForwardShape<decltype(width)::value, decltype(t)>;
            // At most 16 workgroups of 256 lanes a CU, which keep their weights
            // and biases over their rows: 4096 x 8192 bf16 26 us against 27 with
            // a workgroup for every row, 16384 x 1600 23 against 26.
            const uint32_t most = 256 * 16 * 256 / S::kBlock;
            hipLaunchKernelGGL((lnForwardKernel<decltype(t), decltype(w), S::kLanes, S::kChunks, S::kBlock>),
                               dim3(gridFor(a.rows, S::kBlock / S::kLanes, most)), dim3(S::kBlock), 0, stream, a);
        });
    });
}

hipError_t launchLayerNormBackward(const LayerNormBackward &a, hipStream_t stream) {
    const uint32_t blocks = lnBackwardBlocks(a.rows, a.cols);
    if (a.rows && a.rows <= fewRows(a.cols))
        return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
            byWidth(a.cols, [&](auto width) {
                using S = BackwardShape<decltype(width)::value, decltype(t)>;
                bySlab<S::kCols>(a.rows, [&](auto columns) {
                    constexpr int kSlabCols = decltype(columns)::value;
                    const uint32_t slabs = Slabs<decltype(t), kSlabCols>::workgroups(a.cols);
                    hipLaunchKernelGGL((lnBackwardFewKernel<decltype(t), decltype(w), S::kLanes, S::kChunks, S::kBlock,
                                                            kSlabCols>),
                                       dim3(slabs + gridFor(a.rows, S::kRows, 1024)), dim3(S::kBlock), 0, stream, a,
                                       slabs);
                });
            });
        });
    return byTypes(a.dtype, a.paramDtype, [&](auto t, auto w) {
        using W = decltype(w);
        if (blocks)
            byWidth(a.cols, [&](auto width) {
                using S = BackwardShape<decltype(width)::value, decltype(t)>;
                hipLaunchKernelGGL((lnBackwardKernel<decltype(t), W, S::kLanes, S::kChunks, S::kBlock>), dim3(blocks),
                                   dim3(S::kBlock), 0, stream, a);
            });
        hipLaunchKernelGGL((paramSumKernel<W>), dim3((a.cols + kParamCols - 1) / kParamCols, a.dbias ? 2 : 1),
                           dim3(kParamCols * kParamGroups), 0, stream, a.partials, blocks, 2 * a.cols, a.cols,
                           static_cast<W *>(a.dweight), static_cast<W *>(a.dbias),
                           a.accumulate & BFO_ACCUMULATE_PARAMS);
    });
}

}  // namespace bfo
