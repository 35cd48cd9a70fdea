// bfo_ops.hpp -- limits, partitions and kernel launchers of the training-loop
// operators, shared by their host ABI (bfo_ops.cpp, bfo_block.cpp) and their
// gfx950 kernels (bfo_layernorm.hip, bfo_logits.hip, bfo_rmsnorm.hip,
// bfo_activation.hip, bfo_rotary.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bf16opt.h"

namespace bfo {

// A matrix of rows `stride` elements apart.
struct ConstMatrix {
    const void *p;
    uint64_t stride;
};
struct Matrix {
    void *p;
    uint64_t stride;
};

// Layer norm backward: stage 1 runs lnBackwardBlocks workgroups, each of which
// sums its rows' terms of dweight and dbias into one row of 2 * cols floats of
// the workspace; stage 2 adds those rows.  Few rows (0 workgroups here) take
// one launch without partials.  The partition depends on the sizes only.
uint32_t lnBackwardBlocks(uint64_t rows, uint32_t cols);
inline uint64_t lnWorkspaceBytes(uint64_t rows, uint32_t cols) {
    return uint64_t(lnBackwardBlocks(rows, cols)) * 2 * cols * sizeof(float);
}
// What no call of at most so many rows and columns exceeds.
uint64_t lnWorkspaceBound(uint64_t rows, uint32_t cols);

struct LayerNormForward {
    ConstMatrix x;
    const void *weight, *bias;
    Matrix out;
    float *mean, *rstd;
    uint64_t rows;
    uint32_t cols;
    float eps;
    int dtype, paramDtype;
};
hipError_t launchLayerNormForward(const LayerNormForward &a, hipStream_t stream);

struct LayerNormBackward {
    ConstMatrix dout, x;
    const void *weight;
    const float *mean, *rstd;
    Matrix dx;
    void *dweight, *dbias;
    uint64_t rows;
    uint32_t cols;
    int dtype, paramDtype, accumulate;
    float *partials;
};
hipError_t launchLayerNormBackward(const LayerNormBackward &a, hipStream_t stream);

// True for calls whose matrices of `bytes` in all are loaded and stored
// nontemporally, as they pass through the caches anyway: from half of the last-level
// cache's 256 MB on.  On three sets of inputs in turn, without and with: RMS norm with
// codes 8192 x 4096 bf16 (303 MB) 57.9 and 49.8 us, 4096 rows 31.5 and 26.9, 1024 rows
// the same; gated activation with codes 8192 x 11008 (727 MB) 124 and 115, 2048 rows
// (181 MB) 33.9 and 30.2, its gradient 155 and 145, 42.1 and 36.1, 512 rows (57 MB) 11.0
// and 11.8; rotary 2048 x 64 x 128 (67 MB) 12.0 and 13.1.  With a matrix product that
// reads the norm's output behind it, 8192 rows 261 and 259 us, 2048 76.9 and 77.1.
inline bool streams(uint64_t bytes) { return bytes >= (uint64_t(128) << 20); }

// Codes of a matrix, `stride` bytes from row to row, and their scales.
struct ConstCodes {
    const void *p;
    uint64_t stride;
    const float *scales;
    bool wholeRow;  // one scale a row instead of one a group
};
struct CodeMatrix {
    void *p;
    uint64_t stride;
    float *scales;
};

// RMS norm backward: as layer norm's, with one sum a column.
uint32_t rmsBackwardBlocks(uint64_t rows, uint32_t cols);
inline uint64_t rmsWorkspaceBytes(uint64_t rows, uint32_t cols) {
    return uint64_t(rmsBackwardBlocks(rows, cols)) * cols * sizeof(float);
}
uint64_t rmsWorkspaceBound(uint64_t rows, uint32_t cols);  // as lnWorkspaceBound

struct RmsNormForward {
    ConstMatrix x, residual;
    const void *weight;
    Matrix total, out;
    float *rstd;
    Matrix codes;
    float *scales;
    int codeType, codesOfOut;
    uint32_t group;  // BFO_GROUP, or 0: the whole row
    uint64_t rows;
    uint32_t cols;
    float eps;
    int dtype, paramDtype;
};
hipError_t launchRmsNormForward(const RmsNormForward &a, hipStream_t stream);

struct RmsNormBackward {
    ConstMatrix dout, x, codes;
    const float *scales;
    int codeType;
    uint32_t group;
    const void *weight;
    const float *rstd;
    Matrix dx;
    void *dweight;
    Matrix out;
    uint64_t rows;
    uint32_t cols;
    int dtype, paramDtype, accumulate;
    float *partials;
};
hipError_t launchRmsNormBackward(const RmsNormBackward &a, hipStream_t stream);

// Division of numbers below 2^31 by a constant from 1 to 2^31: with s the bits of
// by - 1, (n * (floor(2^(31 + s) / by) + 1)) >> (31 + s) is the quotient, as the
// factor is off by at most 2^s / 2^(31 + s) of itself.
struct FastDivide {
    uint32_t by, factor, shift;
    FastDivide() = default;
    explicit FastDivide(uint32_t d) : by(d), shift(31) {
        while (shift < 62 && (uint64_t(1) << (shift - 31)) < d) ++shift;
        factor = uint32_t((uint64_t(1) << shift) / d + 1);
    }
    __host__ __device__ uint32_t divide(uint32_t n) const { return uint32_t(uint64_t(n) * factor >> shift); }
};

// The rows' groups of columns, `count` in all (at most 2^31).
struct GroupGrid {
    uint32_t cols, count;
    FastDivide perRow;
};

// Beside the kinds and code types of the ABI: codes by themselves, and none.
constexpr int kIdentity = -1, kNoCodes = -1;

struct ActivationForward {
    ConstMatrix gate, up;
    Matrix out;
    CodeMatrix gateCodes, upCodes;
    int codeType;
    GroupGrid grid;
    int kind, dtype;
};
hipError_t launchActivationForward(const ActivationForward &a, hipStream_t stream);

struct ActivationBackward {
    ConstMatrix dout, gate, up;
    ConstCodes gateCodes, upCodes;
    int codeType;
    Matrix dgate, dup, out;
    GroupGrid grid;
    int kind, dtype;
};
hipError_t launchActivationBackward(const ActivationBackward &a, hipStream_t stream);

struct Rotary {
    const void *x;
    uint64_t xToken, xHead;
    void *out;
    uint64_t outToken, outHead;
    uint64_t tokens;
    uint32_t heads, headDim, rotated;
    const double *frequencies;
    const int32_t *positions;
    uint64_t period;
    float amplitude;
    int backward;
    // Set by the launch: a workgroup's tokens and heads, the blocks of heads, the
    // workgroups' work in all, and the items of work a head is cut into.
    uint32_t tokensAtOnce, units;
    FastDivide headsAtOnce, headBlocks, itemsPerHead, pairsPerToken;
};
hipError_t launchRotary(const Rotary &a, int dtype, int layout, hipStream_t stream);

// The scale of a difference of scores, as (x part - m part) rest: by halves below
// 1, where a difference past binary32 may have a product that is not.
struct DifferenceScale {
    float part, rest;
};
inline DifferenceScale differenceScale(float scale) {
    return scale < 1.0f ? DifferenceScale{0.5f, 2.0f * scale} : DifferenceScale{1.0f, scale};
}

// The forward pass over the scores: token log probabilities (count == 0) and
// distillation (count > 0; top == 0).
struct LogitsForward {
    ConstMatrix logits;
    uint64_t rows;
    uint32_t vocab;
    float scale;
    DifferenceScale difference;
    const int32_t *targets;
    float *logprob, *stats, *entropy;
    uint32_t top;
    int32_t *topIndex;
    float *topLogprob;
    const int32_t *teacherIndex;
    const float *teacherLogits;
    uint32_t count;
    float *kl;
    void *workspace;
};
uint64_t logitsWorkspaceBytes(uint64_t rows, uint32_t vocab, uint32_t top);
uint64_t logitsWorkspaceBound(uint64_t rows, uint32_t vocab, uint32_t top);  // as lnWorkspaceBound
hipError_t launchLogitsForward(const LogitsForward &a, int dtype, hipStream_t stream);

struct LogitsBackward {
    ConstMatrix logits;
    Matrix dlogits;
    uint64_t rows;
    uint32_t vocab, width;
    float scale;
    DifferenceScale difference;
    const int32_t *targets;
    const float *stats, *entropy, *dlogprob, *dentropy;
    const int32_t *teacherIndex;
    const float *teacherLogits;
    uint32_t count;
    const float *dkl;
};
hipError_t launchLogitsBackward(const LogitsBackward &a, int dtype, hipStream_t stream);

}  // namespace bfo
