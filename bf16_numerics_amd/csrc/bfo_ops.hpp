// bfo_ops.hpp -- limits, partitions and kernel launchers of the training-loop
// operators, shared by their host ABI (bfo_ops.cpp) and their gfx950 kernels
// (bfo_layernorm.hip, bfo_logits.hip).
#pragma once

#include <hip/hip_runtime_api.h>
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
