// bfo_ops.cpp -- host side of the training-loop operators declared in
// include/bf16opt.h: argument checks and the kernel launches on the caller's
// stream.
#include <cmath>

#include "bfo_args.hpp"
#include "bfo_ops.hpp"

namespace {

using namespace bfo;

int checkLayerNorm(uint32_t cols, int dtype, int paramDtype) {
    if (!knownType(dtype) || !knownType(paramDtype) || cols == 0) return BFO_EINVAL;
    return cols > BFO_LAYERNORM_MAX_COLS ? BFO_ERANGE : BFO_OK;
}

int checkLogits(uint32_t vocab, int dtype, float scale) {
    if (!knownType(dtype) || vocab == 0 || !(scale > 0.0f) || !std::isfinite(scale)) return BFO_EINVAL;
    return vocab > BFO_VOCAB_MAX ? BFO_ERANGE : BFO_OK;
}

int forwardPass(const bfo::LogitsForward &a, int dtype, void *stream) {
    Rows logits;
    int rc = matrix(a.logits.p, a.logits.stride, a.rows, a.vocab, dtype, logits);
    if (rc != BFO_OK) return rc;
    if (!allAligned({a.targets, a.logprob, a.stats, a.entropy, a.topIndex, a.topLogprob, a.teacherIndex,
                     a.teacherLogits, a.kl},
                    4) ||
        !alignedTo(a.workspace, 16))
        return BFO_EMISALIGNED;
    const uint64_t R = a.rows, need = bfo::logitsWorkspaceBytes(R, a.vocab, a.top);
    if (need && !a.workspace) return BFO_EINVAL;
    const Use use[] = {reads(a.targets, 4 * R),
                       writes(a.logprob, 4 * R),
                       writes(a.stats, 8 * R),
                       writes(a.entropy, 4 * R),
                       writes(a.topIndex, 4 * R * a.top),
                       writes(a.topLogprob, 4 * R * a.top),
                       reads(a.teacherIndex, 4 * R * a.count),
                       reads(a.teacherLogits, 4 * R * a.count),
                       writes(a.kl, 4 * R),
                       writes(a.workspace, need)};
    if (conflict(use) || conflict(logits, false, use)) return BFO_EINVAL;
    return done(bfo::launchLogitsForward(a, dtype, static_cast<hipStream_t>(stream)));
}

int backwardPass(const bfo::LogitsBackward &a, int dtype, void *stream) {
    if (a.width < a.vocab) return BFO_EINVAL;
    if (a.width > BFO_VOCAB_MAX) return BFO_ERANGE;
    Rows logits, dlogits;
    int rc = matrix(a.logits.p, a.logits.stride, a.rows, a.vocab, dtype, logits);
    if (rc == BFO_OK) rc = matrix(a.dlogits.p, a.dlogits.stride, a.rows, a.width, dtype, dlogits);
    if (rc != BFO_OK) return rc;
    if (!allAligned({a.targets, a.stats, a.entropy, a.dlogprob, a.dentropy, a.teacherIndex, a.teacherLogits, a.dkl},
                    4))
        return BFO_EMISALIGNED;
    const uint64_t R = a.rows;
    const Use use[] = {reads(a.targets, 4 * R),
                       reads(a.stats, 8 * R),
                       reads(a.entropy, 4 * R),
                       reads(a.dlogprob, 4 * R),
                       reads(a.dentropy, 4 * R),
                       reads(a.teacherIndex, 4 * R * a.count),
                       reads(a.teacherLogits, 4 * R * a.count),
                       reads(a.dkl, 4 * R)};
    const bool inPlace = logits.p == dlogits.p && logits.stride == dlogits.stride;
    if ((!inPlace && overlap(logits, dlogits)) || conflict(dlogits, true, use)) return BFO_EINVAL;
    return done(bfo::launchLogitsBackward(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int layernorm_forward(const void *x, uint64_t x_stride, const void *weight, const void *bias, void *out,
                      uint64_t out_stride, float *mean, float *rstd, uint64_t rows, uint32_t cols, float eps,
                      int dtype, int param_dtype, void *stream) {
    int rc = checkLayerNorm(cols, dtype, param_dtype);
    if (rc != BFO_OK) return rc;
    if (!(eps >= 0.0f) || !std::isfinite(eps) || !weight) return BFO_EINVAL;
    Rows in, res;
    rc = matrix(x, x_stride, rows, cols, dtype, in);
    if (rc == BFO_OK) rc = matrix(out, out_stride, rows, cols, dtype, res);
    if (rc != BFO_OK) return rc;
    if (!allAligned({weight, bias}, sizeOf(param_dtype)) || !allAligned({mean, rstd}, 4)) return BFO_EMISALIGNED;
    const uint64_t pb = cols * sizeOf(param_dtype);
    const Use use[] = {reads(weight, pb), reads(bias, pb), writes(mean, 4 * rows), writes(rstd, 4 * rows)};
    if (conflict(use) || conflict(in, false, use) || conflict(res, true, use) || overlap(in, res)) return BFO_EINVAL;
    const bfo::LayerNormForward a{{x, x_stride}, weight, bias, {out, out_stride}, mean, rstd, rows, cols, eps,
                                  dtype,         param_dtype};
    return done(bfo::launchLayerNormForward(a, static_cast<hipStream_t>(stream)));
}

int bfo_layernorm_workspace_bytes(uint64_t rows, uint32_t cols, uint64_t *bytes) {
    if (!bytes || cols == 0) return BFO_EINVAL;
    if (cols > BFO_LAYERNORM_MAX_COLS || rows > kMaxRows) return BFO_ERANGE;
    *bytes = bfo::lnWorkspaceBound(rows, cols);
    return BFO_OK;
}

int layernorm_backward(const void *dout, uint64_t dout_stride, const void *x, uint64_t x_stride,
                       const void *weight, const float *mean, const float *rstd, void *dx, uint64_t dx_stride,
                       void *dweight, void *dbias, uint64_t rows, uint32_t cols, int dtype, int param_dtype,
                       int accumulate, void *workspace, void *stream) {
    int rc = checkLayerNorm(cols, dtype, param_dtype);
    if (rc != BFO_OK) return rc;
    if ((accumulate & ~(BFO_ACCUMULATE_DX | BFO_ACCUMULATE_PARAMS)) || !weight || !dweight) return BFO_EINVAL;
    Rows g, in, res;
    rc = matrix(dout, dout_stride, rows, cols, dtype, g);
    if (rc == BFO_OK) rc = matrix(x, x_stride, rows, cols, dtype, in);
    if (rc == BFO_OK) rc = matrix(dx, dx_stride, rows, cols, dtype, res);
    if (rc != BFO_OK) return rc;
    if (rows && (!mean || !rstd)) return BFO_EINVAL;
    const uint64_t need = bfo::lnWorkspaceBytes(rows, cols);
    if (need && !workspace) return BFO_EINVAL;
    if (!allAligned({weight, dweight, dbias}, sizeOf(param_dtype)) || !allAligned({mean, rstd}, 4) ||
        !alignedTo(workspace, 16))
        return BFO_EMISALIGNED;
    const uint64_t pb = cols * sizeOf(param_dtype);
    const Use use[] = {reads(weight, pb),
                       reads(mean, 4 * rows),
                       reads(rstd, 4 * rows),
                       writes(dweight, pb),
                       writes(dbias, pb),
                       writes(workspace, need)};
    if (conflict(use) || conflict(g, false, use) || conflict(in, false, use) || conflict(res, true, use) ||
        overlap(g, res) || overlap(in, res))
        return BFO_EINVAL;
    const bfo::LayerNormBackward a{{dout, dout_stride}, {x, x_stride}, weight, mean, rstd, {dx, dx_stride}, dweight,
                                   dbias, rows, cols, dtype, param_dtype, accumulate,
                                   static_cast<float *>(workspace)};
    return done(bfo::launchLayerNormBackward(a, static_cast<hipStream_t>(stream)));
}

int bfo_logits_workspace_bytes(uint64_t rows, uint32_t vocab, uint32_t top, uint64_t *bytes) {
    if (!bytes || vocab == 0 || top > vocab) return BFO_EINVAL;
    if (vocab > BFO_VOCAB_MAX || top > BFO_TOP_MAX || rows > kMaxRows) return BFO_ERANGE;
    *bytes = bfo::logitsWorkspaceBound(rows, vocab, top);
    return BFO_OK;
}

int token_logprobs_forward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, int dtype,
                           float scale, const int32_t *targets, float *logprob, float *stats, float *entropy,
                           uint32_t top, int32_t *top_index, float *top_logprob, void *workspace, void *stream) {
    const int rc = checkLogits(vocab, dtype, scale);
    if (rc != BFO_OK) return rc;
    if (top > BFO_TOP_MAX) return BFO_ERANGE;
    if (top > vocab) return BFO_EINVAL;
    if (rows && ((targets != nullptr) != (logprob != nullptr) || (top != 0) != (top_index != nullptr) ||
                 (top != 0) != (top_logprob != nullptr)))
        return BFO_EINVAL;
    const bfo::LogitsForward a{{logits, stride}, rows, vocab, scale, bfo::differenceScale(scale), targets, logprob,
                               stats, entropy, top, top_index, top_logprob, nullptr, nullptr, 0, nullptr, workspace};
    return forwardPass(a, dtype, stream);
}

int token_logprobs_backward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, uint32_t width,
                            int dtype, float scale, const int32_t *targets, const float *stats,
                            const float *entropy, const float *dlogprob, const float *dentropy, void *dlogits,
                            uint64_t dlogits_stride, void *stream) {
    const int rc = checkLogits(vocab, dtype, scale);
    if (rc != BFO_OK) return rc;
    if (rows && ((targets != nullptr) != (dlogprob != nullptr) || (entropy != nullptr) != (dentropy != nullptr) ||
                 (!targets && !entropy) || !stats))
        return BFO_EINVAL;
    const bfo::LogitsBackward a{{logits, stride}, {dlogits, dlogits_stride}, rows, vocab, width, scale,
                                bfo::differenceScale(scale), targets, stats, entropy, dlogprob, dentropy, nullptr,
                                nullptr, 0, nullptr};
    return backwardPass(a, dtype, stream);
}

int distill_forward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, int dtype, float scale,
                    const int32_t *teacher_index, const float *teacher_logits, uint32_t count,
                    const int32_t *targets, float *kl, float *logprob, float *stats, void *workspace,
                    void *stream) {
    const int rc = checkLogits(vocab, dtype, scale);
    if (rc != BFO_OK) return rc;
    if (count == 0) return BFO_EINVAL;
    if (count > BFO_TOP_MAX) return BFO_ERANGE;
    if (rows && (!teacher_index || !teacher_logits || !kl || (targets != nullptr) != (logprob != nullptr)))
        return BFO_EINVAL;
    const bfo::LogitsForward a{{logits, stride}, rows, vocab, scale, bfo::differenceScale(scale), targets, logprob,
                               stats, nullptr, 0, nullptr, nullptr, teacher_index, teacher_logits, count, kl,
                               workspace};
    return forwardPass(a, dtype, stream);
}

int distill_backward(const void *logits, uint64_t stride, uint64_t rows, uint32_t vocab, uint32_t width,
                     int dtype, float scale, const int32_t *teacher_index, const float *teacher_logits,
                     uint32_t count, const int32_t *targets, const float *stats, const float *dkl,
                     const float *dlogprob, void *dlogits, uint64_t dlogits_stride, void *stream) {
    const int rc = checkLogits(vocab, dtype, scale);
    if (rc != BFO_OK) return rc;
    if (count == 0) return BFO_EINVAL;
    if (count > BFO_TOP_MAX) return BFO_ERANGE;
    if (rows && (!teacher_index || !teacher_logits || !dkl || !stats || (targets != nullptr) != (dlogprob != nullptr)))
        return BFO_EINVAL;
    const bfo::LogitsBackward a{{logits, stride}, {dlogits, dlogits_stride}, rows, vocab, width, scale,
                                bfo::differenceScale(scale), targets, stats, nullptr, dlogprob, nullptr,
                                teacher_index, teacher_logits, count, dkl};
    return backwardPass(a, dtype, stream);
}

}  // extern "C"
