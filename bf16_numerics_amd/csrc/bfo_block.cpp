// bfo_block.cpp -- host side of the operators between a transformer block's
// matrix products (include/bf16opt.h): argument checks and the kernel launches
// on the caller's stream.
#include <cmath>

#include "bfo_args.hpp"
#include "bfo_ops.hpp"

namespace {

using namespace bfo;

constexpr uint64_t kMaxGroups = uint64_t(1) << 31;

bool knownCodes(int type) { return type == BFO_I8 || type == BFO_E4M3; }
uint64_t groupsOf(uint64_t cols, uint32_t group) { return group ? (cols + group - 1) / group : 1; }

// Codes of rows x cols values: both arrays or neither.
int codeMatrix(const void *codes, uint64_t stride, const float *scales, int type, uint64_t rows, uint64_t cols,
               Rows &out) {
    const int rc = optionalMatrix(codes, stride, rows, cols, 1, out);
    if (rc != BFO_OK) return rc;
    if (!codes) return scales ? BFO_EINVAL : BFO_OK;
    if (!scales || !knownCodes(type)) return BFO_EINVAL;
    return alignedTo(scales, 4) ? BFO_OK : BFO_EMISALIGNED;
}

// The first status that is not BFO_OK.
int firstOf(std::initializer_list<int> status) {
    for (int rc : status)
        if (rc != BFO_OK) return rc;
    return BFO_OK;
}

int checkRmsNorm(uint32_t cols, int dtype, int paramDtype) {
    if (!knownType(dtype) || !knownType(paramDtype) || cols == 0) return BFO_EINVAL;
    return cols > BFO_RMSNORM_MAX_COLS ? BFO_ERANGE : BFO_OK;
}

bool knownGroup(uint32_t group) { return group == 0 || group == BFO_GROUP; }

// The groups of rows x cols values.
int groupGrid(uint64_t rows, uint32_t cols, int dtype, GroupGrid &grid) {
    if (!knownType(dtype) || cols == 0) return BFO_EINVAL;
    const uint64_t groups = groupsOf(cols, BFO_GROUP);
    if (cols > BFO_ACTIVATION_MAX_COLS || rows > kMaxGroups / groups) return BFO_ERANGE;
    grid = GroupGrid{cols, uint32_t(rows * groups), FastDivide(uint32_t(groups))};
    return BFO_OK;
}

bool knownKind(int kind) { return kind == BFO_SILU || kind == BFO_GELU; }

int activationForward(ActivationForward a, uint64_t rows, uint32_t cols, void *stream) {
    int rc = groupGrid(rows, cols, a.dtype, a.grid);
    if (rc != BFO_OK) return rc;
    const uint64_t size = sizeOf(a.dtype), scales = 4 * rows * a.grid.perRow.by;
    const bool pack = a.kind == kIdentity, gated = a.up.p != nullptr, coded = a.gateCodes.p != nullptr;
    Rows gate, up, out, gateCodes, upCodes;
    rc = firstOf({matrix(a.gate.p, a.gate.stride, rows, cols, a.dtype, gate),
                  optionalMatrix(a.up.p, a.up.stride, rows, cols, size, up),
                  pack ? optionalMatrix(nullptr, 0, 0, 0, size, out)
                       : matrix(a.out.p, a.out.stride, rows, cols, a.dtype, out),
                  codeMatrix(a.gateCodes.p, a.gateCodes.stride, a.gateCodes.scales, a.codeType, rows, cols, gateCodes),
                  codeMatrix(a.upCodes.p, a.upCodes.stride, a.upCodes.scales, a.codeType, rows, cols, upCodes)});
    if (rc != BFO_OK) return rc;
    if (rows && ((pack && !coded) || (a.upCodes.p != nullptr) != (gated && coded))) return BFO_EINVAL;
    if (!coded) a.codeType = kNoCodes;
    const MatrixUse matrices[] = {{gate, false, true}, {up, false, true}, {out, true, true},
                                  {gateCodes, true, false}, {upCodes, true, false}};
    const Use use[] = {writes(a.gateCodes.scales, scales), writes(a.upCodes.scales, scales)};
    if (conflict(matrices) || conflict(matrices, use)) return BFO_EINVAL;
    return done(launchActivationForward(a, static_cast<hipStream_t>(stream)));
}

// A tokens x heads matrix of heads of `dim` values as one of rows: those of the
// tokens or those of the heads, whichever do not reach into one another.
int headMatrix(const void *p, uint64_t token, uint64_t head, uint64_t tokens, uint64_t heads, uint64_t dim,
               uint64_t size, Rows &out) {
    if (tokens < 2) return matrixOf(p, head, heads, dim, size, out);
    if (heads < 2) return matrixOf(p, token, tokens, dim, size, out);
    if (token > kMaxBytes / size / tokens || head > kMaxBytes / size / heads) return BFO_ERANGE;
    const uint64_t ofToken = (heads - 1) * head + dim, ofHead = (tokens - 1) * token + dim;
    if (head >= dim && token >= ofToken) return matrixOf(p, token, tokens, ofToken, size, out);
    if (token >= dim && head >= ofHead) return matrixOf(p, head, heads, ofHead, size, out);
    return BFO_EINVAL;
}

}  // namespace

extern "C" {

int rmsnorm_forward(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride,
                    const void *weight, void *total, uint64_t total_stride, void *out, uint64_t out_stride,
                    float *rstd, void *codes, uint64_t codes_stride, float *scales, int code_type, int codes_of,
                    uint32_t group, uint64_t rows, uint32_t cols, float eps, int dtype, int param_dtype,
                    void *stream) {
    int rc = checkRmsNorm(cols, dtype, param_dtype);
    if (rc != BFO_OK) return rc;
    if (!(eps >= 0.0f) || !std::isfinite(eps) || !weight || (total && !residual) || (rows && !out && !codes))
        return BFO_EINVAL;
    if (codes && (!knownGroup(group) || (codes_of != BFO_CODES_OF_OUT && codes_of != BFO_CODES_OF_NORMALISED)))
        return BFO_EINVAL;
    const uint64_t size = sizeOf(dtype);
    Rows in, more, sum, res, coded;
    rc = firstOf({matrix(x, x_stride, rows, cols, dtype, in),
                  optionalMatrix(residual, residual_stride, rows, cols, size, more),
                  optionalMatrix(total, total_stride, rows, cols, size, sum),
                  optionalMatrix(out, out_stride, rows, cols, size, res),
                  codeMatrix(codes, codes_stride, scales, code_type, rows, cols, coded)});
    if (rc != BFO_OK) return rc;
    if (!alignedTo(weight, sizeOf(param_dtype)) || !alignedTo(rstd, 4)) return BFO_EMISALIGNED;
    const MatrixUse matrices[] = {{in, false, true}, {more, false, true}, {sum, true, true}, {res, true, false},
                                  {coded, true, false}};
    const Use use[] = {reads(weight, cols * sizeOf(param_dtype)), writes(rstd, 4 * rows),
                       writes(scales, 4 * rows * groupsOf(cols, group))};
    if (conflict(matrices) || conflict(matrices, use)) return BFO_EINVAL;
    const RmsNormForward a{{x, x_stride}, {residual, residual_stride}, weight, {total, total_stride},
                           {out, out_stride}, rstd, {codes, codes_stride}, scales, code_type,
                           codes_of == BFO_CODES_OF_OUT, group, rows, cols, eps, dtype, param_dtype};
    return done(launchRmsNormForward(a, static_cast<hipStream_t>(stream)));
}

int bfo_rmsnorm_workspace_bytes(uint64_t rows, uint32_t cols, uint64_t *bytes) {
    if (!bytes || cols == 0) return BFO_EINVAL;
    if (cols > BFO_RMSNORM_MAX_COLS || rows > kMaxRows) return BFO_ERANGE;
    *bytes = rmsWorkspaceBound(rows, cols);
    return BFO_OK;
}

int rmsnorm_backward(const void *dout, uint64_t dout_stride, const void *x, uint64_t x_stride, const void *codes,
                     uint64_t codes_stride, const float *scales, int code_type, uint32_t group, const void *weight,
                     const float *rstd, void *dx, uint64_t dx_stride, void *dweight, void *out, uint64_t out_stride,
                     uint64_t rows, uint32_t cols, int dtype, int param_dtype, int accumulate, void *workspace,
                     void *stream) {
    int rc = checkRmsNorm(cols, dtype, param_dtype);
    if (rc != BFO_OK) return rc;
    if ((accumulate & ~(BFO_ACCUMULATE_DX | BFO_ACCUMULATE_PARAMS)) || !weight || !dweight || (x && codes) ||
        (rows && !x && !codes) || (codes && !knownGroup(group)))
        return BFO_EINVAL;
    const uint64_t size = sizeOf(dtype);
    Rows g, in, coded, grad, res;
    rc = firstOf({matrix(dout, dout_stride, rows, cols, dtype, g),
                  optionalMatrix(x, x_stride, rows, cols, size, in),
                  codeMatrix(codes, codes_stride, scales, code_type, rows, cols, coded),
                  matrix(dx, dx_stride, rows, cols, dtype, grad),
                  optionalMatrix(out, out_stride, rows, cols, size, res)});
    if (rc != BFO_OK) return rc;
    if (rows && !rstd) return BFO_EINVAL;
    const uint64_t need = rmsWorkspaceBytes(rows, cols), pb = cols * sizeOf(param_dtype);
    if (need && !workspace) return BFO_EINVAL;
    if (!allAligned({weight, dweight}, sizeOf(param_dtype)) || !alignedTo(rstd, 4) || !alignedTo(workspace, 16))
        return BFO_EMISALIGNED;
    const MatrixUse matrices[] = {{g, false, false}, {in, false, false}, {coded, false, false}, {grad, true, false},
                                  {res, true, false}};
    const Use use[] = {reads(weight, pb), reads(rstd, 4 * rows), reads(scales, 4 * rows * groupsOf(cols, group)),
                       writes(dweight, pb), writes(workspace, need)};
    if (conflict(matrices) || conflict(matrices, use)) return BFO_EINVAL;
    const RmsNormBackward a{{dout, dout_stride}, {x, x_stride}, {codes, codes_stride}, scales, code_type, group,
                            weight, rstd, {dx, dx_stride}, dweight, {out, out_stride}, rows, cols, dtype,
                            param_dtype, accumulate, static_cast<float *>(workspace)};
    return done(launchRmsNormBackward(a, static_cast<hipStream_t>(stream)));
}

int activation_forward(const void *gate, uint64_t gate_stride, const void *up, uint64_t up_stride, void *out,
                       uint64_t out_stride, void *gate_codes, uint64_t gate_codes_stride, float *gate_scales,
                       void *up_codes, uint64_t up_codes_stride, float *up_scales, int code_type, uint64_t rows,
                       uint32_t cols, int kind, int dtype, void *stream) {
    if (!knownKind(kind)) return BFO_EINVAL;
    return activationForward({{gate, gate_stride}, {up, up_stride}, {out, out_stride},
                              {gate_codes, gate_codes_stride, gate_scales}, {up_codes, up_codes_stride, up_scales},
                              code_type, {}, kind, dtype},
                             rows, cols, stream);
}

int activation_pack(const void *x, uint64_t x_stride, void *codes, uint64_t codes_stride, float *scales,
                    int code_type, uint64_t rows, uint32_t cols, int dtype, void *stream) {
    return activationForward({{x, x_stride}, {nullptr, 0}, {nullptr, 0}, {codes, codes_stride, scales},
                              {nullptr, 0, nullptr}, code_type, {}, kIdentity, dtype},
                             rows, cols, stream);
}

int activation_backward(const void *dout, uint64_t dout_stride, const void *gate, uint64_t gate_stride,
                        const void *up, uint64_t up_stride, const void *gate_codes, uint64_t gate_codes_stride,
                        const float *gate_scales, const void *up_codes, uint64_t up_codes_stride,
                        const float *up_scales, int code_type, void *dgate, uint64_t dgate_stride, void *dup,
                        uint64_t dup_stride, void *out, uint64_t out_stride, uint64_t rows, uint32_t cols, int kind,
                        int dtype, void *stream) {
    if (!knownKind(kind)) return BFO_EINVAL;
    GroupGrid grid;
    int rc = groupGrid(rows, cols, dtype, grid);
    if (rc != BFO_OK) return rc;
    const uint64_t size = sizeOf(dtype), scales = 4 * rows * grid.perRow.by;
    const bool coded = gate_codes != nullptr, gated = dup != nullptr;
    Rows g, in, more, inCodes, moreCodes, gradIn, gradMore, again;
    rc = firstOf({matrix(dout, dout_stride, rows, cols, dtype, g),
                  optionalMatrix(gate, gate_stride, rows, cols, size, in),
                  optionalMatrix(up, up_stride, rows, cols, size, more),
                  codeMatrix(gate_codes, gate_codes_stride, gate_scales, code_type, rows, cols, inCodes),
                  codeMatrix(up_codes, up_codes_stride, up_scales, code_type, rows, cols, moreCodes),
                  matrix(dgate, dgate_stride, rows, cols, dtype, gradIn),
                  optionalMatrix(dup, dup_stride, rows, cols, size, gradMore),
                  optionalMatrix(out, out_stride, rows, cols, size, again)});
    if (rc != BFO_OK) return rc;
    // The inputs as they were or their codes, and the second of them where its gradient is wanted.
    if (rows && ((gate != nullptr) == coded || (up != nullptr) != (gated && !coded) ||
                 (up_codes != nullptr) != (gated && coded)))
        return BFO_EINVAL;
    const MatrixUse matrices[] = {{g, false, true}, {in, false, true}, {more, false, true},
                                  {inCodes, false, false}, {moreCodes, false, false}, {gradIn, true, true},
                                  {gradMore, true, true}, {again, true, true}};
    const Use use[] = {reads(gate_scales, scales), reads(up_scales, scales)};
    if (conflict(matrices) || conflict(matrices, use)) return BFO_EINVAL;
    const ActivationBackward a{{dout, dout_stride}, {gate, gate_stride}, {up, up_stride},
                               {gate_codes, gate_codes_stride, gate_scales, false},
                               {up_codes, up_codes_stride, up_scales, false}, coded ? code_type : kNoCodes,
                               {dgate, dgate_stride}, {dup, dup_stride}, {out, out_stride}, grid, kind, dtype};
    return done(launchActivationBackward(a, static_cast<hipStream_t>(stream)));
}

int activation_unpack(const void *codes, uint64_t codes_stride, const float *scales, int code_type, uint32_t group,
                      void *out, uint64_t out_stride, uint64_t rows, uint32_t cols, int dtype, void *stream) {
    GroupGrid grid;
    int rc = groupGrid(rows, cols, dtype, grid);
    if (rc != BFO_OK) return rc;
    if (!knownGroup(group) || (rows && !codes)) return BFO_EINVAL;
    Rows in, res;
    rc = firstOf({codeMatrix(codes, codes_stride, scales, code_type, rows, cols, in),
                  matrix(out, out_stride, rows, cols, dtype, res)});
    if (rc != BFO_OK) return rc;
    const MatrixUse matrices[] = {{in, false, false}, {res, true, false}};
    const Use use[] = {reads(scales, 4 * rows * groupsOf(cols, group))};
    if (conflict(matrices) || conflict(matrices, use)) return BFO_EINVAL;
    const ActivationBackward a{{nullptr, 0}, {nullptr, 0}, {nullptr, 0}, {codes, codes_stride, scales, group == 0},
                               {nullptr, 0, nullptr, false}, code_type, {nullptr, 0}, {nullptr, 0},
                               {out, out_stride}, grid, kIdentity, dtype};
    return done(launchActivationBackward(a, static_cast<hipStream_t>(stream)));
}

int bfo_rotary_frequencies(const bfo_rotary_scaling *scaling, uint32_t rotated, double *frequencies) {
    if (!scaling || !frequencies || rotated == 0 || rotated % 2) return BFO_EINVAL;
    if (rotated > BFO_ROTARY_MAX_DIM) return BFO_ERANGE;
    const bfo_rotary_scaling &s = *scaling;
    const bool byParts = s.kind == BFO_ROTARY_BY_TURNS || s.kind == BFO_ROTARY_BY_PAIR;
    if (s.kind < BFO_ROTARY_UNSCALED || s.kind > BFO_ROTARY_BY_PAIR || !(s.base > 1.0) || !std::isfinite(s.base))
        return BFO_EINVAL;
    if (s.kind != BFO_ROTARY_UNSCALED && (!(s.factor >= 1.0) || !std::isfinite(s.factor))) return BFO_EINVAL;
    if (byParts && (!(s.length > 0.0) || !std::isfinite(s.length) || !(s.low > 0.0) || !(s.high > s.low) ||
                    !std::isfinite(s.high)))
        return BFO_EINVAL;
    if (s.kind == BFO_ROTARY_BASE && rotated < 4) return BFO_EINVAL;
    const double kTwoPi = 6.283185307179586476925, r = rotated;
    // The (real) pair that makes `turns` turns over the original length.
    auto pairOf = [&](double turns) {
        return r * (std::log(s.length) - std::log(turns) - std::log(kTwoPi)) / (2.0 * std::log(s.base));
    };
    for (uint32_t i = 0; i < rotated / 2; ++i) {
        double f = std::pow(s.base, -2.0 * i / r);
        if (s.kind == BFO_ROTARY_BASE) f *= std::pow(s.factor, -2.0 * i / (r - 2.0));
        double keep = 1.0;  // how much of the frequency stays; the rest is divided by the factor
        if (s.kind == BFO_ROTARY_LINEAR) keep = 0.0;
        if (s.kind == BFO_ROTARY_BY_TURNS) keep = (s.length * f / kTwoPi - s.low) / (s.high - s.low);
        if (s.kind == BFO_ROTARY_BY_PAIR) keep = (pairOf(s.low) - i) / (pairOf(s.low) - pairOf(s.high));
        keep = !(keep > 0.0) ? 0.0 : keep > 1.0 ? 1.0 : keep;  // no number: a pair at bounds that are one
        frequencies[i] = f * keep + (keep < 1.0 ? f / s.factor * (1.0 - keep) : 0.0);
    }
    return BFO_OK;
}

int rotary_apply(const void *x, uint64_t x_token_stride, uint64_t x_head_stride, void *out,
                 uint64_t out_token_stride, uint64_t out_head_stride, uint64_t tokens, uint32_t heads,
                 uint32_t head_dim, uint32_t rotated, int layout, const double *frequencies,
                 const int32_t *positions, uint64_t period, float amplitude, int backward, int dtype, void *stream) {
    if (!knownType(dtype) || (layout != BFO_ROTARY_HALF && layout != BFO_ROTARY_INTERLEAVED) || !frequencies ||
        rotated == 0 || rotated % 2 || rotated > head_dim || !std::isfinite(amplitude))
        return BFO_EINVAL;
    if (head_dim > BFO_ROTARY_MAX_DIM || heads > BFO_ROTARY_MAX_HEADS || tokens > kMaxRows) return BFO_ERANGE;
    if (!tokens || !heads) return BFO_OK;
    const uint64_t size = sizeOf(dtype);
    Rows in, res;
    const int rc = firstOf({headMatrix(x, x_token_stride, x_head_stride, tokens, heads, head_dim, size, in),
                            headMatrix(out, out_token_stride, out_head_stride, tokens, heads, head_dim, size, res)});
    if (rc != BFO_OK) return rc;
    if (!alignedTo(frequencies, 8) || !alignedTo(positions, 4)) return BFO_EMISALIGNED;
    const bool same = x == out && (tokens < 2 || x_token_stride == out_token_stride) &&
                      (heads < 2 || x_head_stride == out_head_stride);
    const MatrixUse matrices[] = {{in, false, same}, {res, true, same}};
    const Use use[] = {reads(frequencies, 4 * uint64_t(rotated)), reads(positions, 4 * tokens)};
    if (conflict(matrices) || conflict(matrices, use)) return BFO_EINVAL;
    const Rotary a{x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride, tokens, heads, head_dim,
                   rotated, frequencies, positions, period, amplitude, backward != 0, 0, 0, {}, {}, {}, {}};
    return done(launchRotary(a, dtype, layout, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
