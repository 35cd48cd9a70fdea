// bfo_activation.hip -- gfx950 kernels of the feed-forward's activation, gated
// or not, with its inputs kept in 8-bit codes for the backward pass, and of
// codes by themselves.
//
// act(g) = g * sigma(z) with sigma(z) = 1 / (1 + exp(-z)): z = g is SiLU, and
// z = 2 sqrt(2/pi) (g + 0.044715 g^3) GELU in its tanh form, as
// (1 + tanh(u)) / 2 = sigma(2 u).  Its derivative is
// sigma + act * (1 - sigma) * dz/dg.
//
// Rows are cut into groups of 128 columns, the codes' groups; a group is held
// by neighbouring lanes, 16 bytes of it each, and no lane meets another's data
// but for the group's largest value.
//
// Bound by memory: 8192 x 11008 bf16, gated, both inputs kept (727 MB) 115 us,
// 6.3 TB/s, the vector ALUs 53% busy; backward from codes with out again (907 MB)
// 145 us, 6.3 TB/s.  One group a lane's turn: two or four asked for at once 123 and
// 130 us, workgroups of 128, 512 and 1,024 lanes 115, 116 and 122.
#include "bfo_codes.hpp"

namespace bfo {
namespace {

constexpr int kBlock = 256;
constexpr float kSlope = 1.5957691216057308f, kCubic = 0.044715f;  // 2 sqrt(2 / pi)

// exp(-z) as the hardware's power of 2.  A rounding of the exponent -z log2(e) is one
// of the power times |z|, which 16 bits of a result do not show but 32 do: 63 * 2^-24
// of an activation at g = -80.  For fp32 results the power is corrected by what the
// exponent's rounding left, unless it is past the range anyway (infinite, or 0): from
// the product's own rest and log2(e)'s for SiLU, from 64 bits for GELU's cubic.
// Without and with that, gated, codes kept, fp32: 8192 x 11008 199.0 and 198.9 us (GELU
// 198.6 and 199.0), 1003 x 6400 16.6 and 16.8 (GELU 16.6 and 17.3).
template <int kKind, bool kFine>
__device__ __forceinline__ float expNegative(float g, float q) {
    if constexpr (!kFine)
        return exp2Fast(kKind == BFO_SILU ? -kLog2e * g
                                          : g * fmaf(-kLog2e * kSlope * kCubic, q, -kLog2e * kSlope));
    constexpr double kLog2eFull = 1.44269504088896340736, kLinear = -kLog2eFull * 1.5957691216057308;
    float power, left;
    if constexpr (kKind == BFO_SILU) {
        constexpr float kRest = float(kLog2eFull - double(kLog2e));
        power = -kLog2e * g;
        left = fmaf(-kRest, g, fmaf(-kLog2e, g, -power));
    } else {
        const double d = g, whole = d * fma(kLinear * 0.044715, d * d, kLinear);
        power = float(whole);
        left = float(whole - double(power));
    }
    const float e = exp2Fast(power);
    return fabsf(power) < 128.0f ? fmaf(e, left * kLn2, e) : e;
}

// sigma(z), act and its derivative.
template <int kKind, bool kFine>
struct Activation {
    float sigma, act, slope;
    __device__ __forceinline__ explicit Activation(float g) {
        // Above 100, where sigma is 0 or 1, g * g might overflow, and 0 times that be NaN.
        const float q = fminf(g * g, 1e4f);
        // For z below about -88 the exponential is infinite and sigma 0.
        sigma = __builtin_amdgcn_rcpf(1.0f + expNegative<kKind, kFine>(g, q));
        act = g * sigma;
        const float dz = kKind == BFO_SILU ? 1.0f : kSlope * fmaf(3.0f * kCubic, q, 1.0f);
        slope = fmaf(act * (1.0f - sigma), dz, sigma);
    }
};

// Where a lane's columns lie: E of them from `c` on, in group `group` of row `row`.
struct Place {
    uint64_t row;
    uint32_t group;
    int c;
};
template <int E>
__device__ __forceinline__ Place place(const GroupGrid &g, uint32_t index) {
    const uint32_t row = g.perRow.divide(index);
    const uint32_t group = index - row * g.perRow.by;
    return {row, group, int(group) * kGroup + int(threadIdx.x % (kGroup / E)) * E};
}

// v's codes and their group's scale.
template <int kType, Loads kLoads, bool kNontemporal, int E>
__device__ __forceinline__ void writeGroup(const CodeMatrix &m, const Place &p, const GroupGrid &g,
                                           const float (&v)[E]) {
    constexpr int kLanes = kGroup / E;
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) amax = max(amax, absBits(v[e]));
    const CodeScale s = codeScale<kType>(laneMax<kLanes>(amax));
    uint32_t w[E / 4];
    encode<kType, E>(v, s.inverse, w);
    storeCodes<kLoads, kNontemporal, E>(static_cast<uint8_t *>(m.p) + p.row * m.stride, p.c, int(g.cols), w);
    if (threadIdx.x % kLanes == 0) m.scales[p.row * g.perRow.by + p.group] = s.scale;
}

template <typename T, int kKind, bool kGated, int kType, Loads kLoads>
__global__ __launch_bounds__(kBlock) void actForwardKernel(ActivationForward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr uint32_t kAt = kBlock / (kGroup / E);  // groups of a workgroup
    // Of large calls, 8192 x 11008 bf16: two matrices of codes 121 us with plain stores,
    // 115 with nontemporal ones, but one 69.6 and 72.1.
    constexpr bool kStreamCodes = kLoads == kEvenStream && kGated;
    const int C = int(a.grid.cols);
    for (uint32_t i = blockIdx.x * kAt + threadIdx.x / (kGroup / E); i < a.grid.count; i += gridDim.x * kAt) {
        const Place p = place<E>(a.grid, i);
        Chunk<T, E> gate, up;
        loadChunk<kLoads>(gate, static_cast<const T *>(a.gate.p) + p.row * a.gate.stride, p.c, C, true);
        if constexpr (kGated) loadChunk<kLoads>(up, static_cast<const T *>(a.up.p) + p.row * a.up.stride, p.c, C, true);
        settle<kLoads>(gate, p.c, C, true);
        if constexpr (kGated) settle<kLoads>(up, p.c, C, true);
        float g[E], u[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            g[e] = gate[e];
            u[e] = kGated ? up[e] : 1.0f;
        }
        if constexpr (kType != kNoCodes) {
            writeGroup<kType, kLoads, kStreamCodes, E>(a.gateCodes, p, a.grid, g);
            if constexpr (kGated) writeGroup<kType, kLoads, kStreamCodes, E>(a.upCodes, p, a.grid, u);
        }
        if constexpr (kKind != kIdentity) {
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const Activation<kKind, sizeof(T) == 4> f(g[e]);
                y[e] = kGated ? f.act * u[e] : f.act;
            }
            storeChunk<kLoads>(static_cast<T *>(a.out.p) + p.row * a.out.stride, p.c, C, y);
        }
    }
}

// A kept input: the matrix itself or its codes.
template <typename T, int E, Loads kLoads, int kType>
struct Kept {
    uint32_t w[E / 4];
    float scale;
    __device__ __forceinline__ void load(const ConstMatrix &, const ConstCodes &codes, const Place &p,
                                         const GroupGrid &g) {
        loadCodes<kLoads, E>(static_cast<const uint8_t *>(codes.p) + p.row * codes.stride, p.c, int(g.cols), true, w);
        scale = codes.scales[codes.wholeRow ? p.row : p.row * g.perRow.by + p.group];
    }
    __device__ __forceinline__ void values(const Place &p, const GroupGrid &g, float (&v)[E]) {
        settleCodes<kLoads, E>(w, p.c, int(g.cols), true);
        decode<kType, E>(w, scale, v);
    }
};
template <typename T, int E, Loads kLoads>
struct Kept<T, E, kLoads, kNoCodes> {
    Chunk<T, E> raw;
    __device__ __forceinline__ void load(const ConstMatrix &m, const ConstCodes &, const Place &p, const GroupGrid &g) {
        loadChunk<kLoads>(raw, static_cast<const T *>(m.p) + p.row * m.stride, p.c, int(g.cols), true);
    }
    __device__ __forceinline__ void values(const Place &p, const GroupGrid &g, float (&v)[E]) {
        settle<kLoads>(raw, p.c, int(g.cols), true);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = raw[e];
    }
};

template <typename T, int kKind, bool kGated, int kType, Loads kLoads>
__global__ __launch_bounds__(kBlock) void actBackwardKernel(ActivationBackward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr uint32_t kAt = kBlock / (kGroup / E);
    const int C = int(a.grid.cols);
    for (uint32_t i = blockIdx.x * kAt + threadIdx.x / (kGroup / E); i < a.grid.count; i += gridDim.x * kAt) {
        const Place p = place<E>(a.grid, i);
        Kept<T, E, kLoads, kType> gate, up;
        float g[E], u[E], y[E];
        gate.load(a.gate, a.gateCodes, p, a.grid);
        if constexpr (kKind == kIdentity) {
            gate.values(p, a.grid, g);
            storeChunk<kLoads>(static_cast<T *>(a.out.p) + p.row * a.out.stride, p.c, C, g);
            continue;
        } else {
            if constexpr (kGated) up.load(a.up, a.upCodes, p, a.grid);
            Chunk<T, E> d;
            loadChunk<kLoads>(d, static_cast<const T *>(a.dout.p) + p.row * a.dout.stride, p.c, C, true);
            gate.values(p, a.grid, g);
            if constexpr (kGated) up.values(p, a.grid, u);
            settle<kLoads>(d, p.c, C, true);
            float act[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const Activation<kKind, sizeof(T) == 4> f(g[e]);
                act[e] = f.act;
                y[e] = (kGated ? d[e] * u[e] : d[e]) * f.slope;
            }
            storeChunk<kLoads>(static_cast<T *>(a.dgate.p) + p.row * a.dgate.stride, p.c, C, y);
            if constexpr (kGated) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = d[e] * act[e];
                storeChunk<kLoads>(static_cast<T *>(a.dup.p) + p.row * a.dup.stride, p.c, C, y);
            }
            if (a.out.p) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = kGated ? act[e] * u[e] : act[e];
                storeChunk<kLoads>(static_cast<T *>(a.out.p) + p.row * a.out.stride, p.c, C, y);
            }
        }
    }
}

template <int kValue>
using Const = std::integral_constant<int, kValue>;

// f(type, kind, gated, code type, way to load) with the call's values as constants.
template <typename F>
hipError_t byKind(int dtype, int kind, bool gated, int codeType, uint32_t cols, uint64_t bytes, F f) {
    auto coded = [&](auto t, auto k, auto g, auto s) {
        if (codeType == BFO_I8) f(t, k, g, Const<BFO_I8>{}, s);
        else if (codeType == BFO_E4M3) f(t, k, g, Const<BFO_E4M3>{}, s);
        else if constexpr (decltype(k)::value != kIdentity) f(t, k, g, Const<kNoCodes>{}, s);
    };
    auto gates = [&](auto t, auto k, auto s) {
        if constexpr (decltype(k)::value == kIdentity) coded(t, k, std::false_type{}, s);
        else gated ? coded(t, k, std::true_type{}, s) : coded(t, k, std::false_type{}, s);
    };
    auto kinds = [&](auto t, auto s) {
        if (kind == kIdentity) gates(t, Const<kIdentity>{}, s);
        else if (kind == BFO_SILU) gates(t, Const<BFO_SILU>{}, s);
        else gates(t, Const<BFO_GELU>{}, s);
    };
    auto types = [&](auto t) { byLoads<decltype(t)>(cols, bytes, [&](auto loads) { kinds(t, loads); }); };
    if (dtype == BFO_BF16) types(bf16_t(0));
    else types(float(0));
    return hipGetLastError();
}

// At most 2^22 workgroups, so that a launch's lanes can be counted in 32 bits.
template <typename T>
dim3 workgroups(const GroupGrid &g) {
    constexpr uint32_t kAt = kBlock / (kGroup * sizeof(T) / 16);
    const uint32_t n = (g.count + kAt - 1) / kAt, most = 1u << 22;
    return dim3(n < most ? n : most);
}

// Bytes of `matrices` matrices and `codes` matrices in codes.
uint64_t moved(const GroupGrid &g, int dtype, int matrices, int codes) {
    return uint64_t(g.count / g.perRow.by) * g.cols * (matrices * (dtype == BFO_BF16 ? 2 : 4) + codes);
}

}  // namespace

hipError_t launchActivationForward(const ActivationForward &a, hipStream_t stream) {
    if (!a.grid.count) return hipSuccess;
    const int inputs = a.up.p ? 2 : 1;
    const uint64_t bytes = moved(a.grid, a.dtype, inputs + 1, a.codeType == kNoCodes ? 0 : inputs);
    return byKind(a.dtype, a.kind, a.up.p != nullptr, a.codeType, a.grid.cols, bytes,
                  [&](auto t, auto kind, auto gated, auto type, auto loads) {
                      using T = decltype(t);
                      hipLaunchKernelGGL((actForwardKernel<T, decltype(kind)::value, decltype(gated)::value,
                                                           decltype(type)::value, decltype(loads)::value>),
                                         workgroups<T>(a.grid), dim3(kBlock), 0, stream, a);
                  });
}

hipError_t launchActivationBackward(const ActivationBackward &a, hipStream_t stream) {
    if (!a.grid.count) return hipSuccess;
    const int inputs = a.dup.p ? 2 : 1, coded = a.codeType == kNoCodes ? 0 : inputs;
    const uint64_t bytes = moved(a.grid, a.dtype, 1 + inputs - coded + inputs + (a.out.p ? 1 : 0), coded);
    return byKind(a.dtype, a.kind, a.dup.p != nullptr, a.codeType, a.grid.cols, bytes,
                  [&](auto t, auto kind, auto gated, auto type, auto loads) {
                      using T = decltype(t);
                      hipLaunchKernelGGL((actBackwardKernel<T, decltype(kind)::value, decltype(gated)::value,
                                                            decltype(type)::value, decltype(loads)::value>),
                                         workgroups<T>(a.grid), dim3(kBlock), 0, stream, a);
                  });
}

}  // namespace bfo
