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
#include "bfo_codes.hpp"

namespace bfo {
namespace {

constexpr int kBlock = 256;
constexpr float kSlope = 1.5957691216057308f, kCubic = 0.044715f;

// sigma(z), act and its derivative.
template <int kKind>
struct Activation {
    float sigma, act, slope;
    __device__ __forceinline__ explicit Activation(float g) {
        // Above 100, where sigma is 0 or 1, g * g might overflow, and 0 times that be NaN.
        const float q = fminf(g * g, 1e4f);
        const float z = kKind == BFO_SILU ? g : kSlope * g * fmaf(kCubic, q, 1.0f);
        // Below about -88 the exponential is infinite and sigma 0.
        sigma = __builtin_amdgcn_rcpf(1.0f + exp2Fast(-kLog2e * z));
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
template <int kType, int E>
__device__ __forceinline__ void writeGroup(const CodeMatrix &m, const Place &p, const GroupGrid &g, const float (&v)[E]) {
    constexpr int kLanes = kGroup / E;
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) amax = max(amax, absBits(v[e]));
    const CodeScale s = codeScale<kType>(laneMax<kLanes>(amax));
    uint32_t w[E / 4];
    encode<kType, E>(v, s.inverse, w);
    storeCodes<E>(static_cast<uint8_t *>(m.p) + p.row * m.stride, p.c, int(g.cols), w);
    if (threadIdx.x % kLanes == 0) m.scales[p.row * g.perRow.by + p.group] = s.scale;
}

template <typename T, int kKind, bool kGated, int kType>
__global__ __launch_bounds__(kBlock) void actForwardKernel(ActivationForward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr uint32_t kAt = kBlock / (kGroup / E);  // groups of a workgroup
    const int C = int(a.grid.cols);
    for (uint32_t i = blockIdx.x * kAt + threadIdx.x / (kGroup / E); i < a.grid.count; i += gridDim.x * kAt) {
        const Place p = place<E>(a.grid, i);
        Chunk<T, E> gate, up;
        gate.loadRow(static_cast<const T *>(a.gate.p) + p.row * a.gate.stride, p.c, C);
        if constexpr (kGated) up.loadRow(static_cast<const T *>(a.up.p) + p.row * a.up.stride, p.c, C);
        float g[E], u[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            g[e] = gate[e];
            u[e] = kGated ? up[e] : 1.0f;
        }
        if constexpr (kType != kNoCodes) {
            writeGroup<kType, E>(a.gateCodes, p, a.grid, g);
            if constexpr (kGated) writeGroup<kType, E>(a.upCodes, p, a.grid, u);
        }
        if constexpr (kKind != kIdentity) {
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const Activation<kKind> f(g[e]);
                y[e] = kGated ? f.act * u[e] : f.act;
            }
            storeRow(static_cast<T *>(a.out.p) + p.row * a.out.stride, p.c, 0, C, y);
        }
    }
}

// A kept input: the matrix itself or its codes.
template <typename T, int E, int kType>
__device__ __forceinline__ void readKept(const ConstMatrix &m, const ConstCodes &codes, const Place &p,
                                         const GroupGrid &g, float (&v)[E]) {
    const int C = int(g.cols);
    if constexpr (kType == kNoCodes) {
        Chunk<T, E> raw;
        raw.loadRow(static_cast<const T *>(m.p) + p.row * m.stride, p.c, C);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = raw[e];
    } else {
        uint32_t w[E / 4];
        loadCodes<E>(static_cast<const uint8_t *>(codes.p) + p.row * codes.stride, p.c, C, true, w);
        decode<kType, E>(w, codes.scales[codes.wholeRow ? p.row : p.row * g.perRow.by + p.group], v);
    }
}

template <typename T, int kKind, bool kGated, int kType>
__global__ __launch_bounds__(kBlock) void actBackwardKernel(ActivationBackward a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr uint32_t kAt = kBlock / (kGroup / E);
    const int C = int(a.grid.cols);
    for (uint32_t i = blockIdx.x * kAt + threadIdx.x / (kGroup / E); i < a.grid.count; i += gridDim.x * kAt) {
        const Place p = place<E>(a.grid, i);
        float g[E], u[E], y[E];
        readKept<T, E, kType>(a.gate, a.gateCodes, p, a.grid, g);
        if constexpr (kKind == kIdentity) {
            storeRow(static_cast<T *>(a.out.p) + p.row * a.out.stride, p.c, 0, C, g);
            continue;
        } else {
            if constexpr (kGated) readKept<T, E, kType>(a.up, a.upCodes, p, a.grid, u);
            Chunk<T, E> d;
            d.loadRow(static_cast<const T *>(a.dout.p) + p.row * a.dout.stride, p.c, C);
            float act[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const Activation<kKind> f(g[e]);
                act[e] = f.act;
                y[e] = (kGated ? d[e] * u[e] : d[e]) * f.slope;
            }
            storeRow(static_cast<T *>(a.dgate.p) + p.row * a.dgate.stride, p.c, 0, C, y);
            if constexpr (kGated) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = d[e] * act[e];
                storeRow(static_cast<T *>(a.dup.p) + p.row * a.dup.stride, p.c, 0, C, y);
            }
            if (a.out.p) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = kGated ? act[e] * u[e] : act[e];
                storeRow(static_cast<T *>(a.out.p) + p.row * a.out.stride, p.c, 0, C, y);
            }
        }
    }
}

template <int kValue>
using Const = std::integral_constant<int, kValue>;

// f(type, kind, gated, code type) with the call's values as constants.
template <typename F>
hipError_t byKind(int dtype, int kind, bool gated, int codeType, F f) {
    auto coded = [&](auto t, auto k, auto g) {
        if (codeType == BFO_I8) f(t, k, g, Const<BFO_I8>{});
        else if (codeType == BFO_E4M3) f(t, k, g, Const<BFO_E4M3>{});
        else if constexpr (decltype(k)::value != kIdentity) f(t, k, g, Const<kNoCodes>{});
    };
    auto kinds = [&](auto t) {
        if (kind == kIdentity) coded(t, Const<kIdentity>{}, std::false_type{});
        else if (kind == BFO_SILU) gated ? coded(t, Const<BFO_SILU>{}, std::true_type{}) : coded(t, Const<BFO_SILU>{}, std::false_type{});
        else gated ? coded(t, Const<BFO_GELU>{}, std::true_type{}) : coded(t, Const<BFO_GELU>{}, std::false_type{});
    };
    if (dtype == BFO_BF16) kinds(bf16_t(0));
    else kinds(float(0));
    return hipGetLastError();
}

// At most 2^22 workgroups, so that a launch's lanes can be counted in 32 bits.
template <typename T>
dim3 workgroups(const GroupGrid &g) {
    constexpr uint32_t kAt = kBlock / (kGroup * sizeof(T) / 16);
    const uint32_t n = (g.count + kAt - 1) / kAt, most = 1u << 22;
    return dim3(n < most ? n : most);
}

}  // namespace

hipError_t launchActivationForward(const ActivationForward &a, hipStream_t stream) {
    if (!a.grid.count) return hipSuccess;
    return byKind(a.dtype, a.kind, a.up.p != nullptr, a.codeType, [&](auto t, auto kind, auto gated, auto type) {
        using T = decltype(t);
        hipLaunchKernelGGL((actForwardKernel<T, decltype(kind)::value, decltype(gated)::value, decltype(type)::value>),
                           workgroups<T>(a.grid), dim3(kBlock), 0, stream, a);
    });
}

hipError_t launchActivationBackward(const ActivationBackward &a, hipStream_t stream) {
    if (!a.grid.count) return hipSuccess;
    return byKind(a.dtype, a.kind, a.dup.p != nullptr, a.codeType, [&](auto t, auto kind, auto gated, auto type) {
        using T = decltype(t);
        hipLaunchKernelGGL((actBackwardKernel<T, decltype(kind)::value, decltype(gated)::value, decltype(type)::value>),
                           workgroups<T>(a.grid), dim3(kBlock), 0, stream, a);
    });
}

}  // namespace bfo
