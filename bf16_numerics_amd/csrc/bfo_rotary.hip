// bfo_rotary.hip -- gfx950 kernel of rotary positions.
//
// Pair i of a head at position p is turned by the angle p * frequency[i]:
//   (a, b) -> amplitude * (a cos - b sin, a sin + b cos),
// backward by the negative angle, which is the transpose.  Angles are formed
// and reduced to a turn in 64 bits, so that far positions keep them.  A
// wavefront takes a token and a range of its heads: each lane forms the sine
// and cosine of one pair (and of pair + 64, ...) into LDS, then the wavefront
// walks over the heads, 16-byte chunks of both members of the pairs a lane.
#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

constexpr int kBlock = 256, kWaves = kBlock / 64;
constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)

// Rotated pairs that one item of work holds.
template <typename T, bool kHalf>
constexpr int pairsAtOnce() {
    return (kHalf ? 16 : 8) / int(sizeof(T));
}

template <typename T, bool kHalf>
__global__ __launch_bounds__(kBlock) void rotaryKernel(Rotary a) {
    constexpr int E = 16 / int(sizeof(T));
    constexpr int P = pairsAtOnce<T, kHalf>();
    extern __shared__ float turns[];  // a wavefront's cosines, then its sines
    const int lane = int(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int pairs = int(a.rotated / 2), room = (pairs + 7) / 8 * 8;
    float *cosine = turns + wave * 2 * room, *sine = cosine + room;
    const uint32_t first = blockIdx.y * a.headsAtOnce;
    const uint32_t heads = min(a.headsAtOnce, a.heads - first);
    const uint32_t turning = uint32_t(pairs + P - 1) / P, items = heads * a.itemsPerHead.by;
    for (uint64_t token = uint64_t(blockIdx.x) * kWaves + wave; token < a.tokens; token += uint64_t(gridDim.x) * kWaves) {
        const int64_t position = a.positions ? int64_t(a.positions[token]) : int64_t(a.period ? token % a.period : token);
        for (int i = lane; i < pairs; i += 64) {
            double t = double(position) * a.frequencies[i] * kTurn;
            t -= rint(t);
            float s, c;
            sincospif(2.0f * float(t), &s, &c);
            cosine[i] = c * a.amplitude;
            sine[i] = (a.backward ? -s : s) * a.amplitude;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const T *x = static_cast<const T *>(a.x) + token * a.xToken + first * a.xHead;
        T *out = static_cast<T *>(a.out) + token * a.outToken + first * a.outHead;
        for (uint32_t item = lane; item < items; item += 64) {
            const uint32_t head = a.itemsPerHead.divide(item);
            const uint32_t k = item - head * a.itemsPerHead.by;
            const T *in = x + head * a.xHead;
            T *to = out + head * a.outHead;
            if (k >= turning) {  // columns behind the rotated ones
                const int c = int(a.rotated) + int(k - turning) * E;
                Chunk<T, E> v;
                v.loadRow(in, c, int(a.headDim));
                v.storeRow(to, c, int(a.headDim));
                continue;
            }
            const int i = int(k) * P;
            float c[P], s[P];
#pragma unroll
            for (int e = 0; e < P; ++e) c[e] = cosine[i + e], s[e] = sine[i + e];
            if constexpr (kHalf) {
                Chunk<T, E> u, v;
                u.loadRow(in, i, pairs);
                v.loadRow(in + pairs, i, pairs);
                float y[E], z[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    y[e] = fmaf(u[e], c[e], -(v[e] * s[e]));
                    z[e] = fmaf(u[e], s[e], v[e] * c[e]);
                }
                storeRow(to, i, 0, pairs, y);
                storeRow(to + pairs, i, 0, pairs, z);
            } else {
                Chunk<T, E> v;
                v.loadRow(in, 2 * i, 2 * pairs);
                float y[E];
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    y[2 * e] = fmaf(v[2 * e], c[e], -(v[2 * e + 1] * s[e]));
                    y[2 * e + 1] = fmaf(v[2 * e], s[e], v[2 * e + 1] * c[e]);
                }
                storeRow(to, 2 * i, 0, 2 * pairs, y);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, bool kHalf>
void launch(Rotary a, hipStream_t stream) {
    constexpr uint32_t P = pairsAtOnce<T, kHalf>(), E = 16 / sizeof(T);
    const bool inPlace = a.x == a.out;
    const uint32_t turning = (a.rotated / 2 + P - 1) / P;
    const uint32_t per = turning + (inPlace ? 0 : (a.headDim - a.rotated + E - 1) / E);
    a.itemsPerHead = FastDivide(per);
    // A wavefront takes all heads of a token where the tokens fill the chip by
    // themselves, else as few as give each lane one item.
    const uint64_t wanted = a.tokens * a.heads * per / 64 / 8192 + 1;  // items a lane
    uint64_t heads = wanted * 64 / per;
    heads = heads < 1 ? 1 : heads > a.heads ? a.heads : heads;
    a.headsAtOnce = uint32_t(heads);
    const uint64_t tokens = (a.tokens + kWaves - 1) / kWaves, most = 1u << 22;
    const uint32_t room = (a.rotated / 2 + 7) / 8 * 8;
    hipLaunchKernelGGL((rotaryKernel<T, kHalf>), dim3(uint32_t(tokens < most ? tokens : most), (a.heads + a.headsAtOnce - 1) / a.headsAtOnce),
                       dim3(kBlock), kWaves * 2 * room * sizeof(float), stream, a);
}

}  // namespace

hipError_t launchRotary(const Rotary &a, int dtype, int layout, hipStream_t stream) {
    if (!a.tokens || !a.heads) return hipSuccess;
    if (dtype == BFO_BF16) layout == BFO_ROTARY_HALF ? launch<bf16_t, true>(a, stream) : launch<bf16_t, false>(a, stream);
    else layout == BFO_ROTARY_HALF ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
    return hipGetLastError();
}

}  // namespace bfo
