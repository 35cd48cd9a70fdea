// bfo_logits.hip -- gfx950 kernels of the losses over a vocabulary: token log
// probabilities with entropy and top alternatives, distillation from a
// teacher's top logits, and their gradients.
//
// Forward: one workgroup per row, one pass over the row with a running
// maximum, sum of exponentials and sum of their products with the score
// (for the entropy) per lane, joined at the end.  Backward: one pass that
// forms every probability again from the row's maximum and log sum.
#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

constexpr uint32_t kMaxGrid = 1u << 21;

// ---------------------------------------------------------------------------
// Running softmax statistics of raw (unscaled) scores x over some set:
//   m = max x, s = sum 2^((x - m) k), t = sum 2^((x - m) k) (x - m),
// with k = scale * log2(e).  The empty set is {lowest finite, 0, 0}; a set of
// -inf only has s = 0; a NaN or +inf makes s NaN or infinite.
// ---------------------------------------------------------------------------
struct Stat {
    float m, s, t;
};

// The same set with its maximum taken as m >= a.m.
__device__ __forceinline__ Stat raised(const Stat &a, float m, float k) {
    const float d = a.m - m, r = exp2Fast(d * k);
    return {m, a.s * r, r == 0.0f ? 0.0f : r * fmaf(a.s, d, a.t)};
}
__device__ __forceinline__ Stat joined(const Stat &a, const Stat &b, float k) {
    const float m = fmaxf(a.m, b.m);
    const Stat x = raised(a, m, k), y = raised(b, m, k);
    return {m, x.s + y.s, x.t + y.t};
}
__device__ __forceinline__ Stat waveJoined(Stat a, float k) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const Stat b = {__shfl_xor(a.m, d, 64), __shfl_xor(a.s, d, 64), __shfl_xor(a.t, d, 64)};
        a = joined(a, b, k);
    }
    return a;
}

// ---------------------------------------------------------------------------
// Order of scores: larger first, NaN before everything, -0 equal to 0.  A key
// orders like the scores; 0 is below every key.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t keyOf(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float ofKey(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

constexpr int kBlock = 512;             // lanes per row
constexpr int kWaves = kBlock / 64;
constexpr int kGroups = kBlock / 2;     // groups of lanes whose maxima bound the top
constexpr uint32_t kCandidates = 1024;  // scores the top is picked from

struct TopShared {
    alignas(16) uint32_t groupKey[kGroups];
    uint64_t candidate[kCandidates];
    uint32_t histogram[256];
    uint32_t threshold, count, need, digit;
    uint32_t waveCount[kWaves];
};

// The largest 16-bit prefix that at least `top` of the kGroups keys reach:
// a lower bound of the row's top-th key, since every group's key is that of a
// score of its own.  One wavefront, four keys a lane.
__device__ __forceinline__ uint32_t prefixReached(const uint32_t *keys, uint32_t top) {
    const uint4 v = reinterpret_cast<const uint4 *>(keys)[threadIdx.x & 63];
    uint32_t thr = 0;
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t c = thr | (1u << bit);
        const int n = __popcll(__ballot(v.x >= c)) + __popcll(__ballot(v.y >= c)) + __popcll(__ballot(v.z >= c)) +
                      __popcll(__ballot(v.w >= c));
        if (n >= int(top)) thr = c;
    }
    return thr;
}

// The row's exact top, whatever it holds: the top-th key by four rounds of
// 256 bins, then the keys above it and the first equal ones in index order.
// For rows that the bound does not thin out (many equal scores, NaN).
template <typename T>
__device__ void exactTop(const T *row, uint32_t V, uint32_t top, TopShared &sh) {
    uint32_t prefix = 0, need = top;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (uint32_t i = threadIdx.x; i < 256; i += kBlock) sh.histogram[i] = 0;
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < V; c += kBlock) {
            const uint32_t key = keyOf(toFloat(row[c]));
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&sh.histogram[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t d = 255, left = need;
            while (d > 0 && sh.histogram[d] < left) left -= sh.histogram[d--];
            sh.digit = d;
            sh.need = left;
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        need = sh.need;
        __syncthreads();
    }
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    uint32_t equal = 0;  // scores equal to the top-th seen in earlier tiles
    for (uint32_t c0 = 0; c0 < V; c0 += kBlock) {
        const uint32_t c = c0 + threadIdx.x;
        const uint32_t key = c < V ? keyOf(toFloat(row[c])) : 0u;
        const uint64_t same = __ballot(key == prefix);
        if ((threadIdx.x & 63) == 0) sh.waveCount[threadIdx.x >> 6] = uint32_t(__popcll(same));
        __syncthreads();
        uint32_t before = equal, all = equal;
        for (int w = 0; w < kWaves; ++w) {
            if (w < int(threadIdx.x >> 6)) before += sh.waveCount[w];
            all += sh.waveCount[w];
        }
        before += uint32_t(__popcll(same & ((1ull << (threadIdx.x & 63)) - 1)));
        if (key > prefix || (key == prefix && c < V && before < need))
            sh.candidate[atomicAdd(&sh.count, 1u)] = (uint64_t(key) << 32) | (0xFFFFFFFFu - c);
        equal = all;
        __syncthreads();
    }
}

// One pass over the row: E scores of a 16-byte chunk per lane and step.
template <typename T, bool kEntropy>
__device__ __forceinline__ Stat laneStat(const T *row, uint32_t V, float k) {
    constexpr int E = 16 / int(sizeof(T));
    Stat a = {kLowest, 0.0f, 0.0f};
    for (uint32_t c = threadIdx.x * E; c < V; c += kBlock * E) {
        Chunk<T, E> v;
        float x[E];
        v.loadRow(row, c, V);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = c + uint32_t(e) < V ? v[e] : -INFINITY;
        float m = a.m;
#pragma unroll
        for (int e = 0; e < E; e += 2) m = max3(m, x[e], x[e + 1]);
        a = raised(a, m, k);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = x[e] - m, p = exp2Fast(d * k);
            a.s += p;
            if constexpr (kEntropy) a.t = fmaf(p, fmaxf(d, kLowest), a.t);
        }
    }
    return a;
}

struct RowResult {
    float m, s, t, logs, scaled;  // scaled: scale * m
    bool empty, finite;
};
__device__ __forceinline__ RowResult rowResult(const Stat &a, float scale) {
    RowResult r;
    r.m = a.m, r.s = a.s, r.t = a.t;
    r.empty = a.s == 0.0f;
    r.finite = a.s - a.s == 0.0f;
    r.logs = r.empty ? 0.0f : r.finite ? logf(a.s) : NAN;
    r.scaled = r.empty ? -INFINITY : r.finite ? a.m * scale : NAN;
    return r;
}
// log probability of score x.
__device__ __forceinline__ float logProb(const RowResult &r, float x, float scale) {
    if (r.empty) return -INFINITY;
    return r.finite ? (x - r.m) * scale - r.logs : NAN;
}

// The teacher's probabilities of the two entries a lane holds (entries lane
// and lane + 64), over the wavefront; -1 marks no entry.
struct Teacher {
    int id[2];
    float x[2], q[2], logq[2];
    bool any, nan;  // any probability at all; a NaN or +inf among the entries

    __device__ __forceinline__ void load(const int32_t *index, const float *logits, uint32_t count) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t j = (threadIdx.x & 63) + 64 * i;
            id[i] = j < count ? index[j] : -1;
            x[i] = id[i] >= 0 ? logits[j] : -INFINITY;
        }
    }
    __device__ __forceinline__ void softmax(float scale) {
        any = __ballot(id[0] >= 0 || id[1] >= 0) != 0;
        float m = fmaxf(x[0], x[1]);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
        m = fmaxf(m, kLowest);
        float e[2], s = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            e[i] = exp2Fast((x[i] - m) * scale * kLog2e);
            s += e[i];
        }
        s = laneSum<64>(s);
        // Entries of -inf only: no entry at all.
        if (s == 0.0f) any = false;
        nan = !(s - s == 0.0f);
        const float ls = logf(s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            q[i] = any && id[i] >= 0 ? e[i] / s : 0.0f;
            logq[i] = (x[i] - m) * scale - ls;
        }
    }
};

template <typename T, bool kEntropy, bool kTeacher>
__global__ __launch_bounds__(kBlock) void logitsForwardKernel(LogitsForward a) {
    __shared__ Stat stats[kWaves];
    __shared__ TopShared sh;
    const uint32_t V = a.vocab;
    const float k = a.scale * kLog2e;
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *row = static_cast<const T *>(a.logits.p) + r * a.logits.stride;
        const Stat mine = laneStat<T, kEntropy>(row, V, k);
        const Stat wave = waveJoined(mine, k);
        if ((threadIdx.x & 63) == 0) stats[threadIdx.x >> 6] = wave;
        if (a.top) {
            // Lanes without scores hold key 0; one whose maximum may be -inf holds that key.
            uint32_t key = threadIdx.x * (16 / sizeof(T)) < V ? keyOf(mine.m > kLowest ? mine.m : -INFINITY) : 0u;
            key = max(key, uint32_t(__shfl_xor(int(key), 1, 64)));
            if (threadIdx.x % 2 == 0) sh.groupKey[threadIdx.x / 2] = key;
        }
        __syncthreads();
        Stat all = stats[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) all = joined(all, stats[w], k);
        const RowResult res = rowResult(all, a.scale);
        if (threadIdx.x == 0) {
            if (a.stats) a.stats[2 * r] = res.scaled, a.stats[2 * r + 1] = res.logs;
            if (a.logprob) {
                const int t = a.targets[r];
                a.logprob[r] = t < 0 ? 0.0f : uint32_t(t) >= V ? NAN : logProb(res, toFloat(row[t]), a.scale);
            }
            if constexpr (kEntropy) {
                if (a.entropy)
                    a.entropy[r] = res.empty ? 0.0f : res.finite ? res.logs - a.scale * res.t / res.s : NAN;
            }
        }
        if constexpr (kTeacher) {
            if (threadIdx.x < 64) {
                Teacher te;
                te.load(a.teacherIndex + r * a.count, a.teacherLogits + r * a.count, a.count);
                te.softmax(a.scale);
                float kl = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (te.id[i] < 0) continue;
                    if (uint32_t(te.id[i]) >= V) kl = NAN;
                    else if (te.q[i] != 0.0f)
                        kl += te.q[i] * (te.logq[i] - logProb(res, toFloat(row[te.id[i]]), a.scale));
                }
                kl = laneSum<64>(kl);
                if (threadIdx.x == 0) a.kl[r] = kl;
            }
        }
        if (a.top) {
            if (threadIdx.x < 64) {
                const uint32_t thr = prefixReached(sh.groupKey, a.top);
                if (threadIdx.x == 0) sh.threshold = thr, sh.count = 0;
            }
            __syncthreads();
            const uint32_t thr = sh.threshold;
            const bool bounded = res.finite && !res.empty;
            if (bounded && keyOf(mine.m) >= thr) {
                constexpr int E = 16 / int(sizeof(T));
                for (uint32_t c = threadIdx.x * E; c < V; c += kBlock * E) {
                    Chunk<T, E> v;
                    v.loadRow(row, c, V);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const uint32_t key = keyOf(v[e]);
                        if (key >= thr && c + uint32_t(e) < V) {
                            const uint32_t at = atomicAdd(&sh.count, 1u);
                            if (at < kCandidates) sh.candidate[at] = (uint64_t(key) << 32) | (0xFFFFFFFFu - (c + e));
                        }
                    }
                }
            }
            __syncthreads();
            if (!bounded || sh.count > kCandidates) {
                __syncthreads();
                exactTop(row, V, a.top, sh);
            }
            // Keys are unique, so a candidate's place is the number above it.
            const uint32_t n = sh.count;
            for (uint32_t i = threadIdx.x; i < n; i += kBlock) {
                const uint64_t key = sh.candidate[i];
                uint32_t place = 0;
                for (uint32_t j = 0; j < n; ++j) place += sh.candidate[j] > key;
                if (place < a.top) {
                    a.topIndex[r * a.top + place] = int32_t(0xFFFFFFFFu - uint32_t(key));
                    a.topLogprob[r * a.top + place] = logProb(res, ofKey(uint32_t(key >> 32)), a.scale);
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Backward: a workgroup owns a segment of a row's columns.
// ---------------------------------------------------------------------------
constexpr int kBackBlock = 256;
constexpr int kBackChunks = 4;
template <typename T>
constexpr uint32_t backSegment() {
    return kBackBlock * kBackChunks * (16 / sizeof(T));
}

// Teacher entries inside the segment, chained per 16-byte chunk: head[chunk]
// is the first one there, next[entry] the following one, in the entries'
// order, so that equal indexes add in a fixed order.
struct Chains {
    static constexpr uint32_t kNone = 0xFF;
    uint8_t head[kBackBlock * kBackChunks];
    uint8_t next[BFO_TOP_MAX];
    uint32_t column[BFO_TOP_MAX];  // within the segment
    float value[BFO_TOP_MAX];
    float base;
};
static_assert(BFO_TOP_MAX <= 128, "a lane of one wavefront holds two entries");

// One wavefront: writes the chains of the entries with columns in [c0, c1),
// each with its part of the gradient, and the part of the row's `base`.
__device__ __forceinline__ void buildChains(Chains &ch, const Teacher &te, float dkl, uint32_t vocab, uint32_t c0,
                                            uint32_t c1, uint32_t perChunk) {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t below = (1ull << lane) - 1;
    const bool bad = __ballot((te.id[0] >= 0 && uint32_t(te.id[0]) >= vocab) ||
                              (te.id[1] >= 0 && uint32_t(te.id[1]) >= vocab)) != 0;
    const bool in0 = te.id[0] >= 0 && uint32_t(te.id[0]) >= c0 && uint32_t(te.id[0]) < c1;
    const bool in1 = te.id[1] >= 0 && uint32_t(te.id[1]) >= c0 && uint32_t(te.id[1]) < c1;
    const uint64_t m0 = __ballot(in0), m1 = __ballot(in1);
    const uint32_t n0 = uint32_t(__popcll(m0)), n = n0 + uint32_t(__popcll(m1));
    if (in0) {
        const uint32_t at = uint32_t(__popcll(m0 & below));
        ch.column[at] = uint32_t(te.id[0]) - c0;
        ch.value[at] = -dkl * te.q[0];
    }
    if (in1) {
        const uint32_t at = n0 + uint32_t(__popcll(m1 & below));
        ch.column[at] = uint32_t(te.id[1]) - c0;
        ch.value[at] = -dkl * te.q[1];
    }
    if (lane == 0) ch.base = bad || te.nan ? NAN : te.any ? dkl : 0.0f;
    // The wavefront's own LDS writes are read below by its other lanes.
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
    for (uint32_t i = lane; i < n; i += 64) {
        const uint32_t chunk = ch.column[i] / perChunk;
        uint32_t next = Chains::kNone;
        bool first = true;
        for (uint32_t j = 0; j < n; ++j) {
            const bool same = ch.column[j] / perChunk == chunk;
            if (same && j < i) first = false;
            if (same && j > i && next == Chains::kNone) next = j;
        }
        ch.next[i] = uint8_t(next);
        if (first) ch.head[chunk] = uint8_t(i);
    }
}

// Segments run along x, rows along y.
template <typename T, bool kEntropy, bool kTeacher>
__global__ __launch_bounds__(kBackBlock) void logitsBackwardKernel(LogitsBackward a, uint32_t segment) {
    constexpr int E = 16 / int(sizeof(T));
    __shared__ Chains ch;
    const uint32_t V = a.vocab, c0 = blockIdx.x * segment;
    const uint32_t end = min(c0 + segment, a.width);  // the segment's columns: [c0, end)
    for (uint64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const T *row = static_cast<const T *>(a.logits.p) + r * a.logits.stride;
        T *out = static_cast<T *>(a.dlogits.p) + r * a.dlogits.stride;
        const float m = a.stats[2 * r], logs = a.stats[2 * r + 1];
        // dlogits = scale * (p * (base + slope * log p) + what its tokens get)
        int target = -1;
        float hard = 0.0f, base = 0.0f, slope = 0.0f, dkl = 0.0f;
        if (a.targets) {
            target = a.targets[r];
            if (target >= 0) {
                hard = a.dlogprob[r];
                base = uint32_t(target) >= V ? NAN : -hard;
            }
        }
        if constexpr (kEntropy) {
            const float de = a.dentropy[r];
            slope = -de;
            if (de != 0.0f) base -= de * a.entropy[r];
        }
        if constexpr (kTeacher) dkl = a.dkl[r];
        bool live = m != -INFINITY && !(hard == 0.0f && base == 0.0f && slope == 0.0f && dkl == 0.0f);
        Chunk<T, E> v[kBackChunks];
        if (live) {
#pragma unroll
            for (int k = 0; k < kBackChunks; ++k) {
                const uint32_t c = (threadIdx.x + kBackBlock * k) * E;
                if (c < segment) v[k].loadRow(row, c0 + c, V);
            }
        }
        if constexpr (kTeacher) {
            if (live) {
                reinterpret_cast<uint32_t *>(ch.head)[threadIdx.x] = 0xFFFFFFFFu;
                Teacher te;
                if (threadIdx.x < 64) {
                    te.load(a.teacherIndex + r * a.count, a.teacherLogits + r * a.count, a.count);
                    te.softmax(a.scale);
                }
                __syncthreads();
                if (threadIdx.x < 64) buildChains(ch, te, dkl, V, c0, end, E);
                __syncthreads();
                base += ch.base;
                live = !(hard == 0.0f && base == 0.0f && ch.base == 0.0f);
            }
        }
#pragma unroll
        for (int k = 0; k < kBackChunks; ++k) {
            const uint32_t at = (threadIdx.x + kBackBlock * k) * E, c = c0 + at;
            if (at >= segment || c >= end) continue;
            float y[E];
            if (live) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float lp = fmaf(v[k][e], a.scale, -m) - logs;
                    const float p = exp2Fast(lp * kLog2e);
                    // p is 0 well above -1e4, where the product has to be 0 too
                    y[e] = p * (kEntropy ? fmaf(slope, fmaxf(lp, -1e4f), base) : base);
                }
                if constexpr (kTeacher) {
                    uint32_t h = ch.head[threadIdx.x + kBackBlock * k];
                    while (h != Chains::kNone) {
                        const uint32_t col = ch.column[h] - at;
                        const float val = ch.value[h];
#pragma unroll
                        for (int e = 0; e < E; ++e) y[e] += col == uint32_t(e) ? val : 0.0f;
                        h = ch.next[h];
                    }
                }
                if (target >= 0 && uint32_t(target) - c < uint32_t(E)) {
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] += uint32_t(target) - c == uint32_t(e) ? hard : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = c + uint32_t(e) < V ? y[e] * a.scale : 0.0f;
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = 0.0f;
            }
            storeRow(out, c, end, y);
        }
        if constexpr (kTeacher) __syncthreads();
    }
}

template <typename T>
hipError_t forward(const LogitsForward &a, hipStream_t stream) {
    const dim3 grid(uint32_t(a.rows < kMaxGrid ? a.rows : kMaxGrid)), block(kBlock);
    if (a.count) hipLaunchKernelGGL((logitsForwardKernel<T, false, true>), grid, block, 0, stream, a);
    else if (a.entropy) hipLaunchKernelGGL((logitsForwardKernel<T, true, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((logitsForwardKernel<T, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(const LogitsBackward &a, hipStream_t stream) {
    constexpr uint32_t most = backSegment<T>(), line = 128 / sizeof(T);
    // Even segments, each starting on a 128-byte line of the row.
    const uint32_t segments = (a.width + most - 1) / most;
    const uint32_t segment = ((a.width + segments - 1) / segments + line - 1) / line * line;
    const dim3 grid((a.width + segment - 1) / segment, uint32_t(a.rows < 65535 ? a.rows : 65535)), block(kBackBlock);
    if (a.count) hipLaunchKernelGGL((logitsBackwardKernel<T, false, true>), grid, block, 0, stream, a, segment);
    else if (a.dentropy) hipLaunchKernelGGL((logitsBackwardKernel<T, true, false>), grid, block, 0, stream, a, segment);
    else hipLaunchKernelGGL((logitsBackwardKernel<T, false, false>), grid, block, 0, stream, a, segment);
    return hipGetLastError();
}

}  // namespace

uint64_t logitsWorkspaceBytes(uint64_t, uint32_t, uint32_t) { return 0; }

hipError_t launchLogitsForward(const LogitsForward &a, int dtype, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return dtype == BFO_BF16 ? forward<bf16_t>(a, stream) : forward<float>(a, stream);
}

hipError_t launchLogitsBackward(const LogitsBackward &a, int dtype, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return dtype == BFO_BF16 ? backward<bf16_t>(a, stream) : backward<float>(a, stream);
}

}  // namespace bfo
