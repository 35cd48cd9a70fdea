// bfo_logits.hip -- gfx950 kernels of the losses over a vocabulary: token log
// probabilities with entropy and top alternatives, distillation from a
// teacher's top logits, and their gradients.
//
// Forward: one workgroup per row (or per segment of a long one, when there are
// few; a second launch joins those), one pass over the row with a running
// maximum, sum of exponentials and sum of their products with the score (for the
// entropy) per lane, joined at the end.  The best scores are picked from the
// chunks whose kept maximum reaches a bound that at least K scores reach.
// Backward: one pass that forms every probability again from the row's maximum
// and log sum.
//
// On an MI355X, bf16: 8192 x 50257 scores forward in 124 us (6.6 TB/s, bound by
// memory), in 142 with entropy and 20 alternatives (bound by the vector ALUs, 83-88%
// busy), gradient of 8192 x 50304 in 262 us (6.0 TB/s read and written).
#include <type_traits>

#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

constexpr uint32_t kMaxGrid = 1u << 21;

// ---------------------------------------------------------------------------
// Softmax statistics of raw (unscaled) scores x over some set, with
// k = scale * log2(e):
//   m = max x, s = sum 2^(x k - M), t = sum 2^(x k - M) (x k - M).
// While a row is read, M is m k rounded, so that an exponent is one fma; a
// finished Stat has M = m k exactly.  The empty set is {lowest finite, 0, 0}; a
// set of -inf only has s = 0; a NaN or +inf makes s NaN.
// ---------------------------------------------------------------------------
struct Stat {
    float m, s, t;
};

// The rounded M.  Its error is folded into the finished s and t, which needs it
// to be small: rows with |m k| >= kReferenceMost are read again by exactStat.  A
// lane that sees only far lower scores than that (masks of the type's lowest
// value) has them count as 0 by the floor.
constexpr float kReferenceMost = 1024.0f, kReferenceFloor = -2048.0f;
__device__ __forceinline__ float referenceOf(float m, float k) { return fmaxf(m * k, kReferenceFloor); }

// (x - m) times the scale.
__device__ __forceinline__ float scaledDifference(float x, float m, const DifferenceScale &by) {
    return fmaf(x, by.part, -(m * by.part)) * by.rest;
}
// (x - m) k.  From scales of 2^128 / log2(e) on k is infinite, and no reference
// holds (m k is infinite or, for m = 0, NaN): such rows are exactStat's, by this
// product in its parts.
__device__ __forceinline__ float differenceTimesK(float x, float m, float k, float scale) {
    const float d = x - m;
    return k < INFINITY ? d * k : d * scale * kLog2e;
}

// The set's s and t for an M that is `up` larger.
__device__ __forceinline__ Stat raised(const Stat &a, float m, float up) {
    const float r = exp2Fast(-up);
    return {m, a.s * r, r == 0.0f ? 0.0f : r * fmaf(a.s, -up, a.t)};
}
__device__ __forceinline__ Stat raisedReference(const Stat &a, float m, float k) {
    return raised(a, m, referenceOf(m, k) - referenceOf(a.m, k));
}
// The wavefront's statistics, in every lane.
__device__ __forceinline__ Stat waveJoined(const Stat &a, float k) {
    const float m = waveMax(a.m);
    const Stat b = raisedReference(a, m, k);
    return {m, laneSum<64>(b.s), laneSum<64>(b.t)};
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

// A row's workgroup: kBlock lanes take the row in steps of kUnroll 16-byte
// chunks each, whose loads are in flight together.
constexpr int kUnroll = 4;
template <typename T>
constexpr uint32_t chunkElems() {
    return 16 / sizeof(T);
}

// Chunks are cut on 128-byte lines of memory, not from the row's first column
// (8192 x 50257 bf16 of odd rows 129 us for 171): the columns of a row's first line
// that come before the row.  Which lane sums which column thus depends on the row's
// start.
template <typename T>
__device__ __forceinline__ int leadOf(const T *row) {
    return int((reinterpret_cast<uintptr_t>(row) & 127u) / sizeof(T));
}
template <typename T>
constexpr uint32_t kMaxLead = 128 / sizeof(T) - 1;

constexpr uint32_t kNoScores = 0xFFFF;  // upper half of a NaN, which reaches no bound
constexpr int kGroups = 256;           // groups of lanes whose maxima bound the top
// Stretches of a lane's chunks whose maxima are kept.  Stretches of one chunk are
// the best (8192 x 50257 bf16, 20 best, at an earlier step: 157 us, of several 162).
// 28 are seven steps of four chunks, the most steps that leave LDS for the seven
// workgroups a CU has registers for (22 of 160 KB each): one chunk each up to 57,344
// bf16 or 28,672 fp32 scores with 256 lanes.  Longer rows keep a maximum of several:
// 4096 x 128256 bf16 with 20 best 174 us, 6.0 TB/s.
constexpr int kSlots = 28;
constexpr uint32_t kCandidates = 512;  // scores the top is picked from

template <int kBlock>
struct TopShared {
    alignas(16) uint32_t groupKey[kGroups];
    alignas(16) uint64_t candidate[kCandidates];
    uint16_t slotMax[kSlots * kBlock];  // upper halves of the maxima, kNoScores for none
    uint16_t pairs[kCandidates];        // the slots that may hold a candidate
    uint32_t histogram[256];
    float bound;
    uint32_t pairCount, count, need, digit;
    uint32_t waveCount[kBlock / 64];
};

// A lower bound of the row's top-th score: every group's key is that of a score
// of its own, so what `top` of the kGroups keys reach is reached by that many
// scores.  The largest such 14-bit prefix, found below the keys' common one; one
// wavefront, four keys a lane.
__device__ __forceinline__ float boundOf(const uint32_t *keys, uint32_t top) {
    constexpr int kLowBit = 18;
    const uint4 v = reinterpret_cast<const uint4 *>(keys)[threadIdx.x & 63];
    const uint32_t most = waveExtreme<true>(max(max(v.x, v.y), max(v.z, v.w)));
    const uint32_t least = waveExtreme<false>(min(min(v.x, v.y), min(v.z, v.w)));
    const int high = max(31 - __clz(int(most ^ least)), kLowBit - 1);  // the highest bit that differs
    uint32_t bound = most & ~((2u << high) - 1u);
    for (int bit = high; bit >= kLowBit; --bit) {
        const uint32_t c = bound | (1u << bit);
        const int n = __popcll(__ballot(v.x >= c)) + __popcll(__ballot(v.y >= c)) + __popcll(__ballot(v.z >= c)) +
                      __popcll(__ballot(v.w >= c));
        if (n >= int(top)) bound = c;
    }
    return bound <= keyOf(-INFINITY) ? -INFINITY : ofKey(bound);
}

// The row's exact top, whatever it holds: the top-th key by four rounds of
// 256 bins, then the keys above it and the first equal ones in index order.
// For rows that the bound does not thin out (many equal scores, NaN, fewer
// finite scores than asked for).  Five passes of one score a lane: 8192 x 50257
// bf16 of nothing but such rows 5.8 ms against 145 us, one row of 32,000 184 us
// against 9.
template <typename T, int kBlock>
__device__ __noinline__ void exactTop(const T *row, uint32_t V, uint32_t top, TopShared<kBlock> &sh) {
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
        for (int w = 0; w < kBlock / 64; ++w) {
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

// One pass over the row.  The maximum is raised once a step.  With kTop, the maxima of stretches of
// `perSlot` chunks of the lane stay in slotMax.
template <typename T, int kBlock, bool kNontemporal, bool kEntropy, bool kTop>
__device__ __forceinline__ Stat laneStat(const T *row, uint32_t V, float k, uint32_t perSlot, uint16_t *slotMax) {
    constexpr uint32_t E = chunkElems<T>();
    Stat a = {kLowest, 0.0f, 0.0f};
    uint32_t slot = 0, held = 0;
    float stretch = -INFINITY;
    auto endStretch = [&] {
        // + 0 makes -0 the 0 it is equal to
        slotMax[slot * kBlock + threadIdx.x] = uint16_t(__float_as_uint(stretch + 0.0f) >> 16);
        ++slot;
        held = 0;
        stretch = -INFINITY;
    };
    const int lead = leadOf(row), end = int(V) + lead, c = int(threadIdx.x * E);  // columns from the row's line on
    const T *line = row - lead;
    // The wavefront has scores in the chunks that start before waveEnd; in its
    // last step it passes over the others.
    const int waveEnd = end - int(__builtin_amdgcn_readfirstlane(int(threadIdx.x & ~63u)) * E);
    auto step = [&](int c0, auto last) {
        auto gone = [&](int u) { return decltype(last)::value && c0 + int(kBlock * E) * u >= waveEnd; };
        Chunk<T, E> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = c0 + int(kBlock * E) * u;
            v[u].template loadScores<kNontemporal>(line + at, c, lead - at, end - at);
        }
        float m = a.m;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (gone(u)) continue;
            if constexpr (kTop) {
                float top = max3(v[u][0], v[u][1], v[u][2]);
#pragma unroll
                for (int e = 3; e < int(E) - 1; e += 2) top = max3(top, v[u][e], v[u][e + 1]);
                stretch = max3(stretch, top, v[u][E - 1]);
                m = max3(m, stretch, stretch);  // the stretch's earlier scores are in m already
                if (++held == perSlot) endStretch();
            } else {
#pragma unroll
                for (int e = 0; e < int(E); e += 2) m = max3(m, v[u][e], v[u][e + 1]);
            }
        }
        a = raisedReference(a, m, k);
        const float reference = referenceOf(m, k);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (gone(u)) continue;
#pragma unroll
            for (int e = 0; e < int(E); ++e) {
                const float d = fmaf(v[u][e], k, -reference), p = exp2Fast(d);
                a.s += p;
                // p is 0 where d is -inf: their product has to be 0 too
                if constexpr (kEntropy) a.t = fmaf(p, fmaxf(d, kLowest), a.t);
            }
        }
    };
    constexpr int kStep = int(kBlock * E) * kUnroll;
    int c0 = 0;
    for (; c0 + kStep - int(kBlock * E) < waveEnd; c0 += kStep) step(c0, std::false_type{});
    if (c0 < waveEnd) step(c0, std::true_type{});
    if constexpr (kTop) {
        if (held) endStretch();
        for (; slot < uint32_t(kSlots); ++slot) slotMax[slot * kBlock + threadIdx.x] = uint16_t(kNoScores);
    }
    return a;
}

// A number of its own below the counter's new value for each active lane, with
// one atomic a wavefront.
__device__ __forceinline__ uint32_t claimOne(uint32_t *counter) {
    const uint64_t active = __ballot(1);
    const uint32_t before = uint32_t(__popcll(active & ((1ull << (threadIdx.x & 63)) - 1)));
    uint32_t first = 0;
    if (before == 0) first = atomicAdd(counter, uint32_t(__popcll(active)));
    return uint32_t(__builtin_amdgcn_readfirstlane(int(first))) + before;
}

// The workgroup's wavefronts joined, in every lane; `stats` may be used again.
template <int kBlock>
__device__ __forceinline__ Stat blockJoined(const Stat &wave, Stat (&stats)[kBlock / 64], float k) {
    if ((threadIdx.x & 63) == 0) stats[threadIdx.x >> 6] = wave;
    __syncthreads();
    Stat all = stats[0];
#pragma unroll
    for (int w = 1; w < kBlock / 64; ++w) all.m = fmaxf(all.m, stats[w].m);
    all.s = all.t = 0.0f;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) {
        const Stat b = raisedReference(stats[w], all.m, k);
        all.s += b.s;
        all.t += b.t;
    }
    return all;
}

// A finished Stat of a row with maximum m by differences from m, which are
// exact where products with k are not: for the rows that referenceOf is not for.
// (One past binary32 is right as -inf: |m k| >= kReferenceMost leaves no k small
// enough for its exponential to be above 0.)
template <typename T, int kBlock>
__device__ __noinline__ Stat exactStat(const T *row, uint32_t V, float m, float k, float scale,
                                       Stat (&stats)[kBlock / 64]) {
    Stat a = {m, 0.0f, 0.0f};
    for (uint32_t c = threadIdx.x; c < V; c += kBlock) {
        const float d = differenceTimesK(toFloat(row[c]), m, k, scale), p = exp2Fast(d);
        a.s += p;
        a.t = fmaf(p, fmaxf(d, kLowest), a.t);
    }
    a.s = laneSum<64>(a.s);
    a.t = laneSum<64>(a.t);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) stats[threadIdx.x >> 6] = a;
    __syncthreads();
    a.s = a.t = 0.0f;
    for (int w = 0; w < kBlock / 64; ++w) {
        a.s += stats[w].s;
        a.t += stats[w].t;
    }
    return a;
}

template <typename T, int kBlock>
__device__ __forceinline__ Stat finished(const Stat &a, const T *row, uint32_t V, float k, float scale,
                                         Stat (&stats)[kBlock / 64]) {
    if (a.s == 0.0f || !(fabsf(a.m * k) < kReferenceMost)) return exactStat<T, kBlock>(row, V, a.m, k, scale, stats);
    // M's rounding error, an exact difference of less than 2^-13
    return raised(a, a.m, fmaf(a.m, k, -referenceOf(a.m, k)));
}

// The candidates of the row's top: every score that reaches the bound.  False
// if there are too many.
template <typename T, int kBlock>
__device__ __forceinline__ bool gatherCandidates(const T *row, uint32_t V, uint32_t perSlot,
                                                 TopShared<kBlock> &sh) {
    constexpr uint32_t E = chunkElems<T>();
    const float bound = sh.bound;
    uint32_t hits = 0;
#pragma unroll
    for (int slot = 0; slot < kSlots; ++slot) {
        // the maximum cut to its upper half, towards 0: what the bound needs cut the same way or lower; NaN for none
        const float m = __uint_as_float(uint32_t(sh.slotMax[slot * kBlock + threadIdx.x]) << 16);
        hits |= (m >= bound ? 1u : 0u) << slot;
    }
    while (__ballot(hits != 0)) {
        if (hits) {
            const uint32_t n = claimOne(&sh.pairCount);
            if (n < kCandidates) sh.pairs[n] = uint16_t((__ffs(int(hits)) - 1) * kBlock + threadIdx.x);
            hits &= hits - 1;
        }
    }
    __syncthreads();
    const uint32_t pairs = sh.pairCount;
    if (pairs > kCandidates) return false;
    for (uint32_t i = threadIdx.x; i < pairs * perSlot; i += kBlock) {
        const uint32_t at = sh.pairs[i / perSlot], chunk = (at / kBlock) * perSlot + i % perSlot;
        const int c = int((chunk * kBlock + at % kBlock) * E) - leadOf(row);
        if (c >= int(V)) continue;
        Chunk<T, E> v;
        v.loadScores(row, c, 0, int(V));
        uint32_t reached = 0;
#pragma unroll
        for (int e = 0; e < int(E); ++e) reached |= (v[e] >= bound && uint32_t(c + e) < V ? 1u : 0u) << e;
        while (reached) {
            const int at = __ffs(int(reached)) - 1;
            reached &= reached - 1;
            float x = v[0];
#pragma unroll
            for (int e = 1; e < int(E); ++e) x = at == e ? v[e] : x;
            const uint32_t n = claimOne(&sh.count);
            if (n < kCandidates) sh.candidate[n] = (uint64_t(keyOf(x)) << 32) | (0xFFFFFFFFu - uint32_t(c + at));
        }
    }
    __syncthreads();
    return sh.count <= kCandidates;
}

struct Empty {};

struct RowResult {
    float m, s, t, logs, scaled;  // scaled: scale * m
    bool empty, finite;
};
__device__ __forceinline__ RowResult rowResult(const Stat &a, float scale) {
    RowResult r;
    r.m = a.m, r.s = a.s, r.t = a.t;
    // Scores are infinities where their product with the scale is one.
    const float scaled = a.m * scale;
    r.empty = a.s == 0.0f || (a.s > 0.0f && scaled == -INFINITY);
    r.finite = a.s - a.s == 0.0f && scaled < INFINITY;
    r.logs = r.empty ? 0.0f : r.finite ? logf(a.s) : NAN;
    r.scaled = r.empty ? -INFINITY : r.finite ? scaled : NAN;
    return r;
}
// log probability of score x.
__device__ __forceinline__ float logProb(const RowResult &r, float x, const DifferenceScale &by) {
    if (r.empty) return -INFINITY;
    return r.finite ? scaledDifference(x, r.m, by) - r.logs : NAN;
}

__device__ __forceinline__ void writeTop(const LogitsForward &a, uint64_t r, const RowResult &res, uint64_t key,
                                         uint32_t place) {
    a.topIndex[r * a.top + place] = int32_t(0xFFFFFFFFu - uint32_t(key));
    a.topLogprob[r * a.top + place] = logProb(res, ofKey(uint32_t(key >> 32)), a.difference);
}

// Calls put(key, place) for the top: keys are unique, so a candidate's place
// is the number of those above it.
template <int kBlock, typename F>
__device__ __forceinline__ void placeCandidates(const TopShared<kBlock> &sh, uint32_t top, F put) {
    const uint32_t n = sh.count;
    for (uint32_t i = threadIdx.x; i < n; i += kBlock) {
        const uint64_t key = sh.candidate[i];
        const ulonglong2 *pairs = reinterpret_cast<const ulonglong2 *>(sh.candidate);
        uint32_t place = n & 1u ? sh.candidate[n - 1] > key : 0;
#pragma unroll 4
        for (uint32_t j = 0; j < n / 2; ++j) {
            const ulonglong2 other = pairs[j];
            place += other.x > key;
            place += other.y > key;
        }
        if (place < top) put(key, place);
    }
}

// The segments of each row where few rows are split: statistics ({m, s, t, 0})
// and the keys of the segments' tops in the workspace.
struct Segments {
    uint32_t count, length;

    __device__ __forceinline__ float4 *stats(const LogitsForward &a) const {
        return static_cast<float4 *>(a.workspace);
    }
    __device__ __forceinline__ uint64_t *keys(const LogitsForward &a) const {
        return reinterpret_cast<uint64_t *>(stats(a) + a.rows * count);
    }
};
constexpr uint32_t kMaxSegments = 8;

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
    __device__ __forceinline__ void softmax(const DifferenceScale &by) {
        any = __ballot(id[0] >= 0 || id[1] >= 0) != 0;
        const float m = fmaxf(waveMax(fmaxf(x[0], x[1])), kLowest);
        float e[2], s = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            e[i] = exp2Fast(scaledDifference(x[i], m, by) * kLog2e);
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
            logq[i] = scaledDifference(x[i], m, by) - ls;
        }
    }
};

// What the end of a row needs besides its statistics, asked for at its start.
template <typename T, bool kTeacher>
struct RowEnd {
    int target;
    float targetScore;
    Teacher teacher;
    float teacherScore[2];

    __device__ __forceinline__ void load(const LogitsForward &a, uint64_t r, const T *row) {
        const uint32_t V = a.vocab;
        target = a.targets ? a.targets[r] : -1;
        targetScore = target >= 0 && uint32_t(target) < V ? toFloat(row[target]) : 0.0f;
        if constexpr (kTeacher) {
            if (threadIdx.x < 64) {
                teacher.load(a.teacherIndex + r * a.count, a.teacherLogits + r * a.count, a.count);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool token = teacher.id[i] >= 0 && uint32_t(teacher.id[i]) < V;
                    teacherScore[i] = token ? toFloat(row[teacher.id[i]]) : 0.0f;
                }
            }
        }
    }
    // Thread `writer` writes the row's results, the first wavefront those
    // against the teacher.
    __device__ __forceinline__ void write(const LogitsForward &a, uint64_t r, const RowResult &res, bool entropy,
                                          uint32_t writer) {
        const uint32_t V = a.vocab;
        if (threadIdx.x == writer) {
            if (a.stats) a.stats[2 * r] = res.scaled, a.stats[2 * r + 1] = res.logs;
            if (a.logprob)
                a.logprob[r] = target < 0            ? 0.0f
                               : uint32_t(target) >= V ? NAN
                                                       : logProb(res, targetScore, a.difference);
            if (entropy) a.entropy[r] = res.empty ? 0.0f : res.finite ? res.logs - kLn2 * (res.t / res.s) : NAN;
        }
        if constexpr (kTeacher) {
            if (threadIdx.x < 64) {
                teacher.softmax(a.difference);
                float kl = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (teacher.id[i] < 0) continue;
                    if (uint32_t(teacher.id[i]) >= V) kl = NAN;
                    else if (teacher.q[i] != 0.0f)
                        kl += teacher.q[i] * (teacher.logq[i] - logProb(res, teacherScore[i], a.difference));
                }
                kl = laneSum<64>(kl);
                if (threadIdx.x == 0) a.kl[r] = kl;
            }
        }
    }
};

// One workgroup per row, or (kSplit) per segment of a row: then the results are
// the segment's statistics and the keys of its top, in the workspace, for
// logitsJoinKernel.  With a top, 72 registers are enough for seven wavefronts a
// SIMD (odd rows 152 -> 147 us against the compiler's choice; eight lose 4%), but
// with 512 lanes, where two rows a CU are the most, they spill (512 x 32000 13.9
// against 14.6).
template <typename T, int kBlock, bool kNontemporal, bool kEntropy, bool kTop, bool kTeacher, bool kSplit>
__global__ __launch_bounds__(kBlock, kTop ? (kBlock > 256 ? 4 : 7) : 1) void logitsForwardKernel(LogitsForward a, uint32_t perSlot, Segments seg) {
    constexpr uint32_t E = chunkElems<T>();
    __shared__ Stat stats[kBlock / 64];
    __shared__ std::conditional_t<kTop, TopShared<kBlock>, Empty> sh;
    const uint32_t first = kSplit ? blockIdx.y * seg.length : 0;  // the segment's columns: V from `first` on
    const uint32_t V = kSplit ? min(seg.length, a.vocab - first) : a.vocab;
    const float k = a.scale * kLog2e;
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *row = static_cast<const T *>(a.logits.p) + r * a.logits.stride + first;
        RowEnd<T, kTeacher> end;
        if constexpr (!kSplit) end.load(a, r, row);
        uint16_t *slotMax = nullptr;
        if constexpr (kTop) slotMax = sh.slotMax;
        const Stat mine = laneStat<T, kBlock, kNontemporal, kEntropy, kTop>(row, V, k, perSlot, slotMax);
        const Stat wave = waveJoined(mine, k);
        if constexpr (kTop) {
            // Lanes without scores hold key 0; one whose maximum may be -inf holds that key.
            const int c = int(threadIdx.x * E) - leadOf(row);  // its first chunk, whole or not, or its second
            const bool some = (c < int(V) && c + int(E) > 0) || c + int(kBlock * E) < int(V);
            uint32_t key = some ? keyOf(mine.m > kLowest ? mine.m : -INFINITY) : 0u;
#pragma unroll
            for (int d = 1; d < kBlock / kGroups; d *= 2) key = max(key, uint32_t(__shfl_xor(int(key), d, 64)));
            if (threadIdx.x % (kBlock / kGroups) == 0) sh.groupKey[threadIdx.x / (kBlock / kGroups)] = key;
        }
        const Stat all = finished<T, kBlock>(blockJoined<kBlock>(wave, stats, k), row, V, k, a.scale, stats);
        // The last wavefront writes the row's results while the first one looks for
        // the bound of its top.
        const RowResult res = rowResult(all, a.scale);
        if constexpr (kSplit) {
            if (threadIdx.x == kBlock - 64) seg.stats(a)[r * seg.count + blockIdx.y] = {all.m, all.s, all.t, 0.0f};
        } else {
            end.write(a, r, res, kEntropy, kBlock - 64);
        }
        if constexpr (kTop) {
            if (threadIdx.x < 64) {
                const float bound = boundOf(sh.groupKey, a.top);
                if (threadIdx.x == 0) sh.bound = bound, sh.count = sh.pairCount = 0;
            }
            __syncthreads();
            const bool bounded = res.finite && !res.empty;  // the same in every lane
            if (!bounded || !gatherCandidates(row, V, perSlot, sh)) {
                __syncthreads();
                exactTop(row, V, a.top, sh);
            }
            placeCandidates<kBlock>(sh, a.top, [&](uint64_t key, uint32_t place) {
                if constexpr (kSplit) seg.keys(a)[(r * seg.count + blockIdx.y) * a.top + place] = key - first;
                else writeTop(a, r, res, key, place);
            });
        }
        __syncthreads();
    }
}

// The segments of a row joined: their statistics, and the best of their tops,
// where a key's place is its own in its segment's plus, by bisection, the
// number of larger ones in the others'.
constexpr int kJoinBlock = 256;
template <typename T, bool kTeacher>
__global__ __launch_bounds__(kJoinBlock) void logitsJoinKernel(LogitsForward a, Segments seg) {
    __shared__ uint64_t keys[kMaxSegments * BFO_TOP_MAX];
    const uint64_t r = blockIdx.x;
    const float k = a.scale * kLog2e;
    RowEnd<T, kTeacher> end;
    end.load(a, r, static_cast<const T *>(a.logits.p) + r * a.logits.stride);
    const uint32_t count = seg.count * a.top;
    for (uint32_t i = threadIdx.x; i < count; i += kJoinBlock) keys[i] = seg.keys(a)[r * count + i];
    const uint32_t lane = threadIdx.x & 63;
    const float4 part = lane < seg.count ? seg.stats(a)[r * seg.count + lane] : float4{kLowest, 0.0f, 0.0f, 0.0f};
    // finished statistics: M is m k exactly
    Stat all = {waveMax(part.x), 0.0f, 0.0f};
    const float d = all.m - part.x, up = d < INFINITY ? differenceTimesK(all.m, part.x, k, a.scale)
                                                      : scaledDifference(all.m, part.x, a.difference) * kLog2e;
    const Stat mine = raised({part.x, part.y, part.z}, all.m, up);
    all.s = laneSum<64>(mine.s);
    all.t = laneSum<64>(mine.t);
    const RowResult res = rowResult(all, a.scale);
    end.write(a, r, res, a.entropy != nullptr, kJoinBlock - 64);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < count; i += kJoinBlock) {
        const uint64_t key = keys[i];
        const uint32_t own = i / a.top;
        uint32_t place = i % a.top;
        for (uint32_t s = 0; s < seg.count; ++s) {
            uint32_t low = 0, high = s == own ? 0 : a.top;
            while (low < high) {
                const uint32_t mid = (low + high) / 2;
                if (keys[s * a.top + mid] > key) low = mid + 1;
                else high = mid;
            }
            place += low;
        }
        if (place < a.top) writeTop(a, r, res, key, place);
    }
}

// ---------------------------------------------------------------------------
// Backward: a workgroup owns a segment of a row's columns.
// ---------------------------------------------------------------------------
constexpr int kBackBlock = 256;
constexpr int kBackChunks = 4;  // 16-byte chunks per lane
template <typename T>
constexpr uint32_t backSegment() {
    return kBackBlock * kBackChunks * chunkElems<T>();
}

// Teacher entries inside the segment, chained per 16-byte chunk: head[chunk]
// is the first one there, next[entry] the following one, in the entries'
// order, so that equal indexes add in a fixed order.
struct Chains {
    static constexpr uint32_t kNone = 0xFF;
    alignas(4) uint8_t head[kBackBlock * kBackChunks];
    uint8_t next[BFO_TOP_MAX];
    uint32_t column[BFO_TOP_MAX];  // within the segment
    float value[BFO_TOP_MAX];
    float base;
};
static_assert(BFO_TOP_MAX <= 128, "a lane of one wavefront holds two entries");

// One wavefront: writes the chains of the entries with columns in [c0, c1),
// each with its part of the gradient, and the part of the row's `base`.
__device__ __forceinline__ void buildChains(Chains &ch, const Teacher &te, float dkl, uint32_t vocab, int c0, int c1,
                                            uint32_t perChunk) {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t below = (1ull << lane) - 1;
    const bool bad = __ballot((te.id[0] >= 0 && uint32_t(te.id[0]) >= vocab) ||
                              (te.id[1] >= 0 && uint32_t(te.id[1]) >= vocab)) != 0;
    // (without a probability, dkl counts as 0 whatever it is)
    const bool in0 = te.any && te.id[0] >= 0 && te.id[0] >= c0 && te.id[0] < c1;
    const bool in1 = te.any && te.id[1] >= 0 && te.id[1] >= c0 && te.id[1] < c1;
    const uint64_t m0 = __ballot(in0), m1 = __ballot(in1);
    const uint32_t n0 = uint32_t(__popcll(m0)), n = n0 + uint32_t(__popcll(m1));
    if (in0) {
        const uint32_t at = uint32_t(__popcll(m0 & below));
        ch.column[at] = uint32_t(te.id[0] - c0);
        ch.value[at] = -dkl * te.q[0];
    }
    if (in1) {
        const uint32_t at = n0 + uint32_t(__popcll(m1 & below));
        ch.column[at] = uint32_t(te.id[1] - c0);
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

// Segments run along x, rows along y.  Segments are cut on 128-byte lines of
// the output, which is written in whole lines but for the row's ends.
template <typename T, bool kEntropy, bool kTeacher>
__global__ __launch_bounds__(kBackBlock) void logitsBackwardKernel(LogitsBackward a, uint32_t segment) {
    constexpr int E = int(chunkElems<T>());
    __shared__ std::conditional_t<kTeacher, Chains, Empty> ch;
    const int V = int(a.vocab);
    for (uint64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const T *row = static_cast<const T *>(a.logits.p) + r * a.logits.stride;
        T *out = static_cast<T *>(a.dlogits.p) + r * a.dlogits.stride;
        // the segment's columns are those of [c0, end) that are not negative
        const int c0 = int(blockIdx.x * segment) - leadOf(out), end = min(c0 + int(segment), int(a.width));
        const float m = a.stats[2 * r], logs2 = a.stats[2 * r + 1] * kLog2e;
        // dlogits = scale * (p * (base + slope * log2 p) + what its tokens get)
        int target = -1;
        float hard = 0.0f, base = 0.0f, slope = 0.0f, dkl = 0.0f;
        if (a.targets) {
            target = a.targets[r];
            if (target >= 0) {
                hard = a.dlogprob[r];
                base = target >= V ? NAN : -hard;
            }
        }
        if constexpr (kEntropy) {
            const float de = a.dentropy[r];
            slope = -de * kLn2;
            if (de != 0.0f) base -= de * a.entropy[r];
        }
        if constexpr (kTeacher) dkl = a.dkl[r];
        bool live = m != -INFINITY && !(hard == 0.0f && base == 0.0f && slope == 0.0f && dkl == 0.0f);
        const int lane = int(threadIdx.x) * E;
        Chunk<T, E> v[kBackChunks];
        if (live) {
#pragma unroll
            for (int k = 0; k < kBackChunks; ++k) {
                const int at = c0 + kBackBlock * E * k;
                v[k].loadScores(row + at, lane, -at, min(V, end) - at);
            }
        }
        if constexpr (kTeacher) {
            if (live) {
                for (uint32_t i = threadIdx.x; i < sizeof(ch.head) / 4; i += kBackBlock)
                    reinterpret_cast<uint32_t *>(ch.head)[i] = 0xFFFFFFFFu;
                Teacher te;
                if (threadIdx.x < 64) {
                    te.load(a.teacherIndex + r * a.count, a.teacherLogits + r * a.count, a.count);
                    te.softmax(a.difference);
                }
                __syncthreads();
                if (threadIdx.x < 64) buildChains(ch, te, dkl, uint32_t(V), c0, end, E);
                __syncthreads();
                base += ch.base;
                live = !(hard == 0.0f && base == 0.0f && ch.base == 0.0f);
            }
        }
#pragma unroll
        for (int k = 0; k < kBackChunks; ++k) {
            const int at = c0 + kBackBlock * E * k, c = at + lane;
            float y[E];
            if (live) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    // z is rounded before m, itself a rounded z, is taken from it:
                    // the largest z leaves 0, however large.  Columns outside the
                    // vocabulary hold -inf, so p = 0 there.
                    const float z = v[k][e] * a.scale, lp = fmaf(z - m, kLog2e, -logs2);  // log2 p
                    const float p = exp2Fast(lp);
                    // p is 0 well above -1e4, where the product has to be 0 too
                    y[e] = p * (kEntropy ? fmaf(slope, fmaxf(lp, -1e4f), base) : base);
                }
                if constexpr (kTeacher) {
                    if (c < end) {
                        uint32_t h = ch.head[(c - c0) / E];
                        while (h != Chains::kNone) {
                            const int col = int(ch.column[h]) + c0 - c;
                            const float val = ch.value[h];
#pragma unroll
                            for (int e = 0; e < E; ++e) y[e] += col == e ? val : 0.0f;
                            h = ch.next[h];
                        }
                    }
                }
                if (target >= c && target < c + E) {
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] += target - c == e ? hard : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] *= a.scale;
                if (c + E > V) {
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = c + e < V ? y[e] : 0.0f;
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = 0.0f;
            }
            storeRow(out + at, lane, -at, end - at, y);
        }
        if constexpr (kTeacher) __syncthreads();
    }
}

// Few rows of many scores are split, to at most one workgroup a CU and at least
// 16,384 scores a segment; one workgroup reads its row at little more than 20
// GB/s.  One row of 262,144 bf16 scores 15.3 -> 5.6 us, with entropy and 20
// alternatives 22.8 -> 13.0; so 64 rows of 131,072 16.5 -> 14.7.  At 50,257
// scores the second launch costs what the split gains (9.3 -> 10.3), and above 8
// segments joining their tops costs more again (20 us with 16).  A last segment
// still holds more than BFO_TOP_MAX scores.
constexpr uint32_t kSplitRows = 128, kSplitVocab = 65536, kSplitBlocks = 256;
uint32_t mostSegments(uint32_t vocab) {
    if (vocab < kSplitVocab) return 1;
    return vocab / 16384 < kMaxSegments ? vocab / 16384 : kMaxSegments;
}
Segments segmentsOf(uint64_t rows, uint32_t vocab) {
    uint32_t n = rows > kSplitRows ? 1 : mostSegments(vocab);
    if (n * rows > kSplitBlocks) n = uint32_t(kSplitBlocks / rows);
    if (n < 2) return {1, vocab};
    const uint32_t length = ((vocab + n - 1) / n + 63) / 64 * 64;
    return {(vocab + length - 1) / length, length};
}

template <typename T, int kBlock, bool kNontemporal, bool kEntropy, bool kTop, bool kTeacher, bool kSplit>
void forwardOf(const LogitsForward &a, Segments seg, hipStream_t stream) {
    // A lane's chunks, in whole steps, in at most kSlots stretches.
    constexpr uint32_t step = kBlock * chunkElems<T>() * kUnroll;
    const uint32_t perSlot = ((seg.length + kMaxLead<T> + step - 1) / step * kUnroll + kSlots - 1) / kSlots;
    const dim3 grid(uint32_t(a.rows < kMaxGrid ? a.rows : kMaxGrid), seg.count);
    hipLaunchKernelGGL((logitsForwardKernel<T, kBlock, kNontemporal, kEntropy, kTop, kTeacher, kSplit>), grid,
                       dim3(kBlock), 0, stream, a, perSlot, seg);
}

template <typename T, int kBlock, bool kNontemporal, bool kSplit>
hipError_t forwardKind(const LogitsForward &a, Segments seg, hipStream_t stream) {
    if (a.count && !kSplit) forwardOf<T, kBlock, kNontemporal, false, false, !kSplit, kSplit>(a, seg, stream);
    else if (a.entropy && a.top) forwardOf<T, kBlock, kNontemporal, true, true, false, kSplit>(a, seg, stream);
    else if (a.entropy) forwardOf<T, kBlock, kNontemporal, true, false, false, kSplit>(a, seg, stream);
    else if (a.top) forwardOf<T, kBlock, kNontemporal, false, true, false, kSplit>(a, seg, stream);
    else forwardOf<T, kBlock, kNontemporal, false, false, false, kSplit>(a, seg, stream);
    if constexpr (kSplit) {
        const dim3 grid(uint32_t(a.rows)), block(kJoinBlock);
        if (a.count) hipLaunchKernelGGL((logitsJoinKernel<T, true>), grid, block, 0, stream, a, seg);
        else hipLaunchKernelGGL((logitsJoinKernel<T, false>), grid, block, 0, stream, a, seg);
    }
    return hipGetLastError();
}

// Where every CU has a few rows, small workgroups let the ends of some rows hide
// behind the passes of others: 8192 x 50257 bf16 with 20 alternatives 151 us
// with 256 lanes, 186 with 512, without 125 and 134.  With few rows a row's own
// pass counts: 64 x 50257 with 20 alternatives 13.0 us with 256 lanes, 10.6 with
// 512, one row 12.3 and 9.9; 512 x 32000 13.7 and 13.8.  Scores of over 64 MB are
// loaded nontemporally: 8192 x 50257 bf16 141 -> 125 us, fp32 4096 x 50257 138 ->
// 121, 2048 x 32000 bf16 25.5 -> 23.0; below that it gave nothing, and took up to
// 4% where the caches still held them.
template <typename T>
hipError_t forward(const LogitsForward &a, hipStream_t stream) {
    const Segments seg = segmentsOf(a.rows, a.vocab);
    if (seg.count > 1) return forwardKind<T, 512, false, true>(a, seg, stream);
    if (a.rows <= 512) return forwardKind<T, 512, false, false>(a, seg, stream);
    if (a.rows * a.vocab * sizeof(T) <= (uint64_t(64) << 20)) return forwardKind<T, 256, false, false>(a, seg, stream);
    return forwardKind<T, 256, true, false>(a, seg, stream);
}

template <typename T>
hipError_t backward(const LogitsBackward &a, hipStream_t stream) {
    constexpr uint32_t line = 128 / sizeof(T);
    const uint32_t columns = a.width + kMaxLead<T>;
    // Even segments of whole lines.
    const uint32_t segments = (columns + backSegment<T>() - 1) / backSegment<T>();
    const uint32_t segment = ((columns + segments - 1) / segments + line - 1) / line * line;
    const dim3 grid((columns + segment - 1) / segment, uint32_t(a.rows < 65535 ? a.rows : 65535)), block(kBackBlock);
    if (a.count) hipLaunchKernelGGL((logitsBackwardKernel<T, false, true>), grid, block, 0, stream, a, segment);
    else if (a.dentropy) hipLaunchKernelGGL((logitsBackwardKernel<T, true, false>), grid, block, 0, stream, a, segment);
    else hipLaunchKernelGGL((logitsBackwardKernel<T, false, false>), grid, block, 0, stream, a, segment);
    return hipGetLastError();
}

}  // namespace

constexpr uint64_t segmentBytes(uint32_t top) { return sizeof(float4) + top * sizeof(uint64_t); }

uint64_t logitsWorkspaceBytes(uint64_t rows, uint32_t vocab, uint32_t top) {
    const Segments seg = segmentsOf(rows, vocab);
    return seg.count > 1 ? rows * seg.count * segmentBytes(top) : 0;
}

// More rows than are split still cover fewer that are.
uint64_t logitsWorkspaceBound(uint64_t rows, uint32_t vocab, uint32_t top) {
    if (vocab < kSplitVocab) return 0;
    const uint64_t segments = rows * mostSegments(vocab);
    return (segments < kSplitBlocks ? segments : kSplitBlocks) * segmentBytes(top);
}

hipError_t launchLogitsForward(const LogitsForward &a, int dtype, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return dtype == BFO_BF16 ? forward<bf16_t>(a, stream) : forward<float>(a, stream);
}

hipError_t launchLogitsBackward(const LogitsBackward &a, int dtype, hipStream_t stream) {
    if (!a.rows) return hipSuccess;
    return dtype == BFO_BF16 ? backward<bf16_t>(a, stream) : backward<float>(a, stream);
}

}  // namespace bfo
