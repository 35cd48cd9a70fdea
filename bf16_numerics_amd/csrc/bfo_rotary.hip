// bfo_rotary.hip -- gfx950 kernel of rotary positions.
//
// Pair i of a head at position p is turned by the angle p * frequency[i]:
//   (a, b) -> amplitude * (a cos - b sin, a sin + b cos),
// backward by the negative angle, which is the transpose.  Angles are formed
// and reduced to a turn in 64 bits, so that far positions keep them; sines and
// cosines are those of the turn's rest in 32 bits, moved by what its rounding left
// (which is up to 2^-26 of a turn, all of a sine near half a turn).
//
// Bound by memory: every column is read and written once, and the sines are
// shared by a token's heads.  A workgroup takes a token's heads, two 16-byte
// chunks a lane (or several tokens of few heads, or a part of a token of many):
// its lanes first ask for the angles' parts, then for their chunks, and form the
// sines into LDS while those are on their way.  8192 tokens of 64 heads of 128
// bf16 columns: 43.8 us in halves and interleaved, 6.1 TB/s, where a copy of the
// same bytes takes 50.2; a quarter of the columns rotated, in place 17.3, else 56.6.
// Of the larger steps there: a wavefront a token, walking over its heads with the
// sines in its own LDS, 62 us (interleaved 67); four chunks in flight, 54 (56); a
// workgroup a token, 48 (51); angles asked for first, 46; nontemporal, 43.8.
// Workgroups of 256 lanes 47.4, of 1,024 49.9.
#include <type_traits>

#include "bfo_device.hpp"
#include "bfo_ops.hpp"

namespace bfo {
namespace {

constexpr int kBlock = 512;
static_assert(kBlock >= 130, "a head's items fit a workgroup");
constexpr double kRadians = 6.283185307179586476925, kTurn = 1.0 / kRadians;  // of a turn

// What a lane takes at a time: two 16-byte chunks of a head, at column `first` of
// the first half of its rotated columns and at the same of the second one, or so
// of the columns behind them, which are copied.  In halves the two chunks hold the
// members of the same pairs; interleaved, each holds pairs of its own, and where
// their number is odd the halves share the middle one.  (Interleaved, two
// neighbouring chunks a lane leave every store instruction half of each line: 47.2
// us, 53.9 nontemporal.)  A head has at most 130 such items, which fit a workgroup.
// kWhole: the last item of a half starts so much earlier that it ends with it;
// otherwise, for halves of less than a chunk, it ends inside.  What two items share
// is the same in both, and read before either writes.
template <typename T, bool kHalf, bool kWhole, bool kStream>
struct Item {
    static constexpr int E = 16 / int(sizeof(T));
    Chunk<T, E> u, v;

    // A chunk at column c of a head, of which `there` columns are there.
    __device__ __forceinline__ static void get(Chunk<T, E> &w, const T *head, int c, int there) {
        if constexpr (kWhole) w.template load<kStream>(head + c);
        else w.loadRow(head, c, there);
    }
    __device__ __forceinline__ static void put(Chunk<T, E> w, T *head, int c, int there) {
        if constexpr (kStream) w.forget();
        if constexpr (kWhole) w.template store<kStream>(head + c);
        else w.storeRow(head, c, there);
    }
    __device__ __forceinline__ void load(const T *head, int first, int half, int second) {
        get(u, head, first, half);
        get(v, head + second, first, half);
    }
    __device__ __forceinline__ void store(T *head, int first, int half, int second) const {
        put(u, head, first, half);
        put(v, head + second, first, half);
    }
    // The pairs turned, stored.
    __device__ __forceinline__ void turn(const float2 *turns, T *head, int first, int half, int second) const {
        float y[E], z[E];
        if constexpr (kHalf) {
#pragma unroll
            for (int e = 0; e < E; ++e) turnPair(u[e], v[e], turns[first + e], y[e], z[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                turnPair(u[e], u[e + 1], turns[(first + e) / 2], y[e], y[e + 1]);
                turnPair(v[e], v[e + 1], turns[(second + first + e) / 2], z[e], z[e + 1]);
            }
        }
        put(Chunk<T, E>(y), head, first, half);
        put(Chunk<T, E>(z), head + second, first, half);
    }
    __device__ __forceinline__ static void turnPair(float a, float b, float2 t, float &x, float &y) {
        x = fmaf(a, t.x, -(b * t.y));
        y = fmaf(a, t.y, b * t.x);
    }
};

// The columns of each half of the rotated ones (even where pairs lie side by side)
// and of those behind.
template <bool kHalf>
__host__ __device__ uint32_t halfColumns(uint32_t rotated) {
    return kHalf ? rotated / 2 : (rotated / 2 + 1) / 2 * 2;
}
__host__ __device__ inline uint32_t halfBehind(uint32_t behind) { return (behind + 1) / 2; }

// Pairs of a workgroup's tokens at most.  A token's sines take room for a multiple of
// eight pairs: 16 KB of LDS in all where there are as many, and up to 32 KB (512 tokens
// of one to four pairs), of which a CU holds five and its lanes four.
constexpr uint32_t kTurns = 2048;

// kBehind: columns behind the rotated ones are copied.
template <typename T, bool kHalf, bool kWhole, bool kBehind, bool kStream>
__global__ __launch_bounds__(kBlock) void rotaryKernel(Rotary a) {
    constexpr uint32_t E = 16 / sizeof(T);
    extern __shared__ float2 table[];  // every token's cosines and sines
    const uint32_t pairs = a.rotated / 2, room = (pairs + 7) / 8 * 8;
    const uint32_t half = halfColumns<kHalf>(a.rotated), second = a.rotated - half, turning = (half + E - 1) / E;
    // What the angle of a workgroup's pair i is made of, and its cosine and sine.
    struct Angle {
        uint32_t token, pair;
        int32_t position;
        double frequency;
    };
    auto load = [&](uint64_t firstToken, uint32_t i) -> Angle {
        const uint32_t t = a.pairsPerToken.divide(i), pair = i - t * pairs;
        return {t, pair, a.positions ? a.positions[firstToken + t] : 0, a.frequencies[pair]};
    };
    auto put = [&](uint64_t firstToken, const Angle &angle) {
        const uint64_t n = firstToken + angle.token;
        const double position = a.positions ? double(angle.position) : double(a.period ? n % a.period : n);
        double turn = position * angle.frequency * kTurn;
        turn -= rint(turn);
        const float rest = float(turn), left = float((turn - double(rest)) * kRadians);
        float s, c;
        sincospif(2.0f * rest, &s, &c);
        const float sine = fmaf(c, left, s), cosine = fmaf(-s, left, c);
        table[angle.token * room + angle.pair] = {cosine * a.amplitude, (a.backward ? -sine : sine) * a.amplitude};
    };
    for (uint32_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        const uint32_t block = a.headBlocks.divide(unit);
        const uint32_t firstHead = (unit - block * a.headBlocks.by) * a.headsAtOnce.by;
        const uint64_t firstToken = uint64_t(block) * a.tokensAtOnce;
        const uint32_t tokens = uint32_t(min(uint64_t(a.tokensAtOnce), a.tokens - firstToken));
        // The angle's parts first, so that no lane waits for its item before it forms the sine.
        const uint32_t angles = tokens * pairs;
        const Angle angle = load(firstToken, min(threadIdx.x, angles - 1));
        const T *x = static_cast<const T *>(a.x) + firstToken * a.xToken + firstHead * a.xHead;
        T *out = static_cast<T *>(a.out) + firstToken * a.outToken + firstHead * a.outHead;
        const uint32_t row = a.itemsPerHead.divide(threadIdx.x), k = threadIdx.x - row * a.itemsPerHead.by;
        const uint32_t token = a.headsAtOnce.divide(row), head = row - token * a.headsAtOnce.by;
        const bool live = token < tokens && firstHead + head < a.heads;
        const T *from = x + token * a.xToken + head * a.xHead;
        Item<T, kHalf, kWhole, kStream> item;
        // The columns that the item is of, their halves, and its first column in them.
        const bool turns = !kBehind || k < turning;
        const uint32_t start = turns ? 0 : a.rotated, of = turns ? half : halfBehind(a.headDim - a.rotated);
        const uint32_t other = turns ? second : a.headDim - a.rotated - of;
        int at = int((turns ? k : k - turning) * E);
        if constexpr (kWhole) at = min(at, int(of - E));
        if (live) item.load(from + start, at, int(of), int(other));
        if (threadIdx.x < angles) put(firstToken, angle);
        for (uint32_t i = threadIdx.x + kBlock; i < angles; i += kBlock) put(firstToken, load(firstToken, i));
        __syncthreads();
        T *to = out + token * a.outToken + head * a.outHead;
        if (live && turns) item.turn(table + token * room, to, at, int(half), int(second));
        else if (kBehind && live) item.store(to + start, at, int(of), int(other));
        if (unit + gridDim.x < a.units) __syncthreads();
    }
}

template <typename T, bool kHalf>
void launch(Rotary a, hipStream_t stream) {
    constexpr uint32_t E = 16 / sizeof(T);
    const uint32_t pairs = a.rotated / 2, half = halfColumns<kHalf>(a.rotated), turning = (half + E - 1) / E;
    const uint32_t behind = a.x == a.out ? 0 : a.headDim - a.rotated, copied = halfBehind(behind);
    const uint32_t per = turning + (copied + E - 1) / E;
    // A workgroup's tokens and heads: as many as its lanes have items for, the heads of a
    // token in blocks of like size.
    const uint32_t fit = kBlock / per;
    const uint32_t blocks = (a.heads + fit - 1) / fit, heads = (a.heads + blocks - 1) / blocks;
    uint32_t tokens = fit / heads;
    if (tokens > kTurns / pairs) tokens = kTurns / pairs;
    if (tokens > a.tokens) tokens = uint32_t(a.tokens);
    if (tokens < 1) tokens = 1;
    a.itemsPerHead = FastDivide(per);
    a.headsAtOnce = FastDivide(heads);
    a.headBlocks = FastDivide(blocks);
    a.pairsPerToken = FastDivide(pairs);
    a.tokensAtOnce = tokens;
    a.units = uint32_t((a.tokens + tokens - 1) / tokens * blocks);
    const uint32_t lds = tokens * ((pairs + 7) / 8 * 8) * sizeof(float2);
    const dim3 grid(a.units < (1u << 22) ? a.units : 1u << 22);
    auto with = [&](auto whole, auto behind, auto streamed) {
        hipLaunchKernelGGL((rotaryKernel<T, kHalf, decltype(whole)::value, decltype(behind)::value,
                                         decltype(streamed)::value>),
                           grid, dim3(kBlock), lds, stream, a);
    };
    const bool streamed = streams(2 * sizeof(T) * a.tokens * a.heads * (a.rotated + behind));
    constexpr std::true_type yes;
    constexpr std::false_type no;
    // Heads with columns behind are stored in pieces of lines, which nontemporal stores
    // write one by one: 8192 x 64 x 128, a quarter rotated, 56.6 us against 71.
    if (half < E || (behind && copied < E)) with(no, yes, no);
    else if (behind) with(yes, yes, no);
    else streamed ? with(yes, no, yes) : with(yes, no, no);
}

}  // namespace

hipError_t launchRotary(const Rotary &a, int dtype, int layout, hipStream_t stream) {
    if (!a.tokens || !a.heads) return hipSuccess;
    const bool half = layout == BFO_ROTARY_HALF;
    if (dtype == BFO_BF16) half ? launch<bf16_t, true>(a, stream) : launch<bf16_t, false>(a, stream);
    else half ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
    return hipGetLastError();
}

}  // namespace bfo
