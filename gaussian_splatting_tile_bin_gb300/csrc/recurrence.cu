// recurrence.cu -- a gated linear recurrence over the tokens of each item, channel
// by channel, forward and backward.
//
//   a_t = sigmoid(f_t),  h_t = a_t h_(t-1) + (1 - a_t) x_t,  out_t = h_t silu(o_t)
// and with dh_t = dout_t silu(o_t) + a_(t+1) dh_(t+1)
//   dx = dh (1 - a),  df = dh (h_(t-1) - x) a (1 - a),  do = dout h silu'(o).
//
// Bound by HBM.  A block takes a tile of tokens by 32 lanes of channels (128 bytes a
// token), each of its working warps a run of tokens, whose gates stay in registers: a
// run's effect on the state before it is affine, h -> A h + H, and so is a tile's and a
// chain of tiles'.  The tile reads its inputs once, composes its (A, H), takes the state
// in front of it from the tiles before, and runs its tokens from that state.  The
// backward does the same from the end with p_t = a_t dh_t, for which p -> A p + P, and
// computes h again from the forward's states.
//
// The chain.  Tiles are taken from a ticket in the chain's order, so a tile waits only
// for tiles that blocks work on or are done with.  Each publishes its (A, H), the last of
// a group the group's, and again, as a map of no state, once it knows the state behind it.
// A tile folds its group's maps, and takes the state in front of the group from the latest
// group whose state is known and the maps of those behind that: always map by map, so
// that the bits are the same wherever it starts, and results are on every run.  A map is
// one 64-bit word, which is all ones before it is published (no map is: A is never that
// NaN).
//
// A block's warps.  Eight work on runs.  One takes tickets and starts the tiles' copies
// into a ring of stages.  Two follow the chain.  One composes the runs' maps, publishes
// the tile's and hands each run the map of those in front of it.  A working warp composes
// its run of the next tile before it finishes the one of the last: its gates and inputs
// wait in tensor memory (256 columns a block) meanwhile, so that the time that a map takes
// along the chain is spent on work.  The forward's output gates, which only a run's end uses,
// wait in shared memory, where a second ring of copies puts them.
//
// What bounds it, and what the parts are worth (32,640 x 2,048 in bf16 with a gate: four
// arrays of 134 MB forward, 79 us at the copy rate, and seven backward, 138 us): 90 and 168
// us, each byte moved once.  Without any wait along the chain kernels that took 95 and 168 us
// would have taken 86 and 145, bound by HBM; the rest is what a map and a state take through
// L2.  Tiles without a ring and a chain of their own took 170 and 323 us, with them 136 and 299,
// with runs that wait in tensor memory 115 and 213; a chain whose missing words are looked at
// together 102 and 188, and groups that publish their map before their state 95 and 168; the
// forward's runs that keep a and (1 - a) x, and read their gates from shared memory, 90.
//
// Numerics.  With e = exp(-|f|), the smaller of a and 1 - a is e / (1 + e), and the larger 1
// minus it, at least 1/2: both are good to a few ulp of themselves, however far apart they are.
// A step is a h + (1 - a) x with both, wherever it is taken, so that what a gate shuts out
// leaves the rest its bits.  States, maps and gradients along the chain are floats; results
// are rounded once.  exp and reciprocal are the hardware's (2 ulp).
#include <initializer_list>
#include <type_traits>

#include "tensor.cuh"

namespace gsr {
namespace {

constexpr int kWarps = 8;                  // that work on runs
constexpr int kComposeWarp = kWarps, kFetchWarp = kWarps + 1, kChainWarp = kWarps + 2;   // two of the last
constexpr int kThreads = 32 * (kWarps + 4);
constexpr int kBlocks = 2;                 // of an SM
// Registers of a thread: the start's, and after the warps beside the runs have given
// theirs to the others.
constexpr int kStart = 80, kFew = 48, kMany = 96;
static_assert(kWarps == 8 && 4 * kFew + 8 * kMany <= 12 * kStart, "the shares must fit what a block starts with");
constexpr int kGroup = 8;                  // tiles of a group
// Groups that a tile looks back on.  Where many chains share the SMs a few of a chain's
// tiles are under way, and words that are looked at cost time (32,640 x 2,048 in bf16,
// backward: 168 us with 2, 174 to 223 with 3 to 8); where there are few chains most of
// their tiles are, and a state travels by as many groups at a time (32,640 x 64: 20.8 us
// with 2, 14.9 with 8).  The two meet at 4 chains: 25.1 and 23.4 us at 3, 32.1 and 32.5 at
// 4, 36.5 and 37.8 at 5, 53.2 and 55.7 at 8, 92 and 99 at 16; in f32 21.1 and 16.2 at 2,
// 28.9 and 28.4 at 4, 47.9 and 48.7 at 8.
constexpr int kNear = 2, kFar = 8, kManyChains = 4;
constexpr int kColumns = 256, kSlotColumns = kColumns / 2;   // of tensor memory: two tiles' runs
constexpr int kRun = 16, kGradRun = 8;     // tokens of a warp
constexpr int kTile = kWarps * kRun, kGradTile = kWarps * kGradRun;
constexpr int kStages = 2;
constexpr int kRowBytes = 128;             // of a token in a stage
// Up to so many tokens a thread runs them alone.
constexpr int kFewTokens = 16, kFewAhead = 4, kFewThreads = 64;
constexpr int kStateStep = GSR_RECURRENCE_BLOCK;
static_assert(kStateStep % kRun == 0 && kGradTile == kStateStep, "states lie where runs and tiles start");

struct Tokens {
    void *data;
    int64_t batch, token;
};

struct RecurrenceArgs {
    Tokens x, forget, gate, out, dout, dx, dforget, dgate;
    const float *initial;        // backward: dL/dfinal
    float *final, *states;       // backward: dL/dinitial
    const int *lengths;
    int batch, tokens, channels, blocks;
    int tiles, slabs;            // of all tokens, of all channels
    uint32_t work;               // tiles of all items and channels
    int groups, far;             // of all tokens; whether a tile looks back on kFar of them
    int reverse;
    unsigned long long *pairs, *ends;   // published: [batch, slabs, tiles] and [batch, slabs, groups] rows of words
    uint32_t *ticket;            // all ones before the first
    uint32_t *aborted;           // 0 once a wait has run out
    uint32_t *status;
};

// ---- channels --------------------------------------------------------------------------

// A thread's channels: one or a pair, whose arithmetic is one instruction for both.
template <int V>
using Lanes = std::conditional_t<V == 2, float2, float>;

__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return mul2(a, b); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float mad(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 mad(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float minus(float a) { return -a; }
__device__ __forceinline__ float2 minus(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ void fill(float &v, float x) { v = x; }
__device__ __forceinline__ void fill(float2 &v, float x) { v = make_float2(x, x); }
__device__ __forceinline__ float &at(float &v, int) { return v; }
__device__ __forceinline__ float &at(float2 &v, int j) { return j ? v.y : v.x; }
__device__ __forceinline__ float at(const float &v, int) { return v; }
__device__ __forceinline__ float at(const float2 &v, int j) { return j ? v.y : v.x; }

// Bits of a thread's elements of one token: a float, a pair of 16 bits, or one.
template <typename T, int V>
using Raw = std::conditional_t<sizeof(T) * V == 4, uint32_t, uint16_t>;

template <typename T, int V>
__device__ __forceinline__ Lanes<V> value_of(const Raw<T, V> &r)
{
    if constexpr (V == 1) {
        return to_float(*(const T *)&r);
    } else if constexpr (std::is_same_v<T, __half>) {
        return __half22float2(*(const __half2 *)&r);
    } else {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_of(Lanes<V> v)
{
    if constexpr (V == 1) {
        const T t = from_float<T>(v);
        return *(const Raw<T, V> *)&t;
    } else {
        return pack2<T>(v.x, v.y);
    }
}

__device__ __forceinline__ void clear(uint32_t &r) { r = 0; }
__device__ __forceinline__ void clear(uint16_t &r) { r = 0; }

// state -> a state + h
template <int V>
struct Map {
    Lanes<V> a, h;
};

template <int V>
__device__ __forceinline__ Map<V> then(const Map<V> &first, const Map<V> &second)
{
    return {mul(second.a, first.a), mad(second.a, first.h, second.h)};
}

// A map of one channel as a word.
__device__ __forceinline__ unsigned long long word_of(const Map<1> &m)
{
    return (unsigned long long)__float_as_uint(m.h) << 32 | __float_as_uint(m.a);
}
__device__ __forceinline__ Map<1> map_of(unsigned long long w)
{
    return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
constexpr unsigned long long kNoMap = ~0ull;
// The A of a known state, which takes none before it: -0, which no product of gates is.  (A
// product that comes out as 0 still takes its state: one that is not a number stays so.)
constexpr float kNoState = -0.0f;
__device__ __forceinline__ bool is_state(unsigned long long w) { return (uint32_t)w == 0x80000000u; }

// ---- the chain ---------------------------------------------------------------------------

__device__ __forceinline__ void publish(unsigned long long *to, unsigned long long w)
{
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(to), "l"(w) : "memory");
}
__device__ __forceinline__ void look(const unsigned long long *at, unsigned long long &w)
{
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w) : "l"(at) : "memory");
}
// A lane's words of `count` rows, and a wait until they are enough for every lane: looked
// at together until then, those that are missing or (known_only) no map of a known state,
// or until the wait has run out (here or elsewhere).
template <int N>
__device__ __forceinline__ void look(const unsigned long long *at, int stride, int count, unsigned long long (&v)[N])
{
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = kNoMap;
        if (k < count) look(at + k * stride, v[k]);
    }
}

template <int N, typename F>
__device__ __forceinline__ void wait_for(const RecurrenceArgs &a, const unsigned long long *at, int stride, int count,
                                         unsigned long long (&v)[N], bool known_only, F enough)
{
    const long long start = clock64();
    for (int turn = 1;; ++turn) {
        if (__all_sync(~0u, enough())) return;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < count && (known_only ? !is_state(v[k]) : v[k] == kNoMap)) look(at + k * stride, v[k]);
        if (turn % 64 != 0) continue;
        bool stop = *(volatile uint32_t *)a.aborted == 0;
        if (clock64() - start > kWaitCycles) {
            *(volatile uint32_t *)a.aborted = 0;
            *(volatile uint32_t *)a.status = 1;
            stop = true;
        }
        if (__any_sync(~0u, stop)) return;
    }
}

struct Tile {
    int b, slab, index;    // item, channel slab, place along the tokens
    int length, count;     // the item's tokens and tiles
};

// The n-th tile in the order of the chains.
template <bool BACKWARD>
__device__ __forceinline__ Tile tile_at(const RecurrenceArgs &a, uint32_t n)
{
    constexpr int kTokens = BACKWARD ? kGradTile : kTile;
    Tile t;
    const uint32_t chains = (uint32_t)a.batch * a.slabs, place = n / chains, chain = n - place * chains;
    t.b = chain / a.slabs;
    t.slab = chain - t.b * a.slabs;
    t.index = BACKWARD ? a.tiles - 1 - (int)place : (int)place;
    t.length = a.lengths ? min(max(a.lengths[t.b], 0), a.tokens) : a.tokens;
    t.count = (t.length + kTokens - 1) / kTokens;
    return t;
}

// A tile's place in its chain, which the backward starts at the last token; below 0, or
// no less than t.count, for tiles behind an item's tokens.
template <bool BACKWARD>
__device__ __forceinline__ int place_of(const Tile &t)
{
    return BACKWARD ? t.count - 1 - t.index : t.index;
}

template <int V>
__device__ __forceinline__ void store_state(float *to, const Lanes<V> &v)
{
#pragma unroll
    for (int j = 0; j < V; ++j) to[j] = at(v, j);
}

// What a block's warps share.  A tile's part is its number's, modulo 2 or 4: what one
// warp writes for a tile, others have read of the one that used the same place before
// they let the writer go on.
template <int V, int S, bool BACKWARD>
struct Shared {
    Map<V> runs[2][kWarps][32];         // the runs' maps, then in their place those of the runs in front of each
    Map<V> tile[4][32];                 // the tile's
    Lanes<V> carry[4][32];              // the state in front of the tile
    // Backward: H of the runs' forward maps, then h in front of each; x (its elements' bits).
    Lanes<V> h[BACKWARD ? 2 : 1][BACKWARD ? kWarps : 1][32];
    uint32_t x[BACKWARD ? 2 : 1][BACKWARD ? kWarps : 1][BACKWARD ? kGradRun : 1][32];
    Tile tiles[S];
    uint32_t last[S];                   // no tile: the tickets are at an end
    uint64_t known[S], full[S], empty[S];
    uint64_t gate_full[2], gate_empty[2];   // the forward's output gates
    uint64_t runs_ready[2], tile_ready[2], state_ready[2];
    uint32_t aborted, columns;
};

// A warp's arrival: what its lanes have written is there for who waits.
__device__ __forceinline__ void warp_arrive(uint64_t &bar)
{
    __syncwarp();
    if (threadIdx.x % 32 == 0) barrier_arrive(smem_address(&bar));
}

__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFew)); }
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMany)); }

// ---- the warps beside the runs ---------------------------------------------------------

struct Maps {
    CUtensorMap x, forget, gate, dout;
};

// Arrays of a tile that come through the stages.
template <bool GATE, bool BACKWARD>
constexpr int kStaged = BACKWARD ? 3 + (GATE ? 1 : 0) : 2;

// The first token in memory of a tile (below 0 for the last one of a reversed item, perhaps).
__device__ __forceinline__ int first_token(const RecurrenceArgs &a, const Tile &t, int tile_tokens)
{
    return a.reverse ? t.length - (t.index + 1) * tile_tokens : t.index * tile_tokens;
}

__device__ __forceinline__ void copy_tokens(uint32_t to, const CUtensorMap *map, uint32_t bar, int channel, int token, int item)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(to),
        "l"(map), "r"(bar), "r"(channel), "r"(token), "r"(item)
        : "memory");
}

// One lane: tickets in turn, and the copies of their tiles.  The forward's output gates, which
// are used when a run ends, have places of their own, and follow the next tile's inputs.
template <int V, int S, bool GATE, bool COPY, bool BACKWARD>
__device__ __forceinline__ void fetch_tiles(const RecurrenceArgs &a, const Maps &maps, Shared<V, S, BACKWARD> &s, uint32_t stages,
                                            const WaitGuard &guard)
{
    constexpr int kTokens = BACKWARD ? kGradTile : kTile, kBytes = kTokens * kRowBytes;
    constexpr int kArrays = kStaged<GATE, BACKWARD>;
    Tile gated = {};             // whose gates are to come
    uint32_t gates = 0;
    auto copy_gates = [&] {
        if (gated.index >= gated.count) return;
        const uint32_t full = smem_address(&s.gate_full[gates & 1]);
        barrier_wait(smem_address(&s.gate_empty[gates & 1]), gates >> 1 & 1 ^ 1, guard);
        GSR_CANARY(23);
        if (guard.stop()) return;
        barrier_expect(full, kBytes);
        copy_tokens(stages + (S * kArrays + (gates & 1)) * kBytes, &maps.gate, full, gated.slab * 32 * V,
                    first_token(a, gated, kTokens), a.gate.batch ? gated.b : 0);
        ++gates;
    };
    for (uint32_t i = 0;; ++i) {
        const uint32_t n = a.ticket ? atomicAdd(a.ticket, 1u) + 1u : blockIdx.x + i * gridDim.x;
        const uint32_t stage = i % S;
        barrier_wait(smem_address(&s.empty[stage]), i / S & 1 ^ 1, guard);
        const bool last = n >= a.work || guard.stop();
        Tile t = {};
        if (!last) t = tile_at<BACKWARD>(a, n);
        s.tiles[stage] = t;
        s.last[stage] = last;
        barrier_arrive(smem_address(&s.known[stage]));
        if constexpr (COPY) {
            const uint32_t full = smem_address(&s.full[stage]);
            if (t.index < t.count) {
                barrier_expect(full, kArrays * kBytes);
                uint32_t to = stages + stage * kArrays * kBytes;
                const CUtensorMap *order[4] = {&maps.forget, &maps.x, GATE ? &maps.gate : &maps.dout, &maps.dout};
                const Tokens *arrays[4] = {&a.forget, &a.x, GATE ? &a.gate : &a.dout, &a.dout};
#pragma unroll
                for (int k = 0; k < kArrays; ++k, to += kBytes)
                    copy_tokens(to, order[k], full, t.slab * 32 * V, first_token(a, t, kTokens), arrays[k]->batch ? t.b : 0);
            } else if (!last) {
                barrier_arrive(full);
            }
            if constexpr (GATE && !BACKWARD) {
                copy_gates();
                gated = t;
            }
        }
        if (last) return;
    }
}

// Whether a wait of the block has run out, as one answer for the whole warp: lanes that
// each looked for themselves might go different ways, and warp-wide instructions follow.
__device__ __forceinline__ bool warp_stop(const WaitGuard &guard) { return __any_sync(~0u, guard.stop()); }

// Calls f(tile, j) for the block's tiles in turn, j of which with tokens came before, and
// leaves their stages.  (Once a wait has run out there may be no tile where one is looked
// for.)
template <int V, int S, bool BACKWARD, typename F>
__device__ __forceinline__ void each_tile(Shared<V, S, BACKWARD> &s, const WaitGuard &guard, F f)
{
    uint32_t j = 0;
    for (uint32_t i = 0;; ++i) {
        const uint32_t stage = i % S;
        barrier_wait_warp(smem_address(&s.known[stage]), i / S & 1, guard);
        if (warp_stop(guard) || s.last[stage]) return;
        const Tile t = s.tiles[stage];
        warp_arrive(s.empty[stage]);
        f(t, j);
        if (t.index < t.count) ++j;
    }
}

// Composes the runs' maps in order, publishes the tile's, and gives each run the map of
// those in front of it.  It alone reads the state in front of a chain: once the first
// tile's map is out nobody reads that array, in which a block may write the state behind
// the chain.
template <int V, int S, bool BACKWARD>
__device__ __forceinline__ void compose_runs(const RecurrenceArgs &a, Shared<V, S, BACKWARD> &s, const Tile &t, uint32_t j,
                                             const WaitGuard &guard)
{
    const int lane = threadIdx.x % 32, c = min(t.slab * (32 * V) + lane * V, a.channels - V);
    const int place = place_of<BACKWARD>(t);
    if (t.index >= t.count) {
        if (t.length == 0 && t.index == 0 && a.final)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int64_t state = (int64_t)t.b * a.channels + c + k;
                a.final[state] = a.initial ? a.initial[state] : 0.0f;
            }
        return;
    }
    Lanes<V> seed, h;
    fill(seed, 0.0f);
    if (place == 0 && a.initial)
#pragma unroll
        for (int k = 0; k < V; ++k) at(seed, k) = a.initial[(int64_t)t.b * a.channels + c + k];
    if (BACKWARD)
#pragma unroll
        for (int k = 0; k < V; ++k) at(h, k) = a.states[((int64_t)t.b * a.blocks + t.index) * a.channels + c + k];
    barrier_wait_warp(smem_address(&s.runs_ready[j & 1]), j >> 1 & 1, guard);
    GSR_CANARY(26 + j % 4);
    if (BACKWARD)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const Lanes<V> own = s.h[j & 1][w][lane];
            s.h[j & 1][w][lane] = h;
            h = mad(s.runs[j & 1][w][lane].a, h, own);
        }
    Map<V> m;
    fill(m.a, 1.0f);
    fill(m.h, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        Map<V> &place_of_run = s.runs[j & 1][BACKWARD ? kWarps - 1 - w : w][lane];
        const Map<V> own = place_of_run;
        place_of_run = m;
        m = then(m, own);
    }
    if (place + 1 < t.count) {
        Map<V> out = m;
        if (place == 0) {   // as a map of no state
            out.h = mad(out.a, seed, out.h);
            fill(out.a, kNoState);
        }
        unsigned long long *to = a.pairs + (((int64_t)t.b * a.slabs + t.slab) * a.tiles + place) * (32 * V) + lane;
#pragma unroll
        for (int k = 0; k < V; ++k) publish(to + 32 * k, word_of({at(out.a, k), at(out.h, k)}));
    }
    if (place == 0) {
        m.h = mad(m.a, seed, m.h);   // (as published)
        fill(m.a, kNoState);
        s.carry[j & 3][lane] = seed;
    }
    s.tile[j & 3][lane] = m;
    warp_arrive(s.tile_ready[j & 1]);
    warp_arrive(s.state_ready[j & 1]);
}

// The state in front of a group: the latest of the last `count` groups' words that is a
// known state, and the maps from there on.
template <int N>
__device__ __forceinline__ float state_behind(const RecurrenceArgs &a, const unsigned long long *words, int stride, int count,
                                              unsigned long long (&seen)[N])
{
    wait_for(a, words, stride, count, seen, true, [&] {
        bool known = false;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < count) known = is_state(seen[k]) || (known && seen[k] != kNoMap);
        return known;
    });
    float state = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < count) {
            const Map<1> m = map_of(seen[k]);
            state = is_state(seen[k]) ? m.h : fmaf(m.a, state, m.h);
        }
    return state;
}

// Folds the maps that the group's tiles before this one have published, finds the state
// in front of the group, and with both the one in front of the tile; publishes the group's
// map and the state behind it.  A warp for each of a lane's channels.
template <int V, int S, bool BACKWARD>
__device__ __forceinline__ void follow_chain(const RecurrenceArgs &a, Shared<V, S, BACKWARD> &s, const Tile &t, uint32_t j,
                                             const WaitGuard &guard)
{
    constexpr int kRow = 32 * V;
    const int lane = threadIdx.x % 32, channel = threadIdx.x / 32 - kChainWarp, place = place_of<BACKWARD>(t);
    if (t.index >= t.count || channel >= V) return;
    GSR_CANARY(21);
    const int64_t row = (int64_t)t.b * a.slabs + t.slab;
    const int group = place / kGroup, count = place - group * kGroup;
    const unsigned long long *pairs = a.pairs + (row * a.tiles + group * kGroup) * kRow + channel * 32 + lane;
    unsigned long long *ends = a.ends + (row * a.groups + group) * kRow + channel * 32 + lane;
    if (place > 0) {
        unsigned long long seen[kGroup - 1], near[kNear];
        const int nearby = min(group, kNear);
        look(pairs, kRow, count, seen);
        if (!a.far) look(ends - nearby * kRow, kRow, nearby, near);
        wait_for(a, pairs, kRow, count, seen, false, [&] {
            bool all = true;
#pragma unroll
            for (int k = 0; k < kGroup - 1; ++k) all = all && (k >= count || seen[k] != kNoMap);
            return all;
        });
        Map<1> m = {1.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
            if (k < count) m = then(m, map_of(seen[k]));
        const bool closes = count == kGroup - 1 && place + 1 < t.count;
        Map<1> whole = m;
        if (closes) {
            barrier_wait_warp(smem_address(&s.tile_ready[j & 1]), j >> 1 & 1, guard);
            const Map<V> tile = s.tile[j & 3][lane];
            whole = then(m, Map<1>{at(tile.a, channel), at(tile.h, channel)});
            // (The first group's takes no state, whatever its A has become.)
            publish(ends, word_of({group > 0 ? whole.a : kNoState, whole.h}));
        }
        float state = 0.0f;   // (the first group's maps take none)
        if (group > 0) {
            if (a.far) {
                const int back = min(group, kFar);
                unsigned long long far[kFar];
                look(ends - back * kRow, kRow, back, far);
                state = state_behind(a, ends - back * kRow, kRow, back, far);
            } else {
                state = state_behind(a, ends - nearby * kRow, kRow, nearby, near);
            }
            if (closes) publish(ends, word_of({kNoState, mad(whole.a, state, whole.h)}));
        }
        state = mad(m.a, state, m.h);
        GSR_CANARY(22 + j % 4);
        at(s.carry[j & 3][lane], channel) = state;
    }
    // (A barrier for even tiles and one for odd: the working warps look at a tile's when
    // the next one's may be through already.)
    warp_arrive(s.state_ready[j & 1]);
    barrier_wait_warp(smem_address(&s.state_ready[j & 1]), j >> 1 & 1, guard);
}

// ---- runs of tokens ------------------------------------------------------------------------

// A warp's run of an array: a lane's elements of token after token, in the recurrence's
// order.  (Steps are below 2^31 elements, so that an address is one multiply-add.)
template <typename T, int V>
struct Run {
    using R = Raw<T, V>;
    T *at;
    int step;

    __device__ __forceinline__ Run(const RecurrenceArgs &a, const Tokens &t, const Tile &tile, int k, int c)
    {
        at = (T *)t.data + tile.b * t.batch + (int64_t)(a.reverse ? tile.length - 1 - k : k) * t.token + c;
        step = a.reverse ? -(int)t.token : (int)t.token;
    }
    __device__ __forceinline__ R *token(int i) const { return (R *)(at + (int64_t)step * i); }
    // N tokens of which `count` (the same in a warp) are there; the others as 0.
    template <int N>
    __device__ __forceinline__ void load(R (&r)[N], int count) const
    {
        if (count == N) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = *token(i);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                clear(r[i]);
                if (i < count) r[i] = *token(i);
            }
        }
    }
    __device__ __forceinline__ void store(int i, const Lanes<V> &v) const { *token(i) = raw_of<T, V>(v); }
};

__device__ __forceinline__ uint32_t shared_load(uint32_t at)
{
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
    return w;
}
__device__ __forceinline__ void shared_store(uint32_t at, uint32_t w)
{
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
}

// The same of a tile in a stage, a lane's 4 bytes of row after row.
struct StagedRun {
    uint32_t at;
    int step;

    __device__ __forceinline__ StagedRun(const RecurrenceArgs &a, uint32_t stage, int tile_tokens, int first)
    {
        at = stage + (a.reverse ? tile_tokens - 1 - first : first) * kRowBytes + threadIdx.x % 32 * 4;
        step = a.reverse ? -kRowBytes : kRowBytes;
    }
    __device__ __forceinline__ uint32_t word(int i, int array_bytes) const { return shared_load(at + i * step + array_bytes); }
};

template <typename T, int V>
__device__ __forceinline__ void clear_tokens(const Tokens &t, int b, int from, int to, int c)
{
    Raw<T, V> zero;
    clear(zero);
    T *p = (T *)t.data + b * t.batch + (int64_t)from * t.token + c;
    for (int k = from; k < to; ++k, p += t.token) {
        GSR_CANARY_LANES(50);
        *(Raw<T, V> *)p = zero;
    }
}

// A staged word's elements.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_bits(uint32_t w)
{
    return (Raw<T, V>)w;
}

// exp(-x) for x >= 0.  For f32 the product x log2(e) is kept to twice float's length.
template <typename T>
__device__ __forceinline__ float exp_minus(float x)
{
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.9259629911e-8f, kLn2 = 0.69314718056f;
    const float hi = x * -kLog2e;
    if constexpr (sizeof(T) == 2) return exp2_fast(hi);
    const float lo = fmaf(x, -kLog2eLow, fmaf(x, -kLog2e, -hi)), e = exp2_fast(hi);
    return x < 120.0f ? fmaf(e, lo * kLn2, e) : e;   // (beyond, 0; the products may not be finite)
}

// a = sigmoid(f) and s = 1 - a.
template <typename T>
__device__ __forceinline__ void split(float f, float &a, float &s)
{
    const float e = exp_minus<T>(fabsf(f)), small = e * rcp_fast(1.0f + e), large = 1.0f - small;
    a = f < 0.0f ? small : large;
    s = f < 0.0f ? large : small;
}

template <typename T>
__device__ __forceinline__ void split(float2 f, float2 &a, float2 &s)
{
    split<T>(f.x, a.x, s.x);
    split<T>(f.y, a.y, s.y);
}

template <typename T>
__device__ __forceinline__ float sigmoid(float o)
{
    if constexpr (sizeof(T) == 2) return rcp_fast(1.0f + exp2_fast(o * -1.4426950408889634f));
    float a, s;
    split<T>(o, a, s);
    return a;
}

template <typename T>
__device__ __forceinline__ float2 sigmoid(float2 o)
{
    return make_float2(sigmoid<T>(o.x), sigmoid<T>(o.y));
}

// Values of N lanes' words, packed for tensor memory and back.
template <int N>
__device__ __forceinline__ void put(uint32_t *to, const float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = __float_as_uint(v[i]);
}
template <int N>
__device__ __forceinline__ void put(uint32_t *to, const float2 (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        to[2 * i] = __float_as_uint(v[i].x);
        to[2 * i + 1] = __float_as_uint(v[i].y);
    }
}
__device__ __forceinline__ void get(const uint32_t *from, int i, float &v) { v = __uint_as_float(from[i]); }
__device__ __forceinline__ void get(const uint32_t *from, int i, float2 &v)
{
    v = make_float2(__uint_as_float(from[2 * i]), __uint_as_float(from[2 * i + 1]));
}

// 16 columns of the calling thread's lane.
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t at)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
// (As tensor.cuh's: values of a load are used behind its wait.)
__device__ __forceinline__ void pin16(uint32_t (&r)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i += 8)
        asm volatile(""
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                       "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// What a working warp knows of its run.
template <typename T, int V>
struct RunPlace {
    int c, k0, count;      // first channel, first token in the recurrence's order, tokens
    bool mine;             // (other lanes compute the last one's channels, or none)

    __device__ __forceinline__ RunPlace(const RecurrenceArgs &a, const Tile &t, int tile_tokens, int run)
    {
        const int own = t.slab * (32 * V) + threadIdx.x % 32 * V;
        c = min(own, a.channels - V);
        mine = own == c;
        k0 = t.index * tile_tokens + threadIdx.x / 32 * run;
        count = min(max(t.length - k0, 0), run);
    }
};

// ---- forward -----------------------------------------------------------------------------

// Words of a run in tensor memory: a and (1 - a) x, 32 of each at most.  The output gates wait in
// shared memory, in places for two tiles, where their copy has put them, or the warp.
template <typename T, int V, bool GATE, bool COPY, int S>
struct Forward {
    using F = Lanes<V>;
    using R = Raw<T, V>;
    [[maybe_unused]] static constexpr int kTokens = kTile, kLength = kRun, kBytes = kTile * kRowBytes;

    static __device__ __forceinline__ void clear_rest(const RecurrenceArgs &a, const Tile &t)
    {
        const RunPlace<T, V> at(a, t, kTokens, kLength);
        if (at.mine) clear_tokens<T, V>(a.out, t.b, max(at.k0, t.length), min(at.k0 + kLength, a.tokens), at.c);
    }

    // Reads a run, composes its map and leaves it in tensor memory.
    static __device__ __forceinline__ void compose(const RecurrenceArgs &a, Shared<V, S, false> &s, const Tile &t, uint32_t j,
                                                   uint32_t stage, uint32_t gates, uint32_t columns)
    {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const RunPlace<T, V> at(a, t, kTokens, kLength);
        F keep[kLength], enter[kLength];
        uint32_t w0[32], w1[32];
        Map<V> own;
        fill(own.a, 1.0f);
        fill(own.h, 0.0f);
        {
            R f[kLength], x[kLength];
            if constexpr (COPY) {
                const StagedRun staged(a, stage, kTokens, warp * kLength);
#pragma unroll
                for (int i = 0; i < kLength; ++i) {
                    f[i] = raw_bits<T, V>(staged.word(i, 0));
                    x[i] = raw_bits<T, V>(staged.word(i, kBytes));
                }
            } else {
                R o[GATE ? kLength : 1];
                Run<T, V>(a, a.forget, t, at.k0, at.c).load(f, at.count);
                Run<T, V>(a, a.x, t, at.k0, at.c).load(x, at.count);
                // (The gates behind the others: loads would wait for a store to shared memory in
                // front of them, 126 us for 120 of 32,640 x 2,050 in bf16.)
                if constexpr (GATE) {
                    Run<T, V>(a, a.gate, t, at.k0, at.c).load(o, at.count);
#pragma unroll
                    for (int i = 0; i < kLength; ++i) shared_store(gates + i * kRowBytes, o[i]);
                }
            }
            if (at.count == kLength) {
#pragma unroll
                for (int i = 0; i < kLength; ++i) step(f[i], x[i], true, keep[i], enter[i], own);
            } else {
#pragma unroll
                for (int i = 0; i < kLength; ++i) step(f[i], x[i], i < at.count, keep[i], enter[i], own);
            }
        }
        s.runs[j & 1][warp][lane] = own;
        put(w0, keep);
        put(V == 2 ? w1 : w0 + 16, enter);
        tmem_store32(columns, w0);
        if (V == 2) tmem_store32(columns + 32, w1);
        tmem_wait_store();
    }

    static __device__ __forceinline__ void step(R f, R x, bool there, F &keep, F &enter, Map<V> &own)
    {
        F rest;
        split<T>(value_of<T, V>(f), keep, rest);
        enter = mul(rest, value_of<T, V>(x));
        if (!there) {
            fill(keep, 1.0f);
            fill(enter, 0.0f);
        }
        own.h = mad(keep, own.h, enter);
        own.a = mul(keep, own.a);
    }

    // Runs the tokens from the state in front of them.
    static __device__ __forceinline__ void finish(const RecurrenceArgs &a, Shared<V, S, false> &s, const Tile &t, uint32_t j,
                                                  uint32_t gates, uint32_t columns)
    {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const RunPlace<T, V> at(a, t, kTokens, kLength);
        uint32_t w0[32], w1[32];
        tmem_load32(w0, columns);
        if (V == 2) tmem_load32(w1, columns + 32);
        const Map<V> before = s.runs[j & 1][warp][lane];
        F h = mad(before.a, s.carry[j & 3][lane], before.h);
        tmem_wait_load();
        pin(w0);
        if (V == 2) pin(w1);
        if (at.count == 0 || !at.mine) return;
        if (a.states && at.k0 % kStateStep == 0)
            store_state<V>(a.states + ((int64_t)t.b * a.blocks + at.k0 / kStateStep) * a.channels + at.c, h);
        const Run<T, V> out(a, a.out, t, at.k0, at.c);
        // (A few tokens' gates are read ahead of the stores, which none of the reads passes.)
        constexpr int kAhead = 6;
        R o[GATE ? kLength : 1];
        const int gate_step = COPY && a.reverse ? -kRowBytes : kRowBytes;
        auto read = [&](int i) {
            if constexpr (GATE) o[i] = raw_bits<T, V>(shared_load(gates + i * gate_step));
        };
        if constexpr (GATE)
#pragma unroll
            for (int i = 0; i < kAhead; ++i) read(i);
        auto token = [&](int i) {
            if (GATE && i + kAhead < kLength) read(i + kAhead);
            F keep, enter;
            get(w0, i, keep);
            get(V == 2 ? w1 : w0 + 16, i, enter);
            h = mad(keep, h, enter);
            if constexpr (GATE) {
                const F g = value_of<T, V>(o[i]);
                return mul(h, mul(g, sigmoid<T>(g)));
            } else {
                return h;
            }
        };
        if (at.count == kLength) {
#pragma unroll
            for (int i = 0; i < kLength; ++i) out.store(i, token(i));
        } else {
#pragma unroll
            for (int i = 0; i < kLength; ++i) {
                const F y = token(i);
                if (i < at.count) out.store(i, y);
            }
        }
        if (at.k0 + kLength >= t.length) store_state<V>(a.final + (int64_t)t.b * a.channels + at.c, h);
    }
};

// ---- backward ----------------------------------------------------------------------------

// Words of a run in tensor memory: a, 1 - a, dout silu(o) (dL/dh_t without what comes from
// behind) and dout silu'(o), 16 each; x waits in shared memory.  With u_t = a_t (h_(t-1) -
// x_t), dL/df_t = dL/dx_t u_t.  (h_t is x_t + u_t too, but loses a small state beside a large
// x that an open gate keeps out; it is taken as in the forward.)
template <typename T, int V, bool GATE, bool COPY, int S>
struct Backward {
    using F = Lanes<V>;
    using R = Raw<T, V>;
    [[maybe_unused]] static constexpr int kTokens = kGradTile, kLength = kGradRun, kBytes = kGradTile * kRowBytes;

    static __device__ __forceinline__ void clear_rest(const RecurrenceArgs &a, const Tile &t)
    {
        const RunPlace<T, V> at(a, t, kTokens, kLength);
        if (!at.mine) return;
        const int from = max(at.k0, t.length), to = min(at.k0 + kLength, a.tokens);
        clear_tokens<T, V>(a.dx, t.b, from, to, at.c);
        clear_tokens<T, V>(a.dforget, t.b, from, to, at.c);
        if (GATE) clear_tokens<T, V>(a.dgate, t.b, from, to, at.c);
    }

    static __device__ __forceinline__ void park(uint32_t columns, int part, const F (&v)[kLength])
    {
        uint32_t w[16];
        put(w, v);
        if (V == 1)
#pragma unroll
            for (int i = 8; i < 16; ++i) w[i] = 0;
        tmem_store16(columns + 16 * part, w);
    }
    static __device__ __forceinline__ F value(const uint32_t (&w)[16], int i)
    {
        F v;
        get(w, i, v);
        return v;
    }

    static __device__ __forceinline__ void compose(const RecurrenceArgs &a, Shared<V, S, true> &s, const Tile &t, uint32_t j,
                                                   uint32_t stage, uint32_t, uint32_t columns)
    {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const RunPlace<T, V> at(a, t, kTokens, kLength);
        F keep[kLength], rest[kLength], into[kLength], h;
        R x[kLength], f[kLength], dy[kLength], o[GATE ? kLength : 1];
        if constexpr (COPY) {
            const StagedRun staged(a, stage, kTokens, warp * kLength);
#pragma unroll
            for (int i = 0; i < kLength; ++i) {
                f[i] = raw_bits<T, V>(staged.word(i, 0));
                x[i] = raw_bits<T, V>(staged.word(i, kBytes));
                if constexpr (GATE) o[i] = raw_bits<T, V>(staged.word(i, 2 * kBytes));
                dy[i] = raw_bits<T, V>(staged.word(i, (GATE ? 3 : 2) * kBytes));
            }
        } else {
            Run<T, V>(a, a.forget, t, at.k0, at.c).load(f, at.count);
            Run<T, V>(a, a.x, t, at.k0, at.c).load(x, at.count);
            Run<T, V>(a, a.dout, t, at.k0, at.c).load(dy, at.count);
            if constexpr (GATE) Run<T, V>(a, a.gate, t, at.k0, at.c).load(o, at.count);
        }
        if (at.count < kLength)
#pragma unroll
            for (int i = 0; i < kLength; ++i)
                if (i >= at.count) {
                    clear(x[i]);
                    clear(dy[i]);
                    if constexpr (GATE) clear(o[i]);
                }
        if constexpr (GATE) {
            F slope[kLength], one;
            fill(one, 1.0f);
#pragma unroll
            for (int i = 0; i < kLength; ++i) {
                const F d = value_of<T, V>(dy[i]), g = value_of<T, V>(o[i]), r = sigmoid<T>(g), dr = mul(d, r);
                into[i] = mul(dr, g);
                slope[i] = mul(dr, mad(g, add(one, minus(r)), one));
            }
            park(columns, 3, slope);
        } else {
#pragma unroll
            for (int i = 0; i < kLength; ++i) into[i] = value_of<T, V>(dy[i]);
        }
        park(columns, 2, into);
#pragma unroll
        for (int i = 0; i < kLength; ++i) split<T>(value_of<T, V>(f[i]), keep[i], rest[i]);
        if (at.count < kLength)
#pragma unroll
            for (int i = 0; i < kLength; ++i)
                if (i >= at.count) {   // no step (its x and dout are 0)
                    fill(keep[i], 1.0f);
                    fill(rest[i], 0.0f);
                }
        park(columns, 0, keep);
        park(columns, 1, rest);
        Map<V> own;
        fill(h, 0.0f);
        fill(own.a, 1.0f);
        fill(own.h, 0.0f);
#pragma unroll
        for (int i = 0; i < kLength; ++i) {
            s.x[j & 1][warp][i][lane] = x[i];
            h = mad(keep[i], h, mul(rest[i], value_of<T, V>(x[i])));
            own.a = mul(keep[i], own.a);
        }
#pragma unroll
        for (int i = kLength - 1; i >= 0; --i) own.h = mul(keep[i], add(own.h, into[i]));
        s.runs[j & 1][warp][lane] = own;
        s.h[j & 1][warp][lane] = h;
        tmem_wait_store();
    }

    static __device__ __forceinline__ void finish(const RecurrenceArgs &a, Shared<V, S, true> &s, const Tile &t, uint32_t j,
                                                  uint32_t, uint32_t columns)
    {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const RunPlace<T, V> at(a, t, kTokens, kLength);
        uint32_t keep[16], rest[16], into[16];
        F u[kLength], h = s.h[j & 1][warp][lane];
        const Map<V> behind = s.runs[j & 1][warp][lane];
        F p = mad(behind.a, s.carry[j & 3][lane], behind.h);
        {
            uint32_t slope[16];
            tmem_load16(keep, columns);
            tmem_load16(rest, columns + 16);
            if (GATE) tmem_load16(slope, columns + 48);
            tmem_wait_load();
            pin16(keep);
            pin16(rest);
            if (GATE) pin16(slope);
            tmem_load16(into, columns + 32);
            const bool some = at.count > 0 && at.mine;
            const Run<T, V> dg(a, a.dgate, t, at.k0, at.c);
#pragma unroll
            for (int i = 0; i < kLength; ++i) {
                const F x = value_of<T, V>((R)s.x[j & 1][warp][i][lane]);
                u[i] = mul(value(keep, i), add(h, minus(x)));
                h = mad(value(keep, i), h, mul(value(rest, i), x));
                if constexpr (GATE)
                    if (some && i < at.count) {
                        GSR_CANARY_LANES(42 + i);
                        dg.store(i, mul(value(slope, i), h));
                    }
            }
            __syncwarp();   // (lanes behind the channels have not stored)
            tmem_wait_load();
            pin16(into);
            if (!some) return;
        }
        const Run<T, V> dx(a, a.dx, t, at.k0, at.c), df(a, a.dforget, t, at.k0, at.c);
        auto token = [&](int i, bool there) {
            const F dh = add(p, value(into, i)), enter = mul(dh, value(rest, i));
            p = mul(value(keep, i), dh);
            if (!there) return;
            dx.store(i, enter);
            df.store(i, mul(enter, u[i]));
        };
        if (at.count == kLength) {
#pragma unroll
            for (int i = kLength - 1; i >= 0; --i) token(i, true);
        } else {
#pragma unroll
            for (int i = kLength - 1; i >= 0; --i) token(i, i < at.count);
        }
        if (at.k0 == 0 && a.final) store_state<V>(a.final + (int64_t)t.b * a.channels + at.c, p);
    }
};

// A working warp's tiles: the next one's run is composed before the last one's ends.
// gates: the lane's word of its run's first token, of the first of two tiles (in the order of a
// stage's rows where a copy puts them there, in the recurrence's where the warp does).
template <typename Work, int V, int S, bool GATE, bool COPY, bool BACKWARD>
__device__ __forceinline__ void work_tiles(const RecurrenceArgs &a, Shared<V, S, BACKWARD> &s, uint32_t stages, int stage_bytes,
                                           const WaitGuard &guard)
{
    constexpr bool kGates = GATE && COPY && !BACKWARD;
    constexpr int kGateBytes = kTile * kRowBytes;
    const int warp = threadIdx.x / 32, first = warp * kRun;
    const uint32_t gates = stages + (COPY ? S * stage_bytes : 0) + threadIdx.x % 32 * 4 +
                           (COPY && a.reverse ? kTile - 1 - first : first) * kRowBytes;
    const uint32_t columns = s.columns + ((uint32_t)(warp % 4) << 21) + warp / 4 * (kSlotColumns / 2);   // lane << 16
    Tile before = {};
    bool open = false;
    uint32_t j = 0;
    auto finish = [&] {
        const uint32_t k = j - 1;
        GSR_CANARY(34 + k % 4);
        barrier_wait_warp(smem_address(&s.state_ready[k & 1]), k >> 1 & 1, guard);
        if (kGates) barrier_wait_warp(smem_address(&s.gate_full[k & 1]), k >> 1 & 1, guard);
        Work::finish(a, s, before, k, gates + (k & 1) * kGateBytes, columns + (k & 1) * kSlotColumns);
        if (kGates)
            warp_arrive(s.gate_empty[k & 1]);
        else
            __syncwarp();
    };
    for (uint32_t i = 0;; ++i) {
        const uint32_t stage = i % S;
        barrier_wait_warp(smem_address(&s.known[stage]), i / S & 1, guard);
        if (warp_stop(guard) || s.last[stage]) break;
        const Tile t = s.tiles[stage];
        if (t.length < a.tokens) {
            Work::clear_rest(a, t);
            __syncwarp();   // (lanes behind the channels have nothing to clear)
        }
        const bool some = t.index < t.count;
        if (some) {
            if (COPY) barrier_wait_warp(smem_address(&s.full[stage]), i / S & 1, guard);
            GSR_CANARY(30 + j % 4);
            Work::compose(a, s, t, j, stages + stage * stage_bytes, gates + (j & 1) * kGateBytes,
                          columns + (j & 1) * kSlotColumns);
            warp_arrive(s.runs_ready[j & 1]);
        }
        warp_arrive(s.empty[stage]);
        if (open) finish();
        open = some;
        before = t;
        if (some) ++j;
    }
    if (open && !warp_stop(guard)) finish();
}

// COPY: tiles come through the ring of stages; otherwise the runs' warps read them.
template <typename T, int V, bool GATE, bool COPY, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, kBlocks)
    k_recurrence(const RecurrenceArgs a, const __grid_constant__ Maps maps)
{
    grid_dependency_begin();
    constexpr int S = kStages;
    constexpr int kStageBytes = kStaged<GATE, BACKWARD> * (BACKWARD ? kGradTile : kTile) * kRowBytes;
    extern __shared__ unsigned char s_bytes[];
    __shared__ Shared<V, S, BACKWARD> s;
    const uint32_t stages = (smem_address(s_bytes) + 127u) / 128u * 128u;
    const WaitGuard guard = {&s.aborted, a.status};
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        s.aborted = 0;
        for (int k = 0; k < S; ++k) {
            barrier_init(smem_address(&s.known[k]), 1);
            barrier_init(smem_address(&s.full[k]), 1);
            barrier_init(smem_address(&s.empty[k]), kWarps + 3);
        }
        for (int k = 0; k < 2; ++k) {
            barrier_init(smem_address(&s.runs_ready[k]), kWarps);
            barrier_init(smem_address(&s.tile_ready[k]), 1);
            barrier_init(smem_address(&s.state_ready[k]), 1 + V);
            barrier_init(smem_address(&s.gate_full[k]), 1);
            barrier_init(smem_address(&s.gate_empty[k]), kWarps);
        }
        fence_async();
    }
    if (warp == kComposeWarp) tmem_alloc(smem_address(&s.columns), kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp >= kWarps) {
        give_registers();
        if (warp == kFetchWarp) {
            if (threadIdx.x % 32 == 0) fetch_tiles<V, S, GATE, COPY, BACKWARD>(a, maps, s, stages, guard);
            __syncwarp();
        } else if (warp >= kChainWarp) {
            each_tile(s, guard, [&](const Tile &t, uint32_t j) { follow_chain<V, S, BACKWARD>(a, s, t, j, guard); });
        } else if (warp == kComposeWarp) {
            each_tile(s, guard, [&](const Tile &t, uint32_t j) { compose_runs<V, S, BACKWARD>(a, s, t, j, guard); });
        }
    } else {
        take_registers();
        using Work = std::conditional_t<BACKWARD, Backward<T, V, GATE, COPY, S>, Forward<T, V, GATE, COPY, S>>;
        work_tiles<Work, V, S, GATE, COPY, BACKWARD>(a, s, stages, kStageBytes, guard);
    }
    if (s.aborted && a.aborted && threadIdx.x % 32 == 0) *(volatile uint32_t *)a.aborted = 0;
    drain_if_aborted(guard);
    tmem_fence_before();
    __syncthreads();
    if (warp == kComposeWarp) {
        __syncwarp();
        tmem_free(s.columns, kColumns);
    }
}

// ---- few tokens --------------------------------------------------------------------------

// A few tokens of each item, as they come one after the other while a model answers: a
// thread takes a lane's channels of an item, with no chain and nothing shared.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kFewThreads) k_recurrence_few(const RecurrenceArgs a)
{
    grid_dependency_begin();
    using F = Lanes<V>;
    using R = Raw<T, V>;
    const uint32_t lanes = (uint32_t)(a.channels + V - 1) / V, n = blockIdx.x * kFewThreads + threadIdx.x;   // up to 2^32
    if (n >= (uint64_t)lanes * a.batch) return;
    Tile t = {};
    t.b = n / lanes;
    t.length = a.lengths ? min(max(a.lengths[t.b], 0), a.tokens) : a.tokens;
    const int c = (n - t.b * lanes) * V;
    const int64_t at_state = (int64_t)t.b * a.channels + c;
    const Run<T, V> x(a, a.x, t, 0, c), f(a, a.forget, t, 0, c), o(a, a.gate, t, 0, c), out(a, a.out, t, 0, c);
    F h;
#pragma unroll
    for (int j = 0; j < V; ++j) at(h, j) = a.initial ? a.initial[at_state + j] : 0.0f;
    if (a.states && t.length > 0) store_state<V>(a.states + (int64_t)t.b * a.blocks * a.channels + c, h);
    for (int first = 0; first < t.length; first += kFewAhead) {
        R xs[kFewAhead], fs[kFewAhead], os[GATE ? kFewAhead : 1];
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i)
            if (first + i < t.length) {
                xs[i] = *x.token(first + i);
                fs[i] = *f.token(first + i);
                if constexpr (GATE) os[i] = *o.token(first + i);
            }
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            if (first + i >= t.length) continue;
            F keep, rest;
            split<T>(value_of<T, V>(fs[i]), keep, rest);
            h = mad(keep, h, mul(rest, value_of<T, V>(xs[i])));
            if constexpr (GATE) {
                const F g = value_of<T, V>(os[i]);
                out.store(first + i, mul(h, mul(g, sigmoid<T>(g))));
            } else {
                out.store(first + i, h);
            }
        }
    }
    clear_tokens<T, V>(a.out, t.b, t.length, a.tokens, c);
    store_state<V>(a.final + at_state, h);
}

// ---- host --------------------------------------------------------------------------------

Tokens tokens_of(const gsr_heads *t)
{
    return t ? Tokens{t->data, t->batch_stride, t->token_stride} : Tokens{};
}

RecurrenceArgs args_of(const gsr_recurrence &d)
{
    RecurrenceArgs a = {};
    a.lengths = d.lengths;
    a.batch = d.batch;
    a.tokens = d.tokens;
    a.channels = d.channels;
    a.blocks = (d.tokens + kStateStep - 1) / kStateStep;
    a.reverse = d.reverse;
    return a;
}

bool all_arrays(const RecurrenceArgs &a, std::initializer_list<const Tokens *> arrays, int size, int64_t unit)
{
    bool ok = true;
    for (const Tokens *t : arrays)
        if (t->data)
            ok = ok && (uintptr_t)t->data % (unit * size) == 0 && (a.batch == 1 || t->batch % unit == 0) &&
                 (a.tokens == 1 || t->token % unit == 0);
    return ok;
}

template <typename T, int V, bool GATE, bool COPY, bool BACKWARD>
int launch(gsr_ctx *ctx, RecurrenceArgs &a, int dtype, const char *what, cudaStream_t stream)
{
    constexpr int kTokens = BACKWARD ? kGradTile : kTile;
    constexpr int kTiles = (COPY ? kStages * kStaged<GATE, BACKWARD> : 0) + (GATE && !BACKWARD ? 2 : 0);   // of one array
    constexpr int kBytes = kTiles > 0 ? kTiles * kTokens * kRowBytes + 128 : 0;
    Maps maps = {};
    if (COPY) {
        const struct { CUtensorMap *map; const Tokens *t; } inputs[4] = {
            {&maps.x, &a.x}, {&maps.forget, &a.forget}, {&maps.gate, &a.gate}, {&maps.dout, &a.dout}};
        for (const auto &in : inputs)
            if (in.t->data)
                if (int rc = tokens_map(ctx, in.map, in.t->data, dtype, a.channels, a.tokens, a.batch, in.t->token,
                                        in.t->batch, kRowBytes / (int)sizeof(T), kTokens))
                    return rc;
    }
    auto *kernel = k_recurrence<T, V, GATE, COPY, BACKWARD>;
    static OncePerDevice once;
    if (once.due(ctx)) {
        // (A kernel that starts with fewer registers than the shares add up to would wait for them.)
        cudaFuncAttributes attributes;
        if (int rc = cuda_check(ctx, cudaFuncGetAttributes(&attributes, kernel), what)) return rc;
        if (attributes.numRegs < kStart)
            return fail(ctx, GSR_ERR_CUDA, std::string(what) + ": compiled with too few registers");
        if (kBytes > 0)
            if (int rc = cuda_check(ctx, cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
                                    what))
                return rc;
        once.done(ctx);
    }
    const uint32_t most = (uint32_t)(kBlocks * ctx->num_sms);
    return cuda_check(ctx, launch_kernel_smem(ctx, kernel, dim3(a.work < most ? a.work : most), kThreads, kBytes, 1, stream,
                                              a, maps), what);
}

template <typename T, int V, bool BACKWARD>
int run(gsr_ctx *ctx, RecurrenceArgs &a, int dtype, cudaStream_t stream)
{
    const char *what = BACKWARD ? "gated recurrence backward" : "gated recurrence forward";
    constexpr int kTokens = BACKWARD ? kGradTile : kTile, kSlab = 32 * V, kUnit = 16 / (int)sizeof(T);
    a.tiles = (a.tokens + kTokens - 1) / kTokens;
    if (a.tiles == 0) a.tiles = 1;   // for the states of items without tokens
    a.slabs = (a.channels + kSlab - 1) / kSlab;
    a.work = (uint32_t)a.tiles * a.batch * a.slabs;
    if (!BACKWARD && a.tokens <= kFewTokens) {
        const int64_t lanes = (int64_t)a.batch * ((a.channels + V - 1) / V);
        const dim3 grid((unsigned)((lanes + kFewThreads - 1) / kFewThreads));
        return cuda_check(ctx, a.gate.data ? launch_kernel(ctx, k_recurrence_few<T, V, true>, grid, kFewThreads, stream, a)
                                           : launch_kernel(ctx, k_recurrence_few<T, V, false>, grid, kFewThreads, stream, a),
                          what);
    }
    Workspace workspace(ctx, stream);
    const bool chained = a.tiles > 1;
    const size_t chains = (size_t)a.batch * a.slabs;
    a.groups = (a.tiles + kGroup - 1) / kGroup;
    a.far = chains < kManyChains;
    const size_t pairs = chained ? chains * a.tiles * kSlab * sizeof(unsigned long long) : 0;
    const size_t ends = chained ? chains * a.groups * kSlab * sizeof(unsigned long long) : 0;
    const size_t bytes = chained ? pairs + ends + 16 : 0;
    void *work = nullptr;
    if (int rc = workspace.take(bytes, &work)) return rc;
    a.status = ctx->status_dev;
    if (chained) {
        if (int rc = cuda_check(ctx, cudaMemsetAsync(work, 0xff, bytes, stream), what)) return rc;
        a.pairs = (unsigned long long *)work;
        a.ends = a.pairs + pairs / sizeof(unsigned long long);
        a.ticket = (uint32_t *)((unsigned char *)work + pairs + ends);
        a.aborted = a.ticket + 1;
    }
    // Copies of whole tiles where the arrays allow them and a block has more than one to come.
    const bool copy = chained && kSlab * (int)sizeof(T) == kRowBytes &&
                      all_arrays(a, {&a.x, &a.forget, &a.gate, &a.dout}, (int)sizeof(T), kUnit);
    int rc;
    if constexpr (kSlab * (int)sizeof(T) == kRowBytes) {
        if (copy)
            rc = a.gate.data ? launch<T, V, true, true, BACKWARD>(ctx, a, dtype, what, stream)
                             : launch<T, V, false, true, BACKWARD>(ctx, a, dtype, what, stream);
    }
    if (!copy)
        rc = a.gate.data ? launch<T, V, true, false, BACKWARD>(ctx, a, dtype, what, stream)
                         : launch<T, V, false, false, BACKWARD>(ctx, a, dtype, what, stream);
    if (rc != GSR_OK) return rc;
    return workspace.done();
}

// 16-bit elements in pairs where channels and arrays allow it (32,640 x 2,050 in bf16 with a gate,
// which no copies bring: 120 and 214 us; in single elements, x 2,049, 156 and 306).
template <bool BACKWARD>
int dispatch(gsr_ctx *ctx, RecurrenceArgs &a, int dtype, cudaStream_t stream)
{
    if (dtype == GSR_F32) return run<float, 1, BACKWARD>(ctx, a, dtype, stream);
    const bool pairs = a.channels % 2 == 0 && all_arrays(a, {&a.x, &a.forget, &a.gate, &a.out, &a.dout, &a.dx, &a.dforget,
                                                             &a.dgate}, 2, 2);
    if (dtype == GSR_BF16)
        return pairs ? run<__nv_bfloat16, 2, BACKWARD>(ctx, a, dtype, stream)
                     : run<__nv_bfloat16, 1, BACKWARD>(ctx, a, dtype, stream);
    return pairs ? run<__half, 2, BACKWARD>(ctx, a, dtype, stream) : run<__half, 1, BACKWARD>(ctx, a, dtype, stream);
}

}  // namespace

int gated_recurrence_forward(gsr_ctx *ctx, const gsr_recurrence &d, const gsr_heads &x, const gsr_heads &forget,
                             const gsr_heads *gate, const float *initial, const gsr_heads &out, float *final,
                             float *states, cudaStream_t stream)
{
    RecurrenceArgs a = args_of(d);
    a.x = tokens_of(&x);
    a.forget = tokens_of(&forget);
    a.gate = tokens_of(gate);
    a.out = tokens_of(&out);
    a.initial = initial;
    a.final = final;
    a.states = states;
    return dispatch<false>(ctx, a, d.dtype, stream);
}

int gated_recurrence_backward(gsr_ctx *ctx, const gsr_recurrence &d, const gsr_heads &dout, const gsr_heads &x,
                              const gsr_heads &forget, const gsr_heads *gate, const float *states,
                              const float *dfinal, const gsr_heads &dx, const gsr_heads &dforget,
                              const gsr_heads *dgate, float *dinitial, cudaStream_t stream)
{
    RecurrenceArgs a = args_of(d);
    a.dout = tokens_of(&dout);
    a.x = tokens_of(&x);
    a.forget = tokens_of(&forget);
    a.gate = tokens_of(gate);
    a.states = const_cast<float *>(states);
    a.initial = dfinal;
    a.dx = tokens_of(&dx);
    a.dforget = tokens_of(&dforget);
    a.dgate = tokens_of(dgate);
    a.final = dinitial;
    return dispatch<true>(ctx, a, d.dtype, stream);
}

}  // namespace gsr
