// recurrence.cu -- a gated linear recurrence over the tokens of each item, channel
// by channel, forward and backward.
//
//   a_t = sigmoid(f_t),  h_t = a_t h_(t-1) + (1 - a_t) x_t,  out_t = h_t silu(o_t)
// and with dh_t = dout_t silu(o_t) + a_(t+1) dh_(t+1)
//   dx = dh (1 - a),  df = dh (h_(t-1) - x) a (1 - a),  do = dout h silu'(o).
//
// Bound by HBM.  A block takes a tile of tokens by 32 or 64 channels, each warp a run
// of tokens, whose values stay in registers: a run's effect on the state before it is
// affine, h -> A h + H, and so is a warp's, a tile's and a chain of tiles'.  The tile
// reads its inputs once, composes its (A, H), takes the state in front of it from the
// tiles before, and then runs its tokens from that state.  The backward does the same
// from the end with p_t = a_t dh_t, for which p -> A p + P, and computes h again from
// the forward's states.
//
// The chain.  Tiles are taken from a ticket in the chain's order, so a tile waits only
// for blocks that run or have run.  Each publishes its (A, H); every kGroup-th also the
// state behind it, and a tile folds what its group's tiles before it have published:
// the composition does not depend on timing, so results are the same bits on every
// run.  A published pair is one 64-bit word, which is all ones before that (no pair
// is: A is never that NaN).
//
// Numerics.  Of a and 1 - a the smaller one, w <= 1/2, is e / (1 + e) with e =
// exp(-|f|), and a step moves h or x by w times their difference: nothing cancels for
// gates near 0 or 1, and A takes 1 - w as A - w A.
#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 4 * kWarps;         // tiles of a group: four for each warp to fold
constexpr int kRun = 16, kGradRun = 8;     // tokens of a warp
constexpr int kTile = kWarps * kRun, kGradTile = kWarps * kGradRun;
constexpr int kStateStep = GSR_RECURRENCE_BLOCK;
static_assert(kStateStep % kRun == 0 && kGradTile == kStateStep, "states lie where runs and tiles start");
constexpr long long kChainCycles = 4000000000ll;   // of a wait: seconds, where a tile takes microseconds

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
    int reverse;
    unsigned long long *pairs, *ends;   // published: [batch, slabs, tiles] and [batch, slabs, groups] rows of words
    uint32_t *ticket;            // all ones before the first
    uint32_t *aborted;           // 0 once a wait has run out
    uint32_t *status;
};

// ---- the affine maps ------------------------------------------------------------------

struct Map {
    float a, h;   // state -> a state + h
};

__device__ __forceinline__ Map then(const Map &first, const Map &second)
{
    return {second.a * first.a, fmaf(second.a, first.h, second.h)};
}

__device__ __forceinline__ unsigned long long word_of(const Map &m)
{
    return (unsigned long long)__float_as_uint(m.h) << 32 | __float_as_uint(m.a);
}

__device__ __forceinline__ Map map_of(unsigned long long w)
{
    return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

template <int V>
struct Words {
    unsigned long long w[V];
};

__device__ __forceinline__ void publish(unsigned long long *to, const Words<1> &v)
{
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(to), "l"(v.w[0]) : "memory");
}
__device__ __forceinline__ void publish(unsigned long long *to, const Words<2> &v)
{
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(to), "l"(v.w[0]), "l"(v.w[1]) : "memory");
}
__device__ __forceinline__ void look(const unsigned long long *at, Words<1> &v)
{
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v.w[0]) : "l"(at) : "memory");
}
__device__ __forceinline__ void look(const unsigned long long *at, Words<2> &v)
{
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(v.w[0]), "=l"(v.w[1]) : "l"(at) : "memory");
}

template <int V>
__device__ __forceinline__ bool ready(const Words<V> &v)
{
    bool all = true;
#pragma unroll
    for (int j = 0; j < V; ++j) all = all && v.w[j] != ~0ull;
    return all;
}

// Looks until the words are there, or the wait has run out (here or elsewhere).
template <int V>
__device__ __forceinline__ void wait_for(const RecurrenceArgs &a, const unsigned long long *at, Words<V> &v)
{
    if (ready(v)) return;
    const long long start = clock64();
    for (int turn = 1;; ++turn) {
        look(at, v);
        if (ready(v)) return;
        if (turn % 64 != 0) continue;
        if (*(volatile uint32_t *)a.aborted == 0) return;
        if (clock64() - start > kChainCycles) {
            *(volatile uint32_t *)a.aborted = 0;
            *(volatile uint32_t *)a.status = 1;
            return;
        }
    }
}

// ---- tiles -------------------------------------------------------------------------------

struct Tile {
    int b, slab, index;    // item, channel slab, place along the tokens
    int length, count;     // the item's tokens and tiles
};

// A block's tile; the ticket counts in the order of the chains.
__device__ __forceinline__ Tile take_tile(const RecurrenceArgs &a, int tile_tokens, bool backward)
{
    uint32_t n = blockIdx.x;
    if (a.ticket) {
        __shared__ uint32_t s_ticket;
        if (threadIdx.x == 0) s_ticket = atomicAdd(a.ticket, 1u) + 1u;
        __syncthreads();
        n = s_ticket;
    }
    Tile t;
    const uint32_t chains = (uint32_t)a.batch * a.slabs, place = n / chains, chain = n - place * chains;
    t.b = chain / a.slabs;
    t.slab = chain - t.b * a.slabs;
    t.index = backward ? a.tiles - 1 - (int)place : (int)place;
    t.length = a.lengths ? min(max(a.lengths[t.b], 0), a.tokens) : a.tokens;
    t.count = (t.length + tile_tokens - 1) / tile_tokens;
    return t;
}

// A warp's tokens of one array: `from` the first one's address for this lane, in steps
// of `step` elements.  Behind the item's length tokens come in their own order.
struct Walk {
    int64_t first, step;
};

__device__ __forceinline__ Walk walk(const RecurrenceArgs &a, const Tokens &t, const Tile &tile, int k, int c)
{
    const int64_t at = a.reverse ? tile.length - 1 - k : k;
    return {tile.b * t.batch + at * t.token + c, a.reverse ? -t.token : t.token};
}

template <typename T, int V>
__device__ __forceinline__ void clear_tokens(const RecurrenceArgs &a, const Tokens &t, int b, int from, int to, int c)
{
    Vec<T, V> zero;
#pragma unroll
    for (int j = 0; j < V; ++j) zero.e[j] = from_float<T>(0.0f);
    T *at = (T *)t.data + b * t.batch + from * t.token + c;
    for (int k = from; k < to; ++k, at += t.token) *(Vec<T, V> *)at = zero;
}

// The state in front of a chain, read by the warp that publishes the first tile's map
// and handed to the others: once that map is out, nobody reads the array, in which a
// block may write the state behind the chain.
template <int V>
__device__ __forceinline__ void load_seed(const RecurrenceArgs &a, int warp, bool here, int64_t at, float *seed)
{
    if (warp != kWarps - 1) return;
#pragma unroll
    for (int j = 0; j < V; ++j) seed[j] = here && a.initial ? a.initial[at + j] : 0.0f;
}

// The state in front of the block's tile, for this lane's channels.  `tile_map`: the
// tile's own map (warp kWarps - 1 has it); `seed`: the state in front of the first tile.
// place: the tile's in its chain of t.count.
template <int V>
__device__ __forceinline__ void chain(const RecurrenceArgs &a, const Tile &t, int place, const Map (&tile_map)[V],
                                      const float *seed, Map (*s_maps)[32 * V], float (&state)[V])
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < V; ++j) state[j] = seed[j];
    if (t.count == 1) return;
    const int64_t row = (int64_t)t.b * a.slabs + t.slab;
    const int groups = (a.tiles + kGroup - 1) / kGroup, group = place / kGroup;
    unsigned long long *pairs = a.pairs + row * a.tiles * (32 * V) + lane * V;
    unsigned long long *ends = a.ends + row * groups * (32 * V) + lane * V;
    if (warp == kWarps - 1 && place + 1 < t.count) {
        Words<V> w;
#pragma unroll
        for (int j = 0; j < V; ++j) {   // the first tile's, as a map of no state
            const Map m = place == 0 ? Map{0.0f, fmaf(tile_map[j].a, seed[j], tile_map[j].h)} : tile_map[j];
            w.w[j] = word_of(m);
        }
        publish(pairs + (int64_t)place * (32 * V), w);
    }
    if (place == 0) return;
    // Each warp folds four tiles of the group; the first one behind the group's start.
    Map m[V];
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = {1.0f, 0.0f};
    const int first = group * kGroup + 4 * warp;
    Words<V> seen[5];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i < place) look(pairs + (int64_t)(first + i) * (32 * V), seen[i]);
    if (warp == 0 && group > 0) {
        look(ends + (int64_t)group * (32 * V), seen[4]);
        wait_for(a, ends + (int64_t)group * (32 * V), seen[4]);
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = map_of(seen[4].w[j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i < place) {
            wait_for(a, pairs + (int64_t)(first + i) * (32 * V), seen[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = then(m[j], map_of(seen[i].w[j]));
        }
#pragma unroll
    for (int j = 0; j < V; ++j) s_maps[warp][lane * V + j] = m[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        state[j] = 0.0f;   // (the first map of a chain takes no state)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const Map v = s_maps[w][lane * V + j];
            state[j] = fmaf(v.a, state[j], v.h);
        }
    }
    if (warp == kWarps - 1 && place % kGroup == kGroup - 1 && place + 1 < t.count) {
        Words<V> w;
#pragma unroll
        for (int j = 0; j < V; ++j) w.w[j] = word_of({0.0f, fmaf(tile_map[j].a, state[j], tile_map[j].h)});
        publish(ends + (int64_t)(group + 1) * (32 * V), w);
    }
}

// ---- gates -------------------------------------------------------------------------------

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

// The step's weight: the smaller of a and 1 - a, below 0 (or -0) where it is 1 - a.
template <typename T>
__device__ __forceinline__ float gate_weight(float f)
{
    const float e = exp_minus<T>(fabsf(f)), w = e * rcp_fast(1.0f + e);
    return __uint_as_float(__float_as_uint(w) | (~__float_as_uint(f) & 0x80000000u));
}

__device__ __forceinline__ bool keeps(float c) { return __float_as_int(c) < 0; }

// h -> a h + (1 - a) x
__device__ __forceinline__ float step(float c, float h, float x) { return fmaf(c, h - x, keeps(c) ? h : x); }
// v -> a v
__device__ __forceinline__ float keep(float c, float v) { return fmaf(c, v, keeps(c) ? v : 0.0f); }

template <typename T>
__device__ __forceinline__ float sigmoid(float o)
{
    const float e = exp_minus<T>(fabsf(o)), r = rcp_fast(1.0f + e);
    return o < 0.0f ? e * r : r;
}

// ---- forward -----------------------------------------------------------------------------

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, 2) k_recurrence(const RecurrenceArgs a)
{
    grid_dependency_begin();
    __shared__ Map s_maps[2][kWarps][32 * V];
    __shared__ float s_seed[32 * V];
    const Tile t = take_tile(a, kTile, false);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c0 = t.slab * (32 * V) + lane * V;
    const bool mine = c0 < a.channels;
    const int k0 = t.index * kTile + warp * kRun;
    const int count = mine ? min(max(t.length - k0, 0), kRun) : 0;
    if (mine) clear_tokens<T, V>(a, a.out, t.b, max(k0, t.length), min(k0 + kRun, a.tokens), c0);
    const int64_t at_state = (int64_t)t.b * a.channels + c0;
    load_seed<V>(a, warp, mine && t.index == 0, at_state, s_seed + lane * V);
    if (t.index >= t.count) {
        if (t.length == 0 && t.index == 0 && warp == kWarps - 1 && mine)
#pragma unroll
            for (int j = 0; j < V; ++j) a.final[at_state + j] = s_seed[lane * V + j];
        return;
    }

    using Access = Vec<T, V>;
    Access x[kRun], o[kRun];
    float c[kRun][V];
    {
        const Walk wx = walk(a, a.x, t, k0, c0), wf = walk(a, a.forget, t, k0, c0), wo = walk(a, a.gate, t, k0, c0);
        Access f[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (i < count) {
                f[i] = *(const Access *)((const T *)a.forget.data + wf.first + i * wf.step);
                x[i] = *(const Access *)((const T *)a.x.data + wx.first + i * wx.step);
                if (GATE) o[i] = *(const Access *)((const T *)a.gate.data + wo.first + i * wo.step);
            }
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (i >= count) x[i].e[j] = from_float<T>(0.0f);
                c[i][j] = i < count ? gate_weight<T>(to_float(f[i].e[j])) : -0.0f;   // no step
            }
    }
    Map own[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        own[j] = {1.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            own[j].h = step(c[i][j], own[j].h, to_float(x[i].e[j]));
            own[j].a = keep(c[i][j], own[j].a);
        }
        s_maps[0][warp][lane * V + j] = own[j];
    }
    __syncthreads();
    // The warps in front of this one, and for the last warp the tile.
    Map before[V], all[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        before[j] = {1.0f, 0.0f};
        for (int w = 0; w < warp; ++w) before[j] = then(before[j], s_maps[0][w][lane * V + j]);
        all[j] = then(before[j], own[j]);
    }
    float h[V];
    chain<V>(a, t, t.index, all, s_seed + lane * V, s_maps[1], h);
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = fmaf(before[j].a, h[j], before[j].h);
    if (count == 0) return;

    if (a.states && k0 % kStateStep == 0)
#pragma unroll
        for (int j = 0; j < V; ++j)
            a.states[((int64_t)t.b * a.blocks + k0 / kStateStep) * a.channels + c0 + j] = h[j];
    const Walk wy = walk(a, a.out, t, k0, c0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            y[j] = h[j] = step(c[i][j], h[j], to_float(x[i].e[j]));
            if (GATE) {
                const float g = to_float(o[i].e[j]);
                y[j] *= g * sigmoid<T>(g);
            }
        }
        if (i < count) {
            Access out;
            if constexpr (V == 1)
                out.e[0] = from_float<T>(y[0]);
            else
                set_pair(out, 0, make_float2(y[0], y[V - 1]));
            *(Access *)((T *)a.out.data + wy.first + i * wy.step) = out;
        }
    }
    if (k0 < t.length && k0 + kRun >= t.length)
#pragma unroll
        for (int j = 0; j < V; ++j) a.final[at_state + j] = h[j];
}

// ---- backward ----------------------------------------------------------------------------

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, 2) k_recurrence_grad(const RecurrenceArgs a)
{
    grid_dependency_begin();
    __shared__ Map s_maps[2][kWarps][32 * V];
    __shared__ float s_h[kWarps][32 * V], s_seed[32 * V];
    const Tile t = take_tile(a, kGradTile, true);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c0 = t.slab * (32 * V) + lane * V;
    const bool mine = c0 < a.channels;
    const int k0 = t.index * kGradTile + warp * kGradRun;
    const int count = mine ? min(max(t.length - k0, 0), kGradRun) : 0;
    if (mine) {
        const int from = max(k0, t.length), to = min(k0 + kGradRun, a.tokens);
        clear_tokens<T, V>(a, a.dx, t.b, from, to, c0);
        clear_tokens<T, V>(a, a.dforget, t.b, from, to, c0);
        if (GATE) clear_tokens<T, V>(a, a.dgate, t.b, from, to, c0);
    }
    const int64_t at_state = (int64_t)t.b * a.channels + c0;
    const int place = t.count - 1 - t.index;   // in the chain, which starts at the last token
    load_seed<V>(a, warp, mine && (place == 0 || t.length == 0), at_state, s_seed + lane * V);
    if (place < 0) {
        if (t.length == 0 && t.index == 0 && warp == kWarps - 1 && mine && a.final)
#pragma unroll
            for (int j = 0; j < V; ++j) a.final[at_state + j] = s_seed[lane * V + j];
        return;
    }

    using Access = Vec<T, V>;
    Access x[kGradRun], o[kGradRun], dy[kGradRun];
    float c[kGradRun][V], sig[kGradRun][V], before[V];
    {
        const Walk wx = walk(a, a.x, t, k0, c0), wf = walk(a, a.forget, t, k0, c0), wo = walk(a, a.gate, t, k0, c0),
                   wd = walk(a, a.dout, t, k0, c0);
        Access f[kGradRun];
#pragma unroll
        for (int i = 0; i < kGradRun; ++i)
            if (i < count) {
                f[i] = *(const Access *)((const T *)a.forget.data + wf.first + i * wf.step);
                x[i] = *(const Access *)((const T *)a.x.data + wx.first + i * wx.step);
                dy[i] = *(const Access *)((const T *)a.dout.data + wd.first + i * wd.step);
                if (GATE) o[i] = *(const Access *)((const T *)a.gate.data + wo.first + i * wo.step);
            }
#pragma unroll
        for (int j = 0; j < V; ++j)
            before[j] = mine ? a.states[((int64_t)t.b * a.blocks + t.index) * a.channels + c0 + j] : 0.0f;
#pragma unroll
        for (int i = 0; i < kGradRun; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (i >= count) {
                    x[i].e[j] = dy[i].e[j] = from_float<T>(0.0f);
                    if (GATE) o[i].e[j] = from_float<T>(0.0f);
                }
                c[i][j] = i < count ? gate_weight<T>(to_float(f[i].e[j])) : -0.0f;   // no step
                sig[i][j] = GATE ? sigmoid<T>(to_float(o[i].e[j])) : 1.0f;
            }
    }
    // dL/dh_t without what comes from behind.
    auto into = [&](int i, int j) {
        const float d = to_float(dy[i].e[j]);
        return GATE ? d * (to_float(o[i].e[j]) * sig[i][j]) : d;
    };
    Map own[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float h = 0.0f;
        own[j] = {1.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kGradRun; ++i) {
            h = step(c[i][j], h, to_float(x[i].e[j]));
            own[j].a = keep(c[i][j], own[j].a);
        }
#pragma unroll
        for (int i = kGradRun - 1; i >= 0; --i) own[j].h = keep(c[i][j], own[j].h + into(i, j));
        s_maps[0][warp][lane * V + j] = own[j];
        s_h[warp][lane * V + j] = h;
    }
    __syncthreads();
    // h in front of this warp's run; the gradient's map of the warps behind it.  The last
    // warp to fold, of the chain's, is kWarps - 1: it takes the tile's map.
    Map behind[V], all[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        for (int w = 0; w < warp; ++w) before[j] = fmaf(s_maps[0][w][lane * V + j].a, before[j], s_h[w][lane * V + j]);
        behind[j] = {1.0f, 0.0f};
        for (int w = kWarps - 1; w > warp; --w) behind[j] = then(behind[j], s_maps[0][w][lane * V + j]);
        all[j] = own[j];
        if (warp == kWarps - 1)
            for (int w = kWarps - 2; w >= 0; --w) all[j] = then(all[j], s_maps[0][w][lane * V + j]);
    }
    float p[V];
    chain<V>(a, t, place, all, s_seed + lane * V, s_maps[1], p);
    if (count == 0) return;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = fmaf(behind[j].a, p[j], behind[j].h);

    float h[kGradRun + 1][V];   // in front of each token, and behind the last
#pragma unroll
    for (int j = 0; j < V; ++j) {
        h[0][j] = before[j];
#pragma unroll
        for (int i = 0; i < kGradRun; ++i) h[i + 1][j] = step(c[i][j], h[i][j], to_float(x[i].e[j]));
    }
    const Walk wx = walk(a, a.dx, t, k0, c0), wf = walk(a, a.dforget, t, k0, c0), wo = walk(a, a.dgate, t, k0, c0);
#pragma unroll
    for (int i = kGradRun - 1; i >= 0; --i) {
        float gx[V], gf[V], go[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float dh = p[j] + into(i, j), w = fabsf(c[i][j]);
            p[j] = keep(c[i][j], dh);
            gx[j] = dh * (keeps(c[i][j]) ? w : 1.0f - w);
            gf[j] = dh * (h[i][j] - to_float(x[i].e[j])) * fmaf(-w, w, w);
            const float g = to_float(o[i].e[j]), s = sig[i][j];
            go[j] = GATE ? to_float(dy[i].e[j]) * h[i + 1][j] * (s * fmaf(g, 1.0f - s, 1.0f)) : 0.0f;
        }
        if (i >= count) continue;
        auto store = [&](const Tokens &to, const Walk &w, const float (&v)[V]) {
            Access out;
            if constexpr (V == 1)
                out.e[0] = from_float<T>(v[0]);
            else
                set_pair(out, 0, make_float2(v[0], v[V - 1]));
            *(Access *)((T *)to.data + w.first + i * w.step) = out;
        };
        store(a.dx, wx, gx);
        store(a.dforget, wf, gf);
        if (GATE) store(a.dgate, wo, go);
    }
    if (t.index == 0 && warp == 0 && a.final)
#pragma unroll
        for (int j = 0; j < V; ++j) a.final[at_state + j] = p[j];
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

// Whether every array can be accessed in pairs of elements.
bool in_pairs(const RecurrenceArgs &a, int size)
{
    bool ok = a.channels % 2 == 0;
    for (const Tokens *t : {&a.x, &a.forget, &a.gate, &a.out, &a.dout, &a.dx, &a.dforget, &a.dgate})
        if (t->data)
            ok = ok && (uintptr_t)t->data % (2 * size) == 0 && (a.batch == 1 || t->batch % 2 == 0) &&
                 (a.tokens == 1 || t->token % 2 == 0);
    return ok;
}

template <typename T, int V, bool BACKWARD>
int run(gsr_ctx *ctx, RecurrenceArgs &a, cudaStream_t stream)
{
    const char *what = BACKWARD ? "gated recurrence backward" : "gated recurrence forward";
    constexpr int kTokens = BACKWARD ? kGradTile : kTile, kSlab = 32 * V;
    a.tiles = (a.tokens + kTokens - 1) / kTokens;
    if (a.tiles == 0) a.tiles = 1;   // for the states of items without tokens
    a.slabs = (a.channels + kSlab - 1) / kSlab;
    Workspace workspace(ctx, stream);
    if (a.tiles > 1) {
        const size_t chains = (size_t)a.batch * a.slabs, groups = (a.tiles + kGroup - 1) / kGroup;
        const size_t pairs = chains * a.tiles * kSlab * sizeof(unsigned long long);
        const size_t ends = chains * groups * kSlab * sizeof(unsigned long long), bytes = pairs + ends + 16;
        void *work = nullptr;
        if (int rc = workspace.take(bytes, &work)) return rc;
        if (int rc = cuda_check(ctx, cudaMemsetAsync(work, 0xff, bytes, stream), what)) return rc;
        a.pairs = (unsigned long long *)work;
        a.ends = a.pairs + pairs / sizeof(unsigned long long);
        a.ticket = (uint32_t *)((unsigned char *)work + pairs + ends);
        a.aborted = a.ticket + 1;
        a.status = ctx->status_dev;
    }
    void (*kernel)(RecurrenceArgs);
    if constexpr (BACKWARD)
        kernel = a.gate.data ? k_recurrence_grad<T, V, true> : k_recurrence_grad<T, V, false>;
    else
        kernel = a.gate.data ? k_recurrence<T, V, true> : k_recurrence<T, V, false>;
    const dim3 grid((unsigned)((int64_t)a.tiles * a.batch * a.slabs));
    if (int rc = cuda_check(ctx, launch_kernel(ctx, kernel, grid, kThreads, stream, a), what)) return rc;
    return workspace.done();
}

template <bool BACKWARD>
int dispatch(gsr_ctx *ctx, RecurrenceArgs &a, int dtype, cudaStream_t stream)
{
    const bool pairs = in_pairs(a, dtype == GSR_F32 ? 4 : 2);
    if (dtype == GSR_F32)
        return pairs ? run<float, 2, BACKWARD>(ctx, a, stream) : run<float, 1, BACKWARD>(ctx, a, stream);
    if (dtype == GSR_BF16)
        return pairs ? run<__nv_bfloat16, 2, BACKWARD>(ctx, a, stream) : run<__nv_bfloat16, 1, BACKWARD>(ctx, a, stream);
    return pairs ? run<__half, 2, BACKWARD>(ctx, a, stream) : run<__half, 1, BACKWARD>(ctx, a, stream);
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
