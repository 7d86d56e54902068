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
// Numerics.  With e = exp(-|f|), the larger of a and 1 - a is 1 / (1 + e) and the smaller
// e / (1 + e): neither is taken as a difference, so gates near 0 and 1 lose nothing.
#include <type_traits>

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
    uint32_t work;               // their number over all items
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

// Bits of a thread's elements of one token.
template <typename T, int V>
using Raw = std::conditional_t<sizeof(T) * V == 8, uint2, std::conditional_t<sizeof(T) * V == 4, uint32_t, uint16_t>>;

template <typename T, int V>
__device__ __forceinline__ Lanes<V> value_of(const Raw<T, V> &r)
{
    if constexpr (V == 1) {
        return to_float(*(const T *)&r);
    } else if constexpr (sizeof(T) == 4) {
        return make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
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
    } else if constexpr (sizeof(T) == 4) {
        return make_uint2(__float_as_uint(v.x), __float_as_uint(v.y));
    } else {
        return pack2<T>(v.x, v.y);
    }
}

__device__ __forceinline__ void clear(uint2 &r) { r = make_uint2(0, 0); }
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

template <int V>
struct Words {
    unsigned long long w[V];

    __device__ __forceinline__ static Words of(const Map<V> &m)
    {
        Words v;
#pragma unroll
        for (int j = 0; j < V; ++j)
            v.w[j] = (unsigned long long)__float_as_uint(at(m.h, j)) << 32 | __float_as_uint(at(m.a, j));
        return v;
    }
    __device__ __forceinline__ Map<V> map() const
    {
        Map<V> m;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            at(m.a, j) = __uint_as_float((uint32_t)w[j]);
            at(m.h, j) = __uint_as_float((uint32_t)(w[j] >> 32));
        }
        return m;
    }
};

// ---- the chain ---------------------------------------------------------------------------

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

// The n-th tile in the order of the chains.
__device__ __forceinline__ Tile tile_at(const RecurrenceArgs &a, uint32_t n, int tile_tokens, bool backward)
{
    Tile t;
    const uint32_t chains = (uint32_t)a.batch * a.slabs, place = n / chains, chain = n - place * chains;
    t.b = chain / a.slabs;
    t.slab = chain - t.b * a.slabs;
    t.index = backward ? a.tiles - 1 - (int)place : (int)place;
    t.length = a.lengths ? min(max(a.lengths[t.b], 0), a.tokens) : a.tokens;
    t.count = (t.length + tile_tokens - 1) / tile_tokens;
    return t;
}

// The state in front of a chain, read by the warp that publishes the first tile's map
// and handed to the others: once that map is out, nobody reads the array, in which a
// block may write the state behind the chain.
template <int V>
__device__ __forceinline__ void load_seed(const RecurrenceArgs &a, int warp, bool here, int64_t from, Lanes<V> *seed)
{
    if (warp != kWarps - 1) return;
#pragma unroll
    for (int j = 0; j < V; ++j) at(*seed, j) = here && a.initial ? a.initial[from + j] : 0.0f;
}

template <int V>
__device__ __forceinline__ void store_state(float *to, const Lanes<V> &v)
{
#pragma unroll
    for (int j = 0; j < V; ++j) to[j] = at(v, j);
}

// The state in front of the block's tile, for this lane's channels.  `tile_map`: the
// tile's own map (warp kWarps - 1 has it); `seed`: the state in front of the first tile (0 for others).
// place: the tile's in its chain of t.count.
template <int V>
__device__ __forceinline__ Lanes<V> chain(const RecurrenceArgs &a, const Tile &t, int place, const Map<V> &tile_map,
                                          const Lanes<V> &seed, Map<V> (*s_maps)[32])
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (t.count == 1) return seed;
    const int64_t row = (int64_t)t.b * a.slabs + t.slab;
    const int groups = (a.tiles + kGroup - 1) / kGroup, group = place / kGroup;
    unsigned long long *pairs = a.pairs + row * a.tiles * (32 * V) + lane * V;
    unsigned long long *ends = a.ends + row * groups * (32 * V) + lane * V;
    if (warp == kWarps - 1 && place + 1 < t.count) {
        Map<V> m = tile_map;
        if (place == 0) {   // as a map of no state
            m.h = mad(m.a, seed, m.h);
            fill(m.a, 0.0f);
        }
        publish(pairs + (int64_t)place * (32 * V), Words<V>::of(m));
    }
    if (place == 0) return seed;
    // Each warp folds four tiles of the group; the first one behind the group's start.
    Map<V> m;
    fill(m.a, 1.0f);
    fill(m.h, 0.0f);
    const int first = group * kGroup + 4 * warp;
    Words<V> seen[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i < place) look(pairs + (int64_t)(first + i) * (32 * V), seen[i]);
    if (warp == 0 && group > 0) {
        Words<V> end;
        look(ends + (int64_t)group * (32 * V), end);
        wait_for(a, ends + (int64_t)group * (32 * V), end);
        m = end.map();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i < place) {
            wait_for(a, pairs + (int64_t)(first + i) * (32 * V), seen[i]);
            m = then(m, seen[i].map());
        }
    s_maps[warp][lane] = m;
    __syncthreads();
    Lanes<V> state;
    fill(state, 0.0f);   // (the first map of a chain takes no state)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const Map<V> v = s_maps[w][lane];
        state = mad(v.a, state, v.h);
    }
    if (warp == kWarps - 1 && place % kGroup == kGroup - 1 && place + 1 < t.count) {
        fill(m.a, 0.0f);
        m.h = mad(tile_map.a, state, tile_map.h);
        publish(ends + (int64_t)(group + 1) * (32 * V), Words<V>::of(m));
    }
    return state;
}

// ---- runs of tokens ------------------------------------------------------------------------

// A warp's run of an array: a lane's elements of token after token, in the recurrence's
// order.
template <typename T, int V>
struct Run {
    using R = Raw<T, V>;
    T *at;
    int64_t step;

    __device__ __forceinline__ Run(const RecurrenceArgs &a, const Tokens &t, const Tile &tile, int k, int c)
    {
        at = (T *)t.data + tile.b * t.batch + (int64_t)(a.reverse ? tile.length - 1 - k : k) * t.token + c;
        step = a.reverse ? -t.token : t.token;
    }
    // N tokens of which `count` (the same in a warp) are there; the others as 0.
    template <int N>
    __device__ __forceinline__ void load(R (&r)[N], int count) const
    {
        const T *p = at;
        if (count == N) {
#pragma unroll
            for (int i = 0; i < N; ++i, p += step) r[i] = *(const R *)p;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i, p += step) {
                clear(r[i]);
                if (i < count) r[i] = *(const R *)p;
            }
        }
    }
    __device__ __forceinline__ void store(int i, const Lanes<V> &v) const { *(R *)(at + i * step) = raw_of<T, V>(v); }
};

template <typename T, int V>
__device__ __forceinline__ void clear_tokens(const Tokens &t, int b, int from, int to, int c)
{
    Raw<T, V> zero;
    clear(zero);
    T *p = (T *)t.data + b * t.batch + (int64_t)from * t.token + c;
    for (int k = from; k < to; ++k, p += t.token) *(Raw<T, V> *)p = zero;
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
    const float e = exp_minus<T>(fabsf(f)), large = rcp_fast(1.0f + e), small = e * large;
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

// Walks the block's tiles: its own, or tickets as long as there are some.  The next
// ticket is asked for while a tile is worked on.
template <typename F>
__device__ __forceinline__ void for_tiles(const RecurrenceArgs &a, F f)
{
    if (!a.ticket) {
        f(blockIdx.x);
        return;
    }
    __shared__ uint32_t s_ticket[2];
    uint32_t next = 0;
    if (threadIdx.x == 0) next = atomicAdd(a.ticket, 1u) + 1u;
    for (int turn = 0;; turn ^= 1) {
        if (threadIdx.x == 0) s_ticket[turn] = next;
        __syncthreads();   // (also: the last tile's shared memory has been read)
        const uint32_t n = s_ticket[turn];
        if (n >= a.work) return;
        if (threadIdx.x == 0) next = atomicAdd(a.ticket, 1u) + 1u;
        f(n);
    }
}

// ---- forward -----------------------------------------------------------------------------

template <typename T, int V, bool GATE>
__device__ __forceinline__ void forward_tile(const RecurrenceArgs &a, const Tile &t, Map<V> (*s_maps)[kWarps][32],
                                             Lanes<V> *s_seed)
{
    using F = Lanes<V>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int own_c = t.slab * (32 * V) + lane * V, c = min(own_c, a.channels - V);
    const bool mine = own_c == c;   // (other lanes compute the last one's channels)
    const int k0 = t.index * kTile + warp * kRun, count = min(max(t.length - k0, 0), kRun);
    if (mine) clear_tokens<T, V>(a.out, t.b, max(k0, t.length), min(k0 + kRun, a.tokens), c);
    const int64_t at_state = (int64_t)t.b * a.channels + c;
    load_seed<V>(a, warp, t.index == 0, at_state, s_seed + lane);
    if (t.index >= t.count) {
        if (t.length == 0 && t.index == 0 && warp == kWarps - 1 && mine) store_state<V>(a.final + at_state, s_seed[lane]);
        return;
    }

    F keep[kRun], enter[kRun];   // a and (1 - a) x
    Raw<T, V> o[kRun];
    {
        Raw<T, V> x[kRun], f[kRun];
        Run<T, V>(a, a.forget, t, k0, c).load(f, count);
        Run<T, V>(a, a.x, t, k0, c).load(x, count);
        if (GATE) Run<T, V>(a, a.gate, t, k0, c).load(o, count);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            F s;
            split<T>(value_of<T, V>(f[i]), keep[i], s);
            enter[i] = mul(s, value_of<T, V>(x[i]));
        }
        if (count < kRun)
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (i >= count) {   // no step
                    fill(keep[i], 1.0f);
                    fill(enter[i], 0.0f);
                }
    }
    Map<V> own;
    fill(own.a, 1.0f);
    fill(own.h, 0.0f);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        own.h = mad(keep[i], own.h, enter[i]);
        own.a = mul(keep[i], own.a);
    }
    s_maps[0][warp][lane] = own;
    __syncthreads();
    // The warps in front of this one, and with them the tile's map in the last warp.
    Map<V> before;
    fill(before.a, 1.0f);
    fill(before.h, 0.0f);
    for (int w = 0; w < warp; ++w) before = then(before, s_maps[0][w][lane]);
    F h = chain<V>(a, t, t.index, then(before, own), s_seed[lane], s_maps[1]);
    h = mad(before.a, h, before.h);
    if (count == 0 || !mine) return;

    if (a.states && k0 % kStateStep == 0)
        store_state<V>(a.states + ((int64_t)t.b * a.blocks + k0 / kStateStep) * a.channels + c, h);
    const Run<T, V> out(a, a.out, t, k0, c);
    auto token = [&](int i) {
        h = mad(keep[i], h, enter[i]);
        if constexpr (GATE) {
            const F g = value_of<T, V>(o[i]);
            return mul(h, mul(g, sigmoid<T>(g)));
        } else {
            return h;
        }
    };
    if (count == kRun) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) out.store(i, token(i));
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const F y = token(i);
            if (i < count) out.store(i, y);
        }
    }
    if (k0 + kRun >= t.length) store_state<V>(a.final + at_state, h);
}

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, 2) k_recurrence(const RecurrenceArgs a)
{
    grid_dependency_begin();
    __shared__ Map<V> s_maps[2][kWarps][32];
    __shared__ Lanes<V> s_seed[32];
    for_tiles(a, [&](uint32_t n) { forward_tile<T, V, GATE>(a, tile_at(a, n, kTile, false), s_maps, s_seed); });
}

// ---- backward ----------------------------------------------------------------------------

template <typename T, int V, bool GATE>
__device__ __forceinline__ void backward_tile(const RecurrenceArgs &a, const Tile &t, Map<V> (*s_maps)[kWarps][32],
                                              Lanes<V> (*s_h)[32], Lanes<V> *s_seed)
{
    using F = Lanes<V>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int own_c = t.slab * (32 * V) + lane * V, c = min(own_c, a.channels - V);
    const bool mine = own_c == c;
    const int k0 = t.index * kGradTile + warp * kGradRun, count = min(max(t.length - k0, 0), kGradRun);
    if (mine) {
        const int from = max(k0, t.length), to = min(k0 + kGradRun, a.tokens);
        clear_tokens<T, V>(a.dx, t.b, from, to, c);
        clear_tokens<T, V>(a.dforget, t.b, from, to, c);
        if (GATE) clear_tokens<T, V>(a.dgate, t.b, from, to, c);
    }
    const int64_t at_state = (int64_t)t.b * a.channels + c;
    const int place = t.count - 1 - t.index;   // in the chain, which starts at the last token
    load_seed<V>(a, warp, place == 0 || t.length == 0, at_state, s_seed + lane);
    if (place < 0) {
        if (t.length == 0 && t.index == 0 && warp == kWarps - 1 && mine && a.final)
            store_state<V>(a.final + at_state, s_seed[lane]);
        return;
    }

    // dout silu(o): dL/dh_t without what comes from behind; dout silu'(o).
    F keep[kGradRun], rest[kGradRun], into[kGradRun], slope[kGradRun], before;
    Raw<T, V> x[kGradRun];
    {
        Raw<T, V> f[kGradRun], dy[kGradRun], o[kGradRun];
        Run<T, V>(a, a.forget, t, k0, c).load(f, count);
        Run<T, V>(a, a.x, t, k0, c).load(x, count);
        Run<T, V>(a, a.dout, t, k0, c).load(dy, count);
        if (GATE) Run<T, V>(a, a.gate, t, k0, c).load(o, count);
#pragma unroll
        for (int j = 0; j < V; ++j)
            at(before, j) = a.states[((int64_t)t.b * a.blocks + t.index) * a.channels + c + j];
#pragma unroll
        for (int i = 0; i < kGradRun; ++i) {
            split<T>(value_of<T, V>(f[i]), keep[i], rest[i]);
            const F d = value_of<T, V>(dy[i]);
            if constexpr (GATE) {
                const F g = value_of<T, V>(o[i]), s = sigmoid<T>(g);
                into[i] = mul(d, mul(g, s));
                F one;
                fill(one, 1.0f);
                slope[i] = mul(d, mul(s, mad(g, mad(minus(s), one, one), one)));
            } else {
                into[i] = d;
            }
        }
        if (count < kGradRun)
#pragma unroll
            for (int i = 0; i < kGradRun; ++i)
                if (i >= count) {   // no step (its x and dout are 0)
                    fill(keep[i], 1.0f);
                    fill(rest[i], 0.0f);
                }
    }
    Map<V> own;
    F h;
    fill(h, 0.0f);
    fill(own.a, 1.0f);
    fill(own.h, 0.0f);
#pragma unroll
    for (int i = 0; i < kGradRun; ++i) {
        h = mad(keep[i], h, mul(rest[i], value_of<T, V>(x[i])));
        own.a = mul(keep[i], own.a);
    }
#pragma unroll
    for (int i = kGradRun - 1; i >= 0; --i) own.h = mul(keep[i], add(own.h, into[i]));
    s_maps[0][warp][lane] = own;
    s_h[warp][lane] = h;
    __syncthreads();
    // h in front of this warp's run, and the gradient's map of the warps behind it; the
    // tile's map in the warp that publishes.
    for (int w = 0; w < warp; ++w) before = mad(s_maps[0][w][lane].a, before, s_h[w][lane]);
    Map<V> behind, all = own;
    fill(behind.a, 1.0f);
    fill(behind.h, 0.0f);
    for (int w = kWarps - 1; w > warp; --w) behind = then(behind, s_maps[0][w][lane]);
    if (warp == kWarps - 1)
        for (int w = kWarps - 2; w >= 0; --w) all = then(all, s_maps[0][w][lane]);
    F p = chain<V>(a, t, place, all, s_seed[lane], s_maps[1]);
    if (count == 0 || !mine) return;
    p = mad(behind.a, p, behind.h);

    F hs[kGradRun + 1];   // in front of each token, and behind the last
    hs[0] = before;
#pragma unroll
    for (int i = 0; i < kGradRun; ++i) hs[i + 1] = mad(keep[i], hs[i], mul(rest[i], value_of<T, V>(x[i])));
    const Run<T, V> dx(a, a.dx, t, k0, c), df(a, a.dforget, t, k0, c), dg(a, a.dgate, t, k0, c);
    auto token = [&](int i, bool there) {
        const F dh = add(p, into[i]);
        p = mul(keep[i], dh);
        if (!there) return;
        const F enter = mul(dh, rest[i]);
        dx.store(i, enter);
        df.store(i, mul(mul(enter, keep[i]), add(hs[i], minus(value_of<T, V>(x[i])))));
        if constexpr (GATE) dg.store(i, mul(slope[i], hs[i + 1]));
    };
    if (count == kGradRun) {
#pragma unroll
        for (int i = kGradRun - 1; i >= 0; --i) token(i, true);
    } else {
#pragma unroll
        for (int i = kGradRun - 1; i >= 0; --i) token(i, i < count);
    }
    if (k0 == 0 && a.final) store_state<V>(a.final + at_state, p);
}

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(kThreads, 2) k_recurrence_grad(const RecurrenceArgs a)
{
    grid_dependency_begin();
    __shared__ Map<V> s_maps[2][kWarps][32];
    __shared__ Lanes<V> s_h[kWarps][32], s_seed[32];
    for_tiles(a, [&](uint32_t n) { backward_tile<T, V, GATE>(a, tile_at(a, n, kGradTile, true), s_maps, s_h, s_seed); });
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
    a.work = (uint32_t)a.tiles * a.batch * a.slabs;
    const uint32_t most = a.tiles > 1 ? 2u * ctx->num_sms : a.work;
    const dim3 grid(a.work < most ? a.work : most);
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
