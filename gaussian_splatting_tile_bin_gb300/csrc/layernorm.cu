// layernorm.cu -- layer norm over the channels of a row (a token, or a head of a
// token) behind a residual sum, forward and backward.
//
//   total = x + residual,  xh = (total - mean) rstd,  out = xh w + b
// and with g = dout w
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dtotal,  dw = sum dout xh,  db = sum dout.
//
// Bound by HBM.  A row stays in the registers of its team (lanes of a warp, a warp,
// several or two blocks) between the statistics and the result, so every array moves once; a block
// walks rows, and its threads' copies run two or three rows ahead, so that the parameters and,
// backward, the channels' shares of dw and db stay in registers too.  A second kernel adds
// the blocks' shares in order.  32,640 x 2,048 in bf16 behind a residual (four arrays of 134
// MB each way, 79 us at the copy rate): forward 88 us, backward 83 us; without one 42 us of
// 39 and 67 us of 59.  Rows of 128 in f16 (80,000): 6.7 us of 6.0 and 12.3 us of 9.0, of
// which the second kernel's launch is about 3.  Channels that are no multiple of 16 bytes
// take accesses of 4 bytes or one element: 32,640 rows behind a residual in 114 and 141 us at
// 2,050, 183 and 177 at 2,049, bound by the number of accesses.  Rows of more than 8,192
// channels are shared by two blocks (4,000 x 16,384 in bf16: 65 us of 39 and 88 of 58, for what
// sums cost between warps with one row at a time).
//
// Numerics.  The variance is the mean of centred squares, from the registers; sums over
// a row pass a thread's elements and a tree, in a fixed order, all in float.  The norm of a
// sum is that of the rounded sum, which the backward reads.
#include <algorithm>
#include <type_traits>

#include "tensor.cuh"

namespace gsr {
namespace {

constexpr int kRowThreads = 512;   // of a block, one to an SM
// Elements of a thread: parameters, their gradients' sums and a row's inputs stay in
// registers (8 in two blocks an SM: 80,000 x 128 in f16 in 10.2 and 24 us, 6.7 and 12.3 with
// 16; 100,000 x 256 in bf16 in 23 us forward, 15).
constexpr int kElements = 16;

// The rows of one [batch, tokens, heads, channels] array.
struct Rows {
    void *data;
    int64_t batch, token, head;
};

struct LayerArgs {
    Rows x, residual, out, total;   // backward: dout, dtotal, dx, total
    const float *weight, *bias;
    float *mean, *rstd, *dweight, *dbias;
    float2 *partial;                // [blocks, channels]: (sum dout xh, sum dout)
    int batch, tokens, heads, channels;
    uint32_t rows;
    int team;                       // threads of a row
    int blocks;                     // (or pairs of them)
    float eps;
    uint32_t *status;
};

// A row's first element.  `flat`: the rows lie at one stride (one item of one head).
template <typename T>
__device__ __forceinline__ T *row_of(const LayerArgs &a, const Rows &r, uint32_t row, bool flat)
{
    if (flat) return (T *)r.data + row * r.token;
    const uint32_t token = row / (uint32_t)a.heads, item = token / (uint32_t)a.tokens;
    return (T *)r.data + item * r.batch + (token - item * (uint32_t)a.tokens) * r.token +
           (row - token * (uint32_t)a.heads) * r.head;
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w)
{
    return __half22float2(*(const __half2 *)&w);
}

// A thread's elements of a row: N accesses of V, `team` threads apart, taken in pairs.
template <typename T, int V, int N>
struct Part {
    Vec<T, V> v[N];
    static constexpr int kPairs = N * V / 2;
    static_assert(N * V % 2 == 0, "elements come in pairs");

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i].e[j] = from_float<T>(0.0f);
    }
    __device__ __forceinline__ void load(const T *row, const LayerArgs &a, int lane)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * a.team + lane) * V;
            if (c < a.channels) v[i] = *(const Vec<T, V> *)(row + c);
        }
    }
    __device__ __forceinline__ void store(T *row, const LayerArgs &a, int lane) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * a.team + lane) * V;
            if (c < a.channels) *(Vec<T, V> *)(row + c) = v[i];
        }
    }
    __device__ __forceinline__ float2 get(int p) const
    {
        if constexpr (V == 1)
            return make_float2(to_float(v[2 * p].e[0]), to_float(v[(2 * p + 1) % N].e[0]));
        else if constexpr (sizeof(T) == 2)
            return unpack2<T>(((const uint32_t *)&v[p / (V / 2)])[p % (V / 2)]);
        else
            return pair_of(v[p / (V / 2)], p % (V / 2) * 2);
    }
    __device__ __forceinline__ void set(int p, float2 f)
    {
        if constexpr (V == 1) {
            v[2 * p].e[0] = from_float<T>(f.x);
            v[(2 * p + 1) % N].e[0] = from_float<T>(f.y);
        } else {
            set_pair(v[p / (V / 2)], p % (V / 2) * 2, f);
        }
    }
};

// The first channel of a pair, and of its second half.
template <int V>
__device__ __forceinline__ int pair_channel(const LayerArgs &a, int lane, int p, int half)
{
    if (V == 1) return (2 * p + half) * a.team + lane;
    return (p / ((V + 1) / 2) * a.team + lane) * V + p % ((V + 1) / 2) * 2 + half;
}

// A pair of a parameter; `missing` where there is none, 0 behind the channels.
template <int V>
__device__ __forceinline__ float2 parameter(const float *from, const LayerArgs &a, int lane, int p, float missing)
{
    const int c0 = pair_channel<V>(a, lane, p, 0), c1 = pair_channel<V>(a, lane, p, 1);
    float2 f = make_float2(0.0f, 0.0f);
    if constexpr (V > 1) {
        if (c0 < a.channels) f = from ? *(const float2 *)(from + c0) : make_float2(missing, missing);
    } else {
        if (c0 < a.channels) f.x = from ? from[c0] : missing;
        if (c1 < a.channels) f.y = from ? from[c1] : missing;
    }
    return f;
}

// Teams: lanes of a warp, a block's warps, or, for rows of more than 8,192 channels, those of
// two blocks of a cluster (4,000 x 16,384 in bf16 behind a residual in 84 us forward and 102
// backward, without one 65 and 88; a block of 1,024 threads, which has 64 registers a thread
// and spills, took 118 and 231, 66 and 212.  It was faster forward for 5,000 x 9,000 without a
// residual, 63 and 69, and for the single elements of 4,000 x 12,345, 141 and 166).
constexpr int kInWarp = 0, kInBlock = 1, kInTwo = 2;
template <int KIND>
constexpr int kBlocksOf = KIND == kInTwo ? 2 : 1;   // a team's

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// Of a block whose rows another one of its cluster shares.
struct Beside {
    uint64_t full[2];   // the other's sums are there, for either copy
    uint32_t aborted;
};

// Writes to the cluster's other block, where this one's `at` is, and counts the bytes at
// its `bar`.  (No fence: one would wait for the row's stores too, 0.6 us.)
__device__ __forceinline__ uint32_t beside(const void *at)
{
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_address(at)), "r"(blockIdx.x % 2 ^ 1));
    return to;
}
__device__ __forceinline__ void store_beside(const float *at, float v, const uint64_t *bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(beside(at)), "f"(v),
                 "r"(beside(bar))
                 : "memory");
}
__device__ __forceinline__ void store_beside(const float2 *at, float2 v, const uint64_t *bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(beside(at)),
                 "f"(v.x), "f"(v.y), "r"(beside(bar))
                 : "memory");
}

// Sums of a team (of one float or two).  Teams up to a warp: by shuffles.  Wider ones
// meet at a barrier of their own, over shared memory in two copies, so that one
// barrier a sum is enough.  Two blocks write their warps' sums to each other: a copy is
// written again once the other block has all of the sum in between, so behind its reads.
__device__ __forceinline__ void add_lane(float &v, int d) { v += __shfl_xor_sync(~0u, v, d); }
__device__ __forceinline__ void add_lane(float2 &v, int d)
{
    add_lane(v.x, d);
    add_lane(v.y, d);
}
__device__ __forceinline__ float four(const float4 *s) { return s->x + s->y + (s->z + s->w); }
__device__ __forceinline__ float2 four(const float2 (*s)[4])
{
    return make_float2((*s)[0].x + (*s)[1].x + ((*s)[2].x + (*s)[3].x), (*s)[0].y + (*s)[1].y + ((*s)[2].y + (*s)[3].y));
}

__device__ __forceinline__ void team_barrier(int team, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// s_sums: the team's [2][kTeamWarps], 0 behind its warps; turn: which copy.
constexpr int kTeamWarps = 32;

template <int KIND, typename F>
__device__ __forceinline__ F team_sum(F v, const LayerArgs &a, float2 *s_sums, int team, uint32_t &turn, Beside &s_beside)
{
    if constexpr (KIND == kInWarp) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
            if (d < a.team) add_lane(v, d);
    } else {
        using Four = std::conditional_t<std::is_same_v<F, float>, float4, float2[4]>;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) add_lane(v, d);
        const uint32_t copy = turn & 1, parity = turn >> 1 & 1;
        F *s = (F *)(s_sums + copy * kTeamWarps);
        ++turn;
        const int warps = a.team / 32;
        if constexpr (KIND == kInTwo) {
            // (Once a wait has run out the barriers are left as they are, here and, for want
            // of this block's sums, in the other block.)
            const WaitGuard guard = {&s_beside.aborted, a.status};
            uint64_t *full = &s_beside.full[copy];
            GSR_CANARY(38 + copy);
            if (threadIdx.x % 32 == 0 && !guard.stop()) {
                if (threadIdx.x == 0) barrier_expect(smem_address(full), blockDim.x / 32 * sizeof(F));
                F *at = s + (blockIdx.x % 2 * blockDim.x + threadIdx.x) / 32;
                *at = v;
                store_beside(at, v, full);
            }
            __syncthreads();
            barrier_wait_warp(smem_address(full), parity, guard);
            GSR_CANARY(40 + copy);
        } else {
            GSR_CANARY(52 + copy);
            if (threadIdx.x % 32 == 0) s[threadIdx.x / 32 - team * warps] = v;
            team_barrier(team, a.team);
            GSR_CANARY(54 + copy);
        }
        v = four((const Four *)s);
        for (int w = 4; w < warps; w += 4) {
            const F more = four((const Four *)(s + w));
            if constexpr (std::is_same_v<F, float>)
                v += more;
            else
                v = add2(v, more);
        }
    }
    return v;
}

// Clears the sums of the warps that a block's teams do not have.
template <int KIND>
__device__ __forceinline__ void start_sums(float2 *s_all, int teams, Beside &s_beside)
{
    if constexpr (KIND != kInWarp)
        for (int i = threadIdx.x; i < teams * 2 * kTeamWarps; i += blockDim.x) s_all[i] = make_float2(0.0f, 0.0f);
    if constexpr (KIND == kInTwo) {
        if (threadIdx.x == 0) {
            s_beside.aborted = 0;
            for (uint64_t &full : s_beside.full) barrier_init(smem_address(&full), 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        cluster_barrier();
    } else if constexpr (KIND == kInBlock) {
        __syncthreads();
    }
}

// A block leaves once the other one writes to it no more.
template <int KIND>
__device__ __forceinline__ void end_sums(const LayerArgs &a, Beside &s_beside)
{
    if constexpr (KIND == kInTwo) {
        drain_if_aborted({&s_beside.aborted, a.status});
        cluster_barrier();
    }
}

// ---- rows in flight --------------------------------------------------------------------

// A block walks rows, `teams` at a time, and every thread's elements of the next ones
// come through a ring of its own in shared memory (asynchronous copies; no thread
// waits for another): S stages of A arrays, three (two are slower without a residual, 44.1
// to 41.8 us for 32,640 x 2,048 in bf16, four and eight no faster) or what 200 KB hold.  Single elements of
// 2 bytes have no such copies and are read directly (S = 0).
template <typename T, int V, int N, int A>
constexpr int kStages = sizeof(T) * V < 4
                            ? 0
                            : std::min(3, 200 * 1024 / (kRowThreads * A * N * V * (int)sizeof(T)));

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

template <typename T, int V, int N, int A, int S>
struct Ring {
    using Access = Vec<T, V>;
    static constexpr int kStage = A * N * kRowThreads;
    Access *mine;          // the thread's first slot
    const Rows &r0, &r1, &r2;
    bool flat;
    int at = 0;            // of the current stage's first slot

    __device__ __forceinline__ const Rows &array(int k) const { return k == 0 ? r0 : k == 1 ? r1 : r2; }
    __device__ __forceinline__ Access *slot(int k, int i) const { return mine + at + (k * N + i) * kRowThreads; }
    // Starts the copies of a row into the current stage, if there is such a row.
    __device__ __forceinline__ void fetch(const LayerArgs &a, uint32_t row, int lane) const
    {
        if constexpr (S > 0) {
            if (row < a.rows) {
#pragma unroll
                for (int k = 0; k < A; ++k) {
                    const T *from = row_of<T>(a, array(k), row, flat);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int c = (i * a.team + lane) * V;
                        if (c < a.channels) copy_async<sizeof(Access)>(slot(k, i), from + c);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    __device__ __forceinline__ void advance() { at = at + kStage >= S * kStage ? 0 : at + kStage; }
    // Slots behind the channels are 0 from here on.
    __device__ __forceinline__ void start(const LayerArgs &a, uint32_t row, uint32_t stride, int lane)
    {
        for (int k = 0; k < S; ++k) {
            for (int i = 0; i < A * N; ++i)
                if (((i % N) * a.team + lane) * V >= a.channels) *slot(0, i) = Access{};
            fetch(a, row + k * stride, lane);
            advance();
        }
    }
    // The oldest row's elements.  Its stage is free once they have been used.
    __device__ __forceinline__ void take(const LayerArgs &a, uint32_t row, int lane, Part<T, V, N> (&to)[A]) const
    {
        if constexpr (S > 0) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S > 0 ? S - 1 : 0) : "memory");
#pragma unroll
            for (int k = 0; k < A; ++k)
#pragma unroll
                for (int i = 0; i < N; ++i) to[k].v[i] = *slot(k, i);
        } else {
#pragma unroll
            for (int k = 0; k < A; ++k) {
                to[k].clear();
                if (row < a.rows) to[k].load(row_of<T>(a, array(k), row, flat), a, lane);
            }
        }
    }
    // Waits for the copies of rows behind the last.
    __device__ __forceinline__ void finish() const
    {
        if constexpr (S > 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
};

// ---- forward ------------------------------------------------------------------------

// A row's centred squares meet with the next one's sum, so that a team meets once a row (in
// bf16, behind a residual: 21,845 x 3,000 in 83 us, with two meetings 106; 13,107 x 5,000 in
// 96 and 123; x 4,096, x 8,192 and x 2,048 within 10% either way, as DRAM takes four streams;
// without one 8,000 x 8,192 in 51 and 64).  Behind a residual, where the next row is in
// registers, two stages of the ring do.
template <typename T, int V, int N, int A>
constexpr int kForwardStages = std::min(kStages<T, V, N, A>, A > 1 ? 2 : 3);

template <typename T, int V, int N, int KIND, bool SUM>
__global__ void __launch_bounds__(kRowThreads, 1) k_layer_norm(const LayerArgs a)
{
    grid_dependency_begin();
    extern __shared__ __align__(16) unsigned char s_bytes[];   // the teams' sums, then the ring
    __shared__ Beside s_beside;
    using Elements = Part<T, V, N>;
    constexpr int kPairs = Elements::kPairs, A = SUM ? 2 : 1, S = kForwardStages<T, V, N, A>, X = kBlocksOf<KIND>;
    const bool flat = a.batch == 1 && a.heads == 1;
    const int teams = X * blockDim.x / a.team, team = threadIdx.x / a.team;
    const int lane = KIND == kInTwo ? blockIdx.x % 2 * blockDim.x + threadIdx.x : threadIdx.x % a.team;
    const uint32_t block = blockIdx.x / X, stride = gridDim.x / X * (uint32_t)teams;
    float2 *s_sums = (float2 *)s_bytes + team * 2 * kTeamWarps;
    const size_t sum_bytes = KIND != kInWarp ? teams * 2 * kTeamWarps * sizeof(float2) : 0;
    Ring<T, V, N, A, S> ring = {(Vec<T, V> *)(s_bytes + sum_bytes) + threadIdx.x, a.x, a.residual, a.residual, flat};

    // (Below 2^31 rows, steps ahead of them below 2^32.  All teams take the same number of steps.)
    uint32_t row = block * teams + team, first = block * teams;
    ring.start(a, row, stride, lane);
    start_sums<KIND>((float2 *)s_bytes, teams, s_beside);
    float2 weight[kPairs], bias[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        weight[p] = parameter<V>(a.weight, a, lane, p, 1.0f);
        bias[p] = parameter<V>(a.bias, a, lane, p, 0.0f);
    }
    const float share = 1.0f / (float)a.channels;
    const bool full = a.channels == a.team * V * N;
    uint32_t turn = 0;
    // A row's total (stored where its squares are taken) and a thread's share of its sum.
    auto take = [&](uint32_t from, Elements &x) {
        Elements in[A];
        ring.take(a, from, lane, in);
        x = in[0];
        if constexpr (SUM) {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) x.set(p, add2(x.get(p), in[A - 1].get(p)));
        }
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < kPairs; ++p) sum = add2(sum, x.get(p));
        ring.fetch(a, from + S * stride, lane);
        ring.advance();
        return sum.x + sum.y;
    };
    Elements x;
    float mean = team_sum<KIND>(take(row, x), a, s_sums, team, turn, s_beside) * share;
    for (; first < a.rows; first += stride, row += stride) {
        const float2 minus = make_float2(-mean, -mean);
        float2 f[kPairs], sum = make_float2(0.0f, 0.0f);
        if (full) {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                f[p] = add2(x.get(p), minus);
                sum = fma2(f[p], f[p], sum);
            }
        } else {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                f[p] = add2(x.get(p), minus);
                if (pair_channel<V>(a, lane, p, 0) >= a.channels) f[p].x = 0.0f;
                if (pair_channel<V>(a, lane, p, 1) >= a.channels) f[p].y = 0.0f;
                sum = fma2(f[p], f[p], sum);
            }
        }
        float2 sums = make_float2(sum.x + sum.y, 0.0f);
        if (SUM && row < a.rows) x.store(row_of<T>(a, a.total, row, flat), a, lane);
        if (first + stride < a.rows) sums.y = take(row + stride, x);
        sums = team_sum<KIND>(sums, a, s_sums, team, turn, s_beside);
        const float rstd = rsqrtf(sums.x * share + a.eps);
        if (row < a.rows) {
            const float2 scale = make_float2(rstd, rstd);
            Elements y;
#pragma unroll
            for (int p = 0; p < kPairs; ++p) y.set(p, fma2(mul2(f[p], scale), weight[p], bias[p]));
            y.store(row_of<T>(a, a.out, row, flat), a, lane);
            if (lane == 0) {
                a.mean[row] = mean;
                a.rstd[row] = rstd;
            }
        }
        mean = sums.y * share;
    }
    ring.finish();
    end_sums<KIND>(a, s_beside);
}

// ---- backward -----------------------------------------------------------------------

template <typename T, int V, int N, int KIND, bool SUM>
__global__ void __launch_bounds__(kRowThreads, 1) k_layer_norm_grad(const LayerArgs a)
{
    grid_dependency_begin();
    // The teams' sums, then the ring; at the end the block's shares of dw and db.
    extern __shared__ __align__(16) unsigned char s_bytes[];
    __shared__ Beside s_beside;
    float2 *s_work = (float2 *)s_bytes;
    using Elements = Part<T, V, N>;
    constexpr int kPairs = Elements::kPairs, A = SUM ? 3 : 2, S = kStages<T, V, N, A>, X = kBlocksOf<KIND>;
    const bool flat = a.batch == 1 && a.heads == 1;
    const int teams = X * blockDim.x / a.team, team = threadIdx.x / a.team;
    const int lane = KIND == kInTwo ? blockIdx.x % 2 * blockDim.x + threadIdx.x : threadIdx.x % a.team;
    const uint32_t block = blockIdx.x / X, stride = gridDim.x / X * (uint32_t)teams;
    float2 *s_sums = s_work + team * 2 * kTeamWarps;
    const size_t sum_bytes = KIND != kInWarp ? teams * 2 * kTeamWarps * sizeof(float2) : 0;
    Ring<T, V, N, A, S> ring = {(Vec<T, V> *)(s_bytes + sum_bytes) + threadIdx.x, a.total, a.x, a.residual, flat};

    // (As in the forward.)
    uint32_t row = block * teams + team, first = block * teams;
    ring.start(a, row, stride, lane);
    start_sums<KIND>((float2 *)s_bytes, teams, s_beside);
    float2 weight[kPairs], dw[kPairs], db[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        weight[p] = parameter<V>(a.weight, a, lane, p, 1.0f);
        dw[p] = db[p] = make_float2(0.0f, 0.0f);
    }
    const float share = 1.0f / (float)a.channels;
    uint32_t turn = 0;
    float mean = row < a.rows ? a.mean[row] : 0.0f, rstd = row < a.rows ? a.rstd[row] : 0.0f;
    for (; first < a.rows; first += stride, row += stride) {
        Elements in[A];
        ring.take(a, row, lane, in);
        Elements &total = in[0], &dout = in[1];
        const float2 minus = make_float2(-mean, -mean), scale = make_float2(rstd, rstd);
        const uint32_t after = row + stride;
        if (after < a.rows) {
            mean = a.mean[after];
            rstd = a.rstd[after];
        } else {
            mean = rstd = 0.0f;
        }
        if (row >= a.rows) {   // (its stage holds an older row)
            dout.clear();
            total.clear();
        }
        // The second sum is of g (total - mean), and rstd comes behind it: an element of 0 behind
        // the channels then adds g = 0 times -mean.  (Its xh, -mean rstd, may be beyond float's
        // range, and 0 times that is not a number.)
        float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const float2 d = dout.get(p), g = mul2(d, weight[p]);
            const float2 centred = add2(total.get(p), minus), hat = mul2(centred, scale);
            s1 = add2(s1, g);
            s2 = fma2(g, centred, s2);
            dw[p] = fma2(d, hat, dw[p]);
            db[p] = add2(db[p], d);
        }
        ring.fetch(a, row + S * stride, lane);
        ring.advance();
        const float2 m = team_sum<KIND>(make_float2(s1.x + s1.y, s2.x + s2.y), a, s_sums, team, turn, s_beside);
        const float hats = -m.y * share * scale.x;
        const float2 m1 = make_float2(-m.x * share, -m.x * share), m2 = make_float2(hats, hats);
        if (row >= a.rows) continue;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const float2 hat = mul2(add2(total.get(p), minus), scale);
            const float2 d = fma2(hat, m2, fma2(dout.get(p), weight[p], m1));
            total.set(p, SUM ? fma2(d, scale, in[A - 1].get(p)) : mul2(d, scale));
        }
        total.store(row_of<T>(a, a.out, row, flat), a, lane);
    }
    ring.finish();
    end_sums<KIND>(a, s_beside);
    if (!a.partial) return;

    // The block's sums: lanes of a warp that hold the same channels, then teams in order,
    // all of them in shared memory side by side (64 KB, where a team after the other took
    // 8 us of 65,000 x 512's 58).
    if (KIND == kInWarp)
        for (int d = a.team; d < 32; d *= 2)
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                dw[p].x += __shfl_xor_sync(~0u, dw[p].x, d);
                dw[p].y += __shfl_xor_sync(~0u, dw[p].y, d);
                db[p].x += __shfl_xor_sync(~0u, db[p].x, d);
                db[p].y += __shfl_xor_sync(~0u, db[p].y, d);
            }
    const int width = KIND == kInWarp ? 32 : a.team / X, each = 2 * kPairs * width, before = X > 1 ? lane - threadIdx.x : 0;
    const int group = threadIdx.x / width, groups = blockDim.x / width, own = threadIdx.x % width;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        s_work[group * each + 2 * p * width + own] = make_float2(dw[p].x, db[p].x);
        s_work[group * each + (2 * p + 1) * width + own] = make_float2(dw[p].y, db[p].y);
    }
    __syncthreads();
    float2 *out = a.partial + (int64_t)block * a.channels;
    for (int i = threadIdx.x; i < each; i += blockDim.x) {
        const int element = i / width, l = before + i - element * width;
        const int c = pair_channel<V>(a, l, element / 2, element % 2);
        if (l >= a.team || c >= a.channels) continue;
        float2 sum = s_work[i];
        for (int k = 1; k < groups; ++k) sum = add2(sum, s_work[k * each + i]);
        out[c] = sum;
    }
}

// Adds the blocks' sums: 32 channels a block, 32 threads a channel.
constexpr int kParamSlices = 32;

__global__ void __launch_bounds__(32 * kParamSlices) k_layer_norm_params(const LayerArgs a)
{
    grid_dependency_begin();
    __shared__ float2 s_sum[kParamSlices][33];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
    float2 sum = make_float2(0.0f, 0.0f);
    if (c < a.channels)
#pragma unroll 4
        for (int i = slice; i < a.blocks; i += kParamSlices) sum = add2(sum, a.partial[(int64_t)i * a.channels + c]);
    s_sum[slice][threadIdx.x % 32] = sum;
    __syncthreads();
    // A warp takes a channel: its lanes the slices.
    sum = s_sum[threadIdx.x % 32][slice];
    for (int d = 16; d > 0; d /= 2) add_lane(sum, d);
    const int channel = blockIdx.x * 32 + slice;
    if (threadIdx.x % 32 != 0 || channel >= a.channels) return;
    if (a.dweight) a.dweight[channel] = sum.x;
    if (a.dbias) a.dbias[channel] = sum.y;
}

// ---- host ---------------------------------------------------------------------------

Rows rows_of(const gsr_heads *t)
{
    return t ? Rows{t->data, t->batch_stride, t->token_stride, t->head_stride} : Rows{};
}

// Takes dimensions together that every array walks at one stride: heads into
// tokens, then items into tokens.
void collapse(LayerArgs &a)
{
    Rows *arrays[] = {&a.x, &a.residual, &a.out, &a.total};
    bool flat = true;
    for (const Rows *r : arrays)
        if (r->data && a.heads > 1 && a.tokens > 1) flat = flat && r->token == a.heads * r->head;
    if (flat && a.heads > 1) {
        a.tokens *= a.heads;
        a.heads = 1;
        for (Rows *r : arrays) r->token = r->head;
    }
    if (a.heads > 1 || a.batch == 1) return;
    for (const Rows *r : arrays)
        if (r->data && a.tokens > 1) flat = flat && r->batch == a.tokens * r->token;
    if (!flat) return;
    for (Rows *r : arrays)
        if (a.tokens == 1) r->token = r->batch;
    a.tokens *= a.batch;
    a.batch = 1;
}

LayerArgs args_of(const gsr_layer_norm &d)
{
    LayerArgs a = {};
    a.batch = d.batch;
    a.tokens = d.tokens;
    a.heads = d.heads;
    a.channels = d.channels;
    a.rows = (uint32_t)d.batch * (uint32_t)d.tokens * (uint32_t)d.heads;
    a.eps = d.eps;
    return a;
}

// Elements of an access: 16 bytes, or 4 where channels, strides or arrays allow no
// more, or one.
int access_width(const LayerArgs &a, int size)
{
    for (int bytes : {16, 4}) {
        const int v = bytes / size;
        if (v <= 1) break;
        bool ok = a.channels % v == 0;
        for (const float *p : {a.weight, a.bias}) ok = ok && (uintptr_t)p % 8 == 0;   // read in pairs
        for (const Rows *r : {&a.x, &a.residual, &a.out, &a.total})
            if (r->data)
                ok = ok && (uintptr_t)r->data % bytes == 0 && (a.batch == 1 || r->batch % v == 0) &&
                     (a.tokens == 1 || r->token % v == 0) && (a.heads == 1 || r->head % v == 0);
        if (ok) return v;
    }
    return 1;
}

int power_of_two(int n)
{
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// Divides a row over a team, kElements of it to a thread, and the rows over blocks of
// teams; returns a block's teams.  Few rows are spread over the SMs rather than over the
// teams of one block.
int plan_rows(const gsr_ctx *ctx, LayerArgs &a)
{
    const int threads = (a.channels + kElements - 1) / kElements;
    const bool two = threads > kRowThreads;
    const int whole = two ? 64 : 32;
    a.team = threads <= 32 ? power_of_two(threads) : (threads + whole - 1) / whole * whole;
    const uint64_t spread = ((uint64_t)a.rows + ctx->num_sms - 1) / ctx->num_sms;
    int teams = a.team > kRowThreads ? 1 : kRowThreads / a.team;
    while (a.team * teams > 128 && (uint64_t)teams > spread) teams = (teams + 1) / 2;
    if (teams * a.team % 32 != 0) teams = 32 / a.team;   // whole warps
    const uint64_t blocks = ((uint64_t)a.rows + teams - 1) / teams;
    a.blocks = (int)std::min(blocks, (uint64_t)ctx->num_sms / (two ? 2 : 1));
    return teams;
}

// The word that tells of waits between two blocks of a row, where there are any.
int status_of(gsr_ctx *ctx, LayerArgs &a, cudaStream_t stream)
{
    if (a.team <= kRowThreads) return GSR_OK;
    void *none = nullptr;
    const int rc = Workspace(ctx, stream).take(0, &none);
    a.status = ctx->status_dev;
    return rc;
}

template <typename T, int V, int N, int KIND, bool BACKWARD, bool SUM>
cudaError_t launch_rows(gsr_ctx *ctx, LayerArgs &a, int teams, cudaStream_t stream)
{
    constexpr int kArrays = (BACKWARD ? 2 : 1) + SUM;
    constexpr int kInFlight = BACKWARD ? kStages<T, V, N, kArrays> : kForwardStages<T, V, N, kArrays>;
    constexpr size_t kRing = (size_t)kInFlight * kArrays * N * kRowThreads * sizeof(T) * V;
    constexpr size_t kTeamSums = 2 * kTeamWarps * sizeof(float2), kShares = N * V * sizeof(float2);   // of a team, a thread
    const int threads = teams * a.team / kBlocksOf<KIND>;
    const size_t smem = std::max(kRing + (KIND != kInWarp ? teams * kTeamSums : 0), BACKWARD ? threads * kShares : 0);
    void (*kernel)(LayerArgs);
    if constexpr (BACKWARD)
        kernel = k_layer_norm_grad<T, V, N, KIND, SUM>;
    else
        kernel = k_layer_norm<T, V, N, KIND, SUM>;
    static OncePerDevice once;
    if (once.due(ctx)) {
        constexpr size_t kMost = std::max(kRing + (KIND != kInWarp ? kRowThreads / 64 * kTeamSums : 0),
                                          BACKWARD ? kRowThreads * kShares : 0);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (e != cudaSuccess) return e;
        once.done(ctx);
    }
    constexpr unsigned kBlocks = kBlocksOf<KIND>;
    return launch_kernel_smem(ctx, kernel, dim3(a.blocks * kBlocks), threads, smem, kBlocks, stream, a);
}

template <typename T, int V, bool BACKWARD, bool SUM>
cudaError_t dispatch_rows(gsr_ctx *ctx, LayerArgs &a, int teams, cudaStream_t stream)
{
    constexpr int N = kElements / V;
    if (a.team <= 32) return launch_rows<T, V, N, kInWarp, BACKWARD, SUM>(ctx, a, teams, stream);
    if (a.team <= kRowThreads) return launch_rows<T, V, N, kInBlock, BACKWARD, SUM>(ctx, a, teams, stream);
    return launch_rows<T, V, N, kInTwo, BACKWARD, SUM>(ctx, a, teams, stream);
}

template <typename T, int V, bool BACKWARD>
cudaError_t dispatch_sum(gsr_ctx *ctx, LayerArgs &a, int teams, cudaStream_t stream)
{
    return a.residual.data ? dispatch_rows<T, V, BACKWARD, true>(ctx, a, teams, stream)
                           : dispatch_rows<T, V, BACKWARD, false>(ctx, a, teams, stream);
}

// f<T, V>() for the description's type and the arrays' widest access.
template <typename F>
auto with_access(int dtype, const LayerArgs &a, F f)
{
    if (dtype == GSR_F32) {
        if (access_width(a, 4) == 4) return f(float(), std::integral_constant<int, 4>());
        return f(float(), std::integral_constant<int, 1>());
    }
    const int v = access_width(a, 2);
    if (dtype == GSR_BF16) {
        if (v == 8) return f(__nv_bfloat16(), std::integral_constant<int, 8>());
        if (v == 2) return f(__nv_bfloat16(), std::integral_constant<int, 2>());
        return f(__nv_bfloat16(), std::integral_constant<int, 1>());
    }
    if (v == 8) return f(__half(), std::integral_constant<int, 8>());
    if (v == 2) return f(__half(), std::integral_constant<int, 2>());
    return f(__half(), std::integral_constant<int, 1>());
}

}  // namespace

int layer_norm_forward(gsr_ctx *ctx, const gsr_layer_norm &d, const gsr_heads &x, const gsr_heads *residual,
                       const float *weight, const float *bias, const gsr_heads &out, const gsr_heads *total,
                       float *mean, float *rstd, cudaStream_t stream)
{
    LayerArgs a = args_of(d);
    a.x = rows_of(&x);
    a.residual = rows_of(residual);
    a.out = rows_of(&out);
    a.total = rows_of(total);
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    collapse(a);
    const int teams = plan_rows(ctx, a);
    if (int rc = status_of(ctx, a, stream)) return rc;
    const cudaError_t e = with_access(d.dtype, a, [&](auto t, auto v) {
        constexpr int V = decltype(v)::value;
        return dispatch_sum<decltype(t), V, false>(ctx, a, teams, stream);
    });
    return cuda_check(ctx, e, "layer norm forward");
}

int layer_norm_backward(gsr_ctx *ctx, const gsr_layer_norm &d, const gsr_heads &dout, const gsr_heads &total,
                        const float *weight, const float *mean, const float *rstd, const gsr_heads *dtotal,
                        const gsr_heads &dx, float *dweight, float *dbias, cudaStream_t stream)
{
    if (d.batch == 0 || d.tokens == 0 || d.heads == 0) {
        for (float *grad : {dweight, dbias})
            if (grad)
                if (int rc = cuda_check(ctx, cudaMemsetAsync(grad, 0, (size_t)d.channels * sizeof(float), stream),
                                        "layer norm backward"))
                    return rc;
        return GSR_OK;
    }
    LayerArgs a = args_of(d);
    a.x = rows_of(&dout);
    a.residual = rows_of(dtotal);
    a.out = rows_of(&dx);
    a.total = rows_of(&total);
    a.weight = weight;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dweight = dweight;
    a.dbias = dbias;
    collapse(a);
    const int teams = plan_rows(ctx, a);
    if (int rc = status_of(ctx, a, stream)) return rc;
    Workspace workspace(ctx, stream);
    if (dweight || dbias) {
        void *work = nullptr;
        if (int rc = workspace.take((size_t)a.blocks * d.channels * sizeof(float2), &work)) return rc;
        a.partial = (float2 *)work;
    }
    const cudaError_t e = with_access(d.dtype, a, [&](auto t, auto v) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value;
        cudaError_t e = dispatch_sum<T, V, true>(ctx, a, teams, stream);
        if (e == cudaSuccess && a.partial)
            e = launch_kernel(ctx, k_layer_norm_params, dim3((unsigned)((a.channels + 31) / 32)), 32 * kParamSlices,
                              stream, a);
        return e;
    });
    if (int bad = cuda_check(ctx, e, "layer norm backward")) return bad;
    return workspace.done();
}

}  // namespace gsr
