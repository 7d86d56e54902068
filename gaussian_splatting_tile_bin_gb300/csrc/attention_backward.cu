// attention_backward.cu -- cross attention to an encoder's states of another
// length, backward.
//
//   p = exp(s - lse),  dp = do . v,  delta = do . o,  ds = p (dp - delta)
//   dq = scale sum ds k,   dk = scale sum ds q,   dv = sum p do
//
// Two kernels, one whose blocks hold 128 queries and walk the keys (dq) and one
// whose blocks hold 128 keys and walk the queries of every head of the group (dk
// and dv).  Each computes s and dp for itself: seven products instead of five,
// but each gradient is a sum that one accumulator in tensor memory takes in a
// fixed order, with no atomics and no traffic of partial gradients through L2.
//
// In both, two warpgroups take the exponentials and ds, each for half of the
// columns of S and dP, and one thread issues the products.  S of the next step
// runs while ds of this one is computed, so the tensor cores stay busy.  16-bit
// p and ds go back to tensor memory, where the sums' products read them as their
// first operand: over the columns they came from (keys as rows), or into two
// buffers in turn (queries as rows).
//
// Rounding.  p and ds are rounded to the storage type, as the tensor cores take
// operands of one type.  f16 has few exponents: p is held times 2^14 (p <= 1), and
// ds times a power of two that brings its bound, |do| |v| / 2, to f16's largest
// values; both powers are divided out of the float sums at the end.  A query's ds in
// dq takes |do| of its own row, dk's sums over the queries the longest row of the
// group's heads, and |v| is the longest row's of the same item and key head: rows
// that never meet in a product do not cost each other bits.
//
// Bound by the tensor cores: 4,864 queries x 8,192 keys x 16 heads in bf16 take
// 634 to 643 us for all three gradients at head_dim 128 (1,270 TFLOP/s on the five
// products a gradient cannot do without, 1,780 on the seven done, 93% of a large
// library product's rate) and 468 us at 64 (870 and 1,220; by these times a product
// with 64 columns takes that of one with 128), in f16 662 to 675 and 484.  At 4 heads the tensor pipe is active
// 77 and 73% of the two kernels, starts and ends included; DRAM reads are the
// inputs' own 27 MB.  Four warpgroups instead of two take 651 and 477 us; Q and dO
// of the dq kernel in tensor memory, statistics read before the scores' wait and
// dP of the next step ahead of this step's dq were no faster either.
#include <math.h>

#include "attention.cuh"

namespace gsr {
namespace {

constexpr int kRowTile = 128;
constexpr int kGroups = 2;              // warpgroups that compute, each its share of the columns of S and dP
constexpr int kColumnsEach = 128 / kGroups;
constexpr int kComputeWarps = 4 * kGroups;
constexpr int kBackwardThreads = 128 * kGroups + 128;   // and four warps of which one copies and one issues
constexpr float kLog2e = 1.4426950408889634f;

// f16 p is held times this.
template <typename T>
constexpr float kShiftP = std::is_same<T, __half>::value ? 16384.0f : 1.0f;

// ds is held times this, a power of 2, where do's and v's rows are at most this long
// (squared; of 16-bit values, so that their product is in float's range).  |dp| is at
// most the lengths' product B, and a row's ds = p ((1 - p) dp - sum of the others' p dp)
// at most 2 B p (1 - p) <= B / 2 and some 2^-10 B of rounding: below 2^15.1 then.
// So only a B of 2^16 or more, whose ds may pass f16's range, costs small ds bits.
template <typename T>
__device__ __forceinline__ float shift_ds(float dout_length2, float v_length2)
{
    if constexpr (std::is_same<T, __half>::value) {
        const int exponent = __float_as_int(dout_length2 * v_length2) >> 23 & 255;
        if (exponent != 0 && exponent != 255) return __int_as_float((127 + 15 - ((exponent - 127) >> 1)) << 23);
    }
    return 1.0f;
}

// 1 / x of such a power.
__device__ __forceinline__ float inverse_power(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }

struct BackwardArgs {
    CUtensorMap q, k, v, dout;
    Schedule work;
    const float *lse2;           // [batch, q_heads, q_pad]: log2(kShiftP) - lse log2e
    const float *row_delta;      // the same: -do . o
    float *delta;                // the same: -delta times the keys' kernel's shift_ds / kShiftP, left by the dq kernel
    // f16: squared lengths of do's rows (as lse2), and the largest of do's and of v's
    // rows of an item and key head ([batch, kv_heads]).
    const float *dout_length2;
    const float2 *top_length2;
    void *dq, *dk, *dv;
    int64_t dq_item, dq_token, dq_head, dk_item, dk_token, dk_head, dv_item, dv_token, dv_head;
    const int32_t *index;        // original keys of packed ones, [batch, kv_len], or NULL
    float *partial;              // [2 blocks][128][dim] (dq) or [2 blocks][128][2 dim] (dk, dv)
    uint32_t *status;
    int q_len, q_pad, kv_len, q_heads, kv_heads, group, dim;
    int q_tiles;                 // tiles of 128 queries per head
    int q_item, q_head, dout_item, dout_head, k_item, k_head, v_item, v_head;
    bool wide_q, wide_kv;        // the gradients' rows take 32-byte stores
    float scale, scale_log2;
};

template <int HD>
struct BackwardShape {
    static constexpr int kBlocks = HD / 64;
    static constexpr int kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kStages = HD == 128 ? 5 : 8;
    static constexpr int kStatBytes = kRowTile * 4;   // a query tile's lse2 (with Q) or delta (with dO)
    static constexpr int kBarriers = 2 + 2 * kStages + 6;
    static constexpr int kSmemBoth = (2 + kStages) * kTileBytes + kBarriers * 8 + 16;
    static constexpr int kSmemQ = kSmemBoth + kGroups * kStatBytes;   // sums of a row
    static constexpr int kSmemK = kSmemBoth + kStages * kStatBytes;   // statistics of a stage
    static_assert(kSmemK <= 232448 && kSmemQ <= 232448, "more shared memory than a block can have");
    static constexpr int kS = 0, kDp = 128, kOut = 256, kDs = 384;   // tensor memory columns
    static constexpr int kColumns = 512;
};

// Barriers of a block, in shared memory.
template <int HD>
struct Bars {
    uint32_t own, own_free, ring, ring_free, s, dp, s_read, ready, done, p_ready;
    __device__ explicit Bars(uint32_t at)
    {
        own = at;
        own_free = at + 8;
        ring = at + 16;
        ring_free = ring + 8 * BackwardShape<HD>::kStages;
        s = ring_free + 8 * BackwardShape<HD>::kStages;
        dp = s + 8;
        s_read = dp + 8;
        p_ready = s_read;   // queries as rows: scores read; keys as rows: p written
        ready = s_read + 8;
        done = ready + 8;
    }
    __device__ void init() const
    {
        barrier_init(own, 1);
        barrier_init(own_free, 1);
        for (int i = 0; i < BackwardShape<HD>::kStages; ++i) {
            barrier_init(ring + 8 * i, 1);
            barrier_init(ring_free + 8 * i, 1);
        }
        barrier_init(s, 1);
        barrier_init(dp, 1);
        barrier_init(s_read, kComputeWarps);
        barrier_init(ready, kComputeWarps);
        barrier_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
};

__device__ __forceinline__ void copy_bytes(uint32_t to, const void *from, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "l"(from), "r"(bytes), "r"(bar)
                 : "memory");
}

using Columns = uint32_t[kColumnsEach];

// This thread's columns of its lane.
__device__ __forceinline__ void load_columns(Columns &r, uint32_t at)
{
#pragma unroll
    for (int x = 0; x < kColumnsEach; x += 32) tmem_load32(*(uint32_t(*)[32])&r[x], at + x);
    tmem_wait_load();
#pragma unroll
    for (int x = 0; x < kColumnsEach; x += 32) pin(*(uint32_t(*)[32])&r[x]);
}

// Their 16-bit pairs.
__device__ __forceinline__ void store_pairs(uint32_t at, const uint32_t (&r)[32])
{
    tmem_store32(at, r);
    tmem_wait_store();
}
__device__ __forceinline__ float2 pair(const Columns &r, int i)
{
    return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}

// ---- dq: queries as rows -----------------------------------------------------------

template <typename T, int HD>
__global__ void __launch_bounds__(kBackwardThreads, 1) k_attention_grad_q(const __grid_constant__ BackwardArgs a)
{
    grid_dependency_begin();
    using S = BackwardShape<HD>;
    extern __shared__ __align__(1024) unsigned char s_raw[];
    const uint32_t raw = smem_address(s_raw), base = raw;
    if (base % 1024 != 0) {   // the swizzle needs it; there is no room to round up
        *(volatile uint32_t *)a.status = 1;
        return;
    }
    const uint32_t s_own = base, s_ring = base + 2 * S::kTileBytes, at_bars = s_ring + S::kStages * S::kTileBytes;
    const Bars<HD> bar(at_bars);
    const uint32_t tail = at_bars + S::kBarriers * 8;
    uint32_t *s_words = (uint32_t *)(s_raw + (tail - raw));
    float *s_sum = (float *)(s_words + 4);   // [part][row]
    const int warp = (int)uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const WaitGuard guard = {s_words + 1, a.status};
    if (threadIdx.x == 0) {
        s_words[1] = 0;
        bar.init();
    }
    if (warp == kComputeWarps + 2) tmem_alloc(tail, S::kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, s_words[0], 0);
    Walk<QueryLine> walk = walk_share<QueryLine>(a.work);
    Segment g;

    if (warp >= kComputeWarps) {
        give_registers();
        if (warp == kComputeWarps && elect_one()) {
            uint32_t n = 0, seg = 0;
            while (walk.next(g)) {
                if (g.length == 0) continue;
                const int head = g.tile / a.q_tiles, row0 = (g.tile - head * a.q_tiles) * kRowTile;
                const int key_head = head / a.group;
                if (seg > 0) barrier_wait(bar.own_free, (seg - 1) & 1, guard);
                barrier_expect(bar.own, 2 * S::kTileBytes);
                for (int c = 0; c < S::kBlocks; ++c) {
                    copy_box(s_own + c * kBlockBytes, &a.q, bar.own, c * 64, row0, head * a.q_head, g.item * a.q_item);
                    copy_box(s_own + S::kTileBytes + c * kBlockBytes, &a.dout, bar.own, c * 64, row0,
                             head * a.dout_head, g.item * a.dout_item);
                }
                for (int i = g.begin; i < g.end; ++i)
                    for (int half = 0; half < 2; ++half, ++n) {
                        if (guard.stop()) goto done;
                        const uint32_t stage = n % S::kStages, round = n / S::kStages;
                        if (round > 0) barrier_wait(bar.ring_free + 8 * stage, (round - 1) & 1, guard);
                        const uint32_t full = bar.ring + 8 * stage, to = s_ring + stage * S::kTileBytes;
                        barrier_expect(full, S::kTileBytes);
                        for (int c = 0; c < S::kBlocks; ++c)
                            copy_box(to + c * kBlockBytes, half ? &a.v : &a.k, full, c * 64, i * kKeyTile,
                                     key_head * (half ? a.v_head : a.k_head), g.item * (half ? a.v_item : a.k_item));
                    }
                ++seg;
            }
        } else if (warp == kComputeWarps + 1) {
            const bool leader = elect_one();
            const uint32_t form_s = product_form<T>(kKeyTile, false);
            const uint32_t form_o = product_form<T>((a.dim + 15) & ~15, true);
            const int steps = (a.dim + 15) / 16;
            auto stage_at = [&](uint32_t x) { return s_ring + x % S::kStages * S::kTileBytes; };
            auto await = [&](uint32_t x) {
                barrier_wait_warp(bar.ring + 8 * (x % S::kStages), x / S::kStages & 1, guard);
                tmem_fence_after();
            };
            auto release = [&](uint32_t x) { product_commit(leader, bar.ring_free + 8 * (x % S::kStages)); };
            uint32_t n = 0, seg = 0, step = 0;
            while (next_uniform(walk, g)) {
                if (g.length == 0) continue;
                barrier_wait_warp(bar.own, seg & 1, guard);
                const uint32_t s_q = s_own, s_do = s_own + S::kTileBytes;
                // The tile's last step takes the scores of its keys alone.
                const uint32_t form_last = product_form<T>(round_keys(g.length - (g.total - 1) * kKeyTile), false);
                auto scores = [&](uint32_t x, uint32_t form) {
                    await(x);
                    product_rows<HD>(leader, tmem + S::kS, s_q, stage_at(x), form, steps);
                    product_commit(leader, bar.s);
                };
                auto dp = [&](uint32_t x, uint32_t form) {
                    await(x);
                    product_rows<HD>(leader, tmem + S::kDp, s_do, stage_at(x), form, steps);
                    product_commit(leader, bar.dp);
                    release(x);
                };
                const uint32_t form_first = g.begin + 1 < g.total ? form_s : form_last;
                scores(n, form_first);
                dp(n + 1, form_first);
                // The next segment's own tiles arrive while this one's last step is computed.
                if (g.begin + 1 == g.end) product_commit(leader, bar.own_free);
                for (int i = g.begin; i < g.end; ++i, n += 2, ++step) {
                    const bool more = i + 1 < g.end;
                    const uint32_t form_next = i + 2 < g.total ? form_s : form_last;
                    barrier_wait_warp(bar.s_read, step & 1, guard);
                    tmem_fence_after();
                    if (more) scores(n + 2, form_next);
                    barrier_wait_warp(bar.ready, step & 1, guard);
                    tmem_fence_after();
                    product_across(leader, tmem + S::kOut, tmem + S::kDs + (step & 1) * 64, stage_at(n), form_o, i > g.begin);
                    release(n);
                    if (more)
                        dp(n + 3, form_next);
                    else
                        product_commit(leader, bar.done);
                    if (i + 2 == g.end) product_commit(leader, bar.own_free);
                }
                ++seg;
            }
        }
    } else {
        take_registers();
        const int part = warp / 4, column0 = part * kColumnsEach;   // columns of S and dP
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t at_s = tmem + lanes + S::kS + column0, at_dp = tmem + lanes + S::kDp + column0;
        const int row_in_tile = warp % 4 * 32 + lane;
        const float c = a.scale_log2;
        const float2 c2 = make_float2(c, c);
        uint32_t n = 0, seg = 0, step = 0;
        // The next segment's place and statistics are fetched while one is finished.
        bool there = next_uniform(walk, g);
        float lse = 0.0f, delta = 0.0f;
        float length2 = 0.0f;
        float2 top2 = make_float2(0.0f, 0.0f);
        auto statistics = [&](const Segment &t) {
            const int head = t.tile / a.q_tiles;
            return ((int64_t)t.item * a.q_heads + head) * a.q_pad + (t.tile - head * a.q_tiles) * kRowTile + row_in_tile;
        };
        auto fetch = [&] {
            if (!there || g.length == 0) return;
            lse = a.lse2[statistics(g)];
            delta = a.row_delta[statistics(g)];
            if (kShiftP<T> != 1.0f) {
                length2 = a.dout_length2[statistics(g)];
                top2 = a.top_length2[(int64_t)g.item * a.kv_heads + g.tile / a.q_tiles / a.group];
            }
        };
        fetch();
        while (there) {
            const Segment t = g;
            // This row's power for ds, and the one that the keys' kernel takes.
            const float shift = shift_ds<T>(length2, top2.y), shift_keys = shift_ds<T>(top2.x, top2.y);
            const float f_dp = shift / kShiftP<T>;
            const float2 f2 = make_float2(f_dp, f_dp);
            if (t.length > 0) {
                const float2 lse2 = make_float2(lse, lse);
                float2 delta2 = make_float2(delta * f_dp, delta * f_dp);
                if (part == 0 && t.begin == 0 && t.total > 1) a.delta[statistics(t)] = delta * shift_keys / kShiftP<T>;
                for (int i = t.begin; i < t.end; ++i, n += 2, ++step) {
                    Columns r;
                    barrier_wait_warp(bar.s, step & 1, guard);
                    tmem_fence_after();
                    load_columns(r, at_s);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar.s_read);
                    const int valid = t.length - i * kKeyTile;
                    const int mine = valid - column0;   // of this thread's columns
                    float2 p[kColumnsEach / 2];
#pragma unroll
                    for (int y = 0; y < kColumnsEach / 2; ++y) {
                        p[y] = fma2(pair(r, 2 * y), c2, lse2);
                        p[y].x = exp2_fast(p[y].x);
                        p[y].y = exp2_fast(p[y].y);
                    }
                    barrier_wait_warp(bar.dp, step & 1, guard);
                    tmem_fence_after();
                    load_columns(r, at_dp);
                    if (t.total == 1) {
                        // Few keys, whose ds nearly cancel: delta from p and dp themselves, here and
                        // for the key gradients, instead of from the rounded output.
                        float sum = 0.0f;
#pragma unroll
                        for (int y = 0; y < kColumnsEach / 2; ++y)
                            if (y / 8 * 16 < mine) {
                                const float2 e = mul2(p[y], pair(r, 2 * y));
                                sum += (2 * y < mine ? e.x : 0.0f) + (2 * y + 1 < mine ? e.y : 0.0f);
                            }
                        s_sum[part * kRowTile + row_in_tile] = sum;
                        asm volatile("bar.sync 1, %0;" ::"n"(kComputeWarps * 32) : "memory");
                        sum = 0.0f;
#pragma unroll
                        for (int x = 0; x < kGroups; ++x) sum += s_sum[x * kRowTile + row_in_tile];
                        // (The zero rows behind the last query meet an infinite key as NaN.)
                        const float exact = lse == -INFINITY ? 0.0f : -sum / kShiftP<T>;
                        delta2 = make_float2(exact * f_dp, exact * f_dp);
                        if (part == 0) a.delta[statistics(t)] = exact * shift_keys / kShiftP<T>;
                    }
                    uint32_t packed[kColumnsEach / 2];
#pragma unroll
                    for (int y = 0; y < kColumnsEach / 2; ++y) {
                        const float2 ds = mul2(p[y], fma2(pair(r, 2 * y), f2, delta2));
                        packed[y] = pack2<T>(ds.x, ds.y);
                    }
                    if (valid < kKeyTile) {
#pragma unroll
                        for (int y = 0; y < kColumnsEach / 2; ++y)
                            packed[y] = 2 * y + 1 < mine ? packed[y] : 2 * y < mine ? packed[y] & 0xffff : 0;
                        if (part == 0) {
                            barrier_wait_warp(bar.ring + 8 * (n % S::kStages), n / S::kStages & 1, guard);
                            clear_tail<S::kBlocks>(s_raw + (s_ring - raw) + n % S::kStages * S::kTileBytes, row_in_tile, valid);
                        }
                    }
                    __syncwarp();
                    store_pairs(tmem + lanes + S::kDs + (step & 1) * 64 + column0 / 2, packed);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar.ready);
                }
            }
            there = next_uniform(walk, g);
            fetch();
            if (t.length > 0) {
                barrier_wait_warp(bar.done, seg++ & 1, guard);
                tmem_fence_after();
            }
            const float f_out = a.scale * inverse_power(shift);
            const int head = t.tile / a.q_tiles, row = (t.tile - head * a.q_tiles) * kRowTile + row_in_tile;
            T *out = (T *)a.dq + t.item * a.dq_item + (int64_t)row * a.dq_token + head * a.dq_head;
            float *partial = a.partial + ((int64_t)partial_slot(t, blockIdx.x) * kRowTile + row_in_tile) * a.dim;
            for (int x = part * 32; x < HD && x < a.dim; x += kGroups * 32) {
                uint32_t o[32];
                __syncwarp();
                if (t.length > 0) {
                    tmem_load32(o, tmem + lanes + S::kOut + x);
                    tmem_wait_load();
                    pin(o);
                } else {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = 0;
                }
                if (row < a.q_len) {
                    float f[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) f[y] = __uint_as_float(o[y]) * f_out;
                    store_results(out + x, partial + x, t.whole(), a.wide_q, a.dim - x, f);
                }
            }
            tmem_fence_before();
        }
    }
done:
    __syncwarp();
    drain_if_aborted(guard);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    __syncwarp();
    if (warp == kComputeWarps + 2) tmem_free(tmem, S::kColumns);
}

// ---- dk and dv: keys as rows ----------------------------------------------------------

template <typename T, int HD>
__global__ void __launch_bounds__(kBackwardThreads, 1) k_attention_grad_kv(const __grid_constant__ BackwardArgs a)
{
    grid_dependency_begin();
    using S = BackwardShape<HD>;
    constexpr int kOutV = S::kOut, kOutK = S::kOut + HD;
    extern __shared__ __align__(1024) unsigned char s_raw[];
    const uint32_t raw = smem_address(s_raw), base = raw;
    if (base % 1024 != 0) {   // the swizzle needs it; there is no room to round up
        *(volatile uint32_t *)a.status = 1;
        return;
    }
    const uint32_t s_own = base, s_ring = base + 2 * S::kTileBytes, s_stat = s_ring + S::kStages * S::kTileBytes;
    const uint32_t at_bars = s_stat + S::kStages * S::kStatBytes;
    const Bars<HD> bar(at_bars);
    const uint32_t tail = at_bars + S::kBarriers * 8;
    uint32_t *s_words = (uint32_t *)(s_raw + (tail - raw));
    const int warp = (int)uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const WaitGuard guard = {s_words + 1, a.status};
    if (threadIdx.x == 0) {
        s_words[1] = 0;
        bar.init();
    }
    if (warp == kComputeWarps + 2) tmem_alloc(tail, S::kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, s_words[0], 0);
    Walk<KeyLine> walk = walk_share<KeyLine>(a.work);
    Segment g;

    if (warp >= kComputeWarps) {
        give_registers();
        if (warp == kComputeWarps && elect_one()) {
            uint32_t n = 0, seg = 0;
            while (walk.next(g)) {
                if (g.tile * kKeyTile >= g.length) continue;
                if (seg > 0) barrier_wait(bar.own_free, (seg - 1) & 1, guard);
                barrier_expect(bar.own, 2 * S::kTileBytes);
                for (int c = 0; c < S::kBlocks; ++c) {
                    copy_box(s_own + c * kBlockBytes, &a.k, bar.own, c * 64, g.tile * kKeyTile, g.head * a.k_head,
                             g.item * a.k_item);
                    copy_box(s_own + S::kTileBytes + c * kBlockBytes, &a.v, bar.own, c * 64, g.tile * kKeyTile,
                             g.head * a.v_head, g.item * a.v_item);
                }
                for (int i = g.begin; i < g.end; ++i) {
                    const int head = g.head * a.group + i / a.q_tiles, row0 = i % a.q_tiles * kRowTile;
                    for (int half = 0; half < 2; ++half, ++n) {
                        if (guard.stop()) goto done;
                        const uint32_t stage = n % S::kStages, round = n / S::kStages;
                        if (round > 0) barrier_wait(bar.ring_free + 8 * stage, (round - 1) & 1, guard);
                        const uint32_t full = bar.ring + 8 * stage, to = s_ring + stage * S::kTileBytes;
                        barrier_expect(full, S::kTileBytes + S::kStatBytes);
                        for (int c = 0; c < S::kBlocks; ++c)
                            copy_box(to + c * kBlockBytes, half ? &a.dout : &a.q, full, c * 64, row0,
                                     head * (half ? a.dout_head : a.q_head), g.item * (half ? a.dout_item : a.q_item));
                        const int64_t at = ((int64_t)g.item * a.q_heads + head) * a.q_pad + row0;
                        copy_bytes(s_stat + stage * S::kStatBytes, (half ? a.delta : a.lse2) + at, S::kStatBytes,
                                   full);
                    }
                }
                ++seg;
            }
        } else if (warp == kComputeWarps + 1) {
            const bool leader = elect_one();
            const uint32_t form_s = product_form<T>(kRowTile, false);
            const uint32_t form_o = product_form<T>((a.dim + 15) & ~15, true);
            const int steps = (a.dim + 15) / 16;
            auto stage_at = [&](uint32_t x) { return s_ring + x % S::kStages * S::kTileBytes; };
            auto await = [&](uint32_t x) {
                barrier_wait_warp(bar.ring + 8 * (x % S::kStages), x / S::kStages & 1, guard);
                tmem_fence_after();
            };
            auto release = [&](uint32_t x) { product_commit(leader, bar.ring_free + 8 * (x % S::kStages)); };
            uint32_t n = 0, seg = 0, step = 0;
            while (next_uniform(walk, g)) {
                if (g.tile * kKeyTile >= g.length) continue;
                barrier_wait_warp(bar.own, seg & 1, guard);
                auto scores = [&](uint32_t x) {
                    await(x);
                    product_rows<HD>(leader, tmem + S::kS, s_own, stage_at(x), form_s, steps);
                    product_commit(leader, bar.s);
                };
                auto dp = [&](uint32_t x) {
                    await(x);
                    product_rows<HD>(leader, tmem + S::kDp, s_own + S::kTileBytes, stage_at(x), form_s, steps);
                    product_commit(leader, bar.dp);
                };
                scores(n);
                dp(n + 1);
                // The next segment's own tiles arrive while this one's last step is computed.
                if (g.begin + 1 == g.end) product_commit(leader, bar.own_free);
                for (int i = g.begin; i < g.end; ++i, n += 2, ++step) {
                    const bool more = i + 1 < g.end;
                    barrier_wait_warp(bar.p_ready, step & 1, guard);
                    tmem_fence_after();
                    product_across(leader, tmem + kOutV, tmem + S::kS, stage_at(n + 1), form_o, i > g.begin, kGroups);
                    if (more) scores(n + 2);
                    barrier_wait_warp(bar.ready, step & 1, guard);
                    tmem_fence_after();
                    product_across(leader, tmem + kOutK, tmem + S::kDp, stage_at(n), form_o, i > g.begin, kGroups);
                    release(n);
                    release(n + 1);
                    if (more)
                        dp(n + 3);
                    else
                        product_commit(leader, bar.done);
                    if (i + 2 == g.end) product_commit(leader, bar.own_free);
                }
                ++seg;
            }
        }
    } else {
        take_registers();
        const int part = warp / 4, column0 = part * kColumnsEach;   // columns of S and dP
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t at_s = tmem + lanes + S::kS + column0, at_dp = tmem + lanes + S::kDp + column0;
        const int row_in_tile = warp % 4 * 32 + lane;
        const float c = a.scale_log2;
        const float2 c2 = make_float2(c, c);
        uint32_t n = 0, seg = 0, step = 0;
        while (next_uniform(walk, g)) {
            const int row = g.tile * kKeyTile + row_in_tile;        // key (packed)
            const bool any = g.tile * kKeyTile < g.length, live = row < g.length;
            float shift = 1.0f;
            if (kShiftP<T> != 1.0f) {
                const float2 top2 = a.top_length2[(int64_t)g.item * a.kv_heads + g.head];
                shift = shift_ds<T>(top2.x, top2.y);
            }
            const float f_dp = shift / kShiftP<T>, f_k = a.scale * inverse_power(shift);
            constexpr float f_v = 1.0f / kShiftP<T>;
            const float2 f2 = make_float2(f_dp, f_dp);
            if (any) {
                const bool tail_tile = g.length - g.tile * kKeyTile < kKeyTile;
                for (int i = g.begin; i < g.end; ++i, n += 2, ++step) {
                    const float4 *lse4 = (const float4 *)(s_raw + (s_stat - raw) + n % S::kStages * S::kStatBytes) +
                                         column0 / 4;
                    const float4 *delta4 =
                        (const float4 *)(s_raw + (s_stat - raw) + (n + 1) % S::kStages * S::kStatBytes) + column0 / 4;
                    Columns r;
                    uint32_t packed[kColumnsEach / 2];
                    float2 p[kColumnsEach / 2];
                    barrier_wait_warp(bar.ring + 8 * (n % S::kStages), n / S::kStages & 1, guard);   // lse2
                    barrier_wait_warp(bar.s, step & 1, guard);
                    tmem_fence_after();
                    load_columns(r, at_s);
#pragma unroll
                    for (int y = 0; y < kColumnsEach / 2; y += 2) {
                        const float4 l = lse4[y / 2];
                        p[y] = fma2(pair(r, 2 * y), c2, make_float2(l.x, l.y));
                        p[y + 1] = fma2(pair(r, 2 * y + 2), c2, make_float2(l.z, l.w));
                    }
#pragma unroll
                    for (int y = 0; y < kColumnsEach / 2; ++y) {
                        p[y].x = exp2_fast(p[y].x);
                        p[y].y = exp2_fast(p[y].y);
                    }
                    if (tail_tile && !live)
#pragma unroll
                        for (int y = 0; y < kColumnsEach / 2; ++y) p[y] = make_float2(0.0f, 0.0f);
                    // The zero rows behind the last query, whose lse2 is -inf, meet an infinite
                    // key as NaN.  (Found by a value that is there: a count of the queries left
                    // made this kernel 2 to 3% longer, and one branch for both kinds of rows cost
                    // 1 of 15 us where keys are few.)
                    if (lse4[kColumnsEach / 4 - 1].w == -INFINITY) {
#pragma unroll
                        for (int y = 0; y < kColumnsEach / 2; y += 2) {
                            const float4 l = lse4[y / 2];
                            if (l.x == -INFINITY) p[y].x = 0.0f;
                            if (l.y == -INFINITY) p[y].y = 0.0f;
                            if (l.z == -INFINITY) p[y + 1].x = 0.0f;
                            if (l.w == -INFINITY) p[y + 1].y = 0.0f;
                        }
                    }
#pragma unroll
                    for (int y = 0; y < kColumnsEach / 2; ++y) packed[y] = pack2<T>(p[y].x, p[y].y);
                    __syncwarp();
                    store_pairs(at_s, packed);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar.p_ready);
                    barrier_wait_warp(bar.ring + 8 * ((n + 1) % S::kStages), (n + 1) / S::kStages & 1, guard);   // delta
                    barrier_wait_warp(bar.dp, step & 1, guard);
                    tmem_fence_after();
                    load_columns(r, at_dp);
#pragma unroll
                    for (int y = 0; y < kColumnsEach / 2; y += 2) {
                        const float4 d = delta4[y / 2];
                        const float2 one = mul2(p[y], fma2(pair(r, 2 * y), f2, make_float2(d.x, d.y)));
                        const float2 two = mul2(p[y + 1], fma2(pair(r, 2 * y + 2), f2, make_float2(d.z, d.w)));
                        packed[y] = pack2<T>(one.x, one.y);
                        packed[y + 1] = pack2<T>(two.x, two.y);
                    }
                    if (tail_tile && !live)
#pragma unroll
                        for (int y = 0; y < kColumnsEach / 2; ++y) packed[y] = 0;
                    __syncwarp();
                    store_pairs(at_dp, packed);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar.ready);
                }
                barrier_wait_warp(bar.done, seg++ & 1, guard);
                tmem_fence_after();
            }
            // Rows behind the item's keys are zeros; packed ones have no place of their own.
            const bool store = a.index ? live : row < a.kv_len, whole = g.whole();
            const int64_t key = a.index && live ? a.index[(int64_t)g.item * a.kv_len + row] : row;
            T *out_k = (T *)a.dk + g.item * a.dk_item + key * a.dk_token + g.head * a.dk_head;
            T *out_v = (T *)a.dv + g.item * a.dv_item + key * a.dv_token + g.head * a.dv_head;
            float *partial = a.partial + ((int64_t)partial_slot(g, blockIdx.x) * kRowTile + row_in_tile) * 2 * a.dim;
            for (int x = part * 32; x < HD && x < a.dim; x += kGroups * 32) {
                for (int which = 0; which < 2; ++which) {
                    uint32_t o[32];
                    __syncwarp();
                    if (any) {
                        tmem_load32(o, tmem + lanes + (which ? kOutV : kOutK) + x);
                        tmem_wait_load();
                        pin(o);
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = 0;
                    }
                    if (store) {
                        const float factor = which ? f_v : f_k;
                        float f[32];
#pragma unroll
                        for (int y = 0; y < 32; ++y) f[y] = live ? __uint_as_float(o[y]) * factor : 0.0f;
                        store_results((which ? out_v : out_k) + x, partial + which * a.dim + x, whole, a.wide_kv, a.dim - x, f);
                    }
                }
            }
            tmem_fence_before();
        }
    }
done:
    __syncwarp();
    drain_if_aborted(guard);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    __syncwarp();
    if (warp == kComputeWarps + 2) tmem_free(tmem, S::kColumns);
}

// ---- sums of cut tiles' parts -----------------------------------------------------------

constexpr int kSumBlock = 256;

// Adds up the parts of 8 elements at `at` of every slot; parts first - 1 .. last.
template <typename T>
__device__ __forceinline__ void sum_parts(const float *at, int64_t slot_stride, int first, int last, T *out)
{
    const float4 *p = (const float4 *)(at + (2 * first - 1) * slot_stride);
    float4 lo = p[0], hi = p[1];
    for (int b = first; b <= last; ++b) {
        p = (const float4 *)(at + 2 * b * slot_stride);
        const float4 f = p[0], g = p[1];
        lo = make_float4(lo.x + f.x, lo.y + f.y, lo.z + f.z, lo.w + f.w);
        hi = make_float4(hi.x + g.x, hi.y + g.y, hi.z + g.z, hi.w + g.w);
    }
    *(uint4 *)out = make_uint4(pack2<T>(lo.x, lo.y), pack2<T>(lo.z, lo.w), pack2<T>(hi.x, hi.y), pack2<T>(hi.z, hi.w));
}

template <typename T>
__global__ void __launch_bounds__(kSumBlock) k_attention_sum_q(const __grid_constant__ BackwardArgs a, int grid)
{
    grid_dependency_begin();
    Segment g;
    const int first = blockIdx.x + 1, chunks = a.dim / 8;
    int last;
    if (!cut_tile<QueryLine>(a.work, grid, first, g, last)) return;
    const int head = g.tile / a.q_tiles, row0 = (g.tile - head * a.q_tiles) * kRowTile;
    const int i = blockIdx.y * kSumBlock + threadIdx.x, r = i / chunks, c = (i - r * chunks) * 8;
    const int64_t row = row0 + r;
    if (r >= kRowTile || row >= a.q_len) return;
    sum_parts(a.partial + (int64_t)r * a.dim + c, (int64_t)kRowTile * a.dim, first, last,
              (T *)a.dq + g.item * a.dq_item + row * a.dq_token + head * a.dq_head + c);
}

template <typename T>
__global__ void __launch_bounds__(kSumBlock) k_attention_sum_kv(const __grid_constant__ BackwardArgs a, int grid)
{
    grid_dependency_begin();
    Segment g;
    const int first = blockIdx.x + 1, chunks = a.dim / 8;
    int last;
    if (!cut_tile<KeyLine>(a.work, grid, first, g, last)) return;
    const int i = blockIdx.y * kSumBlock + threadIdx.x;
    const int r2 = i / chunks, c = (i - r2 * chunks) * 8, r = r2 >> 1, which = r2 & 1;   // dk, dv
    const int row = g.tile * kKeyTile + r;
    if (r >= kKeyTile || row >= (a.index ? g.length : a.kv_len)) return;
    const int64_t key = a.index ? a.index[(int64_t)g.item * a.kv_len + row] : row;
    T *out = which ? (T *)a.dv + g.item * a.dv_item + key * a.dv_token + g.head * a.dv_head
                   : (T *)a.dk + g.item * a.dk_item + key * a.dk_token + g.head * a.dk_head;
    sum_parts(a.partial + ((int64_t)r * 2 + which) * a.dim + c, (int64_t)kRowTile * 2 * a.dim, first, last, out + c);
}

// ---- statistics of the rows ----------------------------------------------------------------

struct RowArgs {
    gsr_heads out, dout, v;
    const float *lse;
    float *lse2, *delta;
    float *dout_length2;     // f16: squared lengths of dout's rows, and the bits of the largest of them and
    uint2 *top_length2;      // of v's rows by item and key head
    const int32_t *lengths;
    int64_t row_blocks;      // blocks that take the queries' rows; those behind take v's
    int q_len, q_pad, q_heads, kv_len, kv_heads, group, dim;
};

// A block's rows, of one item and head: lanes of a row, 8 elements each, and its place.
template <int LANES>
struct RowPlace {
    static constexpr int kRows = 256 / LANES;
    uint32_t item, head;
    int token, c;
    __device__ RowPlace(uint32_t block, int tokens, int heads)
    {
        const uint32_t each = (uint32_t)(tokens + kRows - 1) / kRows, unit = block / each;
        item = unit / heads;
        head = unit - item * heads;
        token = (int)(block - unit * each) * kRows + threadIdx.x / LANES;
        c = threadIdx.x % LANES * 8;
    }
    template <typename T>
    __device__ Vec<T, 8> load(const gsr_heads &t) const
    {
        return *(const Vec<T, 8> *)((const T *)t.data + item * t.batch_stride + token * t.token_stride +
                                    head * t.head_stride + c);
    }
};

// The sum over a row's lanes.
template <int LANES>
__device__ __forceinline__ float row_sum(float x)
{
    for (int d = LANES / 2; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

// -lse in base 2 with p's shift folded in, -delta, and the lengths of dout's rows and
// of v's valid keys' for ds' shifts; rows behind q_len, and rows without keys, get p = 0.
template <typename T, int LANES>
__global__ void __launch_bounds__(256) k_attention_rows(const RowArgs a)
{
    grid_dependency_begin();
    constexpr bool kLengths = std::is_same<T, __half>::value;
    const bool queries = blockIdx.x < a.row_blocks;
    const RowPlace<LANES> at(queries ? blockIdx.x : blockIdx.x - (uint32_t)a.row_blocks, queries ? a.q_pad : a.kv_len,
                             queries ? a.q_heads : a.kv_heads);
    float length2 = 0.0f;
    if (queries) {
        float sum = 0.0f;
        if (at.token < a.q_len && at.c < a.dim) {
            const Vec<T, 8> o = at.template load<T>(a.out), d = at.template load<T>(a.dout);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum = fmaf(to_float(o.e[e]), to_float(d.e[e]), sum);
                if (kLengths) length2 = fmaf(to_float(d.e[e]), to_float(d.e[e]), length2);
            }
        }
        sum = row_sum<LANES>(sum);
        if (kLengths) length2 = row_sum<LANES>(length2);
        if (at.c == 0) {   // q_pad is a multiple of a block's rows
            const int64_t row = (int64_t)at.item * a.q_heads + at.head, to = row * a.q_pad + at.token;
            float lse = INFINITY;
            if (at.token < a.q_len) {
                lse = a.lse[row * a.q_len + at.token];
                lse = lse == -INFINITY ? INFINITY : lse * kLog2e - log2f(kShiftP<T>);
            }
            a.lse2[to] = -lse;
            a.delta[to] = -sum;
            if (kLengths) a.dout_length2[to] = length2;
        }
    } else {
        if (at.c < a.dim && at.token < item_length(a.lengths, a.kv_len, (int)at.item)) {
            const Vec<T, 8> v = at.template load<T>(a.v);
#pragma unroll
            for (int e = 0; e < 8; ++e) length2 = fmaf(to_float(v.e[e]), to_float(v.e[e]), length2);
        }
        length2 = row_sum<LANES>(length2);
    }
    if constexpr (kLengths) {
        // The largest of all is the same in any order; what is there already needs no atomic.
        __shared__ uint32_t s_top[8];
        uint32_t top = __reduce_max_sync(~0u, __float_as_uint(length2));
        if (threadIdx.x % 32 == 0) s_top[threadIdx.x / 32] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 8; ++w) top = max(top, s_top[w]);
            uint2 *unit = a.top_length2 + (int64_t)at.item * a.kv_heads + (queries ? at.head / a.group : at.head);
            uint32_t *to = queries ? &unit->x : &unit->y;
            if (top > *(volatile uint32_t *)to) atomicMax(to, top);
        }
    }
}

template <typename T, int LANES>
int row_statistics(gsr_ctx *ctx, RowArgs &r, int batch, cudaStream_t stream)
{
    constexpr int kRows = RowPlace<LANES>::kRows;
    static_assert(kRowTile % kRows == 0, "a tile's rows are whole blocks");
    r.row_blocks = (int64_t)batch * r.q_heads * (r.q_pad / kRows);
    int64_t blocks = r.row_blocks;
    if (std::is_same<T, __half>::value) {
        const int64_t units = (int64_t)batch * r.kv_heads;
        blocks += units * ((r.kv_len + kRows - 1) / kRows);
        if (int rc = cuda_check(ctx, cudaMemsetAsync(r.top_length2, 0, units * sizeof(uint2), stream), "k_attention_rows"))
            return rc;
    }
    return cuda_check(ctx, launch_kernel(ctx, k_attention_rows<T, LANES>, dim3((unsigned)blocks), 256, stream, r),
                      "k_attention_rows");
}

// Zeros: rows of one or two arrays of the same shape, all of them or those of
// masked keys; 16 bytes a thread.
__global__ void __launch_bounds__(256) k_attention_zero_rows(gsr_heads t, gsr_heads t2, int64_t items, uint32_t tokens,
                                                             uint32_t heads, uint32_t chunks, const uint8_t *mask,
                                                             const int32_t *lengths)
{
    grid_dependency_begin();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items) return;
    const uint32_t r = (uint32_t)(i / chunks), c = (uint32_t)(i - (int64_t)r * chunks);
    const uint32_t bt = r / heads, h = r - bt * heads, b = bt / tokens, token = bt - b * tokens;
    if (mask && (int)token < item_length(lengths, (int)tokens, (int)b) && mask[(int64_t)b * tokens + token] != 0) return;
    for (const gsr_heads *x : {&t, &t2})
        if (x->data)
            *(uint4 *)((uint16_t *)x->data + b * x->batch_stride + token * x->token_stride + h * x->head_stride + c * 8) =
                make_uint4(0, 0, 0, 0);
}

int zero_rows(gsr_ctx *ctx, const gsr_heads &t, const gsr_heads &t2, const gsr_attention &d, int tokens, int heads,
              bool masked, cudaStream_t stream)
{
    const int chunks = d.head_dim / 8;   // rows are at most 2^31 - 1, as the arguments' check has it
    const int64_t items = (int64_t)d.batch * tokens * heads * chunks;
    if (items == 0) return GSR_OK;
    return cuda_check(ctx, launch_kernel(ctx, k_attention_zero_rows, dim3((unsigned)((items + 255) / 256)), 256, stream,
                                         t, t2, items, (uint32_t)tokens, (uint32_t)heads, (uint32_t)chunks,
                                         masked ? d.key_mask : nullptr, masked ? d.kv_lengths : nullptr),
                      "k_attention_zero_rows");
}

template <typename Kernel>
int launch_big(gsr_ctx *ctx, Kernel *kernel, const char *name, int blocks, int smem, const BackwardArgs &a,
               cudaStream_t stream)
{
    if (int rc = cuda_check(ctx, cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem), name))
        return rc;
    if (int rc = check_registers(ctx, (const void *)kernel, name)) return rc;
    return cuda_check(ctx, launch_kernel_smem(ctx, kernel, dim3((unsigned)blocks), kBackwardThreads, smem, 1, stream, a),
                      name);
}

template <typename T, int HD>
int launch_backward(gsr_ctx *ctx, BackwardArgs &a, const Schedule &by_query, const Schedule &by_key, int blocks_q,
                    int blocks_k, cudaStream_t stream)
{
    // Blocks of a cut tile's sum: its rows' vectors.
    const int vectors = kRowTile * a.dim / 8, each = kSumBlock;
    // Queries first: they leave delta as the keys' kernel takes it.
    a.work = by_query;
    if (int rc = launch_big(ctx, k_attention_grad_q<T, HD>, "k_attention_grad_q", blocks_q, BackwardShape<HD>::kSmemQ, a,
                            stream))
        return rc;
    if (blocks_q > 1 && a.kv_len > kKeyTile)   // tiles of one step are never cut
        if (int rc = cuda_check(ctx, launch_kernel(ctx, k_attention_sum_q<T>,
                                                   dim3((unsigned)blocks_q - 1, (unsigned)((vectors + each - 1) / each)),
                                                   kSumBlock, stream, a, blocks_q),
                                "k_attention_sum_q"))
            return rc;
    a.work = by_key;
    if (int rc = launch_big(ctx, k_attention_grad_kv<T, HD>, "k_attention_grad_kv", blocks_k,
                            BackwardShape<HD>::kSmemK, a, stream))
        return rc;
    if (blocks_k == 1 || by_key.inner == 1) return GSR_OK;
    return cuda_check(ctx, launch_kernel(ctx, k_attention_sum_kv<T>,
                                         dim3((unsigned)blocks_k - 1, (unsigned)((2 * vectors + each - 1) / each)), kSumBlock,
                                         stream, a, blocks_k),
                      "k_attention_sum_kv");
}

template <typename T>
int backward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k, const gsr_heads &v,
             const gsr_heads &out, const float *lse, const gsr_heads &dout, const gsr_heads &dq, const gsr_heads &dk,
             const gsr_heads &dv, cudaStream_t stream)
{
    if (d.kv_len == 0) return zero_rows(ctx, dq, gsr_heads{}, d, d.q_len, d.q_heads, false, stream);
    if (d.q_len == 0) return zero_rows(ctx, dk, dv, d, d.kv_len, d.kv_heads, false, stream);
    BackwardArgs a = {};
    a.q_len = d.q_len;
    a.kv_len = d.kv_len;
    a.q_heads = d.q_heads;
    a.kv_heads = d.kv_heads;
    a.group = d.q_heads / d.kv_heads;
    a.dim = d.head_dim;
    a.q_tiles = (d.q_len + kRowTile - 1) / kRowTile;
    a.q_pad = a.q_tiles * kRowTile;
    a.scale = d.scale;
    a.scale_log2 = d.scale * kLog2e;
    a.dq = dq.data;
    a.dq_item = dq.batch_stride;
    a.dq_token = dq.token_stride;
    a.dq_head = dq.head_stride;
    a.dk = dk.data;
    a.dk_item = dk.batch_stride;
    a.dk_token = dk.token_stride;
    a.dk_head = dk.head_stride;
    a.dv = dv.data;
    a.dv_item = dv.batch_stride;
    a.dv_token = dv.token_stride;
    a.dv_head = dv.head_stride;
    const int key_tiles = (d.kv_len + kKeyTile - 1) / kKeyTile;
    Schedule by_query = {d.batch, d.q_heads * a.q_tiles, 0, 0, d.kv_lengths, d.kv_len};
    Schedule by_key = {d.batch, key_tiles, d.kv_heads, a.group * a.q_tiles, d.kv_lengths, d.kv_len};
    const int64_t line = (int64_t)d.batch * d.q_heads * a.q_tiles * key_tiles;   // both ways
    const int blocks = (int)(line < ctx->num_sms ? line : ctx->num_sms);

    const int64_t rows = (int64_t)d.batch * d.q_heads * a.q_pad;
    const size_t packed = d.key_mask ? round_up(packed_bytes(d), 256) : 0;
    const size_t stats = round_up((size_t)rows * sizeof(float), 512);
    const size_t partial = round_up((size_t)2 * blocks * kRowTile * 2 * d.head_dim * sizeof(float), 256);
    Workspace workspace(ctx, stream);
    void *work;
    const bool lengths = d.dtype == GSR_F16;
    const size_t top = lengths ? (size_t)d.batch * d.kv_heads * sizeof(float2) : 0;
    if (int rc = workspace.take(packed + (lengths ? 4 : 3) * stats + partial + top, &work)) return rc;
    unsigned char *p = (unsigned char *)work + packed;
    float *lse2 = (float *)p, *row_delta = (float *)(p + stats);
    a.partial = (float *)(p + 3 * stats);
    a.lse2 = lse2;
    a.row_delta = row_delta;
    a.delta = (float *)(p + 2 * stats);
    float *dout_length2 = (float *)(p + 3 * stats + partial);
    unsigned char *top_length2 = p + 4 * stats + partial;
    if (lengths) {
        a.dout_length2 = dout_length2;
        a.top_length2 = (const float2 *)top_length2;
    }
    a.status = ctx->status_dev;

    gsr_heads keys = k, values = v;
    if (d.key_mask) {
        Packed pack;
        if (int rc = cuda_check(ctx, pack_keys(ctx, d, k, v, work, &pack, stream), "k_pack_keys")) return rc;
        keys = pack.k;
        values = pack.v;
        by_query.lengths = by_key.lengths = pack.counts;
        a.index = pack.index;
        if (int rc = zero_rows(ctx, dk, dv, d, d.kv_len, d.kv_heads, true, stream)) return rc;
    }
    RowArgs r = {};
    r.out = out;
    r.dout = dout;
    r.v = values;
    r.lengths = by_query.lengths;
    r.lse = lse;
    r.lse2 = lse2;
    r.delta = row_delta;
    r.dout_length2 = dout_length2;
    r.top_length2 = (uint2 *)top_length2;
    r.group = a.group;
    r.q_len = d.q_len;
    r.q_pad = a.q_pad;
    r.q_heads = d.q_heads;
    r.kv_len = d.kv_len;
    r.kv_heads = d.kv_heads;
    r.dim = d.head_dim;
    if (int rc = d.head_dim <= 64 ? row_statistics<T, 8>(ctx, r, d.batch, stream)
                                     : row_statistics<T, 16>(ctx, r, d.batch, stream))
        return rc;

    a.wide_q = rows_of_32_bytes(dq, d.head_dim);
    a.wide_kv = rows_of_32_bytes(dk, d.head_dim) && rows_of_32_bytes(dv, d.head_dim);
    a.q_item = q.batch_stride != 0;
    a.q_head = q.head_stride != 0;
    a.dout_item = dout.batch_stride != 0;
    a.dout_head = dout.head_stride != 0;
    a.k_item = keys.batch_stride != 0;
    a.k_head = keys.head_stride != 0;
    a.v_item = values.batch_stride != 0;
    a.v_head = values.head_stride != 0;
    if (int rc = heads_map(ctx, &a.q, q, d.dtype, d.batch, d.q_len, d.q_heads, d.head_dim, kRowTile)) return rc;
    if (int rc = heads_map(ctx, &a.dout, dout, d.dtype, d.batch, d.q_len, d.q_heads, d.head_dim, kRowTile)) return rc;
    if (int rc = heads_map(ctx, &a.k, keys, d.dtype, d.batch, d.kv_len, d.kv_heads, d.head_dim, kKeyTile)) return rc;
    if (int rc = heads_map(ctx, &a.v, values, d.dtype, d.batch, d.kv_len, d.kv_heads, d.head_dim, kKeyTile)) return rc;
    const int rc = d.head_dim <= 64 ? launch_backward<T, 64>(ctx, a, by_query, by_key, blocks, blocks, stream)
                                    : launch_backward<T, 128>(ctx, a, by_query, by_key, blocks, blocks, stream);
    if (rc) return rc;
    return workspace.done();
}

}  // namespace

int cross_attention_backward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k,
                             const gsr_heads &v, const gsr_heads &out, const float *lse, const gsr_heads &dout,
                             const gsr_heads &dq, const gsr_heads &dk, const gsr_heads &dv, cudaStream_t stream)
{
    return d.dtype == GSR_BF16 ? backward<__nv_bfloat16>(ctx, d, q, k, v, out, lse, dout, dq, dk, dv, stream)
                               : backward<__half>(ctx, d, q, k, v, out, lse, dout, dq, dk, dv, stream);
}

}  // namespace gsr
