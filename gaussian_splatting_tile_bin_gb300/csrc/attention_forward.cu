// attention_forward.cu -- cross attention to an encoder's states of another
// length, forward.
//
//   s = scale q . k,  o = sum exp(s - m) v / l,  l = sum exp(s - m),  lse = m + log l
//
// One pass over the keys with a running reference m and sum l of each row.  A
// block holds two tiles of 128 query rows, each with its own 128 threads (one
// row a thread) and its own score and output accumulators in tensor memory.  One
// thread issues the products: scores S = Q K^T (operands in shared memory) and
// outputs O += P V with P in tensor memory.  While one tile's threads take the
// exponentials, the tensor cores work for the other tile, so both pipes stay busy.
// K and V tiles arrive by bulk tensor copies through a ring of stages.
//
// P has columns of its own at head_dim 64, so the next scores are computed as soon
// as these are read; at 128, where the accumulators fill tensor memory, it
// replaces the scores and the next ones come behind its product.
//
// m starts as the maximum of the row's first 64 keys, to 2^-12 of a power of 2, so
// that this key's P rounds to 1 and a row that it takes is its v.  m moves only when
// 64 keys' sum of exp(s - m) exceeds 2^12, which tells that without a maximum of
// every tile (the comparisons took a third of the softmax' time): the row then takes
// a maximum of these keys, a whole number of powers of 2 higher.  The sum and the output are
// scaled by that power, which rounds nothing, and so is the first half's P, of which
// f16 rounds what falls below its normal range, 2^-14 of the row's largest.  Until
// then P exceeds 1 by at most 2^12, which 16-bit P and float sums hold.  P is rounded
// to the storage type (the tensor cores take 16-bit operands at the full rate); l
// sums the unrounded values in float.
//
// Bound by the tensor cores: 4,864 queries x 8,192 keys x 16 heads in bf16 take
// 182 us at head_dim 128, 1,790 TFLOP/s, 94% of a large library product's rate, and
// 133 us at 64 (1,225 TFLOP/s; a product with 64 columns of output takes the time
// of one with 128).  At 64, scores that waited for P's product took 154 us, four
// tiles with units of 64 keys 192, two tiles with such units 165 to 197, and turns
// that keep the two groups' exponentials apart 183.
#include <math.h>

#include "attention.cuh"

namespace gsr {
namespace {

constexpr int kRowTile = 128;
constexpr int kForwardThreads = 384;   // two row groups of 128; four warps of which one copies and one issues
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLargestSum = 4096.0f;

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t pair)
{
    const Vec<T, 2> v = *(const Vec<T, 2> *)&pair;
    return make_float2(to_float(v.e[0]), to_float(v.e[1]));
}

struct ForwardArgs {
    CUtensorMap q, k, v;
    Schedule work;
    void *out;
    int64_t out_item, out_token, out_head;
    float *lse;
    float *partial;        // [2 blocks][256][dim] of cut tiles
    float *partial_lse;    // [2 blocks][256]
    uint32_t *status;
    int q_len, q_heads, group, dim, row_tiles;
    int q_item, q_head, k_item, k_head, v_item, v_head;   // 0: one array for all items / heads
    bool wide;             // out's rows take 32-byte stores
    float scale_log2;
};

template <int HD>
struct ForwardShape {
    static constexpr int kBlocks = HD / 64;
    static constexpr int kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kStages = HD == 128 ? 5 : 8;
    static constexpr int kBarriers = 2 + 2 * kStages + 8;
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + kBarriers * 8 + 16;
    // Tensor memory columns: two tiles' scores, outputs and P.  Where there is room
    // for P beside the scores, the next scores are computed while P is.
    static constexpr bool kApart = HD <= 64;
    static constexpr int kOut = 256;
    static constexpr int kP = kApart ? kOut + 2 * HD : 0, kPEach = kApart ? 64 : kKeyTile;
    static constexpr int kColumns = 512;
};

template <typename T, int HD>
__global__ void __launch_bounds__(kForwardThreads, 1) k_attention_forward(const __grid_constant__ ForwardArgs a)
{
    grid_dependency_begin();
    using S = ForwardShape<HD>;
    extern __shared__ unsigned char s_raw[];
    const uint32_t raw = smem_address(s_raw);
    const uint32_t base = (raw + 1023) & ~1023u;
    const uint32_t s_q = base, s_kv = base + 2 * S::kTileBytes, bars = s_kv + S::kStages * S::kTileBytes;
    const uint32_t b_q = bars, b_q_free = bars + 8, b_kv = bars + 16, b_kv_free = b_kv + 8 * S::kStages;
    const uint32_t b_s = b_kv_free + 8 * S::kStages, b_p = b_s + 16, b_o = b_p + 16, b_read = b_o + 16, tail = b_read + 16;
    uint32_t *s_words = (uint32_t *)(s_raw + (tail - raw));   // tensor memory base, abort flag
    const int warp = (int)uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const WaitGuard guard = {s_words + 1, a.status};

    if (threadIdx.x == 0) {
        s_words[1] = 0;
        barrier_init(b_q, 1);
        barrier_init(b_q_free, 1);
        for (int i = 0; i < S::kStages; ++i) {
            barrier_init(b_kv + 8 * i, 1);
            barrier_init(b_kv_free + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {   // of a row tile
            barrier_init(b_s + 8 * i, 1);
            barrier_init(b_p + 8 * i, 4);
            barrier_init(b_o + 8 * i, 1);
            barrier_init(b_read + 8 * i, 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (warp == 10) tmem_alloc(tail, S::kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, s_words[0], 0);

    Walk<QueryLine> walk = walk_share<QueryLine>(a.work);
    Segment g;
    const int row_tiles = a.row_tiles;   // of 256 rows, per head

    if (warp >= 8) {
        give_registers();
        if (warp == 8) {
            // ---- copies: Q of a segment, then K and V of every step ----
            if (elect_one()) {
                prefetch_map(&a.q);
                prefetch_map(&a.k);
                prefetch_map(&a.v);
                uint32_t kv = 0, seg = 0;
                while (walk.next(g)) {
                    if (g.length == 0) continue;
                    const int head = g.tile / row_tiles, row0 = (g.tile - head * row_tiles) * 2 * kRowTile;
                    const int tiles = a.q_len - row0 > kRowTile ? 2 : 1;
                    const int key_head = head / a.group;
                    if (seg > 0) barrier_wait(b_q_free, (seg - 1) & 1, guard);
                    barrier_expect(b_q, tiles * S::kTileBytes);
                    for (int t = 0; t < tiles; ++t)
                        for (int c = 0; c < S::kBlocks; ++c)
                            copy_box(s_q + t * S::kTileBytes + c * kBlockBytes, &a.q, b_q, c * 64, row0 + t * kRowTile,
                                     head * a.q_head, g.item * a.q_item);
                    for (int i = g.begin; i < g.end; ++i)
                        for (int half = 0; half < 2; ++half, ++kv) {
                            if (guard.stop()) goto done;
                            const uint32_t stage = kv % S::kStages, round = kv / S::kStages;
                            if (round > 0) barrier_wait(b_kv_free + 8 * stage, (round - 1) & 1, guard);
                            const uint32_t bar = b_kv + 8 * stage, to = s_kv + stage * S::kTileBytes;
                            barrier_expect(bar, S::kTileBytes);
                            for (int c = 0; c < S::kBlocks; ++c)
                                copy_box(to + c * kBlockBytes, half ? &a.v : &a.k, bar, c * 64, i * kKeyTile,
                                         key_head * (half ? a.v_head : a.k_head), g.item * (half ? a.v_item : a.k_item));
                        }
                    ++seg;
                }
            }
        } else if (warp == 9) {
            // ---- products ----
            const bool leader = elect_one();
            const uint32_t form_s = product_form<T>(kKeyTile, false);
            const uint32_t form_o = product_form<T>((a.dim + 15) & ~15, true);
            const int steps = (a.dim + 15) / 16;
            uint32_t kv = 0, seg = 0, p[2] = {0, 0}, read[2] = {0, 0};
            auto stage_at = [&](uint32_t n) { return s_kv + n % S::kStages * S::kTileBytes; };
            auto await = [&](uint32_t n) { barrier_wait_warp(b_kv + 8 * (n % S::kStages), n / S::kStages & 1, guard); };
            auto release = [&](uint32_t n) { product_commit(leader, b_kv_free + 8 * (n % S::kStages)); };
            auto scores = [&](int t, uint32_t n, uint32_t form) {
                if (S::kApart) {
                    if (read[t] > 0) barrier_wait_warp(b_read + 8 * t, (read[t] - 1) & 1, guard);
                    ++read[t];
                    tmem_fence_after();
                }
                product_rows<HD>(leader, tmem + t * kKeyTile, s_q + t * S::kTileBytes, stage_at(n), form, steps);
                product_commit(leader, b_s + 8 * t);
            };
            while (next_uniform(walk, g)) {
                if (g.length == 0) continue;
                const int head = g.tile / row_tiles, row0 = (g.tile - head * row_tiles) * 2 * kRowTile;
                const int tiles = a.q_len - row0 > kRowTile ? 2 : 1;
                barrier_wait_warp(b_q, seg & 1, guard);
                await(kv);
                tmem_fence_after();
                // The tile's last step takes the scores of its keys alone.
                const uint32_t form_last = product_form<T>(round_keys(g.length - (g.total - 1) * kKeyTile), false);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (t < tiles) scores(t, kv, g.begin + 1 < g.total ? form_s : form_last);
                release(kv);
                // The next segment's Q arrives while this one's last keys are worked on.
                if (g.begin + 1 == g.end) product_commit(leader, b_q_free);
                for (int i = g.begin; i < g.end; ++i, kv += 2) {
                    const bool more = i + 1 < g.end;
                    const uint32_t form_next = i + 2 < g.total ? form_s : form_last;
                    if (!S::kApart) await(kv + 1);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t >= tiles) continue;
                        if (S::kApart) {
                            if (more) {
                                if (t == 0) await(kv + 2);
                                scores(t, kv + 2, form_next);
                            }
                            if (t == 0) await(kv + 1);
                        }
                        barrier_wait_warp(b_p + 8 * t, p[t]++ & 1, guard);
                        tmem_fence_after();
                        product_across(leader, tmem + S::kOut + t * HD, tmem + S::kP + t * S::kPEach, stage_at(kv + 1),
                                       form_o, i > g.begin);
                        product_commit(leader, b_o + 8 * t);
                        if (!S::kApart && more) {
                            if (t == 0) await(kv + 2);
                            scores(t, kv + 2, form_next);
                        }
                    }
                    release(kv + 1);
                    if (more) release(kv + 2);
                    if (i + 2 == g.end) product_commit(leader, b_q_free);
                }
                ++seg;
            }
        }
    } else {
        take_registers();
        // ---- softmax: one row a thread ----
        const int t = warp / 4;                                     // row tile
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;     // this warp's lanes of tensor memory
        const uint32_t at_o = tmem + lanes + S::kOut + t * HD;
        const int row_in_tile = warp % 4 * 32 + lane;
        const float c = a.scale_log2;
        const uint32_t at_s = tmem + lanes + t * kKeyTile, at_p = tmem + lanes + S::kP + t * S::kPEach;
        uint32_t kv = 0, n = 0;   // ring position; key tiles this row tile has seen
        while (next_uniform(walk, g)) {
            const int head = g.tile / row_tiles, row0 = (g.tile - head * row_tiles) * 2 * kRowTile + t * kRowTile;
            const int row = row0 + row_in_tile;
            const bool whole = g.whole();
            float m = -INFINITY, l = 0.0f;   // the reference, in powers of 2; the sum
            const bool active = row0 < a.q_len;
            if (g.length > 0 && active) {
                for (int i = g.begin; i < g.end; ++i, ++n) {
                    barrier_wait_warp(b_s + 8 * t, n & 1, guard);
                    tmem_fence_after();
                    uint32_t r[4][32];
                    tmem_load32(r[0], at_s);
                    tmem_load32(r[1], at_s + 32);
                    tmem_wait_load();
                    pin(r[0]);
                    pin(r[1]);
                    const int valid = g.length - i * kKeyTile;
                    const bool ragged = valid < kKeyTile;
                    if (ragged && t == 0) {
                        // What lies behind the item's last key must not meet the zero
                        // probabilities as infinities or NaN.
                        const uint32_t at_v = kv + 2 * (i - g.begin) + 1;
                        barrier_wait_warp(b_kv + 8 * (at_v % S::kStages), at_v / S::kStages & 1, guard);
                        clear_tail<S::kBlocks>(s_raw + (s_kv - raw) + at_v % S::kStages * S::kTileBytes, row_in_tile, valid);
                    }
                    auto clear_ragged = [&](int h) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (h * 64 + x * 32 + y >= valid) r[2 * h + x][y] = __float_as_uint(-INFINITY);
                    };
                    auto largest = [&](int h) {
                        float part[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                part[y % 4] = fmaxf(part[y % 4], __uint_as_float(r[2 * h + x][y]));
                        return fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
                    };
                    // 2^(c s - m) of 64 keys, and their sum.
                    uint32_t packed[2][32];
                    auto exponentials = [&](int h, float shift) {
                        const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                        for (int y = 0; y < 64; y += 2) {
                            float2 e = fma2(make_float2(__uint_as_float(r[2 * h + y / 32][y % 32]),
                                                        __uint_as_float(r[2 * h + y / 32][y % 32 + 1])),
                                            c2, shift2);
                            e.x = exp2_fast(e.x);
                            e.y = exp2_fast(e.y);
                            sum[y / 2 & 1] = add2(sum[y / 2 & 1], e);
                            packed[h][y / 2] = pack2<T>(e.x, e.y);
                        }
                        return (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    };
                    // The products of the keys before are complete.
                    auto await_output = [&] {
                        if (S::kApart && n > 0) {
                            barrier_wait_warp(b_o + 8 * t, (n - 1) & 1, guard);
                            tmem_fence_after();
                        }
                    };
                    // The keys' maximum becomes the reference (at most 1 above it once there was
                    // another), and what was summed before is scaled down.
                    auto first = [](float top) { return rintf(top * 4096.0f) * (1.0f / 4096.0f); };
                    auto raise = [&](int h) {
                        const float top = largest(h) * c;
                        const float down = m == -INFINITY ? INFINITY : fmaxf(ceilf(top - m), 0.0f);   // whole
                        const float next = m == -INFINITY ? first(top) : m + down;
                        const float keep = down > 126.0f ? 0.0f : __int_as_float((127 - (int)down) << 23);
                        m = next;
                        l *= keep;
                        if (h == 1)
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                const float2 e = unpack2<T>(packed[0][y]);
                                packed[0][y] = pack2<T>(e.x * keep, e.y * keep);
                            }
                        if (i > g.begin) {
                            await_output();
                            for (int x = 0; x < HD; x += 32) {
                                uint32_t o[32];
                                tmem_load32(o, at_o + x);
                                tmem_wait_load();
                                pin(o);
#pragma unroll
                                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * keep);
                                tmem_store32(at_o + x, o);
                            }
                        }
                        return exponentials(h, next == -INFINITY ? 0.0f : -next);
                    };
                    auto half = [&](int h) {
                        float sum = exponentials(h, -m);
                        if (__any_sync(~0u, !(sum <= kLargestSum))) {
                            sum = raise(h);
                            if (h == 1 && !S::kApart) tmem_store32(at_p, packed[0]);
                        }
                        l += sum;
                        if (!S::kApart) tmem_store32(at_p + h * 32, packed[h]);
                    };
                    if (ragged) clear_ragged(0);
                    if (i == g.begin) m = first(largest(0) * c);
                    half(0);
                    tmem_load32(r[2], at_s + 64);   // any earlier takes more registers than there are
                    tmem_load32(r[3], at_s + 96);
                    tmem_wait_load();
                    pin(r[2]);
                    pin(r[3]);
                    if (S::kApart) {
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) barrier_arrive(b_read + 8 * t);
                    }
                    if (ragged) clear_ragged(1);
                    half(1);
                    if (S::kApart) {
                        await_output();
                        tmem_store32(at_p, packed[0]);
                        tmem_store32(at_p + 32, packed[1]);
                    }
                    tmem_wait_store();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(b_p + 8 * t);
                }
                barrier_wait_warp(b_o + 8 * t, (n - 1) & 1, guard);
                tmem_fence_after();
            }
            if (g.length > 0) kv += 2 * (g.end - g.begin);
            if (!active) continue;
            const bool store = row < a.q_len;
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            const float lse = m * kLn2 + logf(l);
            const int slot = partial_slot(g, blockIdx.x);
            T *out = (T *)a.out + g.item * a.out_item + (int64_t)row * a.out_token + head * a.out_head;
            float *partial = a.partial + ((int64_t)slot * 2 * kRowTile + t * kRowTile + row_in_tile) * a.dim;
            for (int x = 0; x < HD; x += 32) {
                if (x >= a.dim) break;
                uint32_t o[32];
                __syncwarp();
                if (g.length > 0) {
                    tmem_load32(o, at_o + x);
                    tmem_wait_load();
                    pin(o);
                } else {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = 0;
                }
                if (store) {
                    float f[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) f[y] = inv == 0.0f ? 0.0f : __uint_as_float(o[y]) * inv;
                    store_results<T, true>(out + x, partial + x, whole, a.wide, a.dim - x, f);
                }
            }
            if (store) {
                if (whole)
                    a.lse[((int64_t)g.item * a.q_heads + head) * a.q_len + row] = lse;
                else
                    a.partial_lse[(int64_t)slot * 2 * kRowTile + t * kRowTile + row_in_tile] = lse;
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
    if (warp == 10) tmem_free(tmem, S::kColumns);
}

// Joins the parts of a cut tile: weights exp(lse_part - lse).  Block x handles the
// tile that the start of share x + 1 cuts, if that is the first share to start
// inside it; a thread takes 8 elements of a row (of four rows: 4 us
// longer, each a chain of loads).
constexpr int kJoinBlock = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinBlock) k_attention_join(const __grid_constant__ ForwardArgs a, int grid)
{
    grid_dependency_begin();
    Segment g;
    const int first = blockIdx.x + 1, chunks = a.dim / 8;
    int last;
    if (!cut_tile<QueryLine>(a.work, grid, first, g, last)) return;
    const int head = g.tile / a.row_tiles, row0 = (g.tile - head * a.row_tiles) * 2 * kRowTile;
    constexpr int kRows = 2 * kRowTile;
    const int slot0 = 2 * first - 1;   // then 2 b of the blocks b = first .. last
    const int i = blockIdx.y * kJoinBlock + threadIdx.x, r = i / chunks, c = (i - r * chunks) * 8;
    const int row = row0 + r;
    if (r >= kRows || row >= a.q_len) return;
    const float lse0 = a.partial_lse[(int64_t)slot0 * kRows + r];
    float top = lse0;
    for (int b = first; b <= last; ++b) top = fmaxf(top, a.partial_lse[(int64_t)2 * b * kRows + r]);
    const float shift = top == -INFINITY ? 0.0f : top;
    float total = 0.0f, o[8] = {};
    auto add = [&](int64_t slot, float lse) {
        const float w = expf(lse - shift);
        total += w;
        const float4 *p = (const float4 *)(a.partial + (slot * kRows + r) * a.dim + c);
        const float4 f = p[0], h = p[1];
        if (w != 0.0f) {
            o[0] = fmaf(w, f.x, o[0]);
            o[1] = fmaf(w, f.y, o[1]);
            o[2] = fmaf(w, f.z, o[2]);
            o[3] = fmaf(w, f.w, o[3]);
            o[4] = fmaf(w, h.x, o[4]);
            o[5] = fmaf(w, h.y, o[5]);
            o[6] = fmaf(w, h.z, o[6]);
            o[7] = fmaf(w, h.w, o[7]);
        }
    };
    add(slot0, lse0);
    for (int b = first; b <= last; ++b) add(2 * b, a.partial_lse[(int64_t)2 * b * kRows + r]);
    const float inv = total > 0.0f ? 1.0f / total : (total == 0.0f ? 0.0f : total);
    T *out = (T *)a.out + g.item * a.out_item + (int64_t)row * a.out_token + head * a.out_head + c;
    *(uint4 *)out = make_uint4(pack_average<T>(o[0] * inv, o[1] * inv), pack_average<T>(o[2] * inv, o[3] * inv),
                               pack_average<T>(o[4] * inv, o[5] * inv), pack_average<T>(o[6] * inv, o[7] * inv));
    if (c == 0) a.lse[((int64_t)g.item * a.q_heads + head) * a.q_len + row] = top + logf(total);
}

// Rows of an item without keys.
template <typename T>
__global__ void __launch_bounds__(256) k_attention_no_keys(void *out, int64_t item_stride, int64_t token_stride,
                                                           int64_t head_stride, float *lse, int64_t rows, int q_len,
                                                           int q_heads, int dim)
{
    grid_dependency_begin();
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (r >= rows) return;
    const int64_t i = r % q_len, h = r / q_len % q_heads, b = r / q_len / q_heads;
    T *o = (T *)out + b * item_stride + i * token_stride + h * head_stride;
    for (int c = 0; c < dim; c += 8) *(uint4 *)(o + c) = make_uint4(0, 0, 0, 0);
    if (lse) lse[r] = -INFINITY;
}

template <typename T, int HD>
int launch_forward(gsr_ctx *ctx, ForwardArgs &a, int blocks, cudaStream_t stream)
{
    auto *kernel = k_attention_forward<T, HD>;
    constexpr int smem = ForwardShape<HD>::kSmem;
    if (int rc = cuda_check(ctx, cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                            "k_attention_forward"))
        return rc;
    if (int rc = check_registers(ctx, (const void *)kernel, "k_attention_forward")) return rc;
    if (int rc = cuda_check(ctx, launch_kernel_smem(ctx, kernel, dim3((unsigned)blocks), kForwardThreads, smem, 1, stream, a),
                            "k_attention_forward"))
        return rc;
    if (blocks == 1 || a.work.length <= kKeyTile) return GSR_OK;   // tiles of one step are never cut
    const int vectors = 2 * kRowTile * a.dim / 8, each = kJoinBlock;
    return cuda_check(ctx, launch_kernel(ctx, k_attention_join<T>,
                                         dim3((unsigned)blocks - 1, (unsigned)((vectors + each - 1) / each)), kJoinBlock,
                                         stream, a, blocks),
                      "k_attention_join");
}

template <typename T>
int forward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k, const gsr_heads &v,
            const gsr_heads &out, float *lse, cudaStream_t stream)
{
    if (d.kv_len == 0) {
        const int64_t rows = (int64_t)d.batch * d.q_heads * d.q_len;
        return cuda_check(ctx, launch_kernel(ctx, k_attention_no_keys<T>, dim3((unsigned)((rows + 255) / 256)), 256,
                                             stream, out.data, out.batch_stride, out.token_stride, out.head_stride,
                                             lse, rows, (int)d.q_len, (int)d.q_heads, (int)d.head_dim),
                          "k_attention_no_keys");
    }
    ForwardArgs a = {};
    a.q_len = d.q_len;
    a.q_heads = d.q_heads;
    a.group = d.q_heads / d.kv_heads;
    a.dim = d.head_dim;
    a.row_tiles = (d.q_len + 2 * kRowTile - 1) / (2 * kRowTile);
    a.scale_log2 = d.scale * kLog2e;
    a.out = out.data;
    a.out_item = out.batch_stride;
    a.out_token = out.token_stride;
    a.out_head = out.head_stride;
    a.lse = lse;
    a.work = {d.batch, d.q_heads * a.row_tiles, 0, 0, d.kv_lengths, d.kv_len};
    const int64_t line = (int64_t)d.batch * a.work.tiles * ((d.kv_len + kKeyTile - 1) / kKeyTile);
    const int blocks = (int)(line < ctx->num_sms ? line : ctx->num_sms);
    const size_t rows = (size_t)2 * blocks * 2 * kRowTile;
    const size_t packed = d.key_mask ? round_up(packed_bytes(d), 256) : 0;
    const size_t partial = round_up(rows * d.head_dim * sizeof(float), 256);
    Workspace workspace(ctx, stream);
    void *work;
    if (int rc = workspace.take(packed + partial + rows * sizeof(float), &work)) return rc;
    a.partial = (float *)((unsigned char *)work + packed);
    a.partial_lse = (float *)((unsigned char *)work + packed + partial);
    a.status = ctx->status_dev;
    gsr_heads keys = k, values = v;
    if (d.key_mask) {
        Packed p;
        if (int rc = cuda_check(ctx, pack_keys(ctx, d, k, v, work, &p, stream), "k_pack_keys")) return rc;
        keys = p.k;
        values = p.v;
        a.work.lengths = p.counts;
    }
    a.wide = rows_of_32_bytes(out, d.head_dim);
    a.q_item = q.batch_stride != 0;
    a.q_head = q.head_stride != 0;
    a.k_item = keys.batch_stride != 0;
    a.k_head = keys.head_stride != 0;
    a.v_item = values.batch_stride != 0;
    a.v_head = values.head_stride != 0;
    if (int rc = heads_map(ctx, &a.q, q, d.dtype, d.batch, d.q_len, d.q_heads, d.head_dim, kRowTile)) return rc;
    if (int rc = heads_map(ctx, &a.k, keys, d.dtype, d.batch, d.kv_len, d.kv_heads, d.head_dim, kKeyTile)) return rc;
    if (int rc = heads_map(ctx, &a.v, values, d.dtype, d.batch, d.kv_len, d.kv_heads, d.head_dim, kKeyTile)) return rc;
    const int rc = d.head_dim <= 64 ? launch_forward<T, 64>(ctx, a, blocks, stream)
                                    : launch_forward<T, 128>(ctx, a, blocks, stream);
    if (rc) return rc;
    return workspace.done();
}

}  // namespace

int cross_attention_forward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k,
                            const gsr_heads &v, const gsr_heads &out, float *lse, cudaStream_t stream)
{
    if (d.kv_len > 0 && (int64_t)d.q_len * (d.q_heads / d.kv_heads) <= kFewRows)
        return few_rows_forward(ctx, d, q, k, v, out, lse, stream);
    return d.dtype == GSR_BF16 ? forward<__nv_bfloat16>(ctx, d, q, k, v, out, lse, stream)
                               : forward<__half>(ctx, d, q, k, v, out, lse, stream);
}

}  // namespace gsr
