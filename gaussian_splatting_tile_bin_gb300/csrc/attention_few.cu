// attention_few.cu -- cross attention of few query rows: single tokens, or a few,
// against a long row of keys.
//
//   s = scale q . k,  o = sum exp(s - m) v / l,  lse = m + log l
//
// Bound by HBM: k and v are read once and a row's products are a fraction of a
// tile of the tensor cores.  All query heads of a key head make one block of at
// most 16 rows, so their keys are read once; the keys of an item are split over
// enough blocks to keep copies in flight on every SM, and a second kernel joins
// the blocks' results in order.  In a block one warp copies tiles of 64 keys
// through a ring, four warps take 16 keys of each tile with m16n8k16 products on
// registers (a tcgen05 tile would be at most an eighth full, and would wait on
// tensor memory twice per tile) and keep their own running maximum, sum and
// output, which meet in shared memory at the end.
//
// 4 x 1 token, 16 query heads over 4 key heads of 128, 10,000 keys in bf16 (82 MB):
// 19 us with cold caches, which read those bytes once from DRAM (4.2 TB/s), and 8
// for the join; calls captured one behind the other, which start with part of the
// keys in L2, take 15.75 us, and from Python 21.
#include <math.h>

#include "attention.cuh"

namespace gsr {
namespace {

constexpr int kTileKeys = 64;
constexpr int kWarps = 4;
constexpr int kFewThreads = (kWarps + 1) * 32;
constexpr int kStages = 3;
constexpr float kLog2e = 1.4426950408889634f;

struct FewArgs {
    CUtensorMap k, v;
    const void *q;
    void *out;
    int64_t q_item, q_token, q_head, out_item, out_token, out_head;
    float *lse;
    float *partial;          // [item][key head][split][16][dim]
    float *partial_lse;      // [item][key head][split][16]
    const int32_t *lengths;
    const uint8_t *mask;
    uint32_t *status;
    int q_len, kv_len, q_heads, kv_heads, group, dim, splits;
    int k_item, k_head, v_item, v_head;
    float scale, scale_log2;
    uint32_t zero;           // 0, which the compiler does not know
};

template <int HD>
struct FewShape {
    static constexpr int kBlocks = HD / 64;
    static constexpr int kBlockBytes = kTileKeys * 128;
    static constexpr int kTileBytes = kBlocks * kBlockBytes;          // K or V
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kBars = 2 * kStages * 8;
    static constexpr int kMerge = kWarps * 16 * (HD + 2) * 4;         // after the loop, over the ring
    static_assert(kMerge <= kRing, "the merge reuses the ring");
    static constexpr int kSmem = 1024 + kRing + kBars + 16;
};

__device__ __forceinline__ void load_matrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void load_matrix4_across(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// d += a b: 16 rows, 8 columns, 16 terms.
template <typename T>
__device__ __forceinline__ void product16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
    return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}

__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(~0u, x, 1);
    return x + __shfl_xor_sync(~0u, x, 2);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kFewThreads) k_attention_few(const __grid_constant__ FewArgs a)
{
    grid_dependency_begin();
    using S = FewShape<HD>;
    extern __shared__ unsigned char s_raw[];
    const uint32_t raw = smem_address(s_raw);
    const uint32_t ring = (raw + 1023) & ~1023u, b_full = ring + S::kRing, b_free = b_full + 8 * kStages;
    uint32_t *s_abort = (uint32_t *)(s_raw + (b_free + 8 * kStages - raw));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const WaitGuard guard = {s_abort, a.status};
    if (threadIdx.x == 0) {
        *s_abort = 0;
        for (int i = 0; i < kStages; ++i) {
            barrier_init(b_full + 8 * i, 1);
            barrier_init(b_free + 8 * i, kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    __syncthreads();

    const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int key_head = unit % a.kv_heads, item = unit / a.kv_heads;
    const int length = item_length(a.lengths, a.kv_len, item);
    const int tiles = (length + kTileKeys - 1) / kTileKeys;
    const int first = (int)((int64_t)tiles * split / a.splits), last = (int)((int64_t)tiles * (split + 1) / a.splits);

    // Rows lane / 4 and lane / 4 + 8 of the block; row = token x group + head of the group.
    const int rows = a.q_len * a.group;
    float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

    if (warp == kWarps) {
        if (elect_one()) {
            for (int i = first; i < last; ++i) {
                if (guard.stop()) goto done;
                const int n = i - first, stage = n % kStages, round = n / kStages;
                if (round > 0) barrier_wait(b_free + 8 * stage, (round - 1) & 1, guard);
                const uint32_t bar = b_full + 8 * stage, to = ring + stage * S::kStageBytes;
                barrier_expect(bar, S::kStageBytes);
                for (int c = 0; c < S::kBlocks; ++c) {
                    copy_box(to + c * S::kBlockBytes, &a.k, bar, c * 64, i * kTileKeys, key_head * a.k_head,
                             item * a.k_item);
                    copy_box(to + S::kTileBytes + c * S::kBlockBytes, &a.v, bar, c * 64, i * kTileKeys,
                             key_head * a.v_head, item * a.v_item);
                }
            }
        }
    } else {
        uint32_t q[HD / 16][4];
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = lane / 4 + (e & 1) * 8, c = k * 16 + (lane % 4) * 2 + (e >> 1) * 8;
                q[k][e] = 0;
                if (r < rows && c < a.dim)
                    q[k][e] = *(const uint32_t *)((const T *)a.q + item * a.q_item + (r / a.group) * a.q_token +
                                                  (int64_t)(key_head * a.group + r % a.group) * a.q_head + c);
            }
        const float c = a.scale_log2;
        const int key0 = warp * 16;
        // This lane's row of the 8 x 8 blocks of a tile: keys for K, keys for V.
        const int k_row = key0 + (lane & 7) + (lane >> 4) * 8, k_chunk = lane >> 3 & 1;
        const int v_row = key0 + (lane & 7) + (lane >> 3 & 1) * 8, v_chunk = lane >> 4;
        // Whether one of this warp's 16 keys of a tile takes part, a tile ahead.
        auto takes_part = [&](int tile) {
            const int key = tile * kTileKeys + key0 + (lane & 15);
            if (key >= length) return false;
            return !a.mask || a.mask[(int64_t)item * a.kv_len + key] != 0;
        };
        bool valid = first < last && takes_part(first);
        for (int i = first; i < last; ++i) {
            const int n = i - first, stage = n % kStages;
            const uint32_t live = __ballot_sync(~0u, valid) & 0xffff;
            valid = takes_part(i + 1);
            barrier_wait_warp(b_full + 8 * stage, n / kStages & 1, guard);
            const uint32_t at_k = ring + stage * S::kStageBytes, at_v = at_k + S::kTileBytes;
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                uint32_t b[4];   // keys 0-7: two chunks of 8 dimensions, keys 8-15: two
                const int chunk = (k & 3) * 2 + k_chunk;
                load_matrix4(b, at_k + (k >> 2) * S::kBlockBytes + k_row * 128 + ((chunk ^ (k_row & 7)) << 4));
                product16<T>(s[0], q[k], b[0], b[1]);
                product16<T>(s[1], q[k], b[2], b[3]);
            }
            if (live != 0xffff) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(live >> (t * 8 + (lane % 4) * 2 + (e & 1)) & 1)) s[t][e] = -INFINITY;
            }
            uint32_t p[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float top = quad_max(fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])));
                const float next = fmaxf(m[r], top);
                // The difference first: where the maximum stays, `keep` is 1, and not what
                // the rounding of m c leaves, tile after tile.
                const float from = next == -INFINITY ? 0.0f : next;
                const float keep = exp2_fast((m[r] - from) * c);
                m[r] = next;
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) e[x] = exp2_fast((s[x >> 1][2 * r + (x & 1)] - from) * c);
                l[r] = fmaf(l[r], keep, (e[0] + e[1]) + (e[2] + e[3]));
                p[r] = pack2<T>(e[0], e[1]);
                p[r + 2] = pack2<T>(e[2], e[3]);
#pragma unroll
                for (int x = 0; x < HD / 8; ++x) {
                    o[x][2 * r] *= keep;
                    o[x][2 * r + 1] *= keep;
                }
            }
            // Words of V's operand hold keys 2 (lane % 4) + {0, 1} (+ 8): clear the invalid ones.
            const uint32_t pair0 = live >> ((lane % 4) * 2), pair1 = pair0 >> 8;
            const uint32_t keep0 = (pair0 & 1 ? 0xffffu : 0u) | (pair0 & 2 ? 0xffff0000u : 0u);
            const uint32_t keep1 = (pair1 & 1 ? 0xffffu : 0u) | (pair1 & 2 ? 0xffff0000u : 0u);
            uint32_t seen = p[0];   // of all of K
#pragma unroll
            for (int x = 0; x < HD / 16; ++x) {
                uint32_t b[4];   // dimensions 0-7: keys 0-7 and 8-15, dimensions 8-15: the same
                const int chunk = (x & 3) * 2 + v_chunk;
                load_matrix4_across(b, at_v + (x >> 2) * S::kBlockBytes + v_row * 128 + ((chunk ^ (v_row & 7)) << 4));
                seen |= b[0];
                product16<T>(o[2 * x], p, b[0] & keep0, b[1] & keep1);
                product16<T>(o[2 * x + 1], p, b[2] & keep0, b[3] & keep1);
            }
            // The stage is free once its fragments are in registers, which nothing here
            // waits for: the products may well run behind this point, and a warp that is
            // held up beside another kernel's then reads the next tile.  So the arrival
            // depends on what every load has brought.
            fence_async();
            __syncwarp();
            if (lane == 0) barrier_arrive(b_free + 8 * stage + (seen & a.zero));
        }
    }

done:
    __syncwarp();
    drain_if_aborted(guard);

    // The four warps' parts: [warp][row][dim], then maxima and sums, over the ring
    // (every copy has landed: each was waited for by every warp).
    __syncthreads();
    float *s_o = (float *)(s_raw + (ring - raw)), *s_m = s_o + kWarps * 16 * HD, *s_l = s_m + kWarps * 16;
    if (warp < kWarps) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = lane / 4 + r * 8;
            const float sum = quad_sum(l[r]);
#pragma unroll
            for (int x = 0; x < HD / 8; ++x)
                *(float2 *)&s_o[(warp * 16 + row) * HD + x * 8 + (lane % 4) * 2] = make_float2(o[x][2 * r], o[x][2 * r + 1]);
            if (lane % 4 == 0) {
                s_m[warp * 16 + row] = m[r];
                s_l[warp * 16 + row] = sum;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (HD / 2); i += kFewThreads) {
        const int row = i / (HD / 2), d = i % (HD / 2) * 2;
        if (d >= a.dim) continue;
        float top = -INFINITY;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * 16 + row]);
        const float from = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
        float2 f = make_float2(0.0f, 0.0f);
        for (int w = 0; w < kWarps; ++w) {
            const float weight = exp2_fast((s_m[w * 16 + row] - from) * a.scale_log2);
            const float2 g = *(const float2 *)&s_o[(w * 16 + row) * HD + d];
            sum = fmaf(weight, s_l[w * 16 + row], sum);
            if (weight != 0.0f) f = make_float2(fmaf(weight, g.x, f.x), fmaf(weight, g.y, f.y));
        }
        const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
        f = make_float2(f.x * inv, f.y * inv);
        const float lse = top * a.scale + logf(sum);
        const int token = row / a.group, head = key_head * a.group + row % a.group;
        if (a.splits == 1) {
            *(uint32_t *)((T *)a.out + item * a.out_item + token * a.out_token + head * a.out_head + d) =
                pack_average<T>(f.x, f.y);
            if (d == 0) a.lse[((int64_t)item * a.q_heads + head) * a.q_len + token] = lse;
        } else {
            const int64_t part = (int64_t)blockIdx.x * 16 + row;
            *(float2 *)(a.partial + part * a.dim + d) = f;
            if (d == 0) a.partial_lse[part] = lse;
        }
    }
}

// Joins the splits of a row, one block a row: a warp takes every fourth split, four
// dimensions a lane, and the warps' sums meet in shared memory in their order.
constexpr int kFewJoinWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kFewJoinWarps * 32) k_attention_few_join(const __grid_constant__ FewArgs a)
{
    grid_dependency_begin();
    __shared__ float4 s_o[kFewJoinWarps][32];
    __shared__ float s_total[kFewJoinWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r = blockIdx.x;
    const int per_unit = a.q_len * a.group, row = (int)(r % per_unit);
    const int64_t unit = r / per_unit, item = unit / a.kv_heads;
    const int token = row / a.group, head = (int)(unit % a.kv_heads) * a.group + row % a.group;
    const int64_t part0 = unit * a.splits * 16 + row;
    float top = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.partial_lse[part0 + s * 16]);
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float shift = top == -INFINITY ? 0.0f : top;
    float total = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool mine = lane * 4 < a.dim;
#pragma unroll 4
    for (int s = warp; s < a.splits; s += kFewJoinWarps) {
        const float w = expf(a.partial_lse[part0 + s * 16] - shift);
        total += w;
        if (mine) {
            const float4 f = *(const float4 *)(a.partial + (part0 + s * 16) * a.dim + lane * 4);
            o.x = fmaf(w, f.x, o.x);
            o.y = fmaf(w, f.y, o.y);
            o.z = fmaf(w, f.z, o.z);
            o.w = fmaf(w, f.w, o.w);
        }
    }
    s_o[warp][lane] = o;
    if (lane == 0) s_total[warp] = total;
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < kFewJoinWarps; ++w) {
        const float4 f = s_o[w][lane];
        o = make_float4(o.x + f.x, o.y + f.y, o.z + f.z, o.w + f.w);
        total += s_total[w];
    }
    const float inv = total > 0.0f ? 1.0f / total : (total == 0.0f ? 0.0f : total);
    if (mine)
        *(uint2 *)((T *)a.out + item * a.out_item + token * a.out_token + head * a.out_head + lane * 4) =
            make_uint2(pack_average<T>(o.x * inv, o.y * inv), pack_average<T>(o.z * inv, o.w * inv));
    if (lane == 0) a.lse[(item * a.q_heads + head) * a.q_len + token] = top + logf(total);
}

template <typename T, int HD>
int launch_few(gsr_ctx *ctx, const FewArgs &a, int64_t units, cudaStream_t stream)
{
    auto *kernel = k_attention_few<T, HD>;
    constexpr int smem = FewShape<HD>::kSmem;
    if (int rc = cuda_check(ctx, cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                            "k_attention_few"))
        return rc;
    if (int rc = cuda_check(ctx, launch_kernel_smem(ctx, kernel, dim3((unsigned)(units * a.splits)), kFewThreads, smem, 1,
                                                    stream, a),
                            "k_attention_few"))
        return rc;
    if (a.splits == 1) return GSR_OK;
    const int64_t rows = units * a.q_len * a.group;
    return cuda_check(ctx, launch_kernel(ctx, k_attention_few_join<T>, dim3((unsigned)rows), kFewJoinWarps * 32, stream, a),
                      "k_attention_few_join");
}

}  // namespace

int few_rows_forward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k, const gsr_heads &v,
                     const gsr_heads &out, float *lse, cudaStream_t stream)
{
    FewArgs a = {};
    a.q = q.data;
    a.q_item = q.batch_stride;
    a.q_token = q.token_stride;
    a.q_head = q.head_stride;
    a.out = out.data;
    a.out_item = out.batch_stride;
    a.out_token = out.token_stride;
    a.out_head = out.head_stride;
    a.lse = lse;
    a.lengths = d.kv_lengths;
    a.mask = d.key_mask;
    a.q_len = d.q_len;
    a.kv_len = d.kv_len;
    a.q_heads = d.q_heads;
    a.kv_heads = d.kv_heads;
    a.group = d.q_heads / d.kv_heads;
    a.dim = d.head_dim;
    a.scale = d.scale;
    a.scale_log2 = d.scale * kLog2e;
    a.k_item = k.batch_stride != 0;
    a.k_head = k.head_stride != 0;
    a.v_item = v.batch_stride != 0;
    a.v_head = v.head_stride != 0;
    // Two blocks an SM keep their rings' copies in flight; a split of fewer than
    // four tiles costs more to join than it saves.
    const int64_t units = (int64_t)d.batch * d.kv_heads, tiles = (d.kv_len + kTileKeys - 1) / kTileKeys;
    int64_t splits = 2 * (int64_t)ctx->num_sms / units;
    if (splits > tiles / 4) splits = tiles / 4;
    a.splits = (int)(splits < 1 ? 1 : splits);
    const size_t parts = a.splits > 1 ? (size_t)units * a.splits * 16 : 0;
    const size_t partial = round_up(parts * d.head_dim * sizeof(float), 256);
    Workspace workspace(ctx, stream);
    void *work;
    if (int rc = workspace.take(partial + parts * sizeof(float), &work)) return rc;
    a.partial = (float *)work;
    a.partial_lse = (float *)((unsigned char *)work + partial);
    a.status = ctx->status_dev;
    if (int rc = heads_map(ctx, &a.k, k, d.dtype, d.batch, d.kv_len, d.kv_heads, d.head_dim, kTileKeys)) return rc;
    if (int rc = heads_map(ctx, &a.v, v, d.dtype, d.batch, d.kv_len, d.kv_heads, d.head_dim, kTileKeys)) return rc;
    int rc;
    if (d.dtype == GSR_BF16)
        rc = d.head_dim <= 64 ? launch_few<__nv_bfloat16, 64>(ctx, a, units, stream)
                              : launch_few<__nv_bfloat16, 128>(ctx, a, units, stream);
    else
        rc = d.head_dim <= 64 ? launch_few<__half, 64>(ctx, a, units, stream)
                              : launch_few<__half, 128>(ctx, a, units, stream);
    if (rc) return rc;
    return workspace.done();
}

}  // namespace gsr
