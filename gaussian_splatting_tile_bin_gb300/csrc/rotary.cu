// rotary.cu -- rotary positions with several axes (view, row, column of a patch;
// any coordinates of a Gaussian token), forward and backward.
//
// Pair i of a head turns by theta = p[a(i)] f[i], a(i) the axis whose section
// holds i: (u, v) -> (u cos - v sin, u sin + v cos).  The backward is the
// rotation by -theta, so both directions are one kernel with a sign.
//
// Bound by HBM: every element is read and written once.  A token's sines and
// cosines serve all of its heads, so a block takes a few tokens, evaluates their
// angles once into shared memory while its loads of x are in flight, and turns.
#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kRotaryBlock = 256;
// Items of a thread whose loads are in flight together: 32 bytes of them, so that
// eight blocks fit an SM (one item and eight blocks 29 us, two and six 31, two and
// four 34; 2 x 10,000 x 16 heads x 128 in bf16).
template <int V, bool INTERLEAVED>
constexpr int kRotaryItems = !INTERLEAVED && V > 1 ? 1 : 2;
constexpr int kRotaryTable = 4096;   // (token, pair) angles of a block

// Results pass through L2 without staying: 34 instead of 42 us for the size below.
template <typename A>
__device__ __forceinline__ void store_streaming(A *p, const A &v)
{
    if constexpr (sizeof(A) == 16)
        __stcs((uint4 *)p, *(const uint4 *)&v);
    else
        *p = v;
}

struct RotaryArgs {
    const void *x;
    void *out;
    int64_t x_batch, x_token, x_head, out_batch, out_token, out_head;
    const void *positions;
    const float *frequencies;
    int64_t positions_batch;
    int64_t all_tokens;     // batch * tokens
    int block_runs, slots;  // runs of a block, and threads of a run
    int tokens, heads, block_tokens;
    int pairs, dim;
    int turn_runs, runs;    // runs that turn, and with the copied ones
    int axes, positions_int;
    int section_end[GSR_MAX_AXES];
    float sign;
};

// sin and cos of p * f with the product to twice float's length: hi + lo is the
// exact product (up to the rounding of lo's own small terms), and the rotation
// by lo is applied to the sine and cosine of hi.
__device__ __forceinline__ void sincos_product(float p_hi, float p_lo, float f, float *s, float *c)
{
    const float hi = p_hi * f;
    const float lo = fmaf(p_lo, f, fmaf(p_hi, f, -hi));
    float sh, ch;
    sincosf(hi, &sh, &ch);
    float sl = lo, cl = 1.0f;                    // |lo| < 1e-4: cos lo = 1 within half an ulp
    if (!(fabsf(lo) < 1e-4f)) sincosf(lo, &sl, &cl);
    *s = fmaf(sh, cl, ch * sl);
    *c = fmaf(ch, cl, -sh * sl);
}

// V is the width of an access in elements; a run is V pairs (halves) or V / 2
// pairs (interleaved), one pair with scalar accesses, or V copied dimensions.  An
// item is one run of one head of one token.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryBlock, 8) k_rotary(const RotaryArgs a)
{
    grid_dependency_begin();
    extern __shared__ float2 s_turn[];   // (cos, sin) of [token][pair]
    constexpr int P = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;
    // Vectorised interleaved pairs sit in one access, the others in two.
    constexpr bool kOne = INTERLEAVED && V > 1;
    constexpr int kItems = kRotaryItems<V, INTERLEAVED>;
    using Access = Vec<T, V>;
    const int64_t token0 = (int64_t)blockIdx.x * a.block_tokens;
    const int count = (int)min((int64_t)a.block_tokens, a.all_tokens - token0);
    // A thread keeps its run; its rows (token, head) are `slots` apart.
    const int run = blockIdx.y * a.block_runs + threadIdx.x % a.block_runs, slot = threadIdx.x / a.block_runs;
    const int64_t item0 = token0 / a.tokens;
    const int at0 = (int)(token0 - item0 * a.tokens);
    const bool turns = run < a.turn_runs;
    const int second = INTERLEAVED ? 1 : a.pairs;
    const int d = turns ? (INTERLEAVED ? 2 * P : P) * run : 2 * a.pairs + (run - a.turn_runs) * V;
    const T *x = (const T *)a.x + d;
    T *out = (T *)a.out + d;
    const int step_t = a.slots / a.heads, step_h = a.slots - step_t * a.heads;
    struct Row {
        int t, h;
    };
    auto advance = [&](Row &r) {
        r.t += step_t;
        r.h += step_h;
        if (r.h >= a.heads) {
            r.h -= a.heads;
            ++r.t;
        }
    };
    // Element offset of a row; a block's tokens may run over an item's end.
    auto offset = [&](const Row &r, int64_t batch, int64_t token, int64_t head) {
        int64_t b = item0;
        int at = at0 + r.t;
        if (at >= a.tokens) {
            b += at / a.tokens;
            at %= a.tokens;
        }
        return b * batch + at * token + r.h * head;
    };
    const bool mine = slot < a.slots && run < a.runs;
    Row row = {slot / a.heads, slot - slot / a.heads * a.heads};
    Row rows[kItems];
    Access u[kItems], v[kItems];
    auto load = [&] {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            rows[k] = row;
            advance(row);
            if (mine && rows[k].t < count) {
                const T *from = x + offset(rows[k], a.x_batch, a.x_token, a.x_head);
                u[k] = *(const Access *)from;
                if (!kOne && turns) v[k] = *(const Access *)(from + second);
            }
        }
    };
    load();

    for (int i = threadIdx.x; i < count * a.pairs; i += kRotaryBlock) {
        const int t = i / a.pairs, j = i - t * a.pairs;
        int axis = 0;
#pragma unroll
        for (int k = 0; k < GSR_MAX_AXES - 1; ++k)
            if (k < a.axes - 1 && j >= a.section_end[k]) axis = k + 1;
        const int64_t at = offset({t, 0}, a.positions_batch, a.axes, 0) + axis;
        float hi, lo = 0.0f;
        if (a.positions_int) {
            const int p = ((const int *)a.positions)[at];
            hi = (float)p;
            if (abs(p) >= 1 << 24 || p < -(1 << 24)) lo = (float)((long long)p - (long long)hi);
        } else {
            hi = ((const float *)a.positions)[at];
        }
        float s, c;
        sincos_product(hi, lo, a.frequencies[j], &s, &c);
        s_turn[i] = make_float2(c, s * a.sign);
    }
    __syncthreads();

    for (;;) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (!mine || rows[k].t >= count) continue;
            T *to = out + offset(rows[k], a.out_batch, a.out_token, a.out_head);
            if (turns) {
                const float2 *turn = s_turn + rows[k].t * a.pairs + run * P;
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    T &eu = kOne ? u[k].e[(2 * j) % V] : u[k].e[j % V];
                    T &ev = kOne ? u[k].e[(2 * j + 1) % V] : v[k].e[j % V];
                    const float fu = to_float(eu), fv = to_float(ev);
                    eu = from_float<T>(fmaf(fu, turn[j].x, -fv * turn[j].y));
                    ev = from_float<T>(fmaf(fu, turn[j].y, fv * turn[j].x));
                }
                if (!kOne) store_streaming((Access *)(to + second), v[k]);
            }
            store_streaming((Access *)to, u[k]);
        }
        if (!mine || row.t >= count) break;
        load();
    }
}

template <typename T, int V>
cudaError_t launch_rotary(gsr_ctx *ctx, RotaryArgs &a, bool interleaved, int64_t tokens, cudaStream_t stream)
{
    const int per_run = interleaved ? (V > 1 ? V / 2 : 1) : V;
    a.turn_runs = a.pairs / per_run;
    a.runs = a.turn_runs + (a.dim - 2 * a.pairs) / V;
    a.all_tokens = tokens;
    a.block_runs = a.runs < kRotaryBlock ? a.runs : kRotaryBlock;
    a.slots = kRotaryBlock / a.block_runs;
    // Tokens of a block: two rounds of loads a thread; fewer where that leaves SMs
    // idle, and no more angles than the table holds.
    const int items = interleaved ? kRotaryItems<V, true> : kRotaryItems<V, false>;
    int64_t n = 2 * items * kRotaryBlock / ((int64_t)a.heads * a.runs);
    const int64_t spread = (tokens + 2 * ctx->num_sms - 1) / (2 * ctx->num_sms);
    if (n > spread) n = spread;
    if (a.pairs > 0 && n > kRotaryTable / a.pairs) n = kRotaryTable / a.pairs;
    a.block_tokens = (int)(n < 1 ? 1 : n);
    const dim3 grid((unsigned)((tokens + a.block_tokens - 1) / a.block_tokens),
                    (unsigned)((a.runs + a.block_runs - 1) / a.block_runs));
    const size_t table = (size_t)a.block_tokens * a.pairs * sizeof(float2);
    if (interleaved) return launch_kernel_smem(ctx, k_rotary<T, V, true>, grid, kRotaryBlock, table, 1, stream, a);
    return launch_kernel_smem(ctx, k_rotary<T, V, false>, grid, kRotaryBlock, table, 1, stream, a);
}

// Largest access of at most 16 bytes that divides every offset the kernel forms.
int access_width(const gsr_rotary &d, int pairs, const gsr_heads &x, const gsr_heads &out, int size)
{
    for (int v = 16 / size; v > 1; v /= 2) {
        const int bytes = v * size;
        bool ok = ((uintptr_t)x.data % bytes) == 0 && ((uintptr_t)out.data % bytes) == 0 && d.head_dim % v == 0;
        ok = ok && (d.interleaved ? (2 * pairs) % v == 0 : pairs % v == 0);
        for (const gsr_heads *t : {&x, &out})
            ok = ok && (d.batch == 1 || t->batch_stride % v == 0) && (d.tokens == 1 || t->token_stride % v == 0) &&
                 (d.heads == 1 || t->head_stride % v == 0);
        if (ok) return v;
    }
    return 1;
}

template <typename T>
cudaError_t dispatch_rotary(gsr_ctx *ctx, RotaryArgs &a, const gsr_rotary &d, int width, cudaStream_t stream)
{
    constexpr int kFull = 16 / (int)sizeof(T);
    const int64_t tokens = (int64_t)d.batch * d.tokens;
    if (width == kFull) return launch_rotary<T, kFull>(ctx, a, d.interleaved, tokens, stream);
    if (width == kFull / 2) return launch_rotary<T, kFull / 2>(ctx, a, d.interleaved, tokens, stream);
    return launch_rotary<T, 1>(ctx, a, d.interleaved, tokens, stream);
}

}  // namespace

int rotary(gsr_ctx *ctx, const gsr_rotary &d, const gsr_heads &x, const void *positions, const float *frequencies,
           const gsr_heads &out, float sign, cudaStream_t stream)
{
    RotaryArgs a = {};
    a.x = x.data;
    a.out = out.data;
    a.x_batch = x.batch_stride;
    a.x_token = x.token_stride;
    a.x_head = x.head_stride;
    a.out_batch = out.batch_stride;
    a.out_token = out.token_stride;
    a.out_head = out.head_stride;
    a.positions = positions;
    a.frequencies = frequencies;
    a.positions_batch = d.positions_batch_stride;
    a.tokens = d.tokens;
    a.heads = d.heads;
    a.dim = d.head_dim;
    a.axes = d.axes;
    a.positions_int = d.positions_int;
    a.sign = sign;
    for (int k = 0; k < d.axes; ++k) a.section_end[k] = a.pairs += d.sections[k];
    const int size = d.dtype == GSR_F32 ? 4 : 2;
    const int width = access_width(d, a.pairs, x, out, size);
    cudaError_t e;
    if (d.dtype == GSR_F32)
        e = dispatch_rotary<float>(ctx, a, d, width, stream);
    else if (d.dtype == GSR_BF16)
        e = dispatch_rotary<__nv_bfloat16>(ctx, a, d, width, stream);
    else
        e = dispatch_rotary<__half>(ctx, a, d, width, stream);
    return cuda_check(ctx, e, "k_rotary");
}

}  // namespace gsr
