// rotary.cu -- rotary positions with several axes (view, row, column of a patch;
// any coordinates of a Gaussian token), forward and backward.
//
// Pair i of a head turns by theta = p[a(i)] f[i], a(i) the axis whose section
// holds i: (u, v) -> (u cos - v sin, u sin + v cos).  The backward is the
// rotation by -theta, so both directions are one kernel with a sign.
//
// Bound by HBM: every element is read and written once, and a token's sines and
// cosines serve all of its heads, so a thread owns one run of pairs of a token,
// evaluates their angles once and walks the heads with them.
#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kRotaryBlock = 256;
constexpr int kRotaryHeads = 4;   // heads whose loads are in flight together

struct RotaryArgs {
    const void *x;
    void *out;
    int64_t x_batch, x_token, x_head, out_batch, out_token, out_head;
    const void *positions;
    const float *frequencies;
    int64_t positions_batch;
    int64_t items;          // (token, run) items
    int tokens, heads, heads_per_block;
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
// pairs (interleaved), one pair with scalar accesses.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryBlock) k_rotary(const RotaryArgs a)
{
    grid_dependency_begin();
    constexpr int P = INTERLEAVED ? (V > 1 ? V / 2 : 1) : V;
    using Access = Vec<T, V>;
    const int64_t item = (int64_t)blockIdx.x * kRotaryBlock + threadIdx.x;
    if (item >= a.items) return;
    int64_t token;
    int run;
    if (a.items <= 0x7fffffff) {
        token = (uint32_t)item / (uint32_t)a.runs;
        run = (int)((uint32_t)item - (uint32_t)token * (uint32_t)a.runs);
    } else {
        token = item / a.runs;
        run = (int)(item - token * a.runs);
    }
    const int64_t b = token / a.tokens;
    const int64_t t = token - b * a.tokens;
    const int head0 = blockIdx.y * a.heads_per_block;
    const int head1 = min(a.heads, head0 + a.heads_per_block);
    const T *x = (const T *)a.x + b * a.x_batch + t * a.x_token;
    T *out = (T *)a.out + b * a.out_batch + t * a.out_token;

    if (run >= a.turn_runs) {   // dimensions behind the pairs
        const int d = 2 * a.pairs + (run - a.turn_runs) * V;
        for (int h = head0; h < head1; ++h)
            *(Access *)(out + h * a.out_head + d) = *(const Access *)(x + h * a.x_head + d);
        return;
    }

    float s[P], c[P];
    const int64_t at = b * a.positions_batch + t * a.axes;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int i = run * P + j;
        int axis = 0;
#pragma unroll
        for (int k = 0; k < GSR_MAX_AXES - 1; ++k)
            if (k < a.axes - 1 && i >= a.section_end[k]) axis = k + 1;
        float hi, lo = 0.0f;
        if (a.positions_int) {
            const int p = ((const int *)a.positions)[at + axis];
            hi = (float)p;
            lo = (float)((double)p - (double)hi);
        } else {
            hi = ((const float *)a.positions)[at + axis];
        }
        sincos_product(hi, lo, a.frequencies[i], &s[j], &c[j]);
        s[j] *= a.sign;
    }

    const int first = INTERLEAVED ? run * P * 2 : run * P;
    const int second = INTERLEAVED ? first + 1 : first + a.pairs;
    // Vectorised interleaved pairs sit in one access, the others in two.
    constexpr bool kOne = INTERLEAVED && V > 1;
    for (int h = head0; h < head1; h += kRotaryHeads) {
        Access u[kRotaryHeads], v[kRotaryHeads];
#pragma unroll
        for (int k = 0; k < kRotaryHeads; ++k)
            if (h + k < head1) {
                u[k] = *(const Access *)(x + (h + k) * a.x_head + first);
                if (!kOne) v[k] = *(const Access *)(x + (h + k) * a.x_head + second);
            }
#pragma unroll
        for (int k = 0; k < kRotaryHeads; ++k)
            if (h + k < head1) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    T &eu = kOne ? u[k].e[(2 * j) % V] : u[k].e[j % V];
                    T &ev = kOne ? u[k].e[(2 * j + 1) % V] : v[k].e[j % V];
                    const float fu = to_float(eu), fv = to_float(ev);
                    eu = from_float<T>(fmaf(fu, c[j], -fv * s[j]));
                    ev = from_float<T>(fmaf(fu, s[j], fv * c[j]));
                }
                *(Access *)(out + (h + k) * a.out_head + first) = u[k];
                if (!kOne) *(Access *)(out + (h + k) * a.out_head + second) = v[k];
            }
    }
}

template <typename T, int V>
cudaError_t launch_rotary(gsr_ctx *ctx, RotaryArgs &a, bool interleaved, int64_t tokens, cudaStream_t stream)
{
    const int per_run = interleaved ? (V > 1 ? V / 2 : 1) : V;
    a.turn_runs = a.pairs / per_run;
    a.runs = a.turn_runs + (a.dim - 2 * a.pairs) / V;
    a.items = tokens * a.runs;
    const int64_t blocks = (a.items + kRotaryBlock - 1) / kRotaryBlock;
    // All heads in one thread share its sines and cosines; few tokens spread them
    // over more blocks so that every SM has work.
    const int64_t want = (8 * (int64_t)ctx->num_sms + blocks - 1) / blocks;
    int64_t parts = (a.heads + kRotaryHeads - 1) / kRotaryHeads;
    if (parts > want) parts = want;
    a.heads_per_block = (int)((a.heads + parts - 1) / parts);
    a.heads_per_block = (a.heads_per_block + kRotaryHeads - 1) / kRotaryHeads * kRotaryHeads;
    const dim3 grid((unsigned)blocks, (unsigned)((a.heads + a.heads_per_block - 1) / a.heads_per_block));
    if (interleaved) return launch_kernel(ctx, k_rotary<T, V, true>, grid, kRotaryBlock, stream, a);
    return launch_kernel(ctx, k_rotary<T, V, false>, grid, kRotaryBlock, stream, a);
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
