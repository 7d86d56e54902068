// attention.cu -- cross attention to an encoder's states of another length,
// forward and backward, in its simplest form: one warp per row.
//
//   s = scale q . k over the valid keys,  lse = log sum exp s,  o = sum exp(s - lse) v
//   delta = do . o,  p = exp(s - lse),  ds = p (do . v - delta)
//   dq = scale sum ds k,  dk = scale sum ds q,  dv = sum p do
#include <math.h>

#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDim = GSR_ATTENTION_MAX_HEAD_DIM;
constexpr int kPerLane = kMaxDim / 32;

struct AttentionArgs {
    gsr_attention d;
    gsr_heads q, k, v, out, dout, dq, dk, dv;
    float *lse;
    float *delta;   // [batch, q_heads, q_len]
};

template <typename T>
__device__ __forceinline__ T *row_of(const gsr_heads &t, int64_t b, int64_t i, int64_t h)
{
    return (T *)t.data + b * t.batch_stride + i * t.token_stride + h * t.head_stride;
}

__device__ __forceinline__ bool valid_key(const gsr_attention &d, int64_t b, int j)
{
    if (j >= d.kv_len || (d.kv_lengths && j >= d.kv_lengths[b])) return false;
    return !d.key_mask || d.key_mask[b * d.kv_len + j] != 0;
}

template <typename T>
__device__ __forceinline__ float dot(const float *a, const T *b, int dim)
{
    float s = 0.0f;
    for (int c = 0; c < dim; c += 8) {
        const Vec<T, 8> v = *(const Vec<T, 8> *)(b + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(a[c + e], to_float(v.e[e]), s);
    }
    return s;
}

__device__ __forceinline__ float warp_sum(float x)
{
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

template <typename T>
__device__ __forceinline__ void stage(float *to, const T *from, int dim, int lane)
{
    for (int c = lane; c < dim; c += 32) to[c] = to_float(from[c]);
    __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_attention_grad_rows(const AttentionArgs a)
{
    grid_dependency_begin();
    __shared__ float s_q[kWarps][kMaxDim], s_do[kWarps][kMaxDim];
    const gsr_attention &d = a.d;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * kWarps + warp;
    if (r >= (int64_t)d.batch * d.q_heads * d.q_len) return;
    const int64_t i = r % d.q_len, h = r / d.q_len % d.q_heads, b = r / d.q_len / d.q_heads;
    const int64_t hk = h / (d.q_heads / d.kv_heads);
    stage(s_q[warp], row_of<T>(a.q, b, i, h), d.head_dim, lane);
    stage(s_do[warp], row_of<T>(a.dout, b, i, h), d.head_dim, lane);
    const T *out = row_of<T>(a.out, b, i, h);
    float delta = 0.0f;
    for (int c = lane; c < d.head_dim; c += 32) delta = fmaf(s_do[warp][c], to_float(out[c]), delta);
    delta = warp_sum(delta);
    if (lane == 0) a.delta[r] = delta;
    const float lse = a.lse[r];
    float g[kPerLane] = {};
    for (int j0 = 0; j0 < d.kv_len; j0 += 32) {
        const int j = j0 + lane;
        const bool ok = valid_key(d, b, j);
        const unsigned live = __ballot_sync(~0u, ok);
        float ds = 0.0f;
        if (ok) {
            const float p = expf(d.scale * dot(s_q[warp], row_of<T>(a.k, b, j, hk), d.head_dim) - lse);
            ds = p * (dot(s_do[warp], row_of<T>(a.v, b, j, hk), d.head_dim) - delta);
        }
        for (int n = 0; n < 32; ++n) {
            if (!(live >> n & 1)) continue;
            const float w = __shfl_sync(~0u, ds, n);
            const T *k = row_of<T>(a.k, b, j0 + n, hk);
            for (int e = 0; e < kPerLane; ++e)
                if (lane + 32 * e < d.head_dim) g[e] = fmaf(w, to_float(k[lane + 32 * e]), g[e]);
        }
    }
    T *dq = row_of<T>(a.dq, b, i, h);
    for (int e = 0; e < kPerLane; ++e)
        if (lane + 32 * e < d.head_dim) dq[lane + 32 * e] = from_float<T>(g[e] * d.scale);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_attention_grad_keys(const AttentionArgs a)
{
    grid_dependency_begin();
    __shared__ float s_k[kWarps][kMaxDim], s_v[kWarps][kMaxDim];
    const gsr_attention &d = a.d;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * kWarps + warp;
    if (r >= (int64_t)d.batch * d.kv_heads * d.kv_len) return;
    const int64_t j = r % d.kv_len, hk = r / d.kv_len % d.kv_heads, b = r / d.kv_len / d.kv_heads;
    const int group = d.q_heads / d.kv_heads;
    float gk[kPerLane] = {}, gv[kPerLane] = {};
    if (valid_key(d, b, (int)j)) {
        stage(s_k[warp], row_of<T>(a.k, b, j, hk), d.head_dim, lane);
        stage(s_v[warp], row_of<T>(a.v, b, j, hk), d.head_dim, lane);
        for (int64_t h = hk * group; h < (hk + 1) * group; ++h)
            for (int i0 = 0; i0 < d.q_len; i0 += 32) {
                const int i = i0 + lane;
                float p = 0.0f, ds = 0.0f;
                if (i < d.q_len) {
                    const int64_t at = (b * d.q_heads + h) * d.q_len + i;
                    p = expf(d.scale * dot(s_k[warp], row_of<T>(a.q, b, i, h), d.head_dim) - a.lse[at]);
                    ds = p * (dot(s_v[warp], row_of<T>(a.dout, b, i, h), d.head_dim) - a.delta[at]);
                }
                for (int n = 0; n < 32 && i0 + n < d.q_len; ++n) {
                    const float pn = __shfl_sync(~0u, p, n), dn = __shfl_sync(~0u, ds, n);
                    const T *q = row_of<T>(a.q, b, i0 + n, h), *dout = row_of<T>(a.dout, b, i0 + n, h);
                    for (int e = 0; e < kPerLane; ++e)
                        if (lane + 32 * e < d.head_dim) {
                            gk[e] = fmaf(dn, to_float(q[lane + 32 * e]), gk[e]);
                            gv[e] = fmaf(pn, to_float(dout[lane + 32 * e]), gv[e]);
                        }
                }
            }
    }
    T *dk = row_of<T>(a.dk, b, j, hk), *dv = row_of<T>(a.dv, b, j, hk);
    for (int e = 0; e < kPerLane; ++e)
        if (lane + 32 * e < d.head_dim) {
            dk[lane + 32 * e] = from_float<T>(gk[e] * d.scale);
            dv[lane + 32 * e] = from_float<T>(gv[e]);
        }
}

dim3 warp_grid(int64_t rows) { return dim3((unsigned)((rows + kWarps - 1) / kWarps)); }

}  // namespace

int cross_attention_backward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k,
                             const gsr_heads &v, const gsr_heads &out, const float *lse, const gsr_heads &dout,
                             const gsr_heads &dq, const gsr_heads &dk, const gsr_heads &dv, cudaStream_t stream)
{
    AttentionArgs a = {};
    a.d = d;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dout = dout;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.lse = const_cast<float *>(lse);
    const int64_t rows = (int64_t)d.batch * d.q_heads * d.q_len, keys = (int64_t)d.batch * d.kv_heads * d.kv_len;
    void *work;
    if (int rc = workspace(ctx, (size_t)rows * sizeof(float), stream, &work)) return rc;
    a.delta = (float *)work;
    const bool bf16 = d.dtype == GSR_BF16;
    cudaError_t e = cudaSuccess;
    if (rows > 0)
        e = bf16 ? launch_kernel(ctx, k_attention_grad_rows<__nv_bfloat16>, warp_grid(rows), kWarps * 32, stream, a)
                 : launch_kernel(ctx, k_attention_grad_rows<__half>, warp_grid(rows), kWarps * 32, stream, a);
    if (e == cudaSuccess && keys > 0)
        e = bf16 ? launch_kernel(ctx, k_attention_grad_keys<__nv_bfloat16>, warp_grid(keys), kWarps * 32, stream, a)
                 : launch_kernel(ctx, k_attention_grad_keys<__half>, warp_grid(keys), kWarps * 32, stream, a);
    if (int rc = cuda_check(ctx, e, "cross attention backward")) return rc;
    return workspace_done(ctx, stream);
}

}  // namespace gsr
