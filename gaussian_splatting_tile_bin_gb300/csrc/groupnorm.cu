// groupnorm.cu -- group norm with an activation over channels-last features,
// forward and backward.
//
// Forward: mean and var of each (sample, group), z = (x - mean) rstd w + b,
// out = act(z).  Backward: dz = dout act'(z), xh = (x - mean) rstd and, with M
// elements in a group,
//   dx = rstd (w dz - sum(w dz) / M - xh sum(w dz xh) / M).
//
// Bound by HBM.  Both directions are a pass that reduces over the positions per
// channel, a small kernel that merges the blocks' partial sums into groups, and
// a pass that writes.  Channels stay the fastest axis throughout: a thread owns
// one vector of channels and walks positions, so accesses are contiguous for
// any group width.
//
// Numerics.  The variance is a merge of centred squares: a thread takes the mean
// and the centred squares of kRun values at a time and merges (n, mean, M2)
// pairs by Chan, Golub and LeVeque's formula, which cancels nothing when the
// mean is far from 0.  All merges run in a fixed order.
#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kNormBlock = 256;
constexpr int kRun = 8;          // positions a thread reads at a time
constexpr int kMergeBlock = 128;

struct NormArgs {
    const void *x, *dout;
    void *y;                     // out or dx
    const float *weight, *bias;
    float *mean, *rstd;          // [samples, groups]; read by the backward
    float2 *partial;             // [samples in flight, chunks, channels]: (mean, M2) or (sum dz, sum dz xh)
    float2 *sums;                // [samples, channels] and [samples, groups]: backward's merged sums
    float2 *group_sums;
    float *dweight, *dbias;
    int64_t positions;
    int64_t rows_per_chunk;
    int samples, channels, groups, per_group;
    int chunks;
    int sample0;                 // first sample of this launch
    int vectors;                 // channel vectors a block spans
    float eps;
};

template <typename T>
constexpr bool kFast = sizeof(T) == 2;   // 16-bit outputs hide the fast exponential's 1e-6

template <typename T>
__device__ __forceinline__ float sigmoid_of(float z)
{
    if (kFast<T>) return __fdividef(1.0f, 1.0f + __expf(-z));
    return 1.0f / (1.0f + expf(-z));
}

template <typename T, int ACT>
__device__ __forceinline__ float activate(float z)
{
    if (ACT == GSR_ACT_SILU) {
        // z sigmoid(z); sigmoid underflows to 0 for z < -88, and -inf gives 0 as the limit does.
        const float s = sigmoid_of<T>(z);
        return s == 0.0f ? 0.0f : z * s;
    }
    if (ACT == GSR_ACT_GELU) return 0.5f * z * erfcf(-0.70710678f * z);
    return z;
}

template <typename T, int ACT>
__device__ __forceinline__ float activate_slope(float z)
{
    if (ACT == GSR_ACT_SILU) {
        const float s = sigmoid_of<T>(z);
        return s == 0.0f ? 0.0f : s * (1.0f + z * (1.0f - s));
    }
    if (ACT == GSR_ACT_GELU) {
        const float bell = kFast<T> ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
        return 0.5f * erfcf(-0.70710678f * z) + 0.39894228f * z * bell;
    }
    return 1.0f;
}

struct Moments {
    float n, mean, m2;
};

__device__ __forceinline__ Moments merge(const Moments &a, const Moments &b)
{
    const float n = a.n + b.n;
    if (n == 0.0f) return a;
    const float d = b.mean - a.mean, share = b.n / n;
    return {n, fmaf(d, share, a.mean), a.m2 + b.m2 + d * d * (a.n * share)};
}

// Per channel and chunk of positions: (mean, M2) of x.
template <typename T, int V>
__global__ void __launch_bounds__(kNormBlock) k_norm_moments(const NormArgs a)
{
    grid_dependency_begin();
    __shared__ float s_mean[kNormBlock * V], s_m2[kNormBlock * V], s_n[kNormBlock];
    const int cols = a.vectors;
    const int col = threadIdx.x % cols, row = threadIdx.x / cols, rows = kNormBlock / cols;
    const int vec = blockIdx.z * cols + col;
    const int sample = a.sample0 + blockIdx.y;
    const int64_t p0 = (int64_t)blockIdx.x * a.rows_per_chunk;
    const int64_t p1 = min(a.positions, p0 + a.rows_per_chunk);
    const bool live = row < rows && vec * V < a.channels;
    float mean[V], m2[V];
    float n = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) mean[j] = m2[j] = 0.0f;
    if (live) {
        const T *x = (const T *)a.x + (int64_t)sample * a.positions * a.channels + (int64_t)vec * V;
        int64_t p = p0 + row;
        for (; p + (int64_t)(kRun - 1) * rows < p1; p += (int64_t)kRun * rows) {
            Vec<T, V> v[kRun];
#pragma unroll
            for (int k = 0; k < kRun; ++k) v[k] = *(const Vec<T, V> *)(x + (p + (int64_t)k * rows) * a.channels);
            const float total = n + kRun;
            const float share = kRun / total;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float f[kRun], sum = 0.0f, sq = 0.0f;
#pragma unroll
                for (int k = 0; k < kRun; ++k) sum += f[k] = to_float(v[k].e[j]);
                const float mu = sum * (1.0f / kRun);
#pragma unroll
                for (int k = 0; k < kRun; ++k) sq = fmaf(f[k] - mu, f[k] - mu, sq);
                const float d = mu - mean[j];
                mean[j] = fmaf(d, share, mean[j]);
                m2[j] += fmaf(d * d, n * share, sq);
            }
            n = total;
        }
        for (; p < p1; p += rows) {
            const Vec<T, V> v = *(const Vec<T, V> *)(x + p * a.channels);
            n += 1.0f;
            const float share = 1.0f / n;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = to_float(v.e[j]), d = f - mean[j];
                mean[j] = fmaf(d, share, mean[j]);
                m2[j] = fmaf(d, f - mean[j], m2[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_mean[threadIdx.x * V + j] = mean[j];
        s_m2[threadIdx.x * V + j] = m2[j];
    }
    s_n[threadIdx.x] = n;
    __syncthreads();
    float2 *out = a.partial + ((int64_t)blockIdx.y * a.chunks + blockIdx.x) * a.channels + (int64_t)blockIdx.z * cols * V;
    for (int c = threadIdx.x; c < cols * V && (int)(blockIdx.z * cols * V) + c < a.channels; c += kNormBlock) {
        Moments m = {0.0f, 0.0f, 0.0f};
        for (int r = 0; r < rows; ++r) {
            const int t = r * cols + c / V;
            m = merge(m, {s_n[t], s_mean[t * V + c % V], s_m2[t * V + c % V]});
        }
        out[c] = make_float2(m.mean, m.m2);
    }
}

__device__ __forceinline__ Moments warp_merge(Moments m)
{
    for (int d = 16; d > 0; d /= 2) {
        const Moments o = {__shfl_down_sync(~0u, m.n, d), __shfl_down_sync(~0u, m.mean, d),
                           __shfl_down_sync(~0u, m.m2, d)};
        m = merge(m, o);
    }
    return m;
}

// Merges the chunks' and channels' moments of one (group, sample).
__global__ void __launch_bounds__(kMergeBlock) k_norm_merge(const NormArgs a)
{
    grid_dependency_begin();
    __shared__ Moments s[kMergeBlock / 32];
    const int g = blockIdx.x, sample = a.sample0 + blockIdx.y;
    const float2 *in = a.partial + (int64_t)blockIdx.y * a.chunks * a.channels + g * a.per_group;
    Moments m = {0.0f, 0.0f, 0.0f};
    const int count = a.chunks * a.per_group;
    for (int i = threadIdx.x; i < count; i += kMergeBlock) {
        const int chunk = i / a.per_group, c = i - chunk * a.per_group;
        const float2 v = in[(int64_t)chunk * a.channels + c];
        const float n = (float)(min(a.positions, (chunk + 1) * a.rows_per_chunk) - chunk * a.rows_per_chunk);
        m = merge(m, {n, v.x, v.y});
    }
    m = warp_merge(m);
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kMergeBlock / 32; ++w) m = merge(m, s[w]);
        const float var = m.m2 / ((float)a.per_group * (float)a.positions);
        a.mean[(int64_t)sample * a.groups + g] = m.mean;
        a.rstd[(int64_t)sample * a.groups + g] = 1.0f / sqrtf(var + a.eps);
    }
}

// A thread's channel constants.
template <int V>
struct Channel {
    float mean[V], rstd[V], weight[V], bias[V];
    __device__ __forceinline__ void load(const NormArgs &a, int sample, int c0)
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t at = (int64_t)sample * a.groups + (c0 + j) / a.per_group;
            mean[j] = a.mean[at];
            rstd[j] = a.rstd[at];
            weight[j] = a.weight ? a.weight[c0 + j] : 1.0f;
            bias[j] = a.bias ? a.bias[c0 + j] : 0.0f;
        }
    }
};

// out = act((x - mean) rstd w + b).  Blocks take the chunks from the last to the
// first: what the moments pass read last is what L2 still holds.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kNormBlock) k_norm_apply(const NormArgs a)
{
    grid_dependency_begin();
    const int cols = a.vectors;
    const int col = threadIdx.x % cols, row = threadIdx.x / cols, rows = kNormBlock / cols;
    const int vec = blockIdx.z * cols + col;
    if (row >= rows || vec * V >= a.channels) return;
    const int local = gridDim.y - 1 - blockIdx.y, sample = a.sample0 + local;
    const int64_t p0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * a.rows_per_chunk;
    const int64_t p1 = min(a.positions, p0 + a.rows_per_chunk);
    Channel<V> ch;
    ch.load(a, sample, vec * V);
    float scale[V];
#pragma unroll
    for (int j = 0; j < V; ++j) scale[j] = ch.rstd[j] * ch.weight[j];
    const int64_t base = (int64_t)sample * a.positions * a.channels + (int64_t)vec * V;
    const T *x = (const T *)a.x + base;
    T *y = (T *)a.y + base;
    constexpr int kUnroll = 4;
    for (int64_t p = p0 + row; p < p1; p += (int64_t)kUnroll * rows) {
        Vec<T, V> v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (p + (int64_t)k * rows < p1) v[k] = *(const Vec<T, V> *)(x + (p + (int64_t)k * rows) * a.channels);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (p + (int64_t)k * rows < p1) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[k].e[j] = from_float<T>(
                        activate<T, ACT>(fmaf(to_float(v[k].e[j]) - ch.mean[j], scale[j], ch.bias[j])));
                *(Vec<T, V> *)(y + (p + (int64_t)k * rows) * a.channels) = v[k];
            }
    }
}

// Per channel and chunk: (sum dz, sum dz xh).
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kNormBlock) k_norm_grad_sums(const NormArgs a)
{
    grid_dependency_begin();
    __shared__ float s_b[kNormBlock * V], s_w[kNormBlock * V];
    const int cols = a.vectors;
    const int col = threadIdx.x % cols, row = threadIdx.x / cols, rows = kNormBlock / cols;
    const int vec = blockIdx.z * cols + col;
    const int sample = a.sample0 + blockIdx.y;
    const int64_t p0 = (int64_t)blockIdx.x * a.rows_per_chunk;
    const int64_t p1 = min(a.positions, p0 + a.rows_per_chunk);
    float sb[V], sw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sb[j] = sw[j] = 0.0f;
    if (row < rows && vec * V < a.channels) {
        Channel<V> ch;
        ch.load(a, sample, vec * V);
        const int64_t base = (int64_t)sample * a.positions * a.channels + (int64_t)vec * V;
        const T *x = (const T *)a.x + base, *dout = (const T *)a.dout + base;
        constexpr int kUnroll = 4;
        for (int64_t p = p0 + row; p < p1; p += (int64_t)kUnroll * rows) {
            Vec<T, V> vx[kUnroll], vd[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (p + (int64_t)k * rows < p1) {
                    vx[k] = *(const Vec<T, V> *)(x + (p + (int64_t)k * rows) * a.channels);
                    vd[k] = *(const Vec<T, V> *)(dout + (p + (int64_t)k * rows) * a.channels);
                }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (p + (int64_t)k * rows < p1) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float xh = (to_float(vx[k].e[j]) - ch.mean[j]) * ch.rstd[j];
                        const float dz = to_float(vd[k].e[j]) *
                                         activate_slope<T, ACT>(fmaf(xh, ch.weight[j], ch.bias[j]));
                        sb[j] += dz;
                        sw[j] = fmaf(dz, xh, sw[j]);
                    }
                }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_b[threadIdx.x * V + j] = sb[j];
        s_w[threadIdx.x * V + j] = sw[j];
    }
    __syncthreads();
    float2 *out = a.partial + ((int64_t)blockIdx.y * a.chunks + blockIdx.x) * a.channels + (int64_t)blockIdx.z * cols * V;
    for (int c = threadIdx.x; c < cols * V && (int)(blockIdx.z * cols * V) + c < a.channels; c += kNormBlock) {
        float2 m = make_float2(0.0f, 0.0f);
        for (int r = 0; r < rows; ++r) {
            const int t = (r * cols + c / V) * V + c % V;
            m.x += s_b[t];
            m.y += s_w[t];
        }
        out[c] = m;
    }
}

// Merges the chunks' sums of one (group, sample): per channel for the parameter
// gradients, weighted over the group for dx.
__global__ void __launch_bounds__(kMergeBlock) k_norm_grad_merge(const NormArgs a)
{
    grid_dependency_begin();
    __shared__ float2 s[kMergeBlock];
    const int g = blockIdx.x, sample = a.sample0 + blockIdx.y;
    const float2 *in = a.partial + (int64_t)blockIdx.y * a.chunks * a.channels + g * a.per_group;
    float2 *out = a.sums + (int64_t)sample * a.channels + g * a.per_group;
    // lanes over the group's channels, the rest of the block over chunks
    const int cols = min(a.per_group, 32);
    const int col = threadIdx.x % cols, row = threadIdx.x / cols, rows = kMergeBlock / cols;
    float2 group = make_float2(0.0f, 0.0f);
    for (int c0 = 0; c0 < a.per_group; c0 += cols) {
        float2 m = make_float2(0.0f, 0.0f);
        if (row < rows && c0 + col < a.per_group)
            for (int k = row; k < a.chunks; k += rows) {
                const float2 v = in[(int64_t)k * a.channels + c0 + col];
                m.x += v.x;
                m.y += v.y;
            }
        s[threadIdx.x] = m;
        __syncthreads();
        if (threadIdx.x < cols && c0 + col < a.per_group) {
            m = make_float2(0.0f, 0.0f);
            for (int r = 0; r < rows; ++r) {
                m.x += s[r * cols + col].x;
                m.y += s[r * cols + col].y;
            }
            out[c0 + col] = m;
            const float w = a.weight ? a.weight[g * a.per_group + c0 + col] : 1.0f;
            group.x = fmaf(w, m.x, group.x);
            group.y = fmaf(w, m.y, group.y);
        }
        __syncthreads();
    }
    s[threadIdx.x] = threadIdx.x < cols ? group : make_float2(0.0f, 0.0f);
    __syncthreads();
    if (threadIdx.x == 0) {
        group = s[0];
        for (int k = 1; k < cols; ++k) {
            group.x += s[k].x;
            group.y += s[k].y;
        }
        const float inv = 1.0f / ((float)a.per_group * (float)a.positions);
        a.group_sums[(int64_t)sample * a.groups + g] = make_float2(group.x * inv, group.y * inv);
    }
}

// dx = rstd (w dz - m1 - xh m2).  The blocks of the last launch's first chunk
// also sum the parameter gradients over the samples.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kNormBlock) k_norm_grad_apply(const NormArgs a)
{
    grid_dependency_begin();
    if (blockIdx.x == 0 && blockIdx.y == 0 && a.sample0 + (int)gridDim.y == a.samples) {
        for (int c = blockIdx.z * kNormBlock + threadIdx.x; c < a.channels; c += gridDim.z * kNormBlock) {
            float2 m = make_float2(0.0f, 0.0f);
            for (int n = 0; n < a.samples; ++n) {
                const float2 v = a.sums[(int64_t)n * a.channels + c];
                m.x += v.x;
                m.y += v.y;
            }
            if (a.dbias) a.dbias[c] = m.x;
            if (a.dweight) a.dweight[c] = m.y;
        }
    }
    const int cols = a.vectors;
    const int col = threadIdx.x % cols, row = threadIdx.x / cols, rows = kNormBlock / cols;
    const int vec = blockIdx.z * cols + col;
    if (row >= rows || vec * V >= a.channels) return;
    const int local = gridDim.y - 1 - blockIdx.y, sample = a.sample0 + local;
    const int64_t p0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * a.rows_per_chunk;
    const int64_t p1 = min(a.positions, p0 + a.rows_per_chunk);
    Channel<V> ch;
    ch.load(a, sample, vec * V);
    float m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float2 m = a.group_sums[(int64_t)sample * a.groups + (vec * V + j) / a.per_group];
        m1[j] = m.x;
        m2[j] = m.y;
    }
    const int64_t base = (int64_t)sample * a.positions * a.channels + (int64_t)vec * V;
    const T *x = (const T *)a.x + base, *dout = (const T *)a.dout + base;
    T *y = (T *)a.y + base;
    constexpr int kUnroll = 4;
    for (int64_t p = p0 + row; p < p1; p += (int64_t)kUnroll * rows) {
        Vec<T, V> vx[kUnroll], vd[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (p + (int64_t)k * rows < p1) {
                vx[k] = *(const Vec<T, V> *)(x + (p + (int64_t)k * rows) * a.channels);
                vd[k] = *(const Vec<T, V> *)(dout + (p + (int64_t)k * rows) * a.channels);
            }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (p + (int64_t)k * rows < p1) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (to_float(vx[k].e[j]) - ch.mean[j]) * ch.rstd[j];
                    const float dz =
                        to_float(vd[k].e[j]) * activate_slope<T, ACT>(fmaf(xh, ch.weight[j], ch.bias[j]));
                    const float dxh = fmaf(ch.weight[j], dz, -m1[j]);
                    vx[k].e[j] = from_float<T>(ch.rstd[j] * fmaf(-xh, m2[j], dxh));
                }
                *(Vec<T, V> *)(y + (p + (int64_t)k * rows) * a.channels) = vx[k];
            }
    }
}

// Splits of the positions: enough blocks for every SM, a few runs of rows each.
struct NormPlan {
    int vectors, slabs, chunks, wave;
    int64_t rows_per_chunk;
};

NormPlan norm_plan(const gsr_ctx *ctx, const gsr_group_norm &d, int width, int arrays)
{
    NormPlan p;
    const int vectors = (d.channels + width - 1) / width;
    p.vectors = vectors < kNormBlock ? vectors : kNormBlock;
    p.slabs = (vectors + p.vectors - 1) / p.vectors;
    const int rows = kNormBlock / p.vectors;
    // A wave of samples whose arrays stay in L2 between the two passes over them.
    const int64_t sample_bytes = d.positions * d.channels * (d.dtype == GSR_F32 ? 4 : 2) * arrays;
    constexpr int64_t kL2Share = (int64_t)64 << 20;
    int64_t wave = kL2Share / (sample_bytes > 0 ? sample_bytes : 1);
    wave = wave < 1 ? 1 : wave;
    p.wave = (int)(wave < d.samples ? wave : d.samples);
    if (p.wave > 65535) p.wave = 65535;
    int64_t chunks = (4 * (int64_t)ctx->num_sms + (int64_t)p.wave * p.slabs - 1) / ((int64_t)p.wave * p.slabs);
    const int64_t most = (d.positions + (int64_t)rows * kRun - 1) / ((int64_t)rows * kRun);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    p.rows_per_chunk = (d.positions + chunks - 1) / chunks;
    p.chunks = (int)((d.positions + p.rows_per_chunk - 1) / p.rows_per_chunk);
    return p;
}

int norm_width(const gsr_group_norm &d, const void *x, const void *dout, const void *y)
{
    const int full = d.dtype == GSR_F32 ? 4 : 8;
    const bool ok = d.channels % full == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)dout % 16 == 0 &&
                    (uintptr_t)y % 16 == 0;
    return ok ? full : 1;
}

template <typename T, int V, int ACT>
cudaError_t norm_forward(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    for (a.sample0 = 0; a.sample0 < a.samples; a.sample0 += p.wave) {
        const unsigned n = (unsigned)(a.samples - a.sample0 < p.wave ? a.samples - a.sample0 : p.wave);
        const dim3 grid((unsigned)p.chunks, n, (unsigned)p.slabs);
        cudaError_t e = launch_kernel(ctx, k_norm_moments<T, V>, grid, kNormBlock, stream, a);
        if (e == cudaSuccess) e = launch_kernel(ctx, k_norm_merge, dim3((unsigned)a.groups, n), kMergeBlock, stream, a);
        if (e == cudaSuccess) e = launch_kernel(ctx, k_norm_apply<T, V, ACT>, grid, kNormBlock, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int V, int ACT>
cudaError_t norm_backward(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    for (a.sample0 = 0; a.sample0 < a.samples; a.sample0 += p.wave) {
        const unsigned n = (unsigned)(a.samples - a.sample0 < p.wave ? a.samples - a.sample0 : p.wave);
        const dim3 grid((unsigned)p.chunks, n, (unsigned)p.slabs);
        cudaError_t e = launch_kernel(ctx, k_norm_grad_sums<T, V, ACT>, grid, kNormBlock, stream, a);
        if (e == cudaSuccess)
            e = launch_kernel(ctx, k_norm_grad_merge, dim3((unsigned)a.groups, n), kMergeBlock, stream, a);
        if (e == cudaSuccess) e = launch_kernel(ctx, k_norm_grad_apply<T, V, ACT>, grid, kNormBlock, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int ACT>
cudaError_t dispatch_width(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, int width, bool backward, cudaStream_t s)
{
    constexpr int kFull = 16 / (int)sizeof(T);
    if (width == kFull) return backward ? norm_backward<T, kFull, ACT>(ctx, a, p, s) : norm_forward<T, kFull, ACT>(ctx, a, p, s);
    return backward ? norm_backward<T, 1, ACT>(ctx, a, p, s) : norm_forward<T, 1, ACT>(ctx, a, p, s);
}

template <typename T>
cudaError_t dispatch_act(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, int act, int width, bool backward,
                         cudaStream_t s)
{
    if (act == GSR_ACT_SILU) return dispatch_width<T, GSR_ACT_SILU>(ctx, a, p, width, backward, s);
    if (act == GSR_ACT_GELU) return dispatch_width<T, GSR_ACT_GELU>(ctx, a, p, width, backward, s);
    return dispatch_width<T, GSR_ACT_NONE>(ctx, a, p, width, backward, s);
}

int run_norm(gsr_ctx *ctx, const gsr_group_norm &d, NormArgs &a, bool backward, cudaStream_t stream)
{
    const int width = norm_width(d, a.x, a.dout, a.y);
    const NormPlan p = norm_plan(ctx, d, width, backward ? 3 : 2);
    a.samples = d.samples;
    a.channels = d.channels;
    a.groups = d.groups;
    a.per_group = d.channels / d.groups;
    a.positions = d.positions;
    a.rows_per_chunk = p.rows_per_chunk;
    a.chunks = p.chunks;
    a.vectors = p.vectors;
    a.eps = d.eps;
    const size_t partial = (size_t)p.wave * p.chunks * d.channels * sizeof(float2);
    const size_t sums = backward ? (size_t)d.samples * d.channels * sizeof(float2) : 0;
    const size_t group_sums = backward ? (size_t)d.samples * d.groups * sizeof(float2) : 0;
    void *work;
    if (int rc = workspace(ctx, partial + sums + group_sums, stream, &work)) return rc;
    a.partial = (float2 *)work;
    a.sums = (float2 *)((unsigned char *)work + partial);
    a.group_sums = (float2 *)((unsigned char *)work + partial + sums);
    cudaError_t e;
    if (d.dtype == GSR_F32)
        e = dispatch_act<float>(ctx, a, p, d.activation, width, backward, stream);
    else if (d.dtype == GSR_BF16)
        e = dispatch_act<__nv_bfloat16>(ctx, a, p, d.activation, width, backward, stream);
    else
        e = dispatch_act<__half>(ctx, a, p, d.activation, width, backward, stream);
    if (int rc = cuda_check(ctx, e, backward ? "group norm backward" : "group norm forward")) return rc;
    return workspace_done(ctx, stream);
}

}  // namespace

int group_norm_forward(gsr_ctx *ctx, const gsr_group_norm &d, const void *x, const float *weight, const float *bias,
                       void *out, float *mean, float *rstd, cudaStream_t stream)
{
    NormArgs a = {};
    a.x = x;
    a.y = out;
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    return run_norm(ctx, d, a, false, stream);
}

int group_norm_backward(gsr_ctx *ctx, const gsr_group_norm &d, const void *dout, const void *x, const float *weight,
                        const float *bias, const float *mean, const float *rstd, void *dx, float *dweight,
                        float *dbias, cudaStream_t stream)
{
    if (d.samples == 0 || d.positions == 0) {
        for (float *grad : {dweight, dbias})
            if (grad)
                if (int rc = cuda_check(ctx, cudaMemsetAsync(grad, 0, (size_t)d.channels * sizeof(float), stream),
                                        "group norm backward"))
                    return rc;
        return GSR_OK;
    }
    NormArgs a = {};
    a.x = x;
    a.dout = dout;
    a.y = dx;
    a.weight = weight;
    a.bias = bias;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dweight = dweight;
    a.dbias = dbias;
    return run_norm(ctx, d, a, true, stream);
}

}  // namespace gsr
