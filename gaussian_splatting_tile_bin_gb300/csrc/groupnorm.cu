// groupnorm.cu -- group norm with an activation over channels-last features,
// forward and backward.
//
// Forward: mean and var of each (sample, group), z = (x - mean) rstd w + b,
// out = act(z).  Backward: dz = dout act'(z), xh = (x - mean) rstd and, with M
// elements in a group,
//   dx = rstd (w dz - sum(w dz) / M - xh sum(w dz xh) / M).
//
// Bound by HBM.  Channels stay the fastest axis throughout: a thread owns one
// vector of channels and walks positions, so accesses are contiguous for any
// group width.  Two forms:
//   - resident: a cluster of blocks keeps a sample's slab of whole groups in
//     shared memory between the statistics and the result, one kernel and one
//     read of the inputs.  For slabs that a cluster holds (3 x 6,767 x 96 in f32:
//     14 and 21 us where the passes take 20 and 27).
//   - passes: a pass that reduces over the positions per channel, a small kernel
//     that merges the blocks' partial sums into groups, and a pass that writes
//     and walks back, from what L2 still holds of the first.  Moves 3 arrays
//     forward and 5 backward where 2 and 3 are needed: 4 x 40,000 x 256 in bf16
//     (82 MB an array) takes 47 us, a training step of 4 x 160,000 x 128 (164 MB)
//     226 us.  Of the first one's second pass 32 of 82 MB come from DRAM (of the
//     backward's, 27 MB), the rest from L2; what is written leaves later.
//     GELU in 16 bits is bound by erfcf, not by HBM: 103 us forward.
//
// Numerics.  The variance is a merge of centred squares: a thread takes the mean
// and the centred squares of kRun values at a time and merges (n, mean, M2)
// pairs by Chan, Golub and LeVeque's formula, which cancels nothing when the
// mean is far from 0.  All merges run in a fixed order.
#include <cooperative_groups.h>

#include <algorithm>

#include "decoder.cuh"

namespace gsr {
namespace {

namespace cg = cooperative_groups;

constexpr int kNormBlock = 256;
constexpr int kRun = 8;          // values whose mean and centred squares are taken together
constexpr int kMergeBlock = 256;
// Blocks an SM holds (their rings fill its shared memory): one wave of them takes
// all chunks.
constexpr int kNormOccupancy = 2;

// A result, which nothing here reads again.
template <typename T, int V>
__device__ __forceinline__ void store_last(T *p, const Vec<T, V> &v)
{
    if constexpr (sizeof(T) * V == 16)
        __stcs((uint4 *)p, *(const uint4 *)&v);
    else
        *(Vec<T, V> *)p = v;
}

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

constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(z) = 1 / (1 + 2^(-z log2 e)); 0 where the exponential overflows.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    if constexpr (kFast<T>) {
        const float2 e = mul2(z, make_float2(-kLog2e, -kLog2e));
        const float2 d = add2(make_float2(exp2_fast(e.x), exp2_fast(e.y)), make_float2(1.0f, 1.0f));
        return make_float2(rcp_fast(d.x), rcp_fast(d.y));
    } else {
        return make_float2(1.0f / (1.0f + expf(-z.x)), 1.0f / (1.0f + expf(-z.y)));
    }
}

template <typename T, int ACT>
__device__ __forceinline__ float2 activate2(float2 z)
{
    if constexpr (ACT == GSR_ACT_SILU) return mul2(z, sigmoid2<T>(z));
    if constexpr (ACT == GSR_ACT_GELU)
        return make_float2(0.5f * z.x * erfcf(-0.70710678f * z.x), 0.5f * z.y * erfcf(-0.70710678f * z.y));
    return z;
}

template <typename T>
__device__ __forceinline__ float gelu_slope(float z)
{
    const float bell = kFast<T> ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
    return 0.5f * erfcf(-0.70710678f * z) + 0.39894228f * z * bell;
}

// act'(z): sigmoid + z sigmoid (1 - sigmoid), Phi + z phi, 1.
template <typename T, int ACT>
__device__ __forceinline__ float2 slope2(float2 z)
{
    if constexpr (ACT == GSR_ACT_SILU) {
        const float2 s = sigmoid2<T>(z);
        return fma2(z, fma2(make_float2(-s.x, -s.y), s, s), s);
    }
    if constexpr (ACT == GSR_ACT_GELU) return make_float2(gelu_slope<T>(z.x), gelu_slope<T>(z.y));
    return make_float2(1.0f, 1.0f);
}

struct Moments {
    float n, mean, m2;
};

__device__ __forceinline__ Moments merge(const Moments &a, const Moments &b)
{
    const float n = a.n + b.n;
    if (n == 0.0f) return a;
    const float d = b.mean - a.mean, share = __fdividef(b.n, n);
    return {n, fmaf(d, share, a.mean), a.m2 + b.m2 + d * d * (a.n * share)};
}

// A thread's moments of its V channels, which share n.
template <typename T, int V>
struct ChannelMoments {
    float n = 0.0f, mean[V] = {}, m2[V] = {};
    __device__ __forceinline__ void add(const Vec<T, V>(&v)[kRun])
    {
        const float total = n + kRun, share = __fdividef(kRun, total);
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
    __device__ __forceinline__ void add(const Vec<T, V> &v)
    {
        n += 1.0f;
        const float share = __fdividef(1.0f, n);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float f = to_float(v.e[j]), d = f - mean[j];
            mean[j] = fmaf(d, share, mean[j]);
            m2[j] = fmaf(d, f - mean[j], m2[j]);
        }
    }
};

__device__ __forceinline__ float block_sum(float x, float *s_warp)
{
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
    __syncthreads();
    if (threadIdx.x % 32 == 0) s_warp[threadIdx.x / 32] = x;
    __syncthreads();
    float sum = 0.0f;
    for (int w = 0; w < kMergeBlock / 32; ++w) sum += s_warp[w];
    return sum;
}

// Merges the chunks' and channels' moments of one (group, sample): the weighted
// mean of the means, then M2 = sum (M2_i + n_i (mean_i - mean)^2).
__global__ void __launch_bounds__(kMergeBlock) k_norm_merge(const NormArgs a)
{
    grid_dependency_begin();
    __shared__ float s_warp[kMergeBlock / 32];
    const int g = blockIdx.x, sample = a.sample0 + blockIdx.y;
    const float2 *in = a.partial + (int64_t)blockIdx.y * a.chunks * a.channels + g * a.per_group;
    const float rows = (float)a.rows_per_chunk;
    const float last = (float)(a.positions - (a.chunks - 1) * a.rows_per_chunk);
    const int count = a.chunks * a.per_group;
    auto entry = [&](int i, float &n) {
        const int chunk = (unsigned)i / (unsigned)a.per_group, c = i - chunk * a.per_group;
        n = chunk == a.chunks - 1 ? last : rows;
        return in[(int64_t)chunk * a.channels + c];
    };
    const float total = (float)a.per_group * (float)a.positions;
    float sum = 0.0f;
#pragma unroll 8
    for (int i = threadIdx.x; i < count; i += kMergeBlock) {
        float n;
        const float2 v = entry(i, n);
        sum = fmaf(n / total, v.x, sum);
    }
    const float mean = block_sum(sum, s_warp);
    sum = 0.0f;
#pragma unroll 8
    for (int i = threadIdx.x; i < count; i += kMergeBlock) {
        float n;
        const float2 v = entry(i, n);
        const float d = v.x - mean;
        sum += fmaf(n * d, d, v.y);
    }
    const float m2 = block_sum(sum, s_warp);
    if (threadIdx.x == 0) {
        a.mean[(int64_t)sample * a.groups + g] = mean;
        a.rstd[(int64_t)sample * a.groups + g] = 1.0f / sqrtf(m2 / total + a.eps);
    }
}

// A thread's channel constants, in pairs.
template <int V>
constexpr int kPairs = (V + 1) / 2;

template <int V>
struct Channel {
    float2 minus_mean[kPairs<V>], rstd[kPairs<V>], weight[kPairs<V>], bias[kPairs<V>];
    __device__ __forceinline__ void load(const NormArgs &a, int sample, int c0)
    {
#pragma unroll
        for (int j = 0; j < 2 * kPairs<V>; ++j) {
            const int c = c0 + (j < V ? j : 0);
            const int64_t at = (int64_t)sample * a.groups + c / a.per_group;
            (&minus_mean[j / 2].x)[j % 2] = -a.mean[at];
            (&rstd[j / 2].x)[j % 2] = a.rstd[at];
            (&weight[j / 2].x)[j % 2] = a.weight ? a.weight[c] : 1.0f;
            (&bias[j / 2].x)[j % 2] = a.bias ? a.bias[c] : 0.0f;
        }
    }
    // (x - mean) rstd, and dz = dout act'(xh w + b).
    __device__ __forceinline__ float2 hat(float2 x, int j) const { return mul2(add2(x, minus_mean[j]), rstd[j]); }
    template <typename T, int ACT>
    __device__ __forceinline__ float2 dz(float2 dout, float2 xh, int j) const
    {
        return mul2(dout, slope2<T, ACT>(fma2(xh, weight[j], bias[j])));
    }
};

// What an output needs of its channels.
template <int V>
struct Affine {
    float2 minus_mean[kPairs<V>], scale[kPairs<V>], bias[kPairs<V>];
    __device__ __forceinline__ void from(const Channel<V> &c)
    {
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) {
            minus_mean[j] = c.minus_mean[j];
            scale[j] = mul2(c.rstd[j], c.weight[j]);
            bias[j] = c.bias[j];
        }
    }
    template <typename T, int ACT>
    __device__ __forceinline__ void apply(Vec<T, V> &v) const
    {
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j)
            set_pair(v, 2 * j, activate2<T, ACT>(fma2(add2(pair_of(v, 2 * j), minus_mean[j]), scale[j], bias[j])));
    }
};

// The backward of a vector: sums, and dx = rstd (w dz - m1 - xh m2).
template <int V>
struct Gradient {
    float2 b[kPairs<V>] = {}, w[kPairs<V>] = {};
    template <typename T, int ACT>
    __device__ __forceinline__ void add(const Channel<V> &c, const Vec<T, V> &x, const Vec<T, V> &dout)
    {
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) {
            const float2 xh = c.hat(pair_of(x, 2 * j), j);
            const float2 dz = c.template dz<T, ACT>(pair_of(dout, 2 * j), xh, j);
            b[j] = add2(b[j], dz);
            w[j] = fma2(dz, xh, w[j]);
        }
    }
    __device__ __forceinline__ float sum_b(int j) const { return (&b[j / 2].x)[j % 2]; }
    __device__ __forceinline__ float sum_w(int j) const { return (&w[j / 2].x)[j % 2]; }
};

template <typename T, int V, int ACT>
__device__ __forceinline__ void input_gradient(const Channel<V> &c, const float2 (&m1)[kPairs<V>],
                                               const float2 (&m2)[kPairs<V>], Vec<T, V> &x, const Vec<T, V> &dout)
{
#pragma unroll
    for (int j = 0; j < kPairs<V>; ++j) {
        const float2 xh = c.hat(pair_of(x, 2 * j), j);
        const float2 dz = c.template dz<T, ACT>(pair_of(dout, 2 * j), xh, j);
        const float2 t = fma2(c.weight[j], dz, make_float2(-m1[j].x, -m1[j].y));
        set_pair(x, 2 * j, mul2(c.rstd[j], fma2(make_float2(-xh.x, -xh.y), m2[j], t)));
    }
}

// A thread's rows through a ring of its own in shared memory: asynchronous copies
// of kUnroll rows of each of N arrays, kDepth - 1 batches ahead, so that the loads
// in flight do not depend on registers and no thread waits for another.  f is
// called with a batch: its first row's number, how many rows, and the values.
// Accesses of 2 bytes (which have no such copies) are read directly.
template <int N>
constexpr int kUnroll = 8 / N;
constexpr int kDepth = 2;   // (three and four were no faster: 47.2 and 46.8 us, 232 and 229 us)
static_assert(kUnroll<1> == kRun, "a batch is a run of the moments");

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// Shared memory of a walk: the ring, then the threads' sums in its place.
template <typename T, int V, int N>
constexpr size_t kWalkBytes = std::max((size_t)kNormBlock * sizeof(Vec<T, V>) * kUnroll<N> * kDepth * N,
                                       (size_t)kNormBlock * (2 * V + 1) * sizeof(float));

template <typename T, int V, int N, typename F>
__device__ __forceinline__ void walk_rows(unsigned char *ring, const T *const (&from)[N], int64_t stride, int rows, F f)
{
    using Access = Vec<T, V>;
    Access v[N][kUnroll<N>];
    if constexpr (sizeof(Access) >= 4) {
        Access *mine = (Access *)ring + threadIdx.x;
        auto slot = [&](int batch, int n, int k) { return mine + (((batch % kDepth) * N + n) * kUnroll<N> + k) * kNormBlock; };
        const int batches = (rows + kUnroll<N> - 1) / kUnroll<N>;
        auto issue = [&](int batch) {
#pragma unroll
            for (int k = 0; k < kUnroll<N>; ++k)
                if (batch * kUnroll<N> + k < rows)
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        copy_async<sizeof(Access)>(slot(batch, n, k), from[n] + (int64_t)(batch * kUnroll<N> + k) * stride);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int b = 0; b < kDepth - 1; ++b) issue(b);
        for (int b = 0; b < batches; ++b) {
            issue(b + kDepth - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            const int count = min(kUnroll<N>, rows - b * kUnroll<N>);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int k = 0; k < kUnroll<N>; ++k)
                    if (k < count) v[n][k] = *slot(b, n, k);
            f(b * kUnroll<N>, count, v);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        for (int b = 0; b < rows; b += kUnroll<N>) {
            const int count = min(kUnroll<N>, rows - b);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int k = 0; k < kUnroll<N>; ++k)
                    if (k < count) v[n][k] = *(const Access *)(from[n] + (int64_t)(b + k) * stride);
            f(b, count, v);
        }
    }
}

// The rows of a thread in the chunk, and its place.
template <int V>
struct RowWalk {
    int sample, col, row, rows, vec, left;
    int64_t first, last, stride;        // elements: the first and the last row's vector, and a row's distance
    bool live;
    __device__ RowWalk(const NormArgs &a)
    {
        col = threadIdx.x % a.vectors;
        row = threadIdx.x / a.vectors;
        rows = kNormBlock / a.vectors;
        vec = blockIdx.z * a.vectors + col;
        sample = a.sample0 + blockIdx.y;
        const int64_t p0 = (int64_t)blockIdx.x * a.rows_per_chunk, p1 = min(a.positions, p0 + a.rows_per_chunk);
        left = p0 + row < p1 ? (int)((p1 - p0 - row + rows - 1) / rows) : 0;
        live = row < rows && vec * V < a.channels && left > 0;
        stride = (int64_t)rows * a.channels;
        first = ((int64_t)sample * a.positions + p0 + row) * a.channels + (int64_t)vec * V;
        last = first + (left - 1) * stride;
    }
};

// Per channel and chunk of positions: (mean, M2) of x.
template <typename T, int V>
__global__ void __launch_bounds__(kNormBlock, kNormOccupancy) k_norm_moments(const NormArgs a)
{
    grid_dependency_begin();
    extern __shared__ __align__(16) unsigned char s_raw[];
    const RowWalk<V> at(a);
    ChannelMoments<T, V> own;
    if (at.live) {
        const T *const from[1] = {(const T *)a.x + at.first};
        walk_rows<T, V, 1>(s_raw, from, at.stride, at.left, [&](int, int count, const Vec<T, V>(&v)[1][kUnroll<1>]) {
            if (count == kUnroll<1>) {
                own.add(v[0]);
            } else {
#pragma unroll
                for (int k = 0; k < kUnroll<1>; ++k)
                    if (k < count) own.add(v[0][k]);
            }
        });
    }
    __syncthreads();   // the ring becomes the threads' sums
    float *s_mean = (float *)s_raw, *s_m2 = s_mean + kNormBlock * V, *s_n = s_m2 + kNormBlock * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_mean[threadIdx.x * V + j] = own.mean[j];
        s_m2[threadIdx.x * V + j] = own.m2[j];
    }
    s_n[threadIdx.x] = own.n;
    __syncthreads();
    const int cols = a.vectors, c0 = blockIdx.z * cols * V;
    float2 *out = a.partial + ((int64_t)blockIdx.y * a.chunks + blockIdx.x) * a.channels + c0;
    for (int c = threadIdx.x; c < cols * V && c0 + c < a.channels; c += kNormBlock) {
        Moments m = {0.0f, 0.0f, 0.0f};
        for (int r = 0; r < at.rows; ++r) {
            const int t = r * cols + c / V;
            m = merge(m, {s_n[t], s_mean[t * V + c % V], s_m2[t * V + c % V]});
        }
        out[c] = make_float2(m.mean, m.m2);
    }
}

// out = act((x - mean) rstd w + b), from the last row back: what the first pass
// read last is what L2 still holds.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kNormBlock, kNormOccupancy) k_norm_apply(const NormArgs a)
{
    grid_dependency_begin();
    extern __shared__ __align__(16) unsigned char s_raw[];
    const RowWalk<V> at(a);
    if (!at.live) return;
    Affine<V> affine;
    {
        Channel<V> ch;
        ch.load(a, at.sample, at.vec * V);
        affine.from(ch);
    }
    const T *const from[1] = {(const T *)a.x + at.last};
    T *y = (T *)a.y + at.last;
    walk_rows<T, V, 1>(s_raw, from, -at.stride, at.left, [&](int row, int count, Vec<T, V>(&v)[1][kUnroll<1>]) {
#pragma unroll
        for (int k = 0; k < kUnroll<1>; ++k)
            if (k < count) {
                affine.template apply<T, ACT>(v[0][k]);
                store_last<T, V>(y - (row + k) * at.stride, v[0][k]);
            }
    });
}

// Per channel and chunk: (sum dz, sum dz xh).
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kNormBlock, kNormOccupancy) k_norm_grad_sums(const NormArgs a)
{
    grid_dependency_begin();
    extern __shared__ __align__(16) unsigned char s_raw[];
    const RowWalk<V> at(a);
    Gradient<V> grad;
    if (at.live) {
        Channel<V> ch;
        ch.load(a, at.sample, at.vec * V);
        const T *const from[2] = {(const T *)a.x + at.first, (const T *)a.dout + at.first};
        walk_rows<T, V, 2>(s_raw, from, at.stride, at.left, [&](int, int count, const Vec<T, V>(&v)[2][kUnroll<2>]) {
#pragma unroll
            for (int k = 0; k < kUnroll<2>; ++k)
                if (k < count) grad.template add<T, ACT>(ch, v[0][k], v[1][k]);
        });
    }
    __syncthreads();   // the ring becomes the threads' sums
    float *s_b = (float *)s_raw, *s_w = s_b + kNormBlock * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_b[threadIdx.x * V + j] = grad.sum_b(j);
        s_w[threadIdx.x * V + j] = grad.sum_w(j);
    }
    __syncthreads();
    const int cols = a.vectors, c0 = blockIdx.z * cols * V;
    float2 *out = a.partial + ((int64_t)blockIdx.y * a.chunks + blockIdx.x) * a.channels + c0;
    for (int c = threadIdx.x; c < cols * V && c0 + c < a.channels; c += kNormBlock) {
        float2 m = make_float2(0.0f, 0.0f);
        for (int r = 0; r < at.rows; ++r) {
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
__global__ void __launch_bounds__(kNormBlock, kNormOccupancy) k_norm_grad_apply(const NormArgs a)
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
    extern __shared__ __align__(16) unsigned char s_raw[];
    const RowWalk<V> at(a);
    if (!at.live) return;
    Channel<V> ch;
    ch.load(a, at.sample, at.vec * V);
    float2 m1[kPairs<V>], m2[kPairs<V>];
#pragma unroll
    for (int j = 0; j < 2 * kPairs<V>; ++j) {
        const float2 m = a.group_sums[(int64_t)at.sample * a.groups + (at.vec * V + (j < V ? j : 0)) / a.per_group];
        (&m1[j / 2].x)[j % 2] = m.x;
        (&m2[j / 2].x)[j % 2] = m.y;
    }
    const T *const from[2] = {(const T *)a.x + at.last, (const T *)a.dout + at.last};
    T *y = (T *)a.y + at.last;
    walk_rows<T, V, 2>(s_raw, from, -at.stride, at.left, [&](int row, int count, Vec<T, V>(&v)[2][kUnroll<2>]) {
#pragma unroll
        for (int k = 0; k < kUnroll<2>; ++k)
            if (k < count) {
                input_gradient<T, V, ACT>(ch, m1, m2, v[0][k], v[1][k]);
                store_last<T, V>(y - (row + k) * at.stride, v[0][k]);
            }
    });
}

// ---- resident form ---------------------------------------------------------------

constexpr int kResidentBlock = 512;
constexpr int kResidentChannels = 512;              // of a slab, at most
constexpr int kResidentCluster = 8;
constexpr size_t kResidentData = 172 * 1024;        // of a block's shared memory, at most

struct ResidentArgs {
    NormArgs n;
    int slabs, slab_groups, slab_channels;
    int64_t rows_per_block;
    int row_capacity;                               // rows_per_block, as the shared layout has it
};

__device__ __forceinline__ void copies_done()
{
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

// A block's place: its sample, slab and rows, and a thread's column and rows.
template <int V>
struct Place {
    int sample, slab, cols, col, row, rows, channel0;
    int64_t p0, p1, base;                           // base: element of (p0, this thread's vector)
    bool live;
    __device__ Place(const ResidentArgs &a, int rank, int cluster)
    {
        const int unit = blockIdx.x / cluster;
        sample = unit / a.slabs;
        slab = unit - sample * a.slabs;
        cols = a.slab_channels / V;
        col = threadIdx.x % cols;
        row = threadIdx.x / cols;
        rows = kResidentBlock / cols;
        live = row < rows;
        channel0 = slab * a.slab_channels + col * V;
        p0 = min(a.n.positions, rank * a.rows_per_block);
        p1 = min(a.n.positions, p0 + a.rows_per_block);
        base = ((int64_t)sample * a.n.positions + p0) * a.n.channels + channel0;
    }
    __device__ int count() const { return (int)(p1 - p0); }
};

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kResidentBlock) k_norm_resident(const __grid_constant__ ResidentArgs a)
{
    grid_dependency_begin();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    extern __shared__ __align__(16) unsigned char s_raw[];
    Vec<T, V> *s_x = (Vec<T, V> *)s_raw;                                      // [row_capacity][cols]
    const Place<V> at(a, rank, ranks);
    float *s_mean = (float *)(s_x + (size_t)a.row_capacity * at.cols), *s_m2 = s_mean + kResidentBlock * V;
    float *s_n = s_m2 + kResidentBlock * V;                                   // [kResidentBlock]
    Moments *s_part = (Moments *)(s_n + kResidentBlock);                      // [parts][channels]
    Moments *s_group = s_part + kResidentBlock;                               // [slab_groups]
    float2 *s_stat = (float2 *)(s_group + kResidentChannels);                 // [slab_groups]: mean, rstd
    const T *x = (const T *)a.n.x + at.base;
    const int count = at.count();
    ChannelMoments<T, V> own;
    if (at.live) {
        for (int p = at.row; p < count; p += at.rows)
            copy_async<16>(&s_x[p * at.cols + at.col], x + (int64_t)p * a.n.channels);
        copies_done();
        // A thread reads only what it copied itself.
        int p = at.row;
        for (; p + (kRun - 1) * at.rows < count; p += kRun * at.rows) {
            Vec<T, V> v[kRun];
#pragma unroll
            for (int k = 0; k < kRun; ++k) v[k] = s_x[(p + k * at.rows) * at.cols + at.col];
            own.add(v);
        }
        for (; p < count; p += at.rows) own.add(s_x[p * at.cols + at.col]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_mean[threadIdx.x * V + j] = own.mean[j];
        s_m2[threadIdx.x * V + j] = own.m2[j];
    }
    s_n[threadIdx.x] = own.n;
    __syncthreads();
    const int channels = a.slab_channels, parts = kResidentBlock / channels;
    if ((int)threadIdx.x < parts * channels) {
        const int c = threadIdx.x % channels, part = threadIdx.x / channels;
        Moments m = {0.0f, 0.0f, 0.0f};
        for (int r = part; r < at.rows; r += parts) {
            const int t = r * at.cols + c / V;
            m = merge(m, {s_n[t], s_mean[t * V + c % V], s_m2[t * V + c % V]});
        }
        s_part[threadIdx.x] = m;
    }
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, per_group = a.n.per_group;
    for (int g = warp; g < a.slab_groups; g += kResidentBlock / 32) {
        Moments m = {0.0f, 0.0f, 0.0f};
        for (int i = lane; i < parts * per_group; i += 32) {
            const int part = i / per_group;
            m = merge(m, s_part[part * channels + g * per_group + i - part * per_group]);
        }
        for (int d = 16; d > 0; d /= 2)
            m = merge(m, {__shfl_down_sync(~0u, m.n, d), __shfl_down_sync(~0u, m.mean, d),
                          __shfl_down_sync(~0u, m.m2, d)});
        if (lane == 0) s_group[g] = m;
    }
    cluster.sync();
    for (int g = threadIdx.x; g < a.slab_groups; g += kResidentBlock) {
        Moments m = {0.0f, 0.0f, 0.0f};
        for (int r = 0; r < ranks; ++r) m = merge(m, *cluster.map_shared_rank(&s_group[g], r));
        const float rstd = 1.0f / sqrtf(m.m2 / m.n + a.n.eps);
        s_stat[g] = make_float2(m.mean, rstd);
        if (rank == 0) {
            const int64_t to = (int64_t)at.sample * a.n.groups + at.slab * a.slab_groups + g;
            a.n.mean[to] = m.mean;
            a.n.rstd[to] = rstd;
        }
    }
    __syncthreads();
    if (at.live) {
        Affine<V> affine;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 st = s_stat[(at.col * V + j) / per_group];
            (&affine.minus_mean[j / 2].x)[j % 2] = -st.x;
            (&affine.scale[j / 2].x)[j % 2] = st.y * (a.n.weight ? a.n.weight[at.channel0 + j] : 1.0f);
            (&affine.bias[j / 2].x)[j % 2] = a.n.bias ? a.n.bias[at.channel0 + j] : 0.0f;
        }
        T *y = (T *)a.n.y + at.base;
#pragma unroll 2
        for (int p = at.row; p < count; p += at.rows) {
            Vec<T, V> v = s_x[p * at.cols + at.col];
            affine.template apply<T, ACT>(v);
            *(Vec<T, V> *)(y + (int64_t)p * a.n.channels) = v;
        }
    }
    cluster.sync();   // no block leaves while another may read its shared memory
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kResidentBlock) k_norm_grad_resident(const __grid_constant__ ResidentArgs a)
{
    grid_dependency_begin();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    extern __shared__ __align__(16) unsigned char s_raw[];
    const Place<V> at(a, rank, ranks);
    Vec<T, V> *s_x = (Vec<T, V> *)s_raw, *s_d = s_x + (size_t)a.row_capacity * at.cols;
    float *s_b = (float *)(s_d + (size_t)a.row_capacity * at.cols), *s_w = s_b + kResidentBlock * V;
    float2 *s_part = (float2 *)(s_w + kResidentBlock * V);                    // [parts][channels]
    float2 *s_mine = s_part + kResidentBlock;                                 // [channels] of this block
    float2 *s_all = s_mine + kResidentChannels;                               // [channels] of the cluster
    float2 *s_group = s_all + kResidentChannels;                              // [slab_groups]
    const int count = at.count(), per_group = a.n.per_group;
    const T *x = (const T *)a.n.x + at.base, *dout = (const T *)a.n.dout + at.base;
    Gradient<V> grad;
    Channel<V> ch;
    if (at.live) {
        for (int p = at.row; p < count; p += at.rows) {
            copy_async<16>(&s_x[p * at.cols + at.col], x + (int64_t)p * a.n.channels);
            copy_async<16>(&s_d[p * at.cols + at.col], dout + (int64_t)p * a.n.channels);
        }
        ch.load(a.n, at.sample, at.channel0);
        copies_done();
#pragma unroll 2
        for (int p = at.row; p < count; p += at.rows) {
            grad.template add<T, ACT>(ch, s_x[p * at.cols + at.col], s_d[p * at.cols + at.col]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_b[threadIdx.x * V + j] = grad.sum_b(j);
        s_w[threadIdx.x * V + j] = grad.sum_w(j);
    }
    __syncthreads();
    const int channels = a.slab_channels, parts = kResidentBlock / channels;
    if ((int)threadIdx.x < parts * channels) {
        const int c = threadIdx.x % channels, part = threadIdx.x / channels;
        float2 m = make_float2(0.0f, 0.0f);
        for (int r = part; r < at.rows; r += parts) {
            const int t = (r * at.cols + c / V) * V + c % V;
            m.x += s_b[t];
            m.y += s_w[t];
        }
        s_part[threadIdx.x] = m;
    }
    __syncthreads();
    if ((int)threadIdx.x < channels) {
        float2 m = make_float2(0.0f, 0.0f);
        for (int part = 0; part < parts; ++part) {
            m.x += s_part[part * channels + threadIdx.x].x;
            m.y += s_part[part * channels + threadIdx.x].y;
        }
        s_mine[threadIdx.x] = m;
    }
    cluster.sync();
    if ((int)threadIdx.x < channels) {
        float2 m = make_float2(0.0f, 0.0f);
        for (int r = 0; r < ranks; ++r) {
            const float2 v = *cluster.map_shared_rank(&s_mine[threadIdx.x], r);
            m.x += v.x;
            m.y += v.y;
        }
        const int c = at.slab * channels + threadIdx.x;
        if (rank == 0) a.n.sums[(int64_t)at.sample * a.n.channels + c] = m;
        const float w = a.n.weight ? a.n.weight[c] : 1.0f;
        s_all[threadIdx.x] = make_float2(w * m.x, w * m.y);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < a.slab_groups; g += kResidentBlock) {
        float2 m = make_float2(0.0f, 0.0f);
        for (int c = g * per_group; c < (g + 1) * per_group; ++c) {
            m.x += s_all[c].x;
            m.y += s_all[c].y;
        }
        const float inv = 1.0f / ((float)per_group * (float)a.n.positions);
        s_group[g] = make_float2(m.x * inv, m.y * inv);
    }
    __syncthreads();
    if (at.live) {
        float2 m1[kPairs<V>], m2[kPairs<V>];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 m = s_group[(at.col * V + j) / per_group];
            (&m1[j / 2].x)[j % 2] = m.x;
            (&m2[j / 2].x)[j % 2] = m.y;
        }
        T *y = (T *)a.n.y + at.base;
#pragma unroll 2
        for (int p = at.row; p < count; p += at.rows) {
            Vec<T, V> vx = s_x[p * at.cols + at.col];
            input_gradient<T, V, ACT>(ch, m1, m2, vx, s_d[p * at.cols + at.col]);
            *(Vec<T, V> *)(y + (int64_t)p * a.n.channels) = vx;
        }
    }
    cluster.sync();   // no block leaves while another may read its shared memory
}

// Parameter gradients: the samples' channel sums in order.
__global__ void __launch_bounds__(kNormBlock) k_norm_param_grads(const NormArgs a)
{
    grid_dependency_begin();
    const int c = blockIdx.x * kNormBlock + threadIdx.x;
    if (c >= a.channels) return;
    float2 m = make_float2(0.0f, 0.0f);
    for (int n = 0; n < a.samples; ++n) {
        const float2 v = a.sums[(int64_t)n * a.channels + c];
        m.x += v.x;
        m.y += v.y;
    }
    if (a.dbias) a.dbias[c] = m.x;
    if (a.dweight) a.dweight[c] = m.y;
}

struct ResidentPlan {
    bool fits = false;
    int slab_groups, slabs, cluster;
    int64_t rows;
    size_t smem;
};

// Slabs of whole groups and whole vectors, 64 bytes wide where the groups allow
// (narrower rows waste DRAM sectors), over as few blocks as hold 32 KB each and as
// many as a cluster has.
ResidentPlan resident_plan(const gsr_group_norm &d, int width, bool backward)
{
    ResidentPlan p;
    const int size = d.dtype == GSR_F32 ? 4 : 2, per_group = d.channels / d.groups;
    if (width * size != 16) return p;
    int groups = 1;
    for (; groups <= d.groups; ++groups)
        if (d.groups % groups == 0 && groups * per_group % width == 0 &&
            (groups == d.groups || groups * per_group * size >= 64))
            break;
    const int channels = groups * per_group, arrays = backward ? 2 : 1;
    if (groups > d.groups || channels > kResidentChannels) return p;
    const int64_t row_bytes = (int64_t)channels * size * arrays, bytes = d.positions * row_bytes;
    int64_t cluster = (bytes + 32 * 1024 - 1) / (32 * 1024);
    if (cluster > kResidentCluster) cluster = kResidentCluster;
    const int64_t rows = (d.positions + cluster - 1) / cluster;
    if (rows * row_bytes > (int64_t)kResidentData) return p;
    p.fits = true;
    p.slab_groups = groups;
    p.slabs = d.groups / groups;
    p.cluster = (int)cluster;
    p.rows = rows;
    const size_t sums = (size_t)kResidentBlock * width * 2 * sizeof(float);
    const size_t rest = backward ? (kResidentBlock + 3 * kResidentChannels) * sizeof(float2)
                                 : kResidentBlock * (sizeof(float) + sizeof(Moments)) +
                                       kResidentChannels * (sizeof(Moments) + sizeof(float2));
    p.smem = (size_t)(rows * row_bytes) + sums + rest;
    return p;
}

template <typename Kernel>
cudaError_t launch_cluster(gsr_ctx *ctx, Kernel *kernel, const ResidentPlan &p, const ResidentArgs &a,
                           cudaStream_t stream)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
    if (e != cudaSuccess) return e;
    return launch_kernel_smem(ctx, kernel, dim3((unsigned)((int64_t)a.n.samples * a.slabs * p.cluster)), kResidentBlock,
                              p.smem, (unsigned)p.cluster, stream, a);
}

// ---- host ---------------------------------------------------------------------------

// Splits of the positions: enough blocks for every SM, a few runs of rows each.
struct NormPlan {
    int vectors, slabs, chunks, wave;
    int64_t rows_per_chunk;
};

NormPlan norm_plan(const gsr_ctx *ctx, const gsr_group_norm &d, int width)
{
    NormPlan p;
    const int vectors = (d.channels + width - 1) / width;
    p.vectors = vectors < kNormBlock ? vectors : kNormBlock;
    p.slabs = (vectors + p.vectors - 1) / p.vectors;
    const int rows = kNormBlock / p.vectors;
    p.wave = d.samples < 65535 ? d.samples : 65535;   // samples of a launch (a grid's limit)
    // Narrow accesses hold fewer bytes in flight and fewer registers: more blocks.
    const int blocks = width * (d.dtype == GSR_F32 ? 4 : 2) == 16 ? kNormOccupancy : 3 * kNormOccupancy;
    int64_t chunks = (int64_t)blocks * ctx->num_sms / ((int64_t)p.wave * p.slabs);
    const int64_t most = (d.positions + (int64_t)rows * kRun - 1) / ((int64_t)rows * kRun);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    p.rows_per_chunk = (d.positions + chunks - 1) / chunks;
    p.chunks = (int)((d.positions + p.rows_per_chunk - 1) / p.rows_per_chunk);
    return p;
}

// Elements of an access: 16 bytes, or 4 where the channels or the arrays allow no
// more, or one.
int norm_width(const gsr_group_norm &d, const void *x, const void *dout, const void *y)
{
    const int size = d.dtype == GSR_F32 ? 4 : 2;
    for (int bytes : {16, 4}) {
        const int width = bytes / size;
        if (d.channels % width == 0 && (uintptr_t)x % bytes == 0 && (uintptr_t)dout % bytes == 0 &&
            (uintptr_t)y % bytes == 0)
            return width;
    }
    return 1;
}

// A kernel that walks rows of N arrays.
template <typename T, int V, int N, typename Kernel>
cudaError_t launch_walk(gsr_ctx *ctx, Kernel *kernel, dim3 grid, cudaStream_t stream, const NormArgs &a)
{
    constexpr size_t smem = kWalkBytes<T, V, N>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_kernel_smem(ctx, kernel, grid, kNormBlock, smem, 1, stream, a);
}

template <typename T, int V, int ACT>
cudaError_t norm_forward(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    for (a.sample0 = 0; a.sample0 < a.samples; a.sample0 += p.wave) {
        const unsigned n = (unsigned)(a.samples - a.sample0 < p.wave ? a.samples - a.sample0 : p.wave);
        const dim3 grid((unsigned)p.chunks, n, (unsigned)p.slabs);
        cudaError_t e = launch_walk<T, V, 1>(ctx, k_norm_moments<T, V>, grid, stream, a);
        if (e == cudaSuccess) e = launch_kernel(ctx, k_norm_merge, dim3((unsigned)a.groups, n), kMergeBlock, stream, a);
        if (e == cudaSuccess) e = launch_walk<T, V, 1>(ctx, k_norm_apply<T, V, ACT>, grid, stream, a);
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
        cudaError_t e = launch_walk<T, V, 2>(ctx, k_norm_grad_sums<T, V, ACT>, grid, stream, a);
        if (e == cudaSuccess)
            e = launch_kernel(ctx, k_norm_grad_merge, dim3((unsigned)a.groups, n), kMergeBlock, stream, a);
        if (e == cudaSuccess) e = launch_walk<T, V, 2>(ctx, k_norm_grad_apply<T, V, ACT>, grid, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int V, int ACT>
cudaError_t norm_resident(gsr_ctx *ctx, const NormArgs &n, const ResidentPlan &p, bool backward, cudaStream_t stream)
{
    ResidentArgs a = {};
    a.n = n;
    a.slabs = p.slabs;
    a.slab_groups = p.slab_groups;
    a.slab_channels = p.slab_groups * n.per_group;
    a.rows_per_block = p.rows;
    a.row_capacity = (int)p.rows;
    if (!backward) return launch_cluster(ctx, k_norm_resident<T, V, ACT>, p, a, stream);
    const cudaError_t e = launch_cluster(ctx, k_norm_grad_resident<T, V, ACT>, p, a, stream);
    if (e != cudaSuccess) return e;
    return launch_kernel(ctx, k_norm_param_grads, dim3((unsigned)((n.channels + kNormBlock - 1) / kNormBlock)),
                         kNormBlock, stream, n);
}

template <typename T, int ACT>
cudaError_t dispatch_width(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, const ResidentPlan &r, int width,
                           bool backward, cudaStream_t s)
{
    constexpr int kFull = 16 / (int)sizeof(T);
    if (r.fits) return norm_resident<T, kFull, ACT>(ctx, a, r, backward, s);
    if (width == kFull) return backward ? norm_backward<T, kFull, ACT>(ctx, a, p, s) : norm_forward<T, kFull, ACT>(ctx, a, p, s);
    if constexpr (sizeof(T) == 2)
        if (width == 2) return backward ? norm_backward<T, 2, ACT>(ctx, a, p, s) : norm_forward<T, 2, ACT>(ctx, a, p, s);
    return backward ? norm_backward<T, 1, ACT>(ctx, a, p, s) : norm_forward<T, 1, ACT>(ctx, a, p, s);
}

template <typename T>
cudaError_t dispatch_act(gsr_ctx *ctx, NormArgs &a, const NormPlan &p, const ResidentPlan &r, int act, int width,
                         bool backward, cudaStream_t s)
{
    if (act == GSR_ACT_SILU) return dispatch_width<T, GSR_ACT_SILU>(ctx, a, p, r, width, backward, s);
    if (act == GSR_ACT_GELU) return dispatch_width<T, GSR_ACT_GELU>(ctx, a, p, r, width, backward, s);
    return dispatch_width<T, GSR_ACT_NONE>(ctx, a, p, r, width, backward, s);
}

int run_norm(gsr_ctx *ctx, const gsr_group_norm &d, NormArgs &a, bool backward, cudaStream_t stream)
{
    const int width = norm_width(d, a.x, a.dout, a.y);
    const ResidentPlan r = resident_plan(d, width, backward);
    const NormPlan p = norm_plan(ctx, d, width);
    a.samples = d.samples;
    a.channels = d.channels;
    a.groups = d.groups;
    a.per_group = d.channels / d.groups;
    a.positions = d.positions;
    a.rows_per_chunk = p.rows_per_chunk;
    a.chunks = p.chunks;
    a.vectors = p.vectors;
    a.eps = d.eps;
    const size_t partial = r.fits ? 0 : round_up((size_t)p.wave * p.chunks * d.channels * sizeof(float2), 256);
    const size_t sums = backward ? (size_t)d.samples * d.channels * sizeof(float2) : 0;
    const size_t group_sums = backward ? (size_t)d.samples * d.groups * sizeof(float2) : 0;
    const bool scratch = partial + sums + group_sums > 0;
    Workspace workspace(ctx, stream);
    void *work = nullptr;
    if (scratch)
        if (int rc = workspace.take(partial + sums + group_sums, &work)) return rc;
    a.partial = (float2 *)work;
    a.sums = (float2 *)((unsigned char *)work + partial);
    a.group_sums = (float2 *)((unsigned char *)work + partial + sums);
    cudaError_t e;
    if (d.dtype == GSR_F32)
        e = dispatch_act<float>(ctx, a, p, r, d.activation, width, backward, stream);
    else if (d.dtype == GSR_BF16)
        e = dispatch_act<__nv_bfloat16>(ctx, a, p, r, d.activation, width, backward, stream);
    else
        e = dispatch_act<__half>(ctx, a, p, r, d.activation, width, backward, stream);
    if (int rc = cuda_check(ctx, e, backward ? "group norm backward" : "group norm forward")) return rc;
    return workspace.done();
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
