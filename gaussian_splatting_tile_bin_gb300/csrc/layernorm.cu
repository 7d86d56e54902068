// layernorm.cu -- layer norm over the channels of a row (a token, or a head of a
// token) behind a residual sum, forward and backward.
//
//   total = x + residual,  xh = (total - mean) rstd,  out = xh w + b
// and with g = dout w
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dtotal,  dw = sum dout xh,  db = sum dout.
//
// One warp a row, three passes over it.
#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kRowBlock = 256;

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
    int tokens, heads, channels, rows, blocks;
    float eps;
};

template <typename T>
__device__ __forceinline__ T *row_of(const Rows &r, const LayerArgs &a, int row)
{
    const int token = row / a.heads, head = row - token * a.heads;
    const int b = token / a.tokens, t = token - b * a.tokens;
    return (T *)r.data + b * r.batch + t * r.token + head * r.head;
}

__device__ __forceinline__ float warp_sum(float v)
{
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kRowBlock) k_layer_norm(const LayerArgs a)
{
    grid_dependency_begin();
    const int row = blockIdx.x * (kRowBlock / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (row >= a.rows) return;
    const T *x = row_of<T>(a.x, a, row);
    T *out = row_of<T>(a.out, a, row);
    if (a.residual.data) {
        const T *residual = row_of<T>(a.residual, a, row);
        T *total = row_of<T>(a.total, a, row);
        for (int c = lane; c < a.channels; c += 32) total[c] = from_float<T>(to_float(x[c]) + to_float(residual[c]));
        x = total;
    }
    float sum = 0.0f, square = 0.0f;
    for (int c = lane; c < a.channels; c += 32) sum += to_float(x[c]);
    const float mean = warp_sum(sum) / a.channels;
    for (int c = lane; c < a.channels; c += 32) {
        const float d = to_float(x[c]) - mean;
        square = fmaf(d, d, square);
    }
    const float rstd = 1.0f / sqrtf(warp_sum(square) / a.channels + a.eps);
    for (int c = lane; c < a.channels; c += 32)
        out[c] = from_float<T>(fmaf((to_float(x[c]) - mean) * rstd, a.weight ? a.weight[c] : 1.0f,
                                    a.bias ? a.bias[c] : 0.0f));
    if (lane == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowBlock) k_layer_norm_grad(const LayerArgs a)
{
    grid_dependency_begin();
    const int row = blockIdx.x * (kRowBlock / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (row >= a.rows) return;
    const T *total = row_of<T>(a.total, a, row), *dout = row_of<T>(a.x, a, row);
    const T *dtotal = a.residual.data ? row_of<T>(a.residual, a, row) : nullptr;
    T *dx = row_of<T>(a.out, a, row);
    const float mean = a.mean[row], rstd = a.rstd[row], share = 1.0f / a.channels;
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = lane; c < a.channels; c += 32) {
        const float xh = (to_float(total[c]) - mean) * rstd, g = to_float(dout[c]) * (a.weight ? a.weight[c] : 1.0f);
        s1 += g;
        s2 = fmaf(g, xh, s2);
    }
    s1 = warp_sum(s1) * share;
    s2 = warp_sum(s2) * share;
    for (int c = lane; c < a.channels; c += 32) {
        const float xh = (to_float(total[c]) - mean) * rstd, g = to_float(dout[c]) * (a.weight ? a.weight[c] : 1.0f);
        float d = rstd * (g - s1 - xh * s2);
        if (dtotal) d += to_float(dtotal[c]);
        dx[c] = from_float<T>(d);
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowBlock) k_layer_norm_sums(const LayerArgs a)
{
    grid_dependency_begin();
    const int c = blockIdx.y * kRowBlock + threadIdx.x;
    if (c >= a.channels) return;
    float2 sum = make_float2(0.0f, 0.0f);
    for (int row = blockIdx.x; row < a.rows; row += a.blocks) {
        const float d = to_float(row_of<T>(a.x, a, row)[c]);
        sum.x = fmaf(d, (to_float(row_of<T>(a.total, a, row)[c]) - a.mean[row]) * a.rstd[row], sum.x);
        sum.y += d;
    }
    a.partial[(int64_t)blockIdx.x * a.channels + c] = sum;
}

__global__ void __launch_bounds__(kRowBlock) k_layer_norm_params(const LayerArgs a)
{
    grid_dependency_begin();
    const int c = blockIdx.x * kRowBlock + threadIdx.x;
    if (c >= a.channels) return;
    float2 sum = make_float2(0.0f, 0.0f);
    for (int i = 0; i < a.blocks; ++i) {
        const float2 v = a.partial[(int64_t)i * a.channels + c];
        sum.x += v.x;
        sum.y += v.y;
    }
    if (a.dweight) a.dweight[c] = sum.x;
    if (a.dbias) a.dbias[c] = sum.y;
}

Rows rows_of(const gsr_heads *t)
{
    return t ? Rows{t->data, t->batch_stride, t->token_stride, t->head_stride} : Rows{};
}

LayerArgs args_of(const gsr_layer_norm &d)
{
    LayerArgs a = {};
    a.tokens = d.tokens;
    a.heads = d.heads;
    a.channels = d.channels;
    a.rows = d.batch * d.tokens * d.heads;
    a.eps = d.eps;
    return a;
}

unsigned row_blocks(const LayerArgs &a) { return (unsigned)(((int64_t)a.rows + kRowBlock / 32 - 1) / (kRowBlock / 32)); }

template <typename T>
cudaError_t run_forward(gsr_ctx *ctx, const LayerArgs &a, cudaStream_t stream)
{
    return launch_kernel(ctx, k_layer_norm<T>, dim3(row_blocks(a)), kRowBlock, stream, a);
}

template <typename T>
cudaError_t run_backward(gsr_ctx *ctx, const LayerArgs &a, cudaStream_t stream)
{
    const unsigned columns = (unsigned)((a.channels + kRowBlock - 1) / kRowBlock);
    cudaError_t e = cudaSuccess;
    if (a.partial) {   // first: dx may take dout's place
        e = launch_kernel(ctx, k_layer_norm_sums<T>, dim3((unsigned)a.blocks, columns), kRowBlock, stream, a);
        if (e == cudaSuccess) e = launch_kernel(ctx, k_layer_norm_params, dim3(columns), kRowBlock, stream, a);
    }
    if (e == cudaSuccess) e = launch_kernel(ctx, k_layer_norm_grad<T>, dim3(row_blocks(a)), kRowBlock, stream, a);
    return e;
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
    cudaError_t e;
    if (d.dtype == GSR_F32)
        e = run_forward<float>(ctx, a, stream);
    else if (d.dtype == GSR_BF16)
        e = run_forward<__nv_bfloat16>(ctx, a, stream);
    else
        e = run_forward<__half>(ctx, a, stream);
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
    a.blocks = a.rows < 2 * ctx->num_sms ? a.rows : 2 * ctx->num_sms;
    Workspace workspace(ctx, stream);
    if (dweight || dbias) {
        void *work = nullptr;
        if (int rc = workspace.take((size_t)a.blocks * d.channels * sizeof(float2), &work)) return rc;
        a.partial = (float2 *)work;
    }
    cudaError_t e;
    if (d.dtype == GSR_F32)
        e = run_backward<float>(ctx, a, stream);
    else if (d.dtype == GSR_BF16)
        e = run_backward<__nv_bfloat16>(ctx, a, stream);
    else
        e = run_backward<__half>(ctx, a, stream);
    if (int rc = cuda_check(ctx, e, "layer norm backward")) return rc;
    return workspace.done();
}

}  // namespace gsr
