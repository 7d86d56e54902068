// decoder.cuh -- the decoder's operators (group norm, rotary positions, cross
// attention): their host sides, and what they share: element types, vector access,
// launches with dynamic shared memory, the workspace.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"

namespace gsr {

// Host sides (validated arguments).
int group_norm_forward(gsr_ctx *ctx, const gsr_group_norm &d, const void *x, const float *weight, const float *bias,
                       void *out, float *mean, float *rstd, cudaStream_t stream);
int group_norm_backward(gsr_ctx *ctx, const gsr_group_norm &d, const void *dout, const void *x, const float *weight,
                        const float *bias, const float *mean, const float *rstd, void *dx, float *dweight,
                        float *dbias, cudaStream_t stream);
// Rotation by +theta (sign = 1) or -theta (sign = -1).
int rotary(gsr_ctx *ctx, const gsr_rotary &d, const gsr_heads &x, const void *positions, const float *frequencies,
           const gsr_heads &out, float sign, cudaStream_t stream);
int cross_attention_forward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k,
                            const gsr_heads &v, const gsr_heads &out, float *lse, cudaStream_t stream);
int cross_attention_backward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k,
                             const gsr_heads &v, const gsr_heads &out, const float *lse, const gsr_heads &dout,
                             const gsr_heads &dq, const gsr_heads &dk, const gsr_heads &dv, cudaStream_t stream);

// launch_kernel with smem bytes of dynamic shared memory, and in clusters of
// `cluster` blocks.
template <typename... Params, typename... Args>
cudaError_t launch_kernel_smem(gsr_ctx *ctx, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                               unsigned cluster, cudaStream_t stream, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = ctx->opt_pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    ++ctx->launches;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs, one instruction for both.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\n"
        "mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 d, a, b;\n"
        "mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Two values as a 16-bit pair, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// V elements moved as one access of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// Elements i and i + 1 of an access as floats (0 behind an access of one).
template <typename T, int V>
__device__ __forceinline__ float2 pair_of(const Vec<T, V> &v, int i)
{
    return make_float2(to_float(v.e[i]), V > 1 ? to_float(v.e[(i + 1) % V]) : 0.0f);
}
template <typename T, int V>
__device__ __forceinline__ void set_pair(Vec<T, V> &v, int i, float2 f)
{
    if constexpr (sizeof(T) == 2 && V > 1) {
        *(uint32_t *)&v.e[i] = pack2<T>(f.x, f.y);
    } else {
        v.e[i] = from_float<T>(f.x);
        if (V > 1) v.e[(i + 1) % V] = from_float<T>(f.y);
    }
}

// Scratch memory for a call's launches on `stream`.  take() grows the context's
// arena and makes `stream` wait for the last call that used it; done() marks this
// call's use.  A call that fails in between has perhaps launched work that uses the
// memory, so its use is marked on the way out.  take() of 0 bytes orders nothing.
class Workspace {
public:
    Workspace(gsr_ctx *ctx, cudaStream_t stream) : ctx_(ctx), stream_(stream) {}
    ~Workspace();
    Workspace(const Workspace &) = delete;
    int take(size_t bytes, void **out);
    int done();

private:
    int mark();
    gsr_ctx *ctx_;
    cudaStream_t stream_;
    bool used_ = false;
};

// GSR_ERR_CUDA, once, if a kernel's bounded wait ran out in an earlier call, as far
// as that has run.
int check_status(gsr_ctx *ctx);

inline size_t round_up(size_t n, size_t unit) { return (n + unit - 1) / unit * unit; }

}  // namespace gsr
