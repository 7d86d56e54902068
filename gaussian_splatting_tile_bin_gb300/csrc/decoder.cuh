// decoder.cuh -- helpers shared by the decoder's operators (group norm, rotary
// positions, cross attention): element types, vector access, the workspace.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"

namespace gsr {

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

// V elements moved as one access of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// Scratch memory of `bytes` for the launches that follow on `stream`, and the
// mark after them.  workspace() grows the context's arena and makes `stream`
// wait for the last call that used it on another stream.
int workspace(gsr_ctx *ctx, size_t bytes, cudaStream_t stream, void **out);
int workspace_done(gsr_ctx *ctx, cudaStream_t stream);

// GSR_ERR_CUDA, once, if a kernel's bounded wait ran out in an earlier call.
int check_status(gsr_ctx *ctx);

inline size_t round_up(size_t n, size_t unit) { return (n + unit - 1) / unit * unit; }

}  // namespace gsr
