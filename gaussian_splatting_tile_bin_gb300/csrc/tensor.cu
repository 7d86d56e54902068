// tensor.cu -- tensor maps, and the packing of masked keys for the attention kernels.
#include "attention.cuh"

namespace gsr {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once per process (an entry point, the same for every device).
EncodeTiled encoder()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

constexpr int kPackBlock = 1024;

// Item b's kept keys in ascending order, and how many they are.
__global__ void __launch_bounds__(kPackBlock) k_pack_index(const uint8_t *mask, const int32_t *lengths, int kv_len,
                                                           int32_t *counts, int32_t *index)
{
    grid_dependency_begin();
    __shared__ int s_warp[kPackBlock / 32];
    const int b = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int length = item_length(lengths, kv_len, b);
    mask += (int64_t)b * kv_len;
    index += (int64_t)b * kv_len;
    int base = 0;
    for (int j0 = 0; j0 < length; j0 += kPackBlock) {
        const int j = j0 + threadIdx.x;
        const bool keep = j < length && mask[j] != 0;
        const unsigned votes = __ballot_sync(~0u, keep);
        if (lane == 0) s_warp[warp] = __popc(votes);
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kPackBlock / 32; ++w) {
            if (w < warp) before += s_warp[w];
            all += s_warp[w];
        }
        if (keep) index[base + before + __popc(votes & ((1u << lane) - 1))] = j;
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) counts[b] = base;
}

// Copies the kept keys' rows of k and v, 16 bytes a thread.
__global__ void __launch_bounds__(256) k_pack_rows(gsr_heads k, gsr_heads v, uint4 *to_k, uint4 *to_v, int64_t items,
                                                   int kv_len, int heads, int chunks, const int32_t *counts,
                                                   const int32_t *index)
{
    grid_dependency_begin();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items) return;
    const int c = (int)(i % chunks);
    const int64_t row = i / chunks;              // [item][head][token]
    const int t = (int)(row % kv_len);
    const int h = (int)(row / kv_len % heads);
    const int64_t b = row / kv_len / heads;
    if (t >= counts[b]) return;
    const int64_t j = index[b * kv_len + t];
    to_k[i] = *(const uint4 *)((const uint16_t *)k.data + b * k.batch_stride + j * k.token_stride + h * k.head_stride +
                               c * 8);
    to_v[i] = *(const uint4 *)((const uint16_t *)v.data + b * v.batch_stride + j * v.token_stride + h * v.head_stride +
                               c * 8);
}

}  // namespace

int check_registers(gsr_ctx *ctx, const void *kernel, const char *name)
{
    cudaFuncAttributes attributes;
    if (int rc = cuda_check(ctx, cudaFuncGetAttributes(&attributes, kernel), name)) return rc;
    if (attributes.numRegs < kStartRegisters)
        return fail(ctx, GSR_ERR_CUDA, std::string(name) + " was compiled to start with too few registers");
    return GSR_OK;
}

int heads_map(gsr_ctx *ctx, CUtensorMap *map, const gsr_heads &t, int dtype, int64_t batch, int64_t tokens,
              int64_t heads, int dim, int rows)
{
    const EncodeTiled encode = encoder();
    if (!encode) return fail(ctx, GSR_ERR_CUDA, "the driver offers no cuTensorMapEncodeTiled");
    // Extents of 1 may carry any stride; give them one the encoder takes.
    const int64_t dense = round_up(dim * 2, 16);
    auto bytes = [&](int64_t extent, int64_t stride) { return (cuuint64_t)(extent > 1 && stride > 0 ? stride * 2 : dense); };
    const cuuint64_t extents[4] = {(cuuint64_t)dim, (cuuint64_t)tokens,
                                   (cuuint64_t)(t.head_stride != 0 ? heads : 1),
                                   (cuuint64_t)(t.batch_stride != 0 ? batch : 1)};
    const cuuint64_t strides[3] = {bytes(tokens, t.token_stride), bytes(heads, t.head_stride),
                                   bytes(batch, t.batch_stride)};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, dtype == GSR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              4, t.data, extents, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ctx, GSR_ERR_CUDA, "cuTensorMapEncodeTiled: error " + std::to_string((int)r));
    return GSR_OK;
}

size_t packed_bytes(const gsr_attention &d)
{
    const size_t rows = (size_t)d.batch * d.kv_heads * d.kv_len * d.head_dim * 2;
    return 2 * round_up(rows, 256) + round_up((size_t)d.batch * 4, 256) + (size_t)d.batch * d.kv_len * 4;
}

cudaError_t pack_keys(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &k, const gsr_heads &v, void *work,
                      Packed *out, cudaStream_t stream)
{
    const size_t rows = round_up((size_t)d.batch * d.kv_heads * d.kv_len * d.head_dim * 2, 256);
    unsigned char *p = (unsigned char *)work;
    out->k = {p, (int64_t)d.kv_heads * d.kv_len * d.head_dim, d.head_dim, (int64_t)d.kv_len * d.head_dim};
    out->v = out->k;
    out->v.data = p + rows;
    out->counts = (int32_t *)(p + 2 * rows);
    out->index = (int32_t *)(p + 2 * rows + round_up((size_t)d.batch * 4, 256));
    cudaError_t e = launch_kernel(ctx, k_pack_index, dim3((unsigned)d.batch), kPackBlock, stream, d.key_mask,
                                  d.kv_lengths, (int)d.kv_len, out->counts, out->index);
    const int chunks = d.head_dim / 8;
    const int64_t items = (int64_t)d.batch * d.kv_heads * d.kv_len * chunks;
    if (e == cudaSuccess)
        e = launch_kernel(ctx, k_pack_rows, dim3((unsigned)((items + 255) / 256)), 256, stream, k, v,
                          (uint4 *)out->k.data, (uint4 *)out->v.data, items, (int)d.kv_len, (int)d.kv_heads, chunks,
                          (const int32_t *)out->counts, (const int32_t *)out->index);
    return e;
}

}  // namespace gsr
