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
constexpr int kPackKeys = 8;   // neighbouring keys of a thread

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
    for (int j0 = 0; j0 < length; j0 += kPackBlock * kPackKeys) {
        const int j = j0 + threadIdx.x * kPackKeys;
        uint32_t keep = 0;
#pragma unroll
        for (int k = 0; k < kPackKeys; ++k)
            if (j + k < length && mask[j + k] != 0) keep |= 1u << k;
        const int mine = __popc(keep);
        int before = mine;                                   // inclusive over the warp
        for (int d = 1; d < 32; d *= 2) {
            const int other = __shfl_up_sync(~0u, before, d);
            if (lane >= d) before += other;
        }
        if (lane == 31) s_warp[warp] = before;
        __syncthreads();
        int all = s_warp[lane];                              // as many warps as lanes
        for (int d = 1; d < 32; d *= 2) {
            const int other = __shfl_up_sync(~0u, all, d);
            if (lane >= d) all += other;
        }
        const int warps_before = __shfl_sync(~0u, all, warp) - s_warp[warp];
        int at = base + warps_before + before - mine;
#pragma unroll
        for (int k = 0; k < kPackKeys; ++k)
            if (keep >> k & 1) index[at++] = j + k;
        base += __shfl_sync(~0u, all, 31);
        __syncthreads();
    }
    if (threadIdx.x == 0) counts[b] = base;
}
static_assert(kPackBlock / 32 == 32, "one warp scans the warps' counts");

// Copies the kept keys' rows of k and v, 16 bytes a thread; block y is the
// head, z the item; rows of a head lie one behind the other.
__global__ void __launch_bounds__(256) k_pack_rows(gsr_heads k, gsr_heads v, uint4 *to_k, uint4 *to_v, int kv_len,
                                                   int heads, int chunks, const int32_t *counts, const int32_t *index)
{
    grid_dependency_begin();
    const int i = blockIdx.x * 256 + threadIdx.x, t = i / chunks, c = i - t * chunks;
    const int64_t b = blockIdx.z, h = blockIdx.y;
    if (t >= counts[b]) return;
    const int64_t j = index[b * kv_len + t], to = (b * heads + h) * ((int64_t)kv_len * chunks) + i;
    to_k[to] = *(const uint4 *)((const uint16_t *)k.data + b * k.batch_stride + j * k.token_stride + h * k.head_stride +
                                c * 8);
    to_v[to] = *(const uint4 *)((const uint16_t *)v.data + b * v.batch_stride + j * v.token_stride + h * v.head_stride +
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

int tokens_map(gsr_ctx *ctx, CUtensorMap *map, void *data, int dtype, int64_t channels, int64_t tokens, int64_t batch,
               int64_t token_stride, int64_t batch_stride, int box_channels, int box_tokens)
{
    const EncodeTiled encode = encoder();
    if (!encode) return fail(ctx, GSR_ERR_CUDA, "the driver offers no cuTensorMapEncodeTiled");
    const int64_t size = dtype == GSR_F32 ? 4 : 2, items = batch_stride != 0 ? batch : 1;
    const cuuint64_t extents[3] = {(cuuint64_t)channels, (cuuint64_t)tokens, (cuuint64_t)items};
    // (An extent of 1 may carry any stride; give it one the encoder takes.)
    const cuuint64_t strides[2] = {(cuuint64_t)(token_stride * size),
                                   (cuuint64_t)(items > 1 ? batch_stride * size : token_stride * size)};
    const cuuint32_t box[3] = {(cuuint32_t)box_channels, (cuuint32_t)box_tokens, 1}, one[3] = {1, 1, 1};
    const CUtensorMapDataType type = dtype == GSR_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == GSR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = encode(map, type, 3, data, extents, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
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
    // Items beyond a grid's z go in further launches.
    for (int b = 0; e == cudaSuccess && b < d.batch; b += 65535) {
        const int n = d.batch - b < 65535 ? d.batch - b : 65535;
        gsr_heads kb = k, vb = v;
        kb.data = (uint16_t *)k.data + b * k.batch_stride;
        vb.data = (uint16_t *)v.data + b * v.batch_stride;
        const int64_t first = (int64_t)b * d.kv_heads * d.kv_len * chunks;
        e = launch_kernel(ctx, k_pack_rows, dim3((unsigned)(((int64_t)d.kv_len * chunks + 255) / 256),
                                                 (unsigned)d.kv_heads, (unsigned)n),
                          256, stream, kb, vb, (uint4 *)out->k.data + first, (uint4 *)out->v.data + first, (int)d.kv_len,
                          (int)d.kv_heads, chunks, (const int32_t *)out->counts + b,
                          (const int32_t *)out->index + (int64_t)b * d.kv_len);
    }
    return e;
}

}  // namespace gsr
