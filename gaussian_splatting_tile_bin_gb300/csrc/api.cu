// api.cu -- the extern "C" surface of libgsr.so: argument checks, the device
// guard, error reporting and the context / arena lifetime.  The operations
// themselves live in bin.cu and raster.cu.
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <new>
#include <string>

#include "decoder.cuh"

namespace gsr {

int fail(gsr_ctx *ctx, int code, const std::string &msg)
{
    if (ctx) ctx->err = msg;
    return code;
}

int cuda_check(gsr_ctx *ctx, cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return GSR_OK;
    return fail(ctx, GSR_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

namespace {

// Makes the context's device current for the lifetime of the guard.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            cudaGetLastError();
            prev = -1;
        }
        if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// An NVTX range named after the entry point, for profilers' timelines (a no-op
// unless a tool is attached).
struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_bins(gsr_ctx *ctx, const gsr_bins *bins, int32_t n)
{
    if (!bins) return fail(ctx, GSR_ERR_INVALID_ARG, "bins is NULL");
    if (bins->n != n) return fail(ctx, GSR_ERR_INVALID_ARG, "n differs from the n the bins were built from");
    if (bins->width < 1 || bins->height < 1 || bins->width > GSR_MAX_IMAGE_SIDE ||
        bins->height > GSR_MAX_IMAGE_SIDE)
        return fail(ctx, GSR_ERR_INVALID_ARG, "bins carry an invalid image size");
    if (bins->tiles_x != (bins->width + GSR_TILE - 1) / GSR_TILE ||
        bins->tiles_y != (bins->height + GSR_TILE - 1) / GSR_TILE)
        return fail(ctx, GSR_ERR_INVALID_ARG, "bins carry an inconsistent tile grid");
    if (!bins->tile_ranges || (n > 0 && bins->num_pairs > 0 && !bins->sorted_idx))
        return fail(ctx, GSR_ERR_INVALID_ARG, "bins hold NULL arrays");
    return GSR_OK;
}

}  // namespace
}  // namespace gsr

using namespace gsr;

extern "C" {

int gsr_create(gsr_ctx **out, int device)
{
    if (!out) return GSR_ERR_INVALID_ARG;
    *out = nullptr;
    int count = 0;
    if (cudaGetDeviceCount(&count) != cudaSuccess) {
        cudaGetLastError();
        return GSR_ERR_CUDA;
    }
    if (device < 0 || device >= count) return GSR_ERR_INVALID_ARG;
    // Grid sizes of the grid-stride kernels are multiples of the SM count.
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return GSR_ERR_CUDA;
    }
    gsr_ctx *ctx = new (std::nothrow) gsr_ctx();
    if (!ctx) return GSR_ERR_OOM;
    ctx->device = device;
    ctx->num_sms = sms;
    *out = ctx;
    return GSR_OK;
}

void gsr_destroy(gsr_ctx *ctx)
{
    if (!ctx) return;
    {
        DeviceGuard g(ctx->device);
        for (int b = 0; b < 3; ++b) {
            cudaFree(ctx->pairs.k[b]);
            cudaFree(ctx->pairs.v[b]);
        }
        cudaFree(ctx->rects);
        for (int b = 0; b < 3; ++b) {
            cudaFree(ctx->depth.k[b]);
            cudaFree(ctx->depth.v[b]);
        }
        cudaFree(ctx->blk_sums);
        cudaFree(ctx->ranges);
        cudaFree(ctx->radix_counts);
        cudaFree(ctx->radix_totals);
        cudaFree(ctx->scalars);
        cudaFree(ctx->grad_acc);
        cudaFree(ctx->bwd_tile_cost);
        cudaFree(ctx->det_escale);
        cudaFree(ctx->bnd);
        cudaFree(ctx->bwd_items);
        cudaFree(ctx->fwd_items);
        cudaFree(ctx->work);
        while (gsr::Outgrown *kept = ctx->outgrown) {
            ctx->outgrown = kept->next;
            cudaFree(kept->buffer);
            delete kept;
        }
        if (ctx->status_host) cudaFreeHost(ctx->status_host);
        if (ctx->work_event) cudaEventDestroy(ctx->work_event);
        while (gsr::CaptureMark *mark = ctx->captures) {
            ctx->captures = mark->next;
            if (mark->event) cudaEventDestroy(mark->event);
            delete mark;
        }
        if (ctx->host_total) cudaFreeHost(ctx->host_total);
    }
    delete ctx;
}

const char *gsr_last_error(const gsr_ctx *ctx) { return ctx ? ctx->err.c_str() : "NULL context"; }

int gsr_set_option(gsr_ctx *ctx, int option, int value)
{
    if (!ctx) return GSR_ERR_INVALID_ARG;
    if (value != 0 && value != 1) return fail(ctx, GSR_ERR_INVALID_ARG, "option value must be 0 or 1");
    switch (option) {
    case GSR_OPT_BWD_WARP_SKIP: ctx->opt_warp_skip = value; return GSR_OK;
    case GSR_OPT_BWD_LAST_CONTRIB: ctx->opt_last_contrib = value; return GSR_OK;
    case GSR_OPT_WARP_CULL: ctx->opt_warp_cull = value; return GSR_OK;
    case GSR_OPT_PDL: ctx->opt_pdl = value; return GSR_OK;
    case GSR_OPT_FAIL_NEXT_ALLOC: ctx->fail_next_alloc = value; return GSR_OK;
    case GSR_OPT_DETERMINISTIC: ctx->opt_deterministic = value; return GSR_OK;
    case GSR_OPT_BWD_PER_SPLAT: ctx->opt_bwd_per_splat = value; return GSR_OK;
    case GSR_OPT_SPLIT: ctx->opt_split = value; return GSR_OK;
    case GSR_OPT_SPLIT_FORWARD: ctx->opt_split_forward = value; return GSR_OK;
    default: return fail(ctx, GSR_ERR_INVALID_ARG, "unknown option " + std::to_string(option));
    }
}

uint64_t gsr_launch_count(const gsr_ctx *ctx) { return ctx ? ctx->launches : 0; }

int gsr_bin_splats(gsr_ctx *ctx, const gsr_splat2d *splats, const float *depths, int32_t n,
                   int32_t width, int32_t height, void *stream, gsr_bins *out)
{
    gsr::Range range("gsr_bin_splats");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (!out) return fail(ctx, GSR_ERR_INVALID_ARG, "out is NULL");
    if (n < 0 || n > GSR_MAX_SPLATS) return fail(ctx, GSR_ERR_INVALID_ARG, "n out of range");
    if (width < 1 || height < 1 || width > GSR_MAX_IMAGE_SIDE || height > GSR_MAX_IMAGE_SIDE)
        return fail(ctx, GSR_ERR_INVALID_ARG, "width/height out of range");
    if (n > 0 && (!splats || !depths)) return fail(ctx, GSR_ERR_INVALID_ARG, "splats/depths is NULL");
    if (!aligned(splats, 4) || !aligned(depths, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "splats/depths must be 4-byte aligned");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    return gsr::bin_splats(ctx, reinterpret_cast<const float *>(splats), depths, n, width, height,
                           (cudaStream_t)stream, out);
}

int gsr_rasterize_forward(gsr_ctx *ctx, const gsr_splat2d *splats, int32_t n, const gsr_bins *bins,
                          float *out_rgbw, float *final_T, uint32_t *last_contrib, void *stream)
{
    gsr::Range range("gsr_rasterize_forward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    int rc = check_bins(ctx, bins, n);
    if (rc) return rc;
    if (!out_rgbw || !final_T || !last_contrib)
        return fail(ctx, GSR_ERR_INVALID_ARG, "an output pointer is NULL");
    if (n > 0 && bins->num_pairs > 0 && !splats) return fail(ctx, GSR_ERR_INVALID_ARG, "splats is NULL");
    if (!aligned(out_rgbw, 16) || !aligned(final_T, 4) || !aligned(last_contrib, 4) ||
        !aligned(splats, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "misaligned buffer (out_rgbw needs 16 bytes)");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    return gsr::rasterize_forward(ctx, reinterpret_cast<const float *>(splats), bins, out_rgbw, final_T,
                                  last_contrib, (cudaStream_t)stream);
}

int gsr_rasterize_backward(gsr_ctx *ctx, const gsr_splat2d *splats, int32_t n, const gsr_bins *bins,
                           const float *dl_dout, const float *final_T, const uint32_t *last_contrib,
                           float *grad, void *stream)
{
    gsr::Range range("gsr_rasterize_backward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    int rc = check_bins(ctx, bins, n);
    if (rc) return rc;
    if (!dl_dout || !final_T || !last_contrib || (n > 0 && !grad))
        return fail(ctx, GSR_ERR_INVALID_ARG, "an input/output pointer is NULL");
    if (n > 0 && bins->num_pairs > 0 && !splats) return fail(ctx, GSR_ERR_INVALID_ARG, "splats is NULL");
    if (!aligned(dl_dout, 16) || !aligned(final_T, 4) || !aligned(last_contrib, 4) ||
        !aligned(grad, 4) || !aligned(splats, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "misaligned buffer (dl_dout needs 16 bytes)");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (n == 0) return GSR_OK;
    return gsr::rasterize_backward(ctx, reinterpret_cast<const float *>(splats), n, bins, dl_dout,
                                   final_T, last_contrib, grad, (cudaStream_t)stream);
}

int gsr_rasterize_backward_noalloc(gsr_ctx *ctx, const gsr_splat2d *splats, int32_t n,
                                   const gsr_bins *bins, const float *dl_dout, const float *final_T,
                                   const uint32_t *last_contrib, float *grad, void *stream)
{
    gsr::Range range("gsr_rasterize_backward_noalloc");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (n < 0 || n > GSR_NOALLOC_MAX_SPLATS)
        return fail(ctx, GSR_ERR_INVALID_ARG,
                    "n = " + std::to_string(n) + " is outside [0, GSR_NOALLOC_MAX_SPLATS = " +
                        std::to_string(GSR_NOALLOC_MAX_SPLATS) + "]");
    int rc = check_bins(ctx, bins, n);
    if (rc) return rc;
    if (!dl_dout || !final_T || !last_contrib || (n > 0 && !grad))
        return fail(ctx, GSR_ERR_INVALID_ARG, "an input/output pointer is NULL");
    if (n > 0 && bins->num_pairs > 0 && !splats) return fail(ctx, GSR_ERR_INVALID_ARG, "splats is NULL");
    if (!aligned(dl_dout, 16) || !aligned(final_T, 4) || !aligned(last_contrib, 4) ||
        !aligned(grad, 4) || !aligned(splats, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "misaligned buffer (dl_dout needs 16 bytes)");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (n == 0) return GSR_OK;
    return gsr::rasterize_backward_noalloc(ctx, reinterpret_cast<const float *>(splats), n, bins,
                                           dl_dout, final_T, last_contrib, grad,
                                           (cudaStream_t)stream);
}

int gsr_get_bin_stats(gsr_ctx *ctx, gsr_bin_stats *out)
{
    if (!ctx || !out) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    DeviceGuard g(ctx->device);
    *out = gsr_bin_stats{};
    out->capacity = ctx->cap_pairs;
    uint32_t status = GSR_OK;
    int rc = gsr::bin_result(ctx, &out->num_pairs, &status, &out->emitting);
    if (rc) return rc;
    int tile_bits = 0, tile_digits = 0;
    rc = gsr::bin_pass_masks(ctx, &out->depth_pass_mask, &out->tile_pass_mask, &tile_bits, &tile_digits);
    if (rc) return rc;
    out->tile_digit_bits = tile_bits;
    out->tile_digits = tile_digits;
    out->radix_passes = __builtin_popcount(out->depth_pass_mask) + __builtin_popcount(out->tile_pass_mask);
    return GSR_OK;
}

int gsr_reserve_pairs(gsr_ctx *ctx, uint64_t max_pairs)
{
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (max_pairs > (uint64_t)GSR_MAX_PAIRS)
        return fail(ctx, GSR_ERR_INVALID_ARG, "max_pairs exceeds GSR_MAX_PAIRS");
    ctx->reserved_pairs = max_pairs;
    return GSR_OK;
}

int gsr_num_pairs(gsr_ctx *ctx, uint32_t *out)
{
    if (!ctx || !out) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    uint32_t status = GSR_OK;
    int rc = gsr::bin_result(ctx, out, &status, nullptr);
    if (rc) return rc;
    if (status != GSR_OK)
        return fail(ctx, GSR_ERR_TOO_MANY_PAIRS,
                    "the last binning needed " + std::to_string(*out) + " tile pairs, more than the arena's " +
                        std::to_string(ctx->cap_pairs) + ": its bins are empty");
    return GSR_OK;
}

int gsr_exp_neg(gsr_ctx *ctx, const float *s, float *out, int32_t n, void *stream)
{
    gsr::Range range("gsr_exp_neg");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (n < 0) return fail(ctx, GSR_ERR_INVALID_ARG, "n < 0");
    if (n > 0 && (!s || !out)) return fail(ctx, GSR_ERR_INVALID_ARG, "s/out is NULL");
    if (!aligned(s, 4) || !aligned(out, 4)) return fail(ctx, GSR_ERR_INVALID_ARG, "s/out must be 4-byte aligned");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (n == 0) return GSR_OK;
    return gsr::exp_neg_eval(ctx, s, out, n, (cudaStream_t)stream);
}

int gsr_peak_kernel(gsr_ctx *ctx, int kind, int32_t iters, float *sink, uint64_t *lane_ops, void *stream)
{
    gsr::Range range("gsr_peak_kernel");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (kind != GSR_PEAK_FFMA && kind != GSR_PEAK_EX2) return fail(ctx, GSR_ERR_INVALID_ARG, "unknown peak kind");
    if (iters < 1 || iters > (1 << 24)) return fail(ctx, GSR_ERR_INVALID_ARG, "iters outside [1, 2^24]");
    if (!sink || !lane_ops) return fail(ctx, GSR_ERR_INVALID_ARG, "sink/lane_ops is NULL");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    return gsr::peak_kernel(ctx, kind, iters, sink, lane_ops, (cudaStream_t)stream);
}

}  // extern "C"

namespace {

int check_projection(gsr_ctx *ctx, const void *gauss, int32_t n, const gsr_camera *cam, const void *a,
                     const void *b)
{
    if (!cam) return fail(ctx, GSR_ERR_INVALID_ARG, "camera is NULL");
    if (n < 0 || n > GSR_MAX_SPLATS) return fail(ctx, GSR_ERR_INVALID_ARG, "n out of range");
    if (n > 0 && (!gauss || !a || !b)) return fail(ctx, GSR_ERR_INVALID_ARG, "an array is NULL");
    if (!aligned(gauss, 4) || !aligned(a, 4) || !aligned(b, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "arrays must be 4-byte aligned");
    const float *f = reinterpret_cast<const float *>(cam);
    for (size_t k = 0; k < sizeof(gsr_camera) / sizeof(float); ++k)
        if (!std::isfinite(f[k])) return fail(ctx, GSR_ERR_INVALID_ARG, "camera field not finite");
    if (!(cam->z_near > 0.0f)) return fail(ctx, GSR_ERR_INVALID_ARG, "camera z_near must be > 0");
    if (!(cam->eps >= 0.0f)) return fail(ctx, GSR_ERR_INVALID_ARG, "camera eps must be >= 0");
    return GSR_OK;
}

}  // namespace

extern "C" {

int gsr_project_forward(gsr_ctx *ctx, const gsr_gaussian3d *gauss, int32_t n, const gsr_camera *camera,
                        gsr_splat2d *splats, float *depths, void *stream)
{
    gsr::Range range("gsr_project_forward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_projection(ctx, gauss, n, camera, splats, depths)) return rc;
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (n == 0) return GSR_OK;
    return gsr::project_forward(ctx, reinterpret_cast<const float *>(gauss), n, *camera,
                                reinterpret_cast<float *>(splats), depths, (cudaStream_t)stream);
}

int gsr_project_backward(gsr_ctx *ctx, const gsr_gaussian3d *gauss, int32_t n, const gsr_camera *camera,
                         const float *dl_dsplat, float *dl_dgauss, void *stream)
{
    gsr::Range range("gsr_project_backward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_projection(ctx, gauss, n, camera, dl_dsplat, dl_dgauss)) return rc;
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (n == 0) return GSR_OK;
    return gsr::project_backward(ctx, reinterpret_cast<const float *>(gauss), n, *camera, dl_dsplat, dl_dgauss,
                                 (cudaStream_t)stream);
}

}  // extern "C"

namespace {

size_t element_size(int dtype) { return dtype == GSR_F32 ? 4 : 2; }

bool known_dtype(int dtype) { return dtype == GSR_F32 || dtype == GSR_BF16 || dtype == GSR_F16; }

int check_group_norm(gsr_ctx *ctx, const gsr_group_norm *d, const void *x, const float *weight, const float *bias,
                     const void *y, const float *mean, const float *rstd)
{
    if (!d) return fail(ctx, GSR_ERR_INVALID_ARG, "desc is NULL");
    if (!known_dtype(d->dtype)) return fail(ctx, GSR_ERR_INVALID_ARG, "unknown dtype");
    if (d->activation != GSR_ACT_NONE && d->activation != GSR_ACT_SILU && d->activation != GSR_ACT_GELU)
        return fail(ctx, GSR_ERR_INVALID_ARG, "unknown activation");
    if (d->samples < 0 || d->positions < 0) return fail(ctx, GSR_ERR_INVALID_ARG, "a size is negative");
    if (d->channels < 1 || d->channels > GSR_MAX_CHANNELS)
        return fail(ctx, GSR_ERR_INVALID_ARG, "channels outside [1, GSR_MAX_CHANNELS]");
    if (d->groups < 1 || d->channels % d->groups != 0)
        return fail(ctx, GSR_ERR_INVALID_ARG, "groups must divide channels");
    if (d->positions > ((int64_t)1 << 40) / d->channels || d->samples > (1 << 20))
        return fail(ctx, GSR_ERR_INVALID_ARG, "samples or positions too large");
    if (!std::isfinite(d->eps) || !(d->eps > 0.0f))
        return fail(ctx, GSR_ERR_INVALID_ARG, "eps must be finite and > 0");
    if (d->samples == 0 || d->positions == 0) return GSR_OK;
    if (!x || !y || !mean || !rstd) return fail(ctx, GSR_ERR_INVALID_ARG, "an array is NULL");
    const size_t size = element_size(d->dtype);
    if (!aligned(x, size) || !aligned(y, size) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "an array is not aligned to its element");
    return GSR_OK;
}

// Sizes and strides of one [batch, tokens, heads, head_dim] array.
int check_heads(gsr_ctx *ctx, const gsr_heads *t, const char *name, int64_t batch, int64_t tokens, int64_t heads,
                size_t align, int64_t stride_unit, bool output)
{
    const std::string who(name);
    if (!t) return fail(ctx, GSR_ERR_INVALID_ARG, who + " is NULL");
    if (batch == 0 || tokens == 0 || heads == 0) return GSR_OK;
    if (!t->data) return fail(ctx, GSR_ERR_INVALID_ARG, who + ".data is NULL");
    if (!aligned(t->data, align))
        return fail(ctx, GSR_ERR_INVALID_ARG, who + " must be " + std::to_string(align) + "-byte aligned");
    const struct { int64_t extent, stride; const char *what; bool shared; } dims[3] = {
        {batch, t->batch_stride, "batch", true}, {tokens, t->token_stride, "token", false},
        {heads, t->head_stride, "head", true}};
    for (const auto &dim : dims) {
        if (dim.extent <= 1) continue;
        if (dim.stride < 0 || dim.stride > ((int64_t)1 << 38) || dim.stride % stride_unit != 0)
            return fail(ctx, GSR_ERR_INVALID_ARG, who + ": the " + dim.what + " stride must be a multiple of " +
                                                      std::to_string(stride_unit) + " in [0, 2^38]");
        if (dim.stride == 0 && (output || !dim.shared))
            return fail(ctx, GSR_ERR_INVALID_ARG, who + ": the " + dim.what + " stride must not be 0");
    }
    return GSR_OK;
}

int check_rotary(gsr_ctx *ctx, const gsr_rotary *d, const gsr_heads *x, const void *positions,
                 const float *frequencies, const gsr_heads *out)
{
    if (!d) return fail(ctx, GSR_ERR_INVALID_ARG, "desc is NULL");
    if (!known_dtype(d->dtype)) return fail(ctx, GSR_ERR_INVALID_ARG, "unknown dtype");
    if (d->batch < 0 || d->tokens < 0) return fail(ctx, GSR_ERR_INVALID_ARG, "a size is negative");
    if ((int64_t)d->batch * d->tokens > GSR_MAX_TOKENS)
        return fail(ctx, GSR_ERR_INVALID_ARG, "batch * tokens above GSR_MAX_TOKENS");
    if (d->heads < 1 || d->heads > GSR_MAX_HEADS)
        return fail(ctx, GSR_ERR_INVALID_ARG, "heads outside [1, GSR_MAX_HEADS]");
    if (d->head_dim < 1 || d->head_dim > GSR_MAX_HEAD_DIM)
        return fail(ctx, GSR_ERR_INVALID_ARG, "head_dim outside [1, GSR_MAX_HEAD_DIM]");
    if (d->axes < 1 || d->axes > GSR_MAX_AXES) return fail(ctx, GSR_ERR_INVALID_ARG, "axes outside [1, GSR_MAX_AXES]");
    int64_t pairs = 0;
    for (int a = 0; a < d->axes; ++a) {
        if (d->sections[a] < 0) return fail(ctx, GSR_ERR_INVALID_ARG, "a section is negative");
        pairs += d->sections[a];
    }
    if (2 * pairs > d->head_dim) return fail(ctx, GSR_ERR_INVALID_ARG, "the sections hold more pairs than head_dim");
    if (d->positions_batch_stride < 0 || d->positions_batch_stride > ((int64_t)1 << 38))
        return fail(ctx, GSR_ERR_INVALID_ARG, "positions_batch_stride outside [0, 2^38]");
    const size_t size = element_size(d->dtype);
    if (int rc = check_heads(ctx, x, "x", d->batch, d->tokens, d->heads, size, 1, false)) return rc;
    if (int rc = check_heads(ctx, out, "out", d->batch, d->tokens, d->heads, size, 1, true)) return rc;
    if (d->batch > 0 && d->tokens > 0 && pairs > 0) {
        if (!positions || !frequencies) return fail(ctx, GSR_ERR_INVALID_ARG, "positions or frequencies is NULL");
        if (!aligned(positions, 4) || !aligned(frequencies, 4))
            return fail(ctx, GSR_ERR_INVALID_ARG, "positions and frequencies must be 4-byte aligned");
    }
    return GSR_OK;
}

int check_attention(gsr_ctx *ctx, const gsr_attention *d)
{
    if (!d) return fail(ctx, GSR_ERR_INVALID_ARG, "desc is NULL");
    if (d->dtype != GSR_BF16 && d->dtype != GSR_F16)
        return fail(ctx, GSR_ERR_INVALID_ARG, "attention takes GSR_BF16 or GSR_F16");
    if (d->batch < 0 || d->q_len < 0 || d->kv_len < 0) return fail(ctx, GSR_ERR_INVALID_ARG, "a size is negative");
    if (d->kv_heads < 1 || d->q_heads < 1 || d->q_heads > GSR_MAX_HEADS || d->q_heads % d->kv_heads != 0)
        return fail(ctx, GSR_ERR_INVALID_ARG, "q_heads must be a multiple of kv_heads, in [1, GSR_MAX_HEADS]");
    if (d->head_dim < 8 || d->head_dim > GSR_ATTENTION_MAX_HEAD_DIM || d->head_dim % 8 != 0)
        return fail(ctx, GSR_ERR_INVALID_ARG,
                    "head_dim must be a multiple of 8 in [8, GSR_ATTENTION_MAX_HEAD_DIM]");
    if (!std::isfinite(d->scale) || !(d->scale > 0.0f))
        return fail(ctx, GSR_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (d->batch > (1 << 16) || d->q_len > (1 << 24) || d->kv_len > (1 << 24))
        return fail(ctx, GSR_ERR_INVALID_ARG, "batch above 2^16 or a length above 2^24");
    constexpr int64_t kMost = 0x7fffffff;
    if ((int64_t)d->batch * d->q_len > kMost / d->q_heads || (int64_t)d->batch * d->kv_len > kMost / d->kv_heads)
        return fail(ctx, GSR_ERR_INVALID_ARG, "batch * heads * length above 2^31 - 1");
    // Steps of 128 x 128 scores, the unit in which the kernels divide their work.
    const int64_t row_tiles = (int64_t)d->batch * d->q_heads * (((int64_t)d->q_len + 127) / 128);
    if (((int64_t)d->kv_len + 127) / 128 > kMost / (row_tiles > 1 ? row_tiles : 1))
        return fail(ctx, GSR_ERR_INVALID_ARG, "2^31 steps of 128 x 128 scores or more");
    if (!aligned(d->kv_lengths, 4)) return fail(ctx, GSR_ERR_INVALID_ARG, "kv_lengths must be 4-byte aligned");
    return GSR_OK;
}

int check_query(gsr_ctx *ctx, const gsr_attention *d, const gsr_heads *t, const char *name, bool output)
{
    return check_heads(ctx, t, name, d->batch, d->q_len, d->q_heads, 16, 8, output);
}

int check_key(gsr_ctx *ctx, const gsr_attention *d, const gsr_heads *t, const char *name, bool output)
{
    return check_heads(ctx, t, name, d->batch, d->kv_len, d->kv_heads, 16, 8, output);
}

}  // namespace

extern "C" {

int gsr_synchronize(gsr_ctx *ctx, void *stream)
{
    gsr::Range range("gsr_synchronize");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = cuda_check(ctx, cudaStreamSynchronize((cudaStream_t)stream), "gsr_synchronize")) return rc;
    return gsr::check_status(ctx);
}

int gsr_group_norm_forward(gsr_ctx *ctx, const gsr_group_norm *desc, const void *x, const float *weight,
                           const float *bias, void *out, float *mean, float *rstd, void *stream)
{
    gsr::Range range("gsr_group_norm_forward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_group_norm(ctx, desc, x, weight, bias, out, mean, rstd)) return rc;
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = gsr::check_status(ctx)) return rc;
    if (desc->samples == 0 || desc->positions == 0) return GSR_OK;
    return gsr::group_norm_forward(ctx, *desc, x, weight, bias, out, mean, rstd, (cudaStream_t)stream);
}

int gsr_group_norm_backward(gsr_ctx *ctx, const gsr_group_norm *desc, const void *dl_dout, const void *x,
                            const float *weight, const float *bias, const float *mean, const float *rstd,
                            void *dl_dx, float *dl_dweight, float *dl_dbias, void *stream)
{
    gsr::Range range("gsr_group_norm_backward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_group_norm(ctx, desc, x, weight, bias, dl_dx, mean, rstd)) return rc;
    if (desc->samples > 0 && desc->positions > 0 && !dl_dout)
        return fail(ctx, GSR_ERR_INVALID_ARG, "dl_dout is NULL");
    if (!aligned(dl_dout, element_size(desc->dtype)) || !aligned(dl_dweight, 4) || !aligned(dl_dbias, 4))
        return fail(ctx, GSR_ERR_INVALID_ARG, "an array is not aligned to its element");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = gsr::check_status(ctx)) return rc;
    return gsr::group_norm_backward(ctx, *desc, dl_dout, x, weight, bias, mean, rstd, dl_dx, dl_dweight, dl_dbias,
                                    (cudaStream_t)stream);
}

int gsr_rotary_forward(gsr_ctx *ctx, const gsr_rotary *desc, const gsr_heads *x, const void *positions,
                       const float *frequencies, const gsr_heads *out, void *stream)
{
    gsr::Range range("gsr_rotary_forward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_rotary(ctx, desc, x, positions, frequencies, out)) return rc;
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = gsr::check_status(ctx)) return rc;
    if (desc->batch == 0 || desc->tokens == 0) return GSR_OK;
    return gsr::rotary(ctx, *desc, *x, positions, frequencies, *out, 1.0f, (cudaStream_t)stream);
}

int gsr_rotary_backward(gsr_ctx *ctx, const gsr_rotary *desc, const gsr_heads *dl_dout, const void *positions,
                        const float *frequencies, const gsr_heads *dl_dx, void *stream)
{
    gsr::Range range("gsr_rotary_backward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_rotary(ctx, desc, dl_dout, positions, frequencies, dl_dx)) return rc;
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = gsr::check_status(ctx)) return rc;
    if (desc->batch == 0 || desc->tokens == 0) return GSR_OK;
    return gsr::rotary(ctx, *desc, *dl_dout, positions, frequencies, *dl_dx, -1.0f, (cudaStream_t)stream);
}

int gsr_cross_attention_forward(gsr_ctx *ctx, const gsr_attention *desc, const gsr_heads *q, const gsr_heads *k,
                                const gsr_heads *v, const gsr_heads *out, float *lse, void *stream)
{
    gsr::Range range("gsr_cross_attention_forward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_attention(ctx, desc)) return rc;
    if (int rc = check_query(ctx, desc, q, "q", false)) return rc;
    if (int rc = check_key(ctx, desc, k, "k", false)) return rc;
    if (int rc = check_key(ctx, desc, v, "v", false)) return rc;
    if (int rc = check_query(ctx, desc, out, "out", true)) return rc;
    if (desc->batch == 0 || desc->q_len == 0) return GSR_OK;
    if (!lse || !aligned(lse, 4)) return fail(ctx, GSR_ERR_INVALID_ARG, "lse is NULL or misaligned");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = gsr::check_status(ctx)) return rc;
    return gsr::cross_attention_forward(ctx, *desc, *q, *k, *v, *out, lse, (cudaStream_t)stream);
}

int gsr_cross_attention_backward(gsr_ctx *ctx, const gsr_attention *desc, const gsr_heads *q, const gsr_heads *k,
                                 const gsr_heads *v, const gsr_heads *out, const float *lse,
                                 const gsr_heads *dl_dout, const gsr_heads *dl_dq, const gsr_heads *dl_dk,
                                 const gsr_heads *dl_dv, void *stream)
{
    gsr::Range range("gsr_cross_attention_backward");
    if (!ctx) return GSR_ERR_INVALID_ARG;
    ctx->err.clear();
    if (int rc = check_attention(ctx, desc)) return rc;
    if (int rc = check_query(ctx, desc, q, "q", false)) return rc;
    if (int rc = check_key(ctx, desc, k, "k", false)) return rc;
    if (int rc = check_key(ctx, desc, v, "v", false)) return rc;
    if (int rc = check_query(ctx, desc, out, "out", false)) return rc;
    if (int rc = check_query(ctx, desc, dl_dout, "dl_dout", false)) return rc;
    if (int rc = check_query(ctx, desc, dl_dq, "dl_dq", true)) return rc;
    if (int rc = check_key(ctx, desc, dl_dk, "dl_dk", true)) return rc;
    if (int rc = check_key(ctx, desc, dl_dv, "dl_dv", true)) return rc;
    if (desc->batch == 0 || (desc->q_len == 0 && desc->kv_len == 0)) return GSR_OK;
    if (desc->q_len > 0 && (!lse || !aligned(lse, 4)))
        return fail(ctx, GSR_ERR_INVALID_ARG, "lse is NULL or misaligned");
    DeviceGuard g(ctx->device);
    if (!g.ok) return fail(ctx, GSR_ERR_CUDA, "cannot select the context's device");
    if (int rc = gsr::check_status(ctx)) return rc;
    return gsr::cross_attention_backward(ctx, *desc, *q, *k, *v, *out, lse, *dl_dout, *dl_dq, *dl_dk, *dl_dv,
                                         (cudaStream_t)stream);
}

}  // extern "C"

static_assert(sizeof(gsr_splat2d) == 36, "Splat2D is 9 floats");
static_assert(sizeof(gsr_gaussian3d) == GSR_GAUSSIAN_FLOATS * 4, "a Gaussian is 14 floats");
static_assert(sizeof(gsr_camera) == 18 * 4, "a camera is 18 floats");
