// decoder.cu -- the workspace of the decoder's operators: scratch memory that
// one call at a time uses, grown like the rest of the context's arena.
#include <new>

#include "decoder.cuh"

namespace gsr {
namespace {

CaptureMark *find_capture(const gsr_ctx *ctx, unsigned long long id)
{
    CaptureMark *mark = ctx->captures;
    while (mark && mark->id != id) mark = mark->next;
    return mark;
}

}  // namespace

int Workspace::take(size_t bytes, void **out)
{
    gsr_ctx *ctx = ctx_;
    const cudaStream_t stream = stream_;
    *out = nullptr;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (int rc = cuda_check(ctx, cudaStreamGetCaptureInfo(stream, &capture, &id), "workspace stream")) return rc;
    if (bytes > ctx->cap_work) {
        if (capture != cudaStreamCaptureStatusNone)
            return fail(ctx, GSR_ERR_CUDA, "the workspace must grow during a capture: make one such call before it");
        // Queued work of an earlier call may still use the old buffer, and the replays
        // of a graph that captured a call will, as long as the graph lives.
        if (int rc = cuda_check(ctx, cudaDeviceSynchronize(), "workspace growth")) return rc;
        if (ctx->work_captured) {
            Outgrown *kept = new (std::nothrow) Outgrown{ctx->work, ctx->outgrown};
            if (!kept) return fail(ctx, GSR_ERR_OOM, "cannot keep the workspace that captured graphs hold");
            ctx->outgrown = kept;
        } else {
            cudaFree(ctx->work);
        }
        ctx->work = nullptr;
        ctx->work_captured = false;
        ctx->cap_work = 0;
        const size_t grown = round_up(bytes, (size_t)1 << 20);
        void *p = nullptr;
        if (device_alloc(ctx, &p, grown) != cudaSuccess) {
            cudaGetLastError();
            return fail(ctx, GSR_ERR_OOM, "cannot grow the workspace to " + std::to_string(grown) + " bytes");
        }
        ctx->work = (unsigned char *)p;
        ctx->cap_work = grown;
        ctx->work_pending = false;
    }
    if (!ctx->status_host) {
        if (capture != cudaStreamCaptureStatusNone)
            return fail(ctx, GSR_ERR_CUDA, "the workspace must be made before a capture: make one such call before it");
        void *host = nullptr, *dev = nullptr;
        if (int rc = cuda_check(ctx, cudaHostAlloc(&host, sizeof(uint32_t), cudaHostAllocMapped), "status word"))
            return rc;
        *(uint32_t *)host = 0;
        if (int rc = cuda_check(ctx, cudaHostGetDevicePointer(&dev, host, 0), "status word")) {
            cudaFreeHost(host);
            return rc;
        }
        ctx->status_host = (uint32_t *)host;
        ctx->status_dev = (uint32_t *)dev;
    }
    *out = ctx->work;
    if (bytes == 0) return GSR_OK;
    // A captured call is ordered with the others of its capture (on the same stream
    // too: a stream that is being captured cannot be asked for its number); the events
    // of live streams and of other captures stay out of it.
    if (capture != cudaStreamCaptureStatusNone) {
        ctx->work_captured = true;
        const CaptureMark *mark = find_capture(ctx, id);
        if (mark && mark->event)
            if (int rc = cuda_check(ctx, cudaStreamWaitEvent(stream, mark->event, 0), "workspace order")) return rc;
    } else if (ctx->work_pending) {
        unsigned long long number = 0;
        if (int rc = cuda_check(ctx, cudaStreamGetId(stream, &number), "workspace stream")) return rc;
        if (ctx->work_stream != number)
            if (int rc = cuda_check(ctx, cudaStreamWaitEvent(stream, ctx->work_event, 0), "workspace order")) return rc;
    }
    used_ = true;
    return GSR_OK;
}

int Workspace::done()
{
    if (!used_) return GSR_OK;
    used_ = false;
    return mark();
}

Workspace::~Workspace()
{
    if (!used_) return;
    std::string reason;            // of the failure, which an error of the mark's must not replace
    reason.swap(ctx_->err);
    mark();
    reason.swap(ctx_->err);
}

int Workspace::mark()
{
    gsr_ctx *ctx = ctx_;
    const cudaStream_t stream = stream_;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (int rc = cuda_check(ctx, cudaStreamGetCaptureInfo(stream, &capture, &id), "workspace stream")) return rc;
    cudaEvent_t *event = &ctx->work_event;
    if (capture != cudaStreamCaptureStatusNone) {
        CaptureMark *mark = find_capture(ctx, id);
        if (!mark) {
            mark = new (std::nothrow) CaptureMark{id, nullptr, ctx->captures};
            if (!mark) return fail(ctx, GSR_ERR_OOM, "cannot note the capture's use of the workspace");
            ctx->captures = mark;
        }
        event = &mark->event;
    }
    if (!*event)
        if (int rc = cuda_check(ctx, cudaEventCreateWithFlags(event, cudaEventDisableTiming), "workspace event"))
            return rc;
    if (int rc = cuda_check(ctx, cudaEventRecord(*event, stream), "workspace event")) return rc;
    if (capture == cudaStreamCaptureStatusNone) {
        ctx->work_pending = true;
        ctx->work_stream = ~0ull;   // no stream's: the next call waits, should the number not be had
        return cuda_check(ctx, cudaStreamGetId(stream, &ctx->work_stream), "workspace stream");
    }
    return GSR_OK;
}

int check_status(gsr_ctx *ctx)
{
    if (!ctx->status_host || *(volatile uint32_t *)ctx->status_host == 0) return GSR_OK;
    *(volatile uint32_t *)ctx->status_host = 0;
    return fail(ctx, GSR_ERR_CUDA, "a kernel of an earlier call gave up waiting for its own copies or products: "
                                   "that call's results are not valid");
}

}  // namespace gsr
