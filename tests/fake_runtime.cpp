// A CUDA runtime that runs nothing: the library's objects linked against it show
// on the CPU what their host code asks of streams, events and memory.
//
// Streams and events carry the launches that are ordered before them (a clock per
// stream).  Every launch counts as a use of the newest device allocation, which in
// a context that has only called the decoder's operators is their workspace.  Two
// uses of one allocation, outside captures or in the same one, that no stream or
// event orders are a conflict, and so is an allocation freed while a captured
// launch holds its address.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdlib>
#include <map>
#include <set>
#include <vector>

namespace {

using Clock = std::map<int, int>;

struct Stream {
    int uid;
    unsigned long long capture = 0;
    Clock seen;
};

struct Event {
    Clock seen;
    unsigned long long capture = 0;
};

struct Use {
    uintptr_t buffer;
    int uid, at;
    unsigned long long capture;
};

std::map<void *, Stream> streams;
std::set<unsigned long long> captures;   // under way
std::vector<uintptr_t> allocations;      // live, oldest first
std::vector<Use> uses;
std::set<uintptr_t> held;                // by captured launches
void *status = nullptr;
int next_uid, next_address, host_allocations, events, conflicts, freed_while_held, pulled_in, launches;
unsigned long long next_capture;
int launch_to_fail, map_to_fail, number_to_fail;

Stream &at(void *handle)
{
    auto found = streams.find(handle);
    if (found == streams.end()) found = streams.emplace(handle, Stream{++next_uid}).first;
    return found->second;
}

void merge(Clock &to, const Clock &from)
{
    for (const auto &s : from)
        if (to[s.first] < s.second) to[s.first] = s.second;
}

cudaError_t work(void *stream)
{
    ++launches;
    if (launch_to_fail > 0 && --launch_to_fail == 0) return cudaErrorLaunchOutOfResources;
    Stream &s = at(stream);
    if (allocations.empty()) return cudaSuccess;
    const uintptr_t buffer = allocations.back();
    for (const Use &u : uses)
        if (u.buffer == buffer && u.capture == s.capture && u.at > s.seen[u.uid]) ++conflicts;
    uses.push_back({buffer, s.uid, ++s.seen[s.uid], s.capture});
    if (s.capture) held.insert(buffer);
    return cudaSuccess;
}

cudaError_t wait(Stream &s, const Event &e, bool asked)
{
    if (e.capture && !captures.count(e.capture)) return cudaErrorCapturedEvent;
    if (e.capture != s.capture) {
        if (s.capture) return e.capture ? cudaErrorStreamCaptureMerge : cudaErrorStreamCaptureIsolation;
        s.capture = e.capture;   // the stream joins the capture
        if (!asked) ++pulled_in;
    }
    merge(s.seen, e.seen);
    return cudaSuccess;
}

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    return map_to_fail > 0 && --map_to_fail == 0 ? CUDA_ERROR_INVALID_VALUE : CUDA_SUCCESS;
}

}  // namespace

extern "C" {

// ---- what a test asks ------------------------------------------------------------

void fake_reset()
{
    streams.clear();
    captures.clear();
    allocations.clear();
    uses.clear();
    held.clear();
    host_allocations = events = 0;
    conflicts = freed_while_held = pulled_in = launches = launch_to_fail = map_to_fail = number_to_fail = 0;
}
int fake_conflicts() { return conflicts; }
int fake_freed_while_held() { return freed_while_held; }
int fake_pulled_in() { return pulled_in; }
int fake_launches() { return launches; }
int fake_live() { return (int)allocations.size() + host_allocations + events; }
int fake_allocations() { return (int)allocations.size(); }
void fake_fail_launch(int n) { launch_to_fail = n; }
void fake_fail_map(int n) { map_to_fail = n; }
void fake_fail_number(int n) { number_to_fail = n; }
void fake_set_status() { *(uint32_t *)status = 1; }
// Another stream under a handle whose stream was destroyed.
void fake_new_stream(void *handle) { streams.erase(handle); }
void fake_begin_capture(void *handle)
{
    at(handle).capture = ++next_capture;
    captures.insert(next_capture);
}
void fake_end_capture(void *handle)
{
    const unsigned long long id = at(handle).capture;
    captures.erase(id);
    for (auto &s : streams)
        if (s.second.capture == id) s.second.capture = 0;
}
// The caller's own edge between two streams: an event recorded on one, waited for by the other.
int fake_edge(void *from, void *to)
{
    const Stream &s = at(from);
    return wait(at(to), Event{s.seen, s.capture}, true);
}

// ---- the runtime -------------------------------------------------------------------

cudaError_t cudaGetDeviceCount(int *n) { return *n = 1, cudaSuccess; }
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "an error of the fake runtime"; }

cudaError_t cudaDeviceSynchronize()
{
    Clock all;
    for (auto &s : streams)
        if (!s.second.capture) merge(all, s.second.seen);
    std::vector<Use> left;
    for (const Use &u : uses)
        if (u.capture) left.push_back(u);
    uses.swap(left);
    for (auto &s : streams)
        if (!s.second.capture) merge(s.second.seen, all);
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }

cudaError_t cudaMalloc(void **p, size_t)
{
    allocations.push_back(((uintptr_t)++next_address) << 40);
    *p = (void *)allocations.back();
    return cudaSuccess;
}
cudaError_t cudaFree(void *p)
{
    for (size_t i = 0; i < allocations.size(); ++i)
        if (allocations[i] == (uintptr_t)p) {
            if (held.count((uintptr_t)p)) ++freed_while_held;
            allocations.erase(allocations.begin() + i);
            break;
        }
    return cudaSuccess;
}
cudaError_t cudaHostAlloc(void **p, size_t bytes, unsigned)
{
    ++host_allocations;
    status = *p = std::calloc(1, bytes);
    return cudaSuccess;
}
cudaError_t cudaHostGetDevicePointer(void **p, void *host, unsigned) { return *p = host, cudaSuccess; }
cudaError_t cudaFreeHost(void *p)
{
    --host_allocations;
    std::free(p);
    return cudaSuccess;
}

cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus *to)
{
    *to = at(s).capture ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t s, cudaStreamCaptureStatus *to, unsigned long long *id,
                                     cudaGraph_t *, const cudaGraphNode_t **, const cudaGraphEdgeData **, size_t *)
{
    *id = at(s).capture;
    return cudaStreamIsCapturing(s, to);
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long *id)
{
    if (at(s).capture) return cudaErrorStreamCaptureUnsupported;
    if (number_to_fail > 0 && --number_to_fail == 0) return cudaErrorUnknown;
    *id = at(s).uid;
    return cudaSuccess;
}

cudaError_t cudaEventCreateWithFlags(cudaEvent_t *e, unsigned)
{
    ++events;
    *e = (cudaEvent_t) new Event;
    return cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t e)
{
    --events;
    delete (Event *)e;
    return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s)
{
    *(Event *)e = {at(s).seen, at(s).capture};
    return cudaSuccess;
}
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned) { return wait(at(s), *(Event *)e, false); }

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **) { return work(c->stream); }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t s) { return work(s); }
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t s) { return work(s); }
cudaError_t cudaMemset(void *, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void *, const void *, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **p, const void *) { return *p = nullptr, cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *)
{
    *a = {};
    a->numRegs = 255;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *found)
{
    *p = (void *)encode;
    *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

// What nvcc's host code calls to register kernels, which never run.
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t *, const void *) { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) { return cudaErrorUnknown; }
unsigned __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return 1; }

}  // extern "C"
