// recurrence.cu -- a gated linear recurrence over the tokens of each item, channel
// by channel, forward and backward.
//
//   a_t = sigmoid(f_t),  h_t = a_t h_(t-1) + (1 - a_t) x_t,  out_t = h_t silu(o_t)
// and with dh_t = dout_t silu(o_t) + a_(t+1) dh_(t+1)
//   dx = dh (1 - a),  df = dh (h_(t-1) - x) a (1 - a),  do = dout h silu'(o).
//
// One thread a channel, token after token.
#include "decoder.cuh"

namespace gsr {
namespace {

constexpr int kSteps = GSR_RECURRENCE_BLOCK;

struct Tokens {
    void *data;
    int64_t batch, token;
};

struct RecurrenceArgs {
    Tokens x, forget, gate, out, dout, dx, dforget, dgate;
    const float *initial;
    float *final, *states;
    const float *dfinal;
    float *dinitial;
    const int *lengths;
    int batch, tokens, channels, blocks, reverse;
};

template <typename T>
__device__ __forceinline__ T *element(const Tokens &t, int b, int token, int c)
{
    return (T *)t.data + b * t.batch + token * t.token + c;
}

__device__ __forceinline__ int item_length(const RecurrenceArgs &a, int b)
{
    return a.lengths ? min(max(a.lengths[b], 0), a.tokens) : a.tokens;
}

template <typename T>
__global__ void __launch_bounds__(128) k_recurrence(const RecurrenceArgs a)
{
    grid_dependency_begin();
    const int c = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
    if (c >= a.channels) return;
    const int length = item_length(a, b);
    float h = a.initial ? a.initial[(int64_t)b * a.channels + c] : 0.0f;
    for (int k = 0; k < length; ++k) {
        if (a.states && k % kSteps == 0) a.states[((int64_t)b * a.blocks + k / kSteps) * a.channels + c] = h;
        const int t = a.reverse ? length - 1 - k : k;
        const float x = to_float(*element<T>(a.x, b, t, c)), f = to_float(*element<T>(a.forget, b, t, c));
        const float keep = 1.0f / (1.0f + expf(-f)), enter = 1.0f / (1.0f + expf(f));
        h = f >= 0.0f ? fmaf(enter, x - h, h) : fmaf(keep, h - x, x);
        float y = h;
        if (a.gate.data) {
            const float o = to_float(*element<T>(a.gate, b, t, c));
            y *= o / (1.0f + expf(-o));
        }
        *element<T>(a.out, b, t, c) = from_float<T>(y);
    }
    for (int t = length; t < a.tokens; ++t) *element<T>(a.out, b, t, c) = from_float<T>(0.0f);
    a.final[(int64_t)b * a.channels + c] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) k_recurrence_grad(const RecurrenceArgs a)
{
    grid_dependency_begin();
    const int c = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
    if (c >= a.channels) return;
    const int length = item_length(a, b);
    float carry = a.dfinal ? a.dfinal[(int64_t)b * a.channels + c] : 0.0f;   // a_(t+1) dh_(t+1)
    for (int block = (length - 1) / kSteps; block >= 0 && length > 0; --block) {
        const int first = block * kSteps, count = min(kSteps, length - first);
        float before[kSteps];
        float h = a.states[((int64_t)b * a.blocks + block) * a.channels + c];
        for (int i = 0; i < count; ++i) {
            const int t = a.reverse ? length - 1 - first - i : first + i;
            const float x = to_float(*element<T>(a.x, b, t, c)), f = to_float(*element<T>(a.forget, b, t, c));
            const float keep = 1.0f / (1.0f + expf(-f)), enter = 1.0f / (1.0f + expf(f));
            before[i] = h;
            h = f >= 0.0f ? fmaf(enter, x - h, h) : fmaf(keep, h - x, x);
        }
        for (int i = count - 1; i >= 0; --i) {
            const int t = a.reverse ? length - 1 - first - i : first + i;
            const float x = to_float(*element<T>(a.x, b, t, c)), f = to_float(*element<T>(a.forget, b, t, c));
            const float keep = 1.0f / (1.0f + expf(-f)), enter = 1.0f / (1.0f + expf(f));
            float dh = to_float(*element<T>(a.dout, b, t, c));
            if (a.gate.data) {
                const float o = to_float(*element<T>(a.gate, b, t, c)), s = 1.0f / (1.0f + expf(-o));
                *element<T>(a.dgate, b, t, c) = from_float<T>(dh * h * (s * fmaf(o, 1.0f - s, 1.0f)));
                dh *= o * s;
            }
            dh += carry;
            *element<T>(a.dx, b, t, c) = from_float<T>(dh * enter);
            *element<T>(a.dforget, b, t, c) = from_float<T>(dh * (before[i] - x) * (keep * enter));
            carry = keep * dh;
            h = before[i];
        }
    }
    for (int t = length; t < a.tokens; ++t) {
        *element<T>(a.dx, b, t, c) = from_float<T>(0.0f);
        *element<T>(a.dforget, b, t, c) = from_float<T>(0.0f);
        if (a.gate.data) *element<T>(a.dgate, b, t, c) = from_float<T>(0.0f);
    }
    if (a.dinitial) a.dinitial[(int64_t)b * a.channels + c] = carry;
}

Tokens tokens_of(const gsr_heads *t)
{
    return t ? Tokens{t->data, t->batch_stride, t->token_stride} : Tokens{};
}

RecurrenceArgs args_of(const gsr_recurrence &d)
{
    RecurrenceArgs a = {};
    a.lengths = d.lengths;
    a.batch = d.batch;
    a.tokens = d.tokens;
    a.channels = d.channels;
    a.blocks = (d.tokens + kSteps - 1) / kSteps;
    a.reverse = d.reverse;
    return a;
}


template <typename K>
int launch(gsr_ctx *ctx, const RecurrenceArgs &a, K *kernel, cudaStream_t stream, const char *what)
{
    return cuda_check(ctx, launch_kernel(ctx, kernel, dim3((unsigned)((a.channels + 127) / 128), (unsigned)a.batch), 128,
                                         stream, a), what);
}

}  // namespace

int gated_recurrence_forward(gsr_ctx *ctx, const gsr_recurrence &d, const gsr_heads &x, const gsr_heads &forget,
                             const gsr_heads *gate, const float *initial, const gsr_heads &out, float *final,
                             float *states, cudaStream_t stream)
{
    RecurrenceArgs a = args_of(d);
    a.x = tokens_of(&x);
    a.forget = tokens_of(&forget);
    a.gate = tokens_of(gate);
    a.out = tokens_of(&out);
    a.initial = initial;
    a.final = final;
    a.states = states;
    if (d.dtype == GSR_F32) return launch(ctx, a, k_recurrence<float>, stream, "gated recurrence forward");
    if (d.dtype == GSR_BF16) return launch(ctx, a, k_recurrence<__nv_bfloat16>, stream, "gated recurrence forward");
    return launch(ctx, a, k_recurrence<__half>, stream, "gated recurrence forward");
}

int gated_recurrence_backward(gsr_ctx *ctx, const gsr_recurrence &d, const gsr_heads &dout, const gsr_heads &x,
                              const gsr_heads &forget, const gsr_heads *gate, const float *states,
                              const float *dfinal, const gsr_heads &dx, const gsr_heads &dforget,
                              const gsr_heads *dgate, float *dinitial, cudaStream_t stream)
{
    RecurrenceArgs a = args_of(d);
    a.dout = tokens_of(&dout);
    a.x = tokens_of(&x);
    a.forget = tokens_of(&forget);
    a.gate = tokens_of(gate);
    a.states = const_cast<float *>(states);
    a.dfinal = dfinal;
    a.dx = tokens_of(&dx);
    a.dforget = tokens_of(&dforget);
    a.dgate = tokens_of(dgate);
    a.dinitial = dinitial;
    if (d.dtype == GSR_F32) return launch(ctx, a, k_recurrence_grad<float>, stream, "gated recurrence backward");
    if (d.dtype == GSR_BF16)
        return launch(ctx, a, k_recurrence_grad<__nv_bfloat16>, stream, "gated recurrence backward");
    return launch(ctx, a, k_recurrence_grad<__half>, stream, "gated recurrence backward");
}

}  // namespace gsr
