// Host side of the token operators declared in include/prism.h: argument validation, the handle
// (sizes, device, workspace) and the launches on the caller's stream.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "prism_tokens.h"

namespace {

thread_local char g_tokens_err[512];

prism_status fail(prism_status s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_tokens_err, sizeof(g_tokens_err), fmt, ap);
    va_end(ap);
    prism_set_error_message(g_tokens_err);
    return s;
}

prism_status cuda_fail(cudaError_t e, const char *what)
{
    (void)cudaGetLastError();  // a recoverable failure is not reported again by a later call's launch check
    return fail(PRISM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Pointer {
    const char *name;
    const void *p;
    size_t align;
    bool required;
};

template <int N>
prism_status check_pointers(const Pointer (&ps)[N])
{
    for (const Pointer &q : ps) {
        if (!q.p && q.required) return fail(PRISM_ERR_INVALID_ARG, "%s must not be NULL", q.name);
        if (q.p && !aligned(q.p, q.align)) return fail(PRISM_ERR_MISALIGNED, "%s is not %d-byte aligned", q.name, (int)q.align);
    }
    return PRISM_OK;
}

// The handle and the number of rows of a call.
prism_status check_call(const prism_tokens_s *t, int n, const char *rows)
{
    if (!t) return fail(PRISM_ERR_INVALID_ARG, "tokens is NULL");
    if (n < 0 || n > t->max_rows)
        return fail(PRISM_ERR_INVALID_ARG, "%s must be in 0 .. max_rows = %d (got %d)", rows, t->max_rows, n);
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != t->device)
        return fail(PRISM_ERR_INVALID_ARG, "current device %d differs from the handle's device %d", dev, t->device);
    return PRISM_OK;
}

prism_status check_sizes8(int N, int K)
{
    if (N < 1 || K < 1) return fail(PRISM_ERR_INVALID_ARG, "N and K must be >= 1 (got %d, %d)", N, K);
    if (K % 16 != 0 || K > 65536 || N > (1 << 30))
        return fail(PRISM_ERR_UNSUPPORTED, "K must be a multiple of 16, at most 65536, and N at most 2^30 (got K=%d, N=%d)", K, N);
    return PRISM_OK;
}

// Above 2^126 the exponentials' scale inv_temperature log2 e overflows.  Below 2^-60 the lowest values, which stand for
// masked tokens, would come within the exponentials' reach of live ones: they are 2^103 apart at least, and 2^43 is far.
prism_status check_temperature(float inv_temperature)
{
    if (!(inv_temperature >= 0x1p-60f && inv_temperature <= 0x1p126f))
        return fail(PRISM_ERR_INVALID_ARG, "inv_temperature must be in 2^-60 .. 2^126 (got %g)", (double)inv_temperature);
    return PRISM_OK;
}

prism_status check_linear(int N, int K, prism_activation act)
{
    if (N < 1 || K < 1) return fail(PRISM_ERR_INVALID_ARG, "N and K must be >= 1 (got %d, %d)", N, K);
    if (N > (1 << 20) || K > (1 << 20)) return fail(PRISM_ERR_UNSUPPORTED, "N and K are at most 2^20 (got %d, %d)", N, K);
    if (act != PRISM_ACT_NONE && act != PRISM_ACT_GELU && act != PRISM_ACT_SILU)
        return fail(PRISM_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    return PRISM_OK;
}

// The form of prism_heads and its backward; fills in what NULL stands for.
prism_status check_heads(const prism_tokens_s *t, const prism_heads_form *f, long long ld, const char *ld_name)
{
    if (!t) return fail(PRISM_ERR_INVALID_ARG, "tokens is NULL");
    if (!f) return fail(PRISM_ERR_INVALID_ARG, "form must not be NULL");
    if (f->B < 0 || f->T < 0 || (long long)f->B * f->T > t->max_rows)
        return fail(PRISM_ERR_INVALID_ARG, "B T must be in 0 .. max_rows = %d (got %d x %d)", t->max_rows, f->B, f->T);
    const prism_status st = check_call(t, f->B * f->T, "B T");
    if (st != PRISM_OK) return st;
    if (f->Hq < 0 || f->Hk < 0 || f->Hv < 0 || (long long)f->Hq + f->Hk + f->Hv < 1)
        return fail(PRISM_ERR_INVALID_ARG, "heads must be >= 0, and one at least (got %d, %d, %d)", f->Hq, f->Hk, f->Hv);
    if ((long long)f->Hq + f->Hk + f->Hv > 65535)
        return fail(PRISM_ERR_UNSUPPORTED, "heads are at most 65535 together (got %d, %d, %d)", f->Hq, f->Hk, f->Hv);
    const bool rows = f->Hq + f->Hk > 0, values = f->Hv > 0;
    if ((rows && f->d < 1) || (values && f->dv < 1)) return fail(PRISM_ERR_INVALID_ARG, "d and dv must be >= 1 (got %d, %d)", f->d, f->dv);
    if ((rows && f->d > prism::kMaxHeadSize) || (values && f->dv > prism::kMaxHeadSize))
        return fail(PRISM_ERR_UNSUPPORTED, "d and dv are at most %d (got %d, %d)", prism::kMaxHeadSize, f->d, f->dv);
    if (f->norm != PRISM_HEADS_PLAIN && f->norm != PRISM_HEADS_UNIT && f->norm != PRISM_HEADS_RMS)
        return fail(PRISM_ERR_INVALID_ARG, "unknown norm %d", (int)f->norm);
    if (!std::isfinite(f->eps) || f->eps < 0.f) return fail(PRISM_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (f->rot < 0 || f->rot % 2 != 0 || (rows && f->rot > f->d))
        return fail(PRISM_ERR_INVALID_ARG, "rot must be even and in 0 .. d = %d (got %d)", f->d, f->rot);
    if (f->rot > 0 && !std::isfinite(f->amplitude)) return fail(PRISM_ERR_INVALID_ARG, "amplitude must be finite");
    const long long width = (rows ? (long long)(f->Hq + f->Hk) * f->d : 0) + (values ? (long long)f->Hv * f->dv : 0);
    if (ld < width) return fail(PRISM_ERR_INVALID_ARG, "%s must be >= the heads' %lld columns (got %lld)", ld_name, width, ld);
    return check_pointers<4>({{"q_weight", f->q_weight, 16, false}, {"k_weight", f->k_weight, 16, false},
                              {"inv_freq", f->inv_freq, 4, f->rot > 0}, {"positions", f->positions, 8, false}});
}

prism::TokenLaunch begin(prism_tokens_s *t, struct CUstream_st *stream)
{
    t->timer.on = t->opt_timing != 0;
    t->timer.reset((cudaStream_t)stream);
    return {t->sm_count, t->d_status, t->opt_wait_ns, &t->timer};
}

prism_status launched(cudaError_t e) { return e == cudaSuccess ? PRISM_OK : cuda_fail(e, "kernel launch"); }

}  // namespace

extern "C" {

prism_status prism_tokens_plan(int max_rows, int D, int V, prism_dtype io, prism_tokens_t *out_tokens)
{
    if (!out_tokens) return fail(PRISM_ERR_INVALID_ARG, "out_tokens is NULL");
    *out_tokens = nullptr;
    if (max_rows < 1 || D < 1 || V < 1)
        return fail(PRISM_ERR_INVALID_ARG, "max_rows, D and V must be >= 1 (got %d, %d, %d)", max_rows, D, V);
    if (io != PRISM_F32 && io != PRISM_BF16) return fail(PRISM_ERR_INVALID_ARG, "unknown io dtype %d", (int)io);
    if (max_rows > (1 << 24) || D > 65536 || V > (1 << 30))
        return fail(PRISM_ERR_UNSUPPORTED, "max_rows is at most 2^24, D at most 65536, V at most 2^30 (got %d, %d, %d)", max_rows,
                    D, V);
    int device = 0, major = 0, minor = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    if (major != 10 || minor != 3)
        return fail(PRISM_ERR_ARCH, "device %d is sm_%d%d; this library is built for sm_103 only", device, major, minor);

    e = prism::embed_prepare();
    if (e == cudaSuccess) e = prism::matmul8_prepare();
    if (e == cudaSuccess) e = prism::logprobs_prepare();
    if (e == cudaSuccess) e = prism::linear_prepare();
    if (e == cudaSuccess) e = prism::sample_prepare();
    if (e != cudaSuccess) return cuda_fail(e, "kernel attribute setup");
    prism_tokens_s *t = new (std::nothrow) prism_tokens_s();
    if (!t) return fail(PRISM_ERR_INVALID_ARG, "out of host memory");
    t->max_rows = max_rows;
    t->D = D;
    t->V = V;
    t->io = t->logits = io;
    t->device = device;
    t->sm_count = sms;
    // one allocation: the status word, then the operators' workspaces
    const size_t embed_bytes = prism::embed_workspace_bytes(max_rows, D, V);
    const size_t norm_bytes = (prism::norm_workspace_bytes(max_rows, D) + 255) & ~(size_t)255;
    t->ws_bytes = 256 + embed_bytes + norm_bytes + prism::heads_workspace_bytes();
    if ((e = cudaMalloc(&t->ws, t->ws_bytes)) != cudaSuccess) {
        delete t;
        return cuda_fail(e, "workspace allocation");
    }
    t->d_status = (int *)t->ws;
    // waited for: streams that do not wait for the default one may use the handle at once
    if ((e = cudaMemset(t->d_status, 0, sizeof(int))) != cudaSuccess || (e = cudaStreamSynchronize(nullptr)) != cudaSuccess) {
        cudaFree(t->ws);
        delete t;
        return cuda_fail(e, "status word init");
    }
    prism::embed_carve(max_rows, V, (char *)t->ws + 256, &t->embed);
    prism::norm_carve(max_rows, D, (char *)t->ws + 256 + embed_bytes, &t->norm);
    t->heads = (float *)((char *)t->ws + 256 + embed_bytes + norm_bytes);
    *out_tokens = t;
    return PRISM_OK;
}

prism_status prism_tokens_set_option(prism_tokens_t t, prism_option opt, long long value)
{
    if (!t) return fail(PRISM_ERR_INVALID_ARG, "tokens is NULL");
    switch (opt) {
    case PRISM_OPT_WAIT_NS:
        if (value < 0) return fail(PRISM_ERR_INVALID_ARG, "wait bound must be >= 0");
        t->opt_wait_ns = value;
        return PRISM_OK;
    case PRISM_OPT_OUT_DTYPE:
        if (value != PRISM_F32 && value != PRISM_BF16) return fail(PRISM_ERR_INVALID_ARG, "unknown out dtype");
        t->logits = (prism_dtype)value;
        return PRISM_OK;
    case PRISM_OPT_TIMING:
        if (value != 0 && value != 1) return fail(PRISM_ERR_INVALID_ARG, "timing must be 0 or 1");
        if (value && !t->have_events) {
            for (int i = 0; i < 2 * prism::kMaxTimedKernels; ++i) {
                const cudaError_t e = cudaEventCreate(&t->timer.ev[i]);
                if (e != cudaSuccess) {
                    for (int j = 0; j < i; ++j) cudaEventDestroy(t->timer.ev[j]);
                    return cuda_fail(e, "event creation");
                }
            }
            t->have_events = true;
        }
        t->opt_timing = value;
        return PRISM_OK;
    default: break;
    }
    return fail(PRISM_ERR_INVALID_ARG, "option %d is not one of a token handle", (int)opt);
}

prism_status prism_tokens_destroy(prism_tokens_t t)
{
    if (!t) return PRISM_OK;
    if (t->have_events)
        for (int i = 0; i < 2 * prism::kMaxTimedKernels; ++i) cudaEventDestroy(t->timer.ev[i]);
    const cudaError_t e = cudaFree(t->ws);
    delete t;
    if (e != cudaSuccess) return cuda_fail(e, "workspace free");
    return PRISM_OK;
}

size_t prism_tokens_workspace_bytes(prism_tokens_t t) { return t ? t->ws_bytes : 0; }

prism_status prism_tokens_last_device_status(prism_tokens_t t)
{
    if (!t) return fail(PRISM_ERR_INVALID_ARG, "tokens is NULL");
    int word = 0;
    cudaError_t e = cudaMemcpy(&word, t->d_status, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "status read");
    if (word == prism::kDevOk) return PRISM_OK;
    if ((e = cudaMemset(t->d_status, 0, sizeof(int))) != cudaSuccess || (e = cudaStreamSynchronize(nullptr)) != cudaSuccess)
        return cuda_fail(e, "status clear");
    if (word == prism::kDevTimeout) return fail(PRISM_ERR_TIMEOUT, "a bounded device wait expired");
    if (word == prism::kDevTemperature) return fail(PRISM_ERR_DEVICE, "a row's inv_temperature was outside 2^-60 .. 2^126 (no token drawn)");
    return fail(PRISM_ERR_DEVICE, "a token id or target was >= V = %d (treated as no token)", t->V);
}

int prism_tokens_kernel_times(prism_tokens_t t, prism_kernel_time *out, int max)
{
    if (!t || max < 0 || (max > 0 && !out)) {
        fail(PRISM_ERR_INVALID_ARG, "bad arguments to prism_tokens_kernel_times");
        return -1;
    }
    const int n = t->timer.n;
    for (int i = 0; i < n && i < max && i < prism::kMaxTimedKernels; ++i) {
        out[i].name = t->timer.names[i];
        out[i].ms = -1.f;
        if (t->timer.on) {
            float ms = 0.f;
            if (cudaEventElapsedTime(&ms, t->timer.ev[2 * i], t->timer.ev[2 * i + 1]) == cudaSuccess) out[i].ms = ms;
        }
    }
    return n;
}

prism_status prism_embed(prism_tokens_t t, int n, const long long *ids, const void *table, long long ld_table, float scale,
                         void *out, struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<3>({{"ids", ids, 8, n > 0}, {"table", table, 16, true}, {"out", out, 16, n > 0}})) != PRISM_OK) return st;
    if (ld_table < t->D) return fail(PRISM_ERR_INVALID_ARG, "ld_table must be >= D = %d (got %lld)", t->D, ld_table);
    const prism::TokenLaunch l = begin(t, stream);
    if (n == 0) return PRISM_OK;
    return launched(prism::embed_forward(t->io, {ids, table, ld_table, scale, out, n, t->D, t->V}, l));
}

prism_status prism_embed_backward(prism_tokens_t t, int n, const long long *ids, const void *dout, float scale, int accumulate,
                                  float *dtable, struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<3>({{"ids", ids, 8, n > 0}, {"dout", dout, 16, n > 0}, {"dtable", dtable, 16, true}})) != PRISM_OK)
        return st;
    const prism::TokenLaunch l = begin(t, stream);
    return launched(prism::embed_backward(t->io, {ids, dout, scale, accumulate != 0, dtable, n, t->D, t->V}, t->embed, l));
}

prism_status prism_norm(prism_tokens_t t, int n, const void *x, const void *residual, const void *weight, float eps, void *sum,
                        void *y, void *y8, float *y_scale, struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<7>({{"x", x, 16, n > 0}, {"residual", residual, 16, false}, {"weight", weight, 16, true},
                                 {"sum", sum, 16, false}, {"y", y, 16, false}, {"y8", y8, 16, false},
                                 {"y_scale", y_scale, 4, false}})) != PRISM_OK)
        return st;
    if (n > 0 && !y && !y8) return fail(PRISM_ERR_INVALID_ARG, "y and y8 must not both be NULL");
    if (!y8 != !y_scale) return fail(PRISM_ERR_INVALID_ARG, "y8 and y_scale come together");
    if (!std::isfinite(eps) || eps < 0.f) return fail(PRISM_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const prism::TokenLaunch l = begin(t, stream);
    if (n == 0) return PRISM_OK;
    return launched(prism::norm_forward(t->io, {x, residual, weight, eps, sum, y, y8, y_scale, n, t->D}, l));
}

prism_status prism_norm_backward(prism_tokens_t t, int n, const void *sum, const void *weight, float eps, const void *dy,
                                 const void *dsum, void *dx, float *dweight, struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<6>({{"sum", sum, 16, n > 0}, {"weight", weight, 16, true}, {"dy", dy, 16, n > 0},
                                 {"dsum", dsum, 16, false}, {"dx", dx, 16, n > 0}, {"dweight", dweight, 4, true}})) != PRISM_OK)
        return st;
    if (!std::isfinite(eps) || eps < 0.f) return fail(PRISM_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const prism::TokenLaunch l = begin(t, stream);
    return launched(prism::norm_backward(t->io, {sum, weight, dy, dsum, eps, dx, dweight, n, t->D}, t->norm, l));
}

prism_status prism_matmul8(prism_tokens_t t, int M, int N, int K, const void *a8, const float *a_scale, const void *w8,
                           const float *w_scale, void *out, struct CUstream_st *stream)
{
    prism_status st = check_call(t, M, "M");
    if (st != PRISM_OK) return st;
    if ((st = check_sizes8(N, K)) != PRISM_OK) return st;
    if ((st = check_pointers<5>({{"a8", a8, 16, M > 0}, {"a_scale", a_scale, 4, M > 0}, {"w8", w8, 16, true},
                                 {"w_scale", w_scale, 4, true}, {"out", out, 16, M > 0}})) != PRISM_OK)
        return st;
    const prism::TokenLaunch l = begin(t, stream);
    if (M == 0) return PRISM_OK;
    return launched(prism::matmul8(t->logits, {a8, a_scale, w8, w_scale, out, M, N, K}, l));
}

prism_status prism_matmul8_weights(prism_tokens_t t, int N, int K, const void *W, void *w8, float *w_scale,
                                   struct CUstream_st *stream)
{
    prism_status st = check_call(t, 0, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_sizes8(N, K)) != PRISM_OK) return st;
    if ((st = check_pointers<3>({{"W", W, 16, true}, {"w8", w8, 16, true}, {"w_scale", w_scale, 4, true}})) != PRISM_OK) return st;
    const prism::TokenLaunch l = begin(t, stream);
    return launched(prism::matmul8_weights(t->io, N, K, W, w8, w_scale, l));
}

prism_status prism_token_logprobs(prism_tokens_t t, int n, const void *logits, long long ld, const long long *targets,
                                  float inv_temperature, int k, float *lse, float *logprob, float *entropy, long long *top_ids,
                                  float *top_logprob, struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<7>({{"logits", logits, 16, n > 0}, {"targets", targets, 8, n > 0 && logprob}, {"lse", lse, 4, false},
                                 {"logprob", logprob, 4, false}, {"entropy", entropy, 4, false}, {"top_ids", top_ids, 8, false},
                                 {"top_logprob", top_logprob, 4, false}})) != PRISM_OK)
        return st;
    if (ld < t->V) return fail(PRISM_ERR_INVALID_ARG, "ld must be >= V = %d (got %lld)", t->V, ld);
    if (k < 0 || k > 32) return fail(PRISM_ERR_INVALID_ARG, "k must be in 0 .. 32 (got %d)", k);
    if ((st = check_temperature(inv_temperature)) != PRISM_OK) return st;
    if (!top_ids && !top_logprob) k = 0;
    const prism::TokenLaunch l = begin(t, stream);
    if (n == 0) return PRISM_OK;
    return launched(prism::logprobs_forward(
        t->logits, {logits, ld, targets, inv_temperature, lse, logprob, entropy, top_ids, top_logprob, n, t->V, k}, l));
}

prism_status prism_token_logprobs_backward(prism_tokens_t t, int n, const void *logits, long long ld, const long long *targets,
                                           float inv_temperature, const float *lse, const float *entropy, const float *dlogprob,
                                           const float *dentropy, void *dlogits, long long ld_d, struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<7>({{"logits", logits, 16, n > 0}, {"targets", targets, 8, n > 0 && dlogprob}, {"lse", lse, 4, n > 0},
                                 {"entropy", entropy, 4, n > 0 && dentropy}, {"dlogprob", dlogprob, 4, false},
                                 {"dentropy", dentropy, 4, false}, {"dlogits", dlogits, 16, n > 0}})) != PRISM_OK)
        return st;
    if (n > 0 && !dlogprob && !dentropy) return fail(PRISM_ERR_INVALID_ARG, "dlogprob and dentropy must not both be NULL");
    if (ld < t->V || ld_d < t->V) return fail(PRISM_ERR_INVALID_ARG, "ld and ld_d must be >= V = %d (got %lld, %lld)", t->V, ld, ld_d);
    if (logits == dlogits && ld != ld_d) return fail(PRISM_ERR_INVALID_ARG, "in place, ld_d must equal ld");
    if ((st = check_temperature(inv_temperature)) != PRISM_OK) return st;
    const prism::TokenLaunch l = begin(t, stream);
    if (n == 0) return PRISM_OK;
    return launched(prism::logprobs_backward(
        t->logits, {logits, ld, targets, inv_temperature, lse, entropy, dlogprob, dentropy, dlogits, ld_d, n, t->V}, l));
}

prism_status prism_linear(prism_tokens_t t, int M, int N, int K, const void *x, const void *W, const void *bias,
                          prism_activation act, const void *residual, void *y, void *pre, struct CUstream_st *stream)
{
    prism_status st = check_call(t, M, "M");
    if (st != PRISM_OK) return st;
    if ((st = check_linear(N, K, act)) != PRISM_OK) return st;
    if ((st = check_pointers<6>({{"x", x, 16, M > 0}, {"W", W, 16, true}, {"bias", bias, 16, false}, {"residual", residual, 16, false},
                                 {"y", y, 16, M > 0}, {"pre", pre, 16, false}})) != PRISM_OK)
        return st;
    if (y && y == pre) return fail(PRISM_ERR_INVALID_ARG, "y and pre must differ");
    const prism::TokenLaunch l = begin(t, stream);
    if (M == 0) return PRISM_OK;
    prism::LinearArgs a{prism::LinearOp::forward, x, W, M, N, K, act};
    a.bias = bias, a.add = residual, a.out = y, a.pre_out = pre;
    return launched(prism::linear(t->io, a, l));
}

prism_status prism_linear_backward(prism_tokens_t t, int M, int N, int K, const void *dy, const void *W, prism_activation act,
                                   const void *pre, const void *dsum, void *dx, struct CUstream_st *stream)
{
    prism_status st = check_call(t, M, "M");
    if (st != PRISM_OK) return st;
    if ((st = check_linear(N, K, act)) != PRISM_OK) return st;
    if ((st = check_pointers<5>({{"dy", dy, 16, M > 0}, {"W", W, 16, true}, {"pre", pre, 16, M > 0 && act != PRISM_ACT_NONE},
                                 {"dsum", dsum, 16, false}, {"dx", dx, 16, M > 0}})) != PRISM_OK)
        return st;
    const prism::TokenLaunch l = begin(t, stream);
    if (M == 0) return PRISM_OK;
    prism::LinearArgs a{prism::LinearOp::backward, dy, W, M, N, K, act};
    a.pre_in = pre, a.add = dsum, a.out = dx;
    return launched(prism::linear(t->io, a, l));
}

prism_status prism_linear_weight_backward(prism_tokens_t t, int M, int N, int K, const void *dy, const void *x, int accumulate,
                                          float *dW, float *dbias, struct CUstream_st *stream)
{
    prism_status st = check_call(t, M, "M");
    if (st != PRISM_OK) return st;
    if ((st = check_linear(N, K, PRISM_ACT_NONE)) != PRISM_OK) return st;
    if ((st = check_pointers<4>({{"dy", dy, 16, M > 0}, {"x", x, 16, M > 0}, {"dW", dW, 16, true}, {"dbias", dbias, 16, false}})) != PRISM_OK)
        return st;
    const prism::TokenLaunch l = begin(t, stream);
    if (M == 0) {
        if (accumulate) return PRISM_OK;
        cudaError_t e = cudaMemsetAsync(dW, 0, sizeof(float) * (size_t)N * K, (cudaStream_t)stream);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)N, (cudaStream_t)stream);
        return e == cudaSuccess ? PRISM_OK : cuda_fail(e, "gradient clear");
    }
    prism::LinearArgs a{prism::LinearOp::weights, dy, x, M, N, K, PRISM_ACT_NONE};
    a.out = dW, a.dbias = dbias, a.accumulate = accumulate != 0;
    return launched(prism::linear(t->io, a, l));
}

prism_status prism_heads(prism_tokens_t t, const prism_heads_form *form, const void *x, long long ld_x, void *q, void *k, void *v,
                         struct CUstream_st *stream)
{
    prism_status st = check_heads(t, form, ld_x, "ld_x");
    if (st != PRISM_OK) return st;
    const bool rows = form->B * form->T > 0;
    if ((st = check_pointers<4>({{"x", x, 16, rows}, {"q", q, 16, rows && form->Hq > 0}, {"k", k, 16, rows && form->Hk > 0},
                                 {"v", v, 16, rows && form->Hv > 0}})) != PRISM_OK)
        return st;
    const prism::TokenLaunch l = begin(t, stream);
    if (!rows) return PRISM_OK;
    return launched(prism::heads_forward(t->io, {*form, x, ld_x, q, k, v}, l));
}

prism_status prism_heads_backward(prism_tokens_t t, const prism_heads_form *form, const void *x, long long ld_x, prism_dtype grads,
                                  const void *dq, const void *dk, const void *dv, void *dx, long long ld_dx, float *dq_weight,
                                  float *dk_weight, struct CUstream_st *stream)
{
    prism_status st = check_heads(t, form, ld_x, "ld_x");
    if (st == PRISM_OK) st = check_heads(t, form, ld_dx, "ld_dx");
    if (st != PRISM_OK) return st;
    if (grads != PRISM_F32 && grads != t->io) return fail(PRISM_ERR_INVALID_ARG, "grads must be float32 or the io dtype");
    const bool rows = form->B * form->T > 0;
    if ((st = check_pointers<7>({{"x", x, 16, rows}, {"dq", dq, 16, rows && form->Hq > 0}, {"dk", dk, 16, rows && form->Hk > 0},
                                 {"dv", dv, 16, rows && form->Hv > 0}, {"dx", dx, 16, rows}, {"dq_weight", dq_weight, 4, false},
                                 {"dk_weight", dk_weight, 4, false}})) != PRISM_OK)
        return st;
    if ((dq_weight && form->Hq == 0) || (dk_weight && form->Hk == 0))
        return fail(PRISM_ERR_INVALID_ARG, "dq_weight and dk_weight need heads of their kind");
    const prism::TokenLaunch l = begin(t, stream);
    return launched(prism::heads_backward(t->io, {*form, x, ld_x, grads, dq, dk, dv, dx, ld_dx, dq_weight, dk_weight}, t->heads, l));
}

prism_status prism_sample(prism_tokens_t t, int n, const void *logits, long long ld, const float *u, const float *inv_temperature,
                          const int *top_k, const float *top_p, const float *min_p, long long *ids, float *logprob, int *kept,
                          struct CUstream_st *stream)
{
    prism_status st = check_call(t, n, "n");
    if (st != PRISM_OK) return st;
    if ((st = check_pointers<9>({{"logits", logits, 16, n > 0}, {"u", u, 4, n > 0}, {"inv_temperature", inv_temperature, 4, false},
                                 {"top_k", top_k, 4, false}, {"top_p", top_p, 4, false}, {"min_p", min_p, 4, false},
                                 {"ids", ids, 8, n > 0}, {"logprob", logprob, 4, false}, {"kept", kept, 4, false}})) != PRISM_OK)
        return st;
    if (ld < t->V) return fail(PRISM_ERR_INVALID_ARG, "ld must be >= V = %d (got %lld)", t->V, ld);
    const prism::TokenLaunch l = begin(t, stream);
    if (n == 0) return PRISM_OK;
    return launched(prism::sample(t->logits, {logits, ld, u, inv_temperature, top_k, top_p, min_p, ids, logprob, kept, n, t->V}, l));
}

}  // extern "C"
