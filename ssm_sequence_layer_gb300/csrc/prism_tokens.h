// Internal declarations of the token operators (embedding, norm, 8-bit product, log probabilities).
#pragma once

#include "prism_internal.h"

namespace prism {

// A launch context: where to record the status and the kernels' times.
struct TokenLaunch {
    int sm_count;
    int *d_status;
    long long wait_ns;
    KernelTimer *timer;
};

// A launch that may begin while the kernel before it in the stream ends, and waits for that kernel's results itself.
// A call's first kernel is launched plainly, but for the weight's gradient of a norm of no rows, which waits like any other.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- embedding (prism_embed.cu) ------------------------------------------------------------------
struct EmbedArgs {
    const long long *ids;
    const void *table;
    long long ld_table;
    float scale;
    void *out;
    int n, D, V;
};
cudaError_t embed_prepare();
cudaError_t embed_forward(prism_dtype io, const EmbedArgs &a, const TokenLaunch &l);

// Workspace of the gradient: the tokens sorted by id and the sums of runs that cross a tile's edge.
struct EmbedWorkspace {
    int *key[2], *pos[2];  // [max_rows] ids (V = no token) and positions, ping-pong of the sort's passes
    int *hist;             // [passes][blocks][bins] digit counts of the sort by a kernel per digit, each at its largest number
    uint32_t *present;     // [V / 32 + 1] a bit for each id that has a token (and for "no token")
    float *part;           // [tiles][2][Dp] sums of a tile's first and last run where it crosses the edge
};
size_t embed_workspace_bytes(int max_rows, int D, int V);
void embed_carve(int max_rows, int V, void *base, EmbedWorkspace *w);
struct EmbedBackwardArgs {
    const long long *ids;
    const void *dout;
    float scale;
    int accumulate;
    float *dtable;
    int n, D, V;
};
cudaError_t embed_backward(prism_dtype io, const EmbedBackwardArgs &a, const EmbedWorkspace &w, const TokenLaunch &l);

// ---- norm (prism_norm.cu) -------------------------------------------------------------------------
struct NormArgs {
    const void *x, *residual, *weight;
    float eps;
    void *sum, *y, *y8;
    float *y_scale;
    int n, D;
};
cudaError_t norm_forward(prism_dtype io, const NormArgs &a, const TokenLaunch &l);

struct NormWorkspace {
    float2 *stats;  // [max_rows] 1 / rms and mean(w dy rh) of each row
    float *part;    // [slabs][D] parts of the weight's gradient
};
size_t norm_workspace_bytes(int max_rows, int D);
void norm_carve(int max_rows, int D, void *base, NormWorkspace *w);
struct NormBackwardArgs {
    const void *sum, *weight, *dy, *dsum;
    float eps;
    void *dx;
    float *dweight;
    int n, D;
};
cudaError_t norm_backward(prism_dtype io, const NormBackwardArgs &a, const NormWorkspace &w, const TokenLaunch &l);

// ---- 8-bit product (prism_matmul8.cu) --------------------------------------------------------------
struct Matmul8Args {
    const void *a8;
    const float *a_scale;
    const void *w8;
    const float *w_scale;
    void *out;
    int M, N, K;
};
cudaError_t matmul8_prepare();
cudaError_t matmul8(prism_dtype out, const Matmul8Args &a, const TokenLaunch &l);
cudaError_t matmul8_weights(prism_dtype io, int N, int K, const void *W, void *w8, float *w_scale, const TokenLaunch &l);

// ---- log probabilities (prism_logprobs.cu) ---------------------------------------------------------
struct LogprobArgs {
    const void *logits;
    long long ld;
    const long long *targets;
    float inv_temperature;
    float *lse, *logprob, *entropy;
    long long *top_ids;
    float *top_logprob;
    int n, V, k;
};
cudaError_t logprobs_prepare();
cudaError_t logprobs_forward(prism_dtype logits, const LogprobArgs &a, const TokenLaunch &l);
struct LogprobBackwardArgs {
    const void *logits;
    long long ld;
    const long long *targets;
    float inv_temperature;
    const float *lse, *entropy, *dlogprob, *dentropy;
    void *dlogits;
    long long ld_d;
    int n, V;
};
cudaError_t logprobs_backward(prism_dtype logits, const LogprobBackwardArgs &a, const TokenLaunch &l);

}  // namespace prism

struct prism_tokens_s {
    int max_rows, D, V;
    prism_dtype io, logits;
    int device, sm_count;
    long long opt_wait_ns, opt_timing;
    prism::KernelTimer timer;
    bool have_events;  // the timer's events exist (created when timing is first switched on)
    int *d_status;
    void *ws;  // device memory (owned)
    size_t ws_bytes;
    prism::EmbedWorkspace embed;
    prism::NormWorkspace norm;
};
