// Log probabilities of given tokens with entropy and top alternatives, and the gradient.
//
// With z = inv_temperature logits, m = max_j z_j, s = sum_j exp(z_j - m), t = sum_j exp(z_j - m) (z_j - m):
//   lse = m + log s,   logprob = z_target - lse,   entropy = log s - t / s
//   dlogits_j = inv_temperature (dlogprob (1_{j = target} - p_j) - dentropy p_j (log p_j + entropy))
// One pass over the row with a running maximum: m, s and t of two parts join as
//   m = max(m1, m2),  f_i = exp(m_i - m),  s = sum f_i s_i,  t = sum f_i (t_i + s_i (m_i - m))
// HBM bounds both directions (a few operations and one exponential per value).
//
// A logit of -inf or of the lowest value (of bfloat16, or below) marks a masked token, and so does a
// product that overflows to -inf: z = -inf there.
#include "io_util.h"
#include "prism_tokens.h"

namespace prism {
namespace logp {

constexpr int kThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

constexpr float kLowest = -3.38953139e38f;  // the lowest bfloat16 value

// z of a logit; -inf for a masked token (NaN stays NaN)
__device__ __forceinline__ float z_of(float x, float c) { return x <= kLowest ? -INFINITY : x * c; }

struct Running {
    float m, s, t;
};
__device__ __forceinline__ Running join(const Running a, const Running b)
{
    Running r;
    r.m = fmaxf(a.m, b.m);
    // a part that holds nothing (m = -inf) has s = t = 0: its factor must be a number
    const float da = a.m == r.m ? 0.f : a.m - r.m, db = b.m == r.m ? 0.f : b.m - r.m;
    const float fa = __expf(da), fb = __expf(db);
    r.s = a.s * fa + b.s * fb;
    r.t = fa * (fa > 0.f ? a.t + a.s * da : 0.f) + fb * (fb > 0.f ? b.t + b.s * db : 0.f);
    return r;
}
__device__ __forceinline__ void add(Running &r, float z)
{
    if (z == -INFINITY) return;  // a masked token
    if (z > r.m) {
        const float d = r.m == -INFINITY ? 0.f : r.m - z, f = r.m == -INFINITY ? 0.f : __expf(d);
        r.t = f > 0.f ? f * (r.t + r.s * d) : 0.f;
        r.s *= f;
        r.m = z;
    }
    const float d = z - r.m, e = __expf(d);  // NaN and +inf give NaN here, as the formulas do
    r.s += e;
    r.t = e == 0.f ? r.t : fmaf(e, d, r.t);
}

// A logit's place in the order of the top: by value (NaN first), then by lowest id.  Larger keys come
// first; 0 stands for nothing (masked tokens never become keys).
__device__ __forceinline__ unsigned long long key_of(float x, int id)
{
    uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // -0 = +0
    b = x != x ? 0xffffffffu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((unsigned long long)b << 32) | (uint32_t)~id;
}

template <typename logit_t>
struct ForwardParams {
    const logit_t *logits;
    const long long *targets;
    float *lse, *logprob, *entropy, *top_logprob;
    long long *top_ids;
    long long ld;
    float inv_temperature;
    int n, V, k;
    int *status;
};

template <typename logit_t>
__global__ void __launch_bounds__(kThreads) forward_kernel(const ForwardParams<logit_t> p)
{
    __shared__ Running parts[kThreads / 32];
    __shared__ unsigned long long best[kThreads / 32];
    __shared__ float m_s, logs_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const logit_t *x = p.logits + row * p.ld;
    Running r{-INFINITY, 0.f, 0.f};
    for (int j = tid; j < p.V; j += kThreads) add(r, z_of(io::ld(x + j), p.inv_temperature));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Running other{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                            __shfl_xor_sync(0xffffffffu, r.t, o)};
        r = lane & o ? join(other, r) : join(r, other);
    }
    if (lane == 0) parts[warp] = r;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kThreads / 32; ++w) r = join(r, parts[w]);
        // logprob = (z - m) - log s rather than z - lse: the difference is exact where z and m are near
        const bool none = r.m == -INFINITY && r.s == 0.f;
        const float m = none ? 0.f : r.m, logs = none ? -INFINITY : logf(r.s);
        m_s = m;
        logs_s = logs;
        if (p.lse) p.lse[row] = m + logs;
        if (p.entropy) p.entropy[row] = none ? 0.f : logs - r.t / r.s;
        if (p.logprob) {
            const long long t = p.targets[row];
            if (t >= p.V) atomicCAS(p.status, 0, kDevBounds);
            float v = 0.f;
            if (t >= 0 && t < p.V) v = none ? -INFINITY : (z_of(io::ld(x + t), p.inv_temperature) - m) - logs;
            p.logprob[row] = v;
        }
    }
    __syncthreads();
    unsigned long long last = ~0ull;
    for (int i = 0; i < p.k; ++i) {
        unsigned long long b = 0;
        for (int j = tid; j < p.V; j += kThreads) {
            const float v = io::ld(x + j);
            if (z_of(v, p.inv_temperature) == -INFINITY) continue;
            const unsigned long long key = key_of(v, j);
            if (key < last && key > b) b = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
        if (lane == 0) best[warp] = b;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) b = max(b, best[w]);
        __syncthreads();
        last = b;
        if (tid == 0) {
            const int id = (int)~(uint32_t)b;
            if (p.top_ids) p.top_ids[row * p.k + i] = b ? id : -1;
            if (p.top_logprob) p.top_logprob[row * p.k + i] = b ? (io::ld(x + id) * p.inv_temperature - m_s) - logs_s : -INFINITY;
        }
    }
}

template <typename logit_t>
struct BackwardParams {
    const logit_t *logits;
    const long long *targets;
    const float *lse, *entropy, *dlogprob, *dentropy;
    logit_t *dlogits;
    long long ld, ld_d;
    float inv_temperature;
    int n, V;
    int *status;
};

template <typename logit_t>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BackwardParams<logit_t> p)
{
    const long long row = blockIdx.x;
    const logit_t *x = p.logits + row * p.ld;
    logit_t *d = p.dlogits + row * p.ld_d;
    const float lse = p.lse[row];
    long long t = p.dlogprob ? p.targets[row] : -1;
    if (t >= p.V) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevBounds);
        t = -1;
    }
    const float dlp = t >= 0 ? p.dlogprob[row] : 0.f;
    const float dh = p.dentropy ? p.dentropy[row] : 0.f, h = p.dentropy ? p.entropy[row] : 0.f;
    for (int j = threadIdx.x; j < p.V; j += kThreads) {
        const float z = z_of(io::ld(x + j), p.inv_temperature);
        float g = 0.f;
        if (z != -INFINITY && lse != -INFINITY) {
            const float lp = z - lse, pr = __expf(lp);
            g = (j == t ? dlp : 0.f) - pr * dlp - (pr == 0.f ? 0.f : dh * pr * (lp + h));
        }
        io::st(d + j, g * p.inv_temperature);
    }
}

template <typename logit_t>
cudaError_t forward(const LogprobArgs &a, const TokenLaunch &l)
{
    const ForwardParams<logit_t> p{(const logit_t *)a.logits, a.targets, a.lse, a.logprob, a.entropy, a.top_logprob, a.top_ids,
                                   a.ld, a.inv_temperature, a.n, a.V, a.k, l.d_status};
    l.timer->begin("token_logprobs");
    forward_kernel<logit_t><<<a.n, kThreads, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

template <typename logit_t>
cudaError_t backward(const LogprobBackwardArgs &a, const TokenLaunch &l)
{
    const BackwardParams<logit_t> p{(const logit_t *)a.logits, a.targets, a.lse, a.entropy, a.dlogprob, a.dentropy,
                                    (logit_t *)a.dlogits, a.ld, a.ld_d, a.inv_temperature, a.n, a.V, l.d_status};
    l.timer->begin("token_logprobs_backward");
    backward_kernel<logit_t><<<a.n, kThreads, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace logp

cudaError_t logprobs_forward(prism_dtype logits, const LogprobArgs &a, const TokenLaunch &l)
{
    return logits == PRISM_BF16 ? logp::forward<__nv_bfloat16>(a, l) : logp::forward<float>(a, l);
}

cudaError_t logprobs_backward(prism_dtype logits, const LogprobBackwardArgs &a, const TokenLaunch &l)
{
    return logits == PRISM_BF16 ? logp::backward<__nv_bfloat16>(a, l) : logp::backward<float>(a, l);
}

}  // namespace prism
