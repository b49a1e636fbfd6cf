// Matrix product with bias, activation and residual in its epilogue, and its gradients.
//
//   forward   pre = x W^T + bias,  y = act(pre) + residual
//   backward  dx = (dy W) act'(pre) + dsum
//   weights   dW (+)= dy^T x,  dbias (+)= sum over rows of dy
#include "io_util.h"
#include "prism_tokens.h"

namespace prism {
namespace lin {

// ---- activations ----------------------------------------------------------------------------------
// Both are within 2^-20 of themselves in relative terms wherever they are normal numbers, also where they are tiny.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 2^(h + l), l small
__device__ __forceinline__ float exp2_of(float h, float l)
{
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(h));
    return fmaf(e, l * 0.69314718f, e);
}
// With a = |z| (cut at 40, where all is decided), E = e^(-a^2 / 2) and Phi(-a) = E R(a): gelu(z) = max(z, 0) - a E R(a) and
// gelu'(z) = [z > 0] -+ E (R(a) - a / sqrt(2 pi)).  R(a) = t P(t), t = 1 / (1 + 0.275 a), P of degree 8 fitted to the scaled complementary error
// function with the least largest relative error, 2^-24; the square's rounding error is carried into the exponential.
__device__ __forceinline__ void gelu_parts(float z, float &a, float &E, float &R)
{
    a = min_nan(fabsf(z), 40.f);
    const float s = a * a, y = s * -0.72134752f;
    E = exp2_of(y, fmaf(s, -0.72134752f, -y) + fmaf(s, -9.6298175e-9f, fmaf(a, a, -s) * -0.72134752f));
    const float t = __fdividef(1.f, fmaf(a, 0.275f, 1.f));
    float q = fmaf(t, 0.027167636901140213f, -0.11067406088113785f);
    q = fmaf(t, q, 0.1301683485507965f);
    q = fmaf(t, q, -0.03515997529029846f);
    q = fmaf(t, q, 0.08800629526376724f);
    q = fmaf(t, q, 0.07893631607294083f);
    q = fmaf(t, q, 0.10219038277864456f);
    q = fmaf(t, q, 0.10965436697006226f);
    q = fmaf(t, q, 0.1097106859087944f);
    R = q * t;
}
// With e = e^-|z| (cut at 120): silu(z) = z / (1 + e) or z e / (1 + e), silu'(z) = that over z + z e / (1 + e)^2
__device__ __forceinline__ void silu_parts(float z, float &a, float &e, float &r)
{
    a = min_nan(fabsf(z), 120.f);
    const float y = a * -1.44269504f;
    e = exp2_of(y, fmaf(a, -1.44269504f, -y) + a * -1.9259630e-8f);
    r = __fdividef(1.f, 1.f + e);
}
template <prism_activation ACT>
__device__ __forceinline__ float act_value(float z)
{
    float a, e, r;
    if constexpr (ACT == PRISM_ACT_GELU) {
        gelu_parts(z, a, e, r);
        return fmaf(-a * e, r, z > 0.f ? z : 0.f);
    } else if constexpr (ACT == PRISM_ACT_SILU) {
        silu_parts(z, a, e, r);
        return z > 0.f ? z * r : -a * e * r;
    } else {
        return z;
    }
}
template <prism_activation ACT>
__device__ __forceinline__ float act_slope(float z)
{
    float a, e, r;
    if constexpr (ACT == PRISM_ACT_GELU) {
        gelu_parts(z, a, e, r);
        const float d = e * fmaf(a, -0.39894228f, r);
        return z > 0.f ? 1.f - d : d;
    } else if constexpr (ACT == PRISM_ACT_SILU) {
        silu_parts(z, a, e, r);
        const float d = a * e * r * r;
        return z > 0.f ? r + d : e * r - d;
    } else {
        return 1.f;
    }
}

// ---- the simplest form: a tile of 64 x 64 per block in registers ------------------------------------
template <typename io_t>
struct Simple {
    const io_t *a, *b;
    long long sai, sak, sbj, sbk;  // A(i, k) = a[i sai + k sak], B(j, k) = b[j sbj + k sbk]
    int I, J, K;
    const io_t *bias, *pre_in, *add;
    void *out;
    io_t *pre_out;
    float *dbias;
    int weights, accumulate;
};

template <typename io_t, prism_activation ACT>
__global__ void __launch_bounds__(256) simple_kernel(const Simple<io_t> p)
{
    constexpr int T = 64, KT = 16;
    __shared__ float as[KT][T + 1], bs[KT][T + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int i0 = blockIdx.x * T, j0 = blockIdx.y * T;
    float c[4][4] = {}, sum[4][4] = {}, bsum = 0.f, bpart = 0.f;
    for (int k0 = 0; k0 < p.K; k0 += KT) {
        for (int e = tid; e < T * KT; e += 256) {
            // neighbouring threads read neighbouring addresses
            const int ia = p.sak == 1 ? e / KT : e % T, ka = p.sak == 1 ? e % KT : e / T;
            as[ka][ia] = i0 + ia < p.I && k0 + ka < p.K ? io::ld(p.a + (i0 + ia) * p.sai + (k0 + ka) * p.sak) : 0.f;
            const int jb = p.sbk == 1 ? e / KT : e % T, kb = p.sbk == 1 ? e % KT : e / T;
            bs[kb][jb] = j0 + jb < p.J && k0 + kb < p.K ? io::ld(p.b + (j0 + jb) * p.sbj + (k0 + kb) * p.sbk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            float x[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = as[k][ty + 16 * u], y[u] = bs[k][tx + 16 * u];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int w = 0; w < 4; ++w) c[u][w] = fmaf(x[u], y[w], c[u][w]);
        }
        if (p.dbias && j0 == 0 && tid < T)
            for (int k = 0; k < KT; ++k) bpart += as[k][tid];
        if (k0 / KT % 16 == 15 || k0 + KT >= p.K) {  // sums of 256 terms, then their sum: long ones keep their last bits
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int w = 0; w < 4; ++w) sum[u][w] += c[u][w], c[u][w] = 0.f;
            bsum += bpart, bpart = 0.f;
        }
        __syncthreads();
    }
    if (p.dbias && j0 == 0 && tid < T && i0 + tid < p.I) p.dbias[i0 + tid] = p.accumulate ? p.dbias[i0 + tid] + bsum : bsum;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int i = i0 + ty + 16 * u, j = j0 + tx + 16 * w;
            if (i >= p.I || j >= p.J) continue;
            const size_t at = (size_t)i * p.J + j;
            float z = sum[u][w];
            if (p.weights) {
                float *to = (float *)p.out + at;
                *to = p.accumulate ? *to + z : z;
                continue;
            }
            if (p.pre_in) {
                z *= act_slope<ACT>(io::ld(p.pre_in + at));
            } else {
                if (p.bias) z += io::ld(p.bias + j);
                if (p.pre_out) io::st(p.pre_out + at, z);
                z = act_value<ACT>(z);
            }
            if (p.add) z += io::ld(p.add + at);
            io::st((io_t *)p.out + at, z);
        }
}

template <typename io_t>
cudaError_t run(const LinearArgs &a, const TokenLaunch &l)
{
    Simple<io_t> p = {};
    p.a = (const io_t *)a.a, p.b = (const io_t *)a.b;
    p.bias = (const io_t *)a.bias, p.add = (const io_t *)a.add, p.out = a.out, p.pre_out = (io_t *)a.pre_out;
    p.dbias = a.dbias, p.accumulate = a.accumulate;
    const char *name = "linear";
    if (a.op == LinearOp::forward) {
        p.sai = a.K, p.sak = 1, p.sbj = a.K, p.sbk = 1, p.I = a.M, p.J = a.N, p.K = a.K;
    } else if (a.op == LinearOp::backward) {
        name = "linear_backward";
        p.sai = a.N, p.sak = 1, p.sbj = 1, p.sbk = a.K, p.I = a.M, p.J = a.K, p.K = a.N;
        if (a.act != PRISM_ACT_NONE) p.pre_in = (const io_t *)a.pre_in;
    } else {
        name = "linear_weights";
        p.sai = 1, p.sak = a.N, p.sbj = 1, p.sbk = a.K, p.I = a.N, p.J = a.K, p.K = a.M, p.weights = 1;
    }
    l.timer->begin(name);
    const dim3 grid((p.I + 63) / 64, (p.J + 63) / 64);
    if (a.act == PRISM_ACT_GELU) simple_kernel<io_t, PRISM_ACT_GELU><<<grid, 256, 0, l.timer->stream>>>(p);
    else if (a.act == PRISM_ACT_SILU) simple_kernel<io_t, PRISM_ACT_SILU><<<grid, 256, 0, l.timer->stream>>>(p);
    else simple_kernel<io_t, PRISM_ACT_NONE><<<grid, 256, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace lin

cudaError_t linear_prepare() { return cudaSuccess; }

cudaError_t linear(prism_dtype io, const LinearArgs &a, const TokenLaunch &l)
{
    return io == PRISM_BF16 ? lin::run<__nv_bfloat16>(a, l) : lin::run<float>(a, l);
}

}  // namespace prism
