// Matrix product of e4m3 operands with a scale for each block of 128, and the weights' layout.
//
//   out[m, j] = sum_b a_scale[m, b] w_scale[j / 128, b] c_b[m, j],   c_b[m, j] = sum_{k in block b} a8[m, k] w8[j, k]
//
// Products of e4m3 values are exact in fp32; the sum over a block is scaled and added in fp32 once per block.
#include "io_util.h"
#include "prism_tokens.h"

namespace prism {
namespace mm8 {

constexpr int kBlock = 128;
constexpr float kMaxE4M3 = 448.f, kMinScale = 1.17549435e-38f;

// two e4m3 values (the first in the low byte) as floats
__device__ __forceinline__ float2 two_e4m3(uint16_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

template <typename out_t>
struct Params {
    const uint8_t *a, *w;
    const float *a_scale, *w_scale;
    out_t *out;
    int M, N, K, KB;
};

constexpr int TM = 64, TN = 64;

template <typename out_t>
__global__ void __launch_bounds__(256) product_any_kernel(const Params<out_t> p)
{
    __shared__ float as[16][TM + 1], ws[16][TN + 1];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n0 = blockIdx.x * TN;
    for (int m0 = blockIdx.y * TM; m0 < p.M; m0 += gridDim.y * TM) {
    float total[4][4] = {};
    for (int b = 0; b < p.KB; ++b) {
        float c[4][4] = {};
        for (int k0 = b * kBlock; k0 < min(p.K, (b + 1) * kBlock); k0 += 16) {
            const int r = tid >> 2, q = (tid & 3) * 4;  // 64 rows, 4 values each
            uint32_t va = 0, vw = 0;
            if (m0 + r < p.M) va = *reinterpret_cast<const uint32_t *>(p.a + (size_t)(m0 + r) * p.K + k0 + q);
            if (n0 + r < p.N) vw = *reinterpret_cast<const uint32_t *>(p.w + (size_t)(n0 + r) * p.K + k0 + q);
            __syncthreads();
            const float2 a0 = two_e4m3((uint16_t)va), a1 = two_e4m3((uint16_t)(va >> 16));
            const float2 w0 = two_e4m3((uint16_t)vw), w1 = two_e4m3((uint16_t)(vw >> 16));
            as[q][r] = a0.x, as[q + 1][r] = a0.y, as[q + 2][r] = a1.x, as[q + 3][r] = a1.y;
            ws[q][r] = w0.x, ws[q + 1][r] = w0.y, ws[q + 2][r] = w1.x, ws[q + 3][r] = w1.y;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[i][j] = fmaf(as[k][ty * 4 + i], ws[k][tx * 4 + j], c[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + ty * 4 + i;
            const float sa = m < p.M ? p.a_scale[(size_t)m * p.KB + b] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                const float sw = n < p.N ? p.w_scale[(size_t)(n / kBlock) * p.KB + b] : 0.f;
                total[i][j] = fmaf(c[i][j], sa * sw, total[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m < p.M && n < p.N) io::st(p.out + (size_t)m * p.N + n, total[i][j]);
        }
    }
}

// A block lays out 128 rows of one block of 128 columns: their largest magnitude, then the values.
template <typename io_t>
__global__ void __launch_bounds__(256) weights_kernel(const io_t *__restrict__ W, uint8_t *__restrict__ w8,
                                                     float *__restrict__ w_scale, int N, int K, int KB)
{
    __shared__ float peaks[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n0 = blockIdx.x * kBlock, k0 = blockIdx.y * kBlock;
    float peak = 0.f;
    for (int i = tid; i < kBlock * kBlock; i += 256) {
        const int n = n0 + i / kBlock, k = k0 + i % kBlock;
        if (n < N && k < K) peak = fmaxf(peak, fabsf(io::ld(W + (size_t)n * K + k)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
    if (lane == 0) peaks[warp] = peak;
    __syncthreads();
    for (int w = 0; w < 8; ++w) peak = fmaxf(peak, peaks[w]);
    const float scale = fmaxf(peak / kMaxE4M3, kMinScale);
    if (tid == 0) w_scale[(size_t)blockIdx.x * KB + blockIdx.y] = scale;
    for (int i = tid; i < kBlock * kBlock; i += 256) {
        const int n = n0 + i / kBlock, k = k0 + i % kBlock;
        if (n >= N || k >= K) continue;
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(io::ld(W + (size_t)n * K + k) / scale));
        w8[(size_t)n * K + k] = (uint8_t)r;
    }
}

template <typename out_t>
cudaError_t product(const Matmul8Args &a, const TokenLaunch &l)
{
    const Params<out_t> p{(const uint8_t *)a.a8, (const uint8_t *)a.w8, a.a_scale, a.w_scale, (out_t *)a.out, a.M, a.N, a.K,
                          (a.K + kBlock - 1) / kBlock};
    l.timer->begin("matmul8");
    product_any_kernel<out_t><<<dim3((a.N + TN - 1) / TN, min((a.M + TM - 1) / TM, 65535)), 256, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace mm8

cudaError_t matmul8(prism_dtype out, const Matmul8Args &a, const TokenLaunch &l)
{
    return out == PRISM_BF16 ? mm8::product<__nv_bfloat16>(a, l) : mm8::product<float>(a, l);
}

cudaError_t matmul8_weights(prism_dtype io, int N, int K, const void *W, void *w8, float *w_scale, const TokenLaunch &l)
{
    const int KB = (K + mm8::kBlock - 1) / mm8::kBlock, NB = (N + mm8::kBlock - 1) / mm8::kBlock;
    l.timer->begin("matmul8_weights");
    if (io == PRISM_BF16)
        mm8::weights_kernel<__nv_bfloat16><<<dim3(NB, KB), 256, 0, l.timer->stream>>>((const __nv_bfloat16 *)W, (uint8_t *)w8, w_scale, N, K, KB);
    else
        mm8::weights_kernel<float><<<dim3(NB, KB), 256, 0, l.timer->stream>>>((const float *)W, (uint8_t *)w8, w_scale, N, K, KB);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace prism
