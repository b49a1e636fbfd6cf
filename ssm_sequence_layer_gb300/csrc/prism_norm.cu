// Root-mean-square norm with the residual's addition, its 8-bit output and its gradient.
//
//   r = x + residual,   q = 1 / sqrt(mean_j r_j^2 + eps),   y_j = r_j q w_j
//   y8 = e4m3(y / s),   s = max(max |y| / 448, 2^-126) over each row's blocks of 128 columns
//   dx = q (w dy - rh mean_j(w_j dy_j rh_j)) + dsum,   rh = r q,   dweight = sum over rows of dy rh
//
// A few operations per value read: HBM bounds both directions.
#include "io_util.h"
#include "prism_tokens.h"

namespace prism {
namespace norm {

constexpr int kThreads = 256;
constexpr int kBlock = 128;  // columns that share a scale
constexpr float kMaxE4M3 = 448.f, kMinScale = 1.17549435e-38f;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// two values to e4m3, round to nearest, the first in the low byte
__device__ __forceinline__ uint16_t e4m3x2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

template <typename io_t>
struct ForwardParams {
    const io_t *x, *residual, *weight;
    io_t *sum, *y;
    uint8_t *y8;
    float *y_scale;
    float eps;
    int n, D;
};

// Any width and alignment: a warp per row, one value per lane at a time, two passes over the row (the
// second one comes from the caches).  Nothing is written before the row has been read to its end, and
// then each value is read before its own place is written, so outputs may take an input's place.
template <typename io_t>
__global__ void __launch_bounds__(kThreads) forward_any_kernel(const ForwardParams<io_t> p)
{
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.n) return;
    const size_t at = (size_t)row * p.D;
    auto sum_at = [&](int c) { return io::ld(p.x + at + c) + (p.residual ? io::ld(p.residual + at + c) : 0.f); };
    float ss = 0.f;
    for (int c = lane; c < p.D; c += 32) {
        const float r = sum_at(c);
        ss = fmaf(r, r, ss);
    }
    const float q = rsqrtf(warp_sum(ss) / (float)p.D + p.eps);
    const int blocks = (p.D + kBlock - 1) / kBlock;
    for (int b = 0; b < blocks; ++b) {
        float y[kBlock / 32], peak = 0.f;
#pragma unroll
        for (int i = 0; i < kBlock / 32; ++i) {
            const int c = b * kBlock + 32 * i + lane;
            y[i] = 0.f;
            if (c < p.D) {
                const float r = sum_at(c);
                y[i] = r * q * io::ld(p.weight + c);
                if (p.sum) io::st(p.sum + at + c, r);
                if (p.y) io::st(p.y + at + c, y[i]);
                peak = fmaxf(peak, fabsf(y[i]));
            }
        }
        if (p.y8) {
            const float scale = fmaxf(warp_max(peak) / kMaxE4M3, kMinScale);
            if (lane == 0) p.y_scale[(size_t)row * blocks + b] = scale;
#pragma unroll
            for (int i = 0; i < kBlock / 32; ++i) {
                const int c = b * kBlock + 32 * i + lane;
                if (c < p.D) p.y8[at + c] = (uint8_t)e4m3x2(y[i] / scale, 0.f);
            }
        }
    }
}

template <typename io_t>
struct BackwardParams {
    const io_t *sum, *weight, *dy, *dsum;
    io_t *dx;
    float2 *stats;  // [n] 1 / rms and mean(w dy rh)
    float *part;  // [slabs][D]
    float *dweight;
    float eps;
    int n, D, slabs;
};

// Per row: q = 1 / rms and mean_j(w dy rh)
template <typename io_t>
__global__ void __launch_bounds__(kThreads) stats_any_kernel(const BackwardParams<io_t> p)
{
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.n) return;
    const size_t at = (size_t)row * p.D;
    float ss = 0.f, along = 0.f;
    for (int c = lane; c < p.D; c += 32) {
        const float r = io::ld(p.sum + at + c);
        ss = fmaf(r, r, ss);
        along = fmaf(io::ld(p.weight + c) * io::ld(p.dy + at + c), r, along);
    }
    const float q = rsqrtf(warp_sum(ss) / (float)p.D + p.eps);
    const float mean = warp_sum(along) * q / (float)p.D;
    if (lane == 0) p.stats[row] = make_float2(q, mean);
}

// dx from the row's statistics; runs after the weight's gradient has read dy, whose place dx may take
template <typename io_t>
__global__ void __launch_bounds__(kThreads) dx_any_kernel(const BackwardParams<io_t> p)
{
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.n) return;
    const size_t at = (size_t)row * p.D;
    const float2 st = p.stats[row];
    for (int c = lane; c < p.D; c += 32) {
        const float rh = io::ld(p.sum + at + c) * st.x;
        float d = st.x * (io::ld(p.weight + c) * io::ld(p.dy + at + c) - rh * st.y);
        if (p.dsum) d += io::ld(p.dsum + at + c);
        io::st(p.dx + at + c, d);
    }
}

// The weight's gradient: a block adds up 32 columns of a slab of rows
template <typename io_t>
__global__ void __launch_bounds__(kThreads) dweight_part_kernel(const BackwardParams<io_t> p)
{
    __shared__ float sums[kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const long long per = ((long long)p.n + p.slabs - 1) / p.slabs, r0 = blockIdx.y * per;
    const long long r1 = min((long long)p.n, r0 + per);
    float acc = 0.f;
    if (c < p.D)
        for (long long r = r0 + warp; r < r1; r += kThreads / 32)
            acc = fmaf(io::ld(p.dy + r * p.D + c), io::ld(p.sum + r * p.D + c) * p.stats[r].x, acc);
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && c < p.D) {
        for (int w = 1; w < kThreads / 32; ++w) acc += sums[w][lane];
        p.part[(size_t)blockIdx.y * p.D + c] = acc;
    }
}

__global__ void __launch_bounds__(kThreads) dweight_kernel(const float *part, float *dweight, int slabs, int D)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= D) return;
    float acc = 0.f;
    for (int s = 0; s < slabs; ++s) acc += part[(size_t)s * D + c];
    dweight[c] = acc;
}

constexpr int kSlabs = 64;

template <typename io_t>
cudaError_t forward(const NormArgs &a, const TokenLaunch &l)
{
    const ForwardParams<io_t> p{(const io_t *)a.x, (const io_t *)a.residual, (const io_t *)a.weight, (io_t *)a.sum,
                                (io_t *)a.y, (uint8_t *)a.y8, a.y_scale, a.eps, a.n, a.D};
    l.timer->begin("norm");
    forward_any_kernel<io_t><<<(a.n + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

template <typename io_t>
cudaError_t backward(const NormBackwardArgs &a, const NormWorkspace &w, const TokenLaunch &l)
{
    const BackwardParams<io_t> p{(const io_t *)a.sum, (const io_t *)a.weight, (const io_t *)a.dy, (const io_t *)a.dsum,
                                 (io_t *)a.dx, w.stats, w.part, a.dweight, a.eps, a.n, a.D, kSlabs};
    cudaStream_t s = l.timer->stream;
    const unsigned rows = (a.n + kThreads / 32 - 1) / (kThreads / 32);
    if (a.n > 0) {
        l.timer->begin("norm_stats");
        stats_any_kernel<io_t><<<rows, kThreads, 0, s>>>(p);
        l.timer->end();
    }
    l.timer->begin("norm_dweight_part");
    dweight_part_kernel<io_t><<<dim3((a.D + 31) / 32, kSlabs), kThreads, 0, s>>>(p);
    l.timer->end();
    if (a.n > 0) {
        l.timer->begin("norm_dx");
        dx_any_kernel<io_t><<<rows, kThreads, 0, s>>>(p);
        l.timer->end();
    }
    l.timer->begin("norm_dweight");
    dweight_kernel<<<(a.D + kThreads - 1) / kThreads, kThreads, 0, s>>>(w.part, a.dweight, kSlabs, a.D);
    l.timer->end();
    return cudaGetLastError();
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace norm

cudaError_t norm_forward(prism_dtype io, const NormArgs &a, const TokenLaunch &l)
{
    return io == PRISM_BF16 ? norm::forward<__nv_bfloat16>(a, l) : norm::forward<float>(a, l);
}

size_t norm_workspace_bytes(int max_rows, int D)
{
    return norm::up256((size_t)max_rows * 8) + norm::up256((size_t)norm::kSlabs * D * 4);
}

void norm_carve(int max_rows, int D, void *base, NormWorkspace *w)
{
    w->stats = (float2 *)base;
    w->part = (float *)((char *)base + norm::up256((size_t)max_rows * 8));
}

cudaError_t norm_backward(prism_dtype io, const NormBackwardArgs &a, const NormWorkspace &w, const TokenLaunch &l)
{
    return io == PRISM_BF16 ? norm::backward<__nv_bfloat16>(a, w, l) : norm::backward<float>(a, w, l);
}

}  // namespace prism
