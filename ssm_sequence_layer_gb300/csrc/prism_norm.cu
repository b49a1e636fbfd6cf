// Root-mean-square norm with the residual's addition, its 8-bit output and its gradient.
//
//   r = x + residual,   q = 1 / sqrt(mean_j r_j^2 + eps),   y_j = r_j q w_j
//   y8 = e4m3(y / s),   s = max(max |y| / 448, 2^-126) over each row's blocks of 128 columns
//   dx = q (w dy - rh mean_j(w_j dy_j rh_j)) + dsum,   rh = r q,   dweight = sum over rows of dy rh
//
// A few operations per value read: HBM bounds both directions.  Sums are fp32 over the unrounded r; outputs are
// rounded once.
#include <type_traits>

#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

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

// 1 / rms as a power of two and a factor in [1, 2).  Rows are multiplied by the power first, which rounds nothing and
// brings them to a size of about one, so that v = (power r) w leaves the range of fp32 only where y = factor v does too.
struct Root {
    float power, factor;
    __device__ __forceinline__ explicit Root(float q)
    {
        const uint32_t b = __float_as_uint(q);
        power = q != q ? q : __uint_as_float(b & 0x7f800000u);  // 0 and infinity stay what they are
        factor = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
    }
};

// The 8-bit values of a block of 128.  A value's e4m3 neighbour is decided by y / scale = v / s with
// s = max |v| / 448, in which 1 / rms cancels.  A rounding error there moves values that lie near the middle between
// two neighbours to the wrong one, so v is held as a product and its rounding error, and the quotient, v times the
// reciprocal of s, is corrected once by the remainder of both, taken with fused operations (P. W. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): what is left are the
// roundings of s and of the result.  (Of 50 million bf16 values the plain sequence of roundings moves 299, this
// one 13.)  Values come in pairs: two operations an instruction.
struct Block {
    float s, inverse;     // max |v| / 448 and its reciprocal
    float factor, scale;  // of the root; the scale that is stored
    // The correction does not apply: s is so small or so large that its reciprocal, a remainder or a product's rounding
    // error is not a normal number, or not a number at all
    bool plain;

    __device__ __forceinline__ Block(float peak, float factor_) : factor(factor_)
    {
        s = peak / kMaxE4M3;
        scale = fmaxf(s * factor, kMinScale);
        plain = !(s >= 0x1p-80f && s <= 0x1p100f);
        inverse = plain ? 1.f / scale : 1.f / s;
    }
    // v and minus its rounding error
    __device__ __forceinline__ float2 quotient(float2 v, float2 minus_low) const
    {
        using namespace io;
        const float2 i2 = make_float2(inverse, inverse), f2 = make_float2(factor, factor);
        if (plain) return mul2(mul2(v, f2), i2);
        const float2 t = mul2(v, i2);
        const float2 rest = fma2(minus_low, make_float2(-1.f, -1.f), fma2(t, make_float2(-s, -s), v));
        return fma2(rest, i2, t);
    }
};
// v = (power r) w, and minus its rounding error
__device__ __forceinline__ float2 product(float2 r, float2 w, float power, float2 &minus_low)
{
    const float2 a = io::mul2(r, make_float2(power, power)), v = io::mul2(a, w);
    minus_low = io::fma2(a, make_float2(-w.x, -w.y), v);
    return v;
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

// Rows of 16-byte units, held in registers: WPR warps per row, UPL units per lane (unit t + 32 WPR j of a row
// belongs to thread t, so a block of 128 columns is the same j of 16 (bf16) or 32 (fp32) neighbouring
// lanes).  Warps walk over the rows; the next row's loads are in flight while a row is worked on, which
// keeps about 60 KB outstanding per SM.  16384 x 768 bf16 with the sum and 8 bits: 18.8 us, 4.7 TB/s (a
// copy of that size reaches about 5; issue slots are 61 % busy); 8192 x 4096 bf16 sum and y 44 us, 6.1 TB/s.
template <typename io_t, int WPR, int UPL>
__global__ void __launch_bounds__(WPR == 1 ? kThreads : 32 * WPR) forward_kernel(const ForwardParams<io_t> p)
{
    constexpr int VEC = 16 / (int)sizeof(io_t), G = 32 * WPR, ROWS = WPR == 1 ? kThreads / 32 : 1;
    constexpr int PER = kBlock / VEC;  // lanes that share a scale
    using U = io::Unit<io_t, VEC>;
    __shared__ float parts[2][WPR];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = WPR == 1 ? lane : (int)threadIdx.x;
    const int units = p.D / VEC, blocks = (p.D + kBlock - 1) / kBlock;
    const long long step = (long long)gridDim.x * ROWS;
    U w[UPL], x[UPL], a[UPL];
    auto load = [&](long long row) {
#pragma unroll
        for (int j = 0; j < UPL; ++j)
            if (t + G * j < units) {
                const size_t at = (size_t)row * p.D + (size_t)(t + G * j) * VEC;
                x[j] = io::load_unit<io_t, VEC>(p.x + at);
                if (p.residual) a[j] = io::load_unit<io_t, VEC>(p.residual + at);
            }
    };
    long long row = (long long)blockIdx.x * ROWS + (WPR == 1 ? warp : 0);
    if (row < p.n) load(row);
#pragma unroll
    for (int j = 0; j < UPL; ++j)
        if (t + G * j < units) w[j] = io::load_unit<io_t, VEC>(p.weight + (size_t)(t + G * j) * VEC);
    for (int turn = 0; row < p.n; row += step, turn ^= 1) {
        float r[UPL][VEC], ss = 0.f;
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[j][e] = 0.f;
            if (t + G * j >= units) continue;
            x[j].get(r[j]);
            if (p.residual) {
                float f[VEC];
                a[j].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) r[j][e] += f[e];
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss = fmaf(r[j][e], r[j][e], ss);
        }
        if (row + step < p.n) load(row + step);
        ss = warp_sum(ss);
        if constexpr (WPR > 1) {
            if (lane == 0) parts[turn][warp] = ss;
            __syncthreads();
            ss = 0.f;
#pragma unroll
            for (int o = 0; o < WPR; ++o) ss += parts[turn][o];
        }
        const Root q(__frsqrt_rn(ss / (float)p.D + p.eps));
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
            const int u = t + G * j;
            const bool mine = u < units;
            const size_t at = (size_t)row * p.D + (size_t)u * VEC;
            float w4[VEC], peak = 0.f;
            float2 v[VEC / 2], low[VEC / 2];  // y without the root's factor, and minus the product's rounding error
#pragma unroll
            for (int e = 0; e < VEC; ++e) w4[e] = 0.f;
            if (mine) w[j].get(w4);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                v[e / 2] = product(make_float2(r[j][e], r[j][e + 1]), make_float2(w4[e], w4[e + 1]), q.power, low[e / 2]);
                peak = fmaxf(peak, fmaxf(fabsf(v[e / 2].x), fabsf(v[e / 2].y)));
            }
            U o;
            if (mine && p.sum) {
                o.set(r[j]);
                io::store_unit<io_t, VEC>(p.sum + at, o);
            }
            if (mine && p.y) {
                float y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; e += 2) y[e] = v[e / 2].x * q.factor, y[e + 1] = v[e / 2].y * q.factor;
                o.set(y);
                io::store_unit<io_t, VEC>(p.y + at, o);
            }
            if (p.y8) {
#pragma unroll
                for (int o2 = PER / 2; o2 > 0; o2 >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o2));
                const Block block(peak, q.factor);
                if (mine) {
                    if (lane % PER == 0) p.y_scale[(size_t)row * blocks + u / PER] = block.scale;
                    uint16_t b[VEC / 2];
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const float2 t = block.quotient(v[e], low[e]);
                        b[e] = e4m3x2(t.x, t.y);
                    }
                    if constexpr (VEC == 8)
                        *reinterpret_cast<uint2 *>(p.y8 + at) = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
                    else
                        *reinterpret_cast<uint32_t *>(p.y8 + at) = b[0] | (uint32_t)b[1] << 16;
                }
            }
        }
    }
}

// Any width and alignment: a warp per row, one value per lane at a time, two passes over the row (the second
// one comes from the caches): 16384 x 770 bf16 33 us, 3.1 TB/s, bound by the instructions that single values take (with the
// row held in registers as much).  Nothing is written before the row has been read to its end, and then each value is read
// before its own place is written, so outputs may take an input's place.
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
    const Root q(__frsqrt_rn(warp_sum(ss) / (float)p.D + p.eps));
    const int blocks = (p.D + kBlock - 1) / kBlock;
    for (int b = 0; b < blocks; ++b) {
        float r[kBlock / 64][2], wt[kBlock / 64][2];  // columns 64 i + lane and 32 further
#pragma unroll
        for (int i = 0; i < kBlock / 64; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = b * kBlock + 64 * i + 32 * h + lane;
                r[i][h] = wt[i][h] = 0.f;
                if (c < p.D) r[i][h] = sum_at(c), wt[i][h] = io::ld(p.weight + c);
            }
        float2 v[kBlock / 64], low[kBlock / 64];
        float peak = 0.f;
#pragma unroll
        for (int i = 0; i < kBlock / 64; ++i) {
            v[i] = product(make_float2(r[i][0], r[i][1]), make_float2(wt[i][0], wt[i][1]), q.power, low[i]);
            peak = fmaxf(peak, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = b * kBlock + 64 * i + 32 * h + lane;
                if (c >= p.D) continue;
                if (p.sum) io::st(p.sum + at + c, r[i][h]);
                if (p.y) io::st(p.y + at + c, (h ? v[i].y : v[i].x) * q.factor);
            }
        }
        if (p.y8) {
            const Block block(warp_max(peak), q.factor);
            if (lane == 0) p.y_scale[(size_t)row * blocks + b] = block.scale;
#pragma unroll
            for (int i = 0; i < kBlock / 64; ++i) {
                const float2 t = block.quotient(v[i], low[i]);
                const uint16_t two = e4m3x2(t.x, t.y);
                const int c = b * kBlock + 64 * i + lane;
                if (c < p.D) p.y8[at + c] = (uint8_t)two;
                if (c + 32 < p.D) p.y8[at + c + 32] = (uint8_t)(two >> 8);
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

// Rows of 16-byte units in registers, as in forward_kernel: one pass gives dx and this block's part of
// the weight's gradient, which each thread holds for its own columns over all rows of the block.  Rows
// that are not made of 16-byte units go through it one value at a time (VEC = 1).  HBM bounds it, with two rows of
// three tensors in flight per warp: 16384 x 768 bf16 21 us and 5 for the join, 16384 x 1024 fp32 47.6 us in all (5.6 TB/s),
// 16384 x 770 bf16 33 us.
template <typename io_t, int WPR, int UPL, int VEC = 16 / (int)sizeof(io_t)>
__global__ void __launch_bounds__(WPR == 1 ? kThreads : 32 * WPR) backward_kernel(const BackwardParams<io_t> p)
{
    constexpr int G = 32 * WPR, ROWS = WPR == 1 ? kThreads / 32 : 1;
    using U = io::Unit<io_t, VEC>;
    __shared__ float2 parts[2][WPR];
    __shared__ float columns[WPR == 1 ? ROWS : 1][WPR == 1 ? G * UPL * VEC : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = WPR == 1 ? lane : (int)threadIdx.x;
    const int units = p.D / VEC;
    const long long step = (long long)gridDim.x * ROWS;
    U w[UPL], x[UPL], a[UPL], b[UPL];
    float acc[UPL][VEC];
    tc::allow_dependent_launch();
    auto load = [&](long long row) {
#pragma unroll
        for (int j = 0; j < UPL; ++j)
            if (t + G * j < units) {
                const size_t at = (size_t)row * p.D + (size_t)(t + G * j) * VEC;
                x[j] = io::load_unit<io_t, VEC>(p.sum + at);
                a[j] = io::load_unit<io_t, VEC>(p.dy + at);
                if (p.dsum) b[j] = io::load_unit<io_t, VEC>(p.dsum + at);
            }
    };
    long long row = (long long)blockIdx.x * ROWS + (WPR == 1 ? warp : 0);
    if (row < p.n) load(row);
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
        if (t + G * j < units) w[j] = io::load_unit<io_t, VEC>(p.weight + (size_t)(t + G * j) * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    }
    for (int turn = 0; row < p.n; row += step, turn ^= 1) {
        float r[UPL][VEC], dy[UPL][VEC];
        U ds[UPL];
        float2 s = make_float2(0.f, 0.f);  // sum r^2, sum w dy r
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
            if (t + G * j >= units) continue;
            x[j].get(r[j]);
            a[j].get(dy[j]);
            ds[j] = b[j];
            float f[VEC];
            w[j].get(f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s.x = fmaf(r[j][e], r[j][e], s.x);
                s.y = fmaf(f[e] * dy[j][e], r[j][e], s.y);
            }
        }
        if (row + step < p.n) load(row + step);
        s.x = warp_sum(s.x);
        s.y = warp_sum(s.y);
        if constexpr (WPR > 1) {
            if (lane == 0) parts[turn][warp] = s;
            __syncthreads();
            s = make_float2(0.f, 0.f);
#pragma unroll
            for (int o = 0; o < WPR; ++o) s.x += parts[turn][o].x, s.y += parts[turn][o].y;
        }
        const float q = __frsqrt_rn(s.x / (float)p.D + p.eps), mean = s.y * q / (float)p.D;
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
            if (t + G * j >= units) continue;
            float f[VEC], d[VEC];
            w[j].get(f);
            if (p.dsum) ds[j].get(d);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float rh = r[j][e] * q;
                acc[j][e] = fmaf(dy[j][e], rh, acc[j][e]);
                const float g = q * (f[e] * dy[j][e] - rh * mean);
                d[e] = p.dsum ? g + d[e] : g;
            }
            U o;
            o.set(d);
            io::store_unit<io_t, VEC>(p.dx + (size_t)row * p.D + (size_t)(t + G * j) * VEC, o);
        }
    }
    float *part = p.part + (size_t)blockIdx.x * p.D;
    if constexpr (WPR == 1) {  // the block's warps add up in order
#pragma unroll
        for (int j = 0; j < UPL; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) columns[warp][(lane + 32 * j) * VEC + e] = acc[j][e];
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int o = 0; o < ROWS; ++o) v += columns[o][c];
            part[c] = v;
        }
    } else {
#pragma unroll
        for (int j = 0; j < UPL; ++j)
            if (t + G * j < units)
#pragma unroll
                for (int e = 0; e < VEC; ++e) part[(size_t)(t + G * j) * VEC + e] = acc[j][e];
    }
}

// Any width and alignment, in three steps.  Per row: q = 1 / rms and mean_j(w dy rh)
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
    const float q = __frsqrt_rn(warp_sum(ss) / (float)p.D + p.eps);
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

// The slabs' parts added up: 32 columns per block, the slabs split over 32 warps and joined in order
constexpr int kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads) dweight_kernel(const float *__restrict__ part, float *dweight, int slabs, int D)
{
    __shared__ float sums[kJoinThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    tc::grid_dependency_wait();
    float acc = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int s = warp; s < slabs; s += kJoinThreads / 32) acc += part[(size_t)s * D + c];
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && c < D) {
        for (int w = 1; w < kJoinThreads / 32; ++w) acc += sums[w][lane];
        dweight[c] = acc;
    }
}

// Blocks of backward_kernel, each with its own part of the weight's gradient: as many as are resident, which takes up
// to 960 blocks of four warps (16384 x 768 fp32: 320 58 us, 640 43 us, 960 41 us), but a part only for rows enough
// (700 x 768 fp32: 320 16.3 us, 700 17.9 us).
constexpr int kSlabs = 320;
constexpr int slabs_max(int D) { return D <= 4096 ? 3 * kSlabs : kSlabs; }
constexpr int kSlabsAny = 64;  // slabs of rows of dweight_part_kernel

// The variant of a width: WPR warps per row and UPL units per lane hold a row of D / VEC units.
// f(WPR, UPL) is called with the smallest that does; false if none does, or rows are not made of units.
// WIDEST: the units per lane of the widest variant (the gradient's registers hold two, the norm's four).
template <int N>
using Int = std::integral_constant<int, N>;
template <int WIDEST, typename F>
bool pick(int D, int vec, F f)
{
    if (D % vec != 0) return false;
    const int units = D / vec;
    if (units <= 32) f(Int<1>(), Int<1>());
    else if (units <= 64) f(Int<1>(), Int<2>());
    else if (units <= 96) f(Int<1>(), Int<3>());
    else if (units <= 128) {
        // the gradient of four units per lane keeps one block per SM (16384 x 512 fp32: 51 us, four warps a row 30 us)
        if constexpr (WIDEST >= 4) f(Int<1>(), Int<4>());
        else f(Int<4>(), Int<1>());
    }
    else if (units <= 256) f(Int<4>(), Int<2>());
    else if (units <= 384) f(Int<4>(), Int<3>());
    else if (units <= 512) f(Int<4>(), Int<4>());
    else if (units <= 1024) f(Int<16>(), Int<2>());
    else {
        if constexpr (WIDEST >= 4) {
            if (units <= 2048) {
                f(Int<16>(), Int<4>());
                return true;
            }
        }
        return false;
    }
    return true;
}

// Blocks of a kernel that walks over the rows: as many as the device holds at a time, no more than rows.
template <auto kernel>
unsigned resident_blocks(int threads, int rows_per_block, int n, int sm_count, int most)
{
    static const int per_sm = [&] {
        int b = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kernel, threads, 0) == cudaSuccess && b > 0 ? b : 1;
    }();
    const long long all = ((long long)n + rows_per_block - 1) / rows_per_block;
    return (unsigned)min(all, min((long long)per_sm * sm_count, (long long)most));
}

template <typename io_t>
cudaError_t forward(const NormArgs &a, const TokenLaunch &l)
{
    const ForwardParams<io_t> p{(const io_t *)a.x, (const io_t *)a.residual, (const io_t *)a.weight, (io_t *)a.sum,
                                (io_t *)a.y, (uint8_t *)a.y8, a.y_scale, a.eps, a.n, a.D};
    l.timer->begin("norm");
    const bool held = pick<4>(a.D, 16 / (int)sizeof(io_t), [&](auto wpr, auto upl) {
        constexpr int WPR = decltype(wpr)::value, UPL = decltype(upl)::value, threads = WPR == 1 ? kThreads : 32 * WPR;
        const unsigned blocks =
            resident_blocks<forward_kernel<io_t, WPR, UPL>>(threads, WPR == 1 ? kThreads / 32 : 1, a.n, l.sm_count, 1 << 30);
        forward_kernel<io_t, WPR, UPL><<<blocks, threads, 0, l.timer->stream>>>(p);
    });
    if (!held) forward_any_kernel<io_t><<<(a.n + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

template <typename io_t>
cudaError_t backward(const NormBackwardArgs &a, const NormWorkspace &w, const TokenLaunch &l)
{
    BackwardParams<io_t> p{(const io_t *)a.sum, (const io_t *)a.weight, (const io_t *)a.dy, (const io_t *)a.dsum,
                           (io_t *)a.dx, w.stats, w.part, a.dweight, a.eps, a.n, a.D, 0};
    cudaStream_t s = l.timer->stream;
    auto go = [&](auto wpr, auto upl, auto vec) {
        constexpr int WPR = decltype(wpr)::value, UPL = decltype(upl)::value, VEC = decltype(vec)::value;
        constexpr int threads = WPR == 1 ? kThreads : 32 * WPR, ROWS = WPR == 1 ? kThreads / 32 : 1;
        const unsigned blocks =
            resident_blocks<backward_kernel<io_t, WPR, UPL, VEC>>(threads, ROWS, a.n, l.sm_count, max(kSlabs, min(slabs_max(a.D), a.n / (4 * ROWS))));
        p.slabs = (int)blocks;
        l.timer->begin("norm_backward");
        backward_kernel<io_t, WPR, UPL, VEC><<<blocks, threads, 0, s>>>(p);
        l.timer->end();
    };
    constexpr int UNIT = 16 / (int)sizeof(io_t);
    bool held = a.n > 0 && pick<2>(a.D, UNIT, [&](auto wpr, auto upl) { go(wpr, upl, Int<UNIT>()); });
    if (!held && a.n > 0 && a.D <= 4096) {  // single values: 8 per thread of one, four or sixteen warps
        if (a.D <= 256) go(Int<1>(), Int<8>(), Int<1>());
        else if (a.D <= 1024) go(Int<4>(), Int<8>(), Int<1>());
        else go(Int<16>(), Int<8>(), Int<1>());
        held = true;
    }
    if (!held && a.n > 0) {
        const unsigned rows = (a.n + kThreads / 32 - 1) / (kThreads / 32);
        p.slabs = min(kSlabsAny, a.n);
        l.timer->begin("norm_stats");
        stats_any_kernel<io_t><<<rows, kThreads, 0, s>>>(p);
        l.timer->end();
        l.timer->begin("norm_dweight_part");
        dweight_part_kernel<io_t><<<dim3((a.D + 31) / 32, p.slabs), kThreads, 0, s>>>(p);
        l.timer->end();
        l.timer->begin("norm_dx");
        dx_any_kernel<io_t><<<rows, kThreads, 0, s>>>(p);
        l.timer->end();
    }
    l.timer->begin("norm_dweight");
    const cudaError_t e = launch_behind(dweight_kernel, dim3((a.D + 31) / 32), kJoinThreads, s, (const float *)w.part, a.dweight, p.slabs, a.D);
    l.timer->end();
    return e == cudaSuccess ? cudaGetLastError() : e;
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace norm

cudaError_t norm_forward(prism_dtype io, const NormArgs &a, const TokenLaunch &l)
{
    return io == PRISM_BF16 ? norm::forward<__nv_bfloat16>(a, l) : norm::forward<float>(a, l);
}

size_t norm_workspace_bytes(int max_rows, int D)
{
    return norm::up256((size_t)max_rows * 8) + norm::up256((size_t)min(norm::slabs_max(D), max_rows) * D * 4);
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
