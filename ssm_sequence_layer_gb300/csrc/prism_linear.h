// The tile kernel of the product with bias, activation and residual and of its gradients: tcgen05 (kind::f16, bf16 operands),
// one output tile of 128 x BN at a time, blocks of 64 in the sum.
//
//   op         A(i, k)          B(j, k)         C(i, j)
//   forward    x[m, k]          W[n, k]         [m, n]   both operands' rows run along the sum (K-major)
//   backward   dy[m, n]         W[n, k]         [m, k]   B's rows run across it (MN-major)
//   weights    dy[m, n]         x[m, k]         [n, k]   both operands' rows run across it
//
// Operands reach shared memory by TMA (bf16 rows whose stride is a multiple of 16 bytes) or through the registers of eight
// warps (SOFT: every other stride, and float32).  A float32 value enters as three bf16 parts, its leading 8 bits, the next 8
// and the last 8, which hold it exactly; of the nine products of parts the six larger ones are summed, so that a product
// is within 2^-21 of itself.
//
// The tensor core cuts its sums off towards zero at each step of 16 terms, which costs long float32 results their last bits (sums over
// 2048 terms in one accumulator: 2 10^-6 off, 256 terms: 3 10^-7, a plain float32 product 2 10^-7).  Where the outputs or the operands
// are float32 an accumulator therefore holds 512 terms at most (256 of float32), and the warps that finish a tile add it to sums in their
// registers while the next ones run into the other accumulator; the five small products of a float32 block have an
// accumulator of their own, whose steps cut off 2^-8 times less.
#pragma once

#include <cudaTypedefs.h>

#include <type_traits>

#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

namespace prism {
namespace lin {

using namespace prism::tc;

// ---- activations ----------------------------------------------------------------------------------
// The values are within 2^-20 of themselves in relative terms wherever they are normal numbers, also where they are tiny; the slopes, each a
// sum of two terms, within 2^-20 of the larger one, so that near their zeros they are no more exact than that.
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

// The same for results that are rounded to bfloat16, two at a time.  R has a polynomial of degree 7 in 1 / (1 + 0.315 a) (2^-21), and the
// exponent's rounding errors are left alone: 2^-20 of the result where |z| < 4, 2^-15 at |z| = 13, where gelu(z) is 10^-37.  Exponentials
// below the smallest normal number are zero, and with them values and slopes below 2^-119 (silu beyond |z| = 87.3, gelu beyond 13.2).
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 exp2_of(float2 y)
{
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
    return e;
}
__device__ __forceinline__ float2 reciprocal(float2 x)
{
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
}
// a = min(|z|, 40), E and -R
__device__ __forceinline__ void gelu_parts(float2 z, float2 &a, float2 &E, float2 &minus_R)
{
    a = make_float2(min_nan(fabsf(z.x), 40.f), min_nan(fabsf(z.y), 40.f));
    E = exp2_of(io::mul2(io::mul2(a, a), both(-0.72134752f)));
    const float2 t = reciprocal(io::fma2(a, both(0.315f), both(1.f)));
    float2 q = io::fma2(t, both(-0.03444384038448334f), both(0.12904778122901917f));
    q = io::fma2(t, q, both(-0.1252608746290207f));
    q = io::fma2(t, q, both(-0.0051743402145802975f));
    q = io::fma2(t, q, both(-0.10147497057914734f));
    q = io::fma2(t, q, both(-0.11121252179145813f));
    q = io::fma2(t, q, both(-0.12581877410411835f));
    q = io::fma2(t, q, both(-0.12566231191158295f));
    minus_R = io::mul2(q, t);
}
__device__ __forceinline__ void silu_parts(float2 z, float2 &a, float2 &e, float2 &r)
{
    a = make_float2(min_nan(fabsf(z.x), 120.f), min_nan(fabsf(z.y), 120.f));
    e = exp2_of(io::mul2(a, both(-1.44269504f)));
    r = reciprocal(io::add2(e, both(1.f)));
}
template <prism_activation ACT>
__device__ __forceinline__ float2 act_value(float2 z)
{
    float2 a, e, r;
    if constexpr (ACT == PRISM_ACT_GELU) {
        gelu_parts(z, a, e, r);
        return io::fma2(io::mul2(a, e), r, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
    } else if constexpr (ACT == PRISM_ACT_SILU) {
        silu_parts(z, a, e, r);
        return io::mul2(r, make_float2(z.x > 0.f ? z.x : -a.x * e.x, z.y > 0.f ? z.y : -a.y * e.y));
    } else {
        return z;
    }
}
template <prism_activation ACT>
__device__ __forceinline__ float2 act_slope(float2 z)
{
    float2 a, e, r;
    if constexpr (ACT == PRISM_ACT_GELU) {
        gelu_parts(z, a, e, r);
        const float2 d = io::mul2(e, io::fma2(a, both(0.39894228f), r));  // minus what the precise form calls d
        return make_float2(z.x > 0.f ? 1.f + d.x : -d.x, z.y > 0.f ? 1.f + d.y : -d.y);
    } else if constexpr (ACT == PRISM_ACT_SILU) {
        silu_parts(z, a, e, r);
        const float2 p = io::mul2(e, r), d = io::mul2(io::mul2(a, p), r);
        return make_float2(z.x > 0.f ? r.x + d.x : p.x - d.x, z.y > 0.f ? r.y + d.y : p.y - d.y);
    } else {
        return both(1.f);
    }
}
// ... of N values, as precise as the type that they go to
template <typename io_t, prism_activation ACT, int N>
__device__ __forceinline__ void to_values(float (&f)[N])
{
    if constexpr (ACT != PRISM_ACT_NONE) {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            if constexpr (sizeof(io_t) == 2) {
                const float2 v = act_value<ACT>(make_float2(f[c], f[c + 1]));
                f[c] = v.x, f[c + 1] = v.y;
            } else {
                f[c] = act_value<ACT>(f[c]), f[c + 1] = act_value<ACT>(f[c + 1]);
            }
        }
    }
}
template <typename io_t, prism_activation ACT, int N>
__device__ __forceinline__ void times_slopes(float (&f)[N], const float (&z)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        if constexpr (sizeof(io_t) == 2) {
            const float2 v = io::mul2(make_float2(f[c], f[c + 1]), act_slope<ACT>(make_float2(z[c], z[c + 1])));
            f[c] = v.x, f[c + 1] = v.y;
        } else {
            f[c] *= act_slope<ACT>(z[c]), f[c + 1] *= act_slope<ACT>(z[c + 1]);
        }
    }
}
template <int N>
__device__ __forceinline__ void plus(float (&f)[N], const float (&g)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 v = io::add2(make_float2(f[c], f[c + 1]), make_float2(g[c], g[c + 1]));
        f[c] = v.x, f[c + 1] = v.y;
    }
}

// ---- the product at hand -----------------------------------------------------------------------------
template <typename io_t>
struct Params {
    const io_t *a, *b;
    long long lda, ldb;  // their row strides
    int I, J, K;         // C is [I, J], the sum runs over K
    prism_activation act;
    const io_t *bias;    // [J]
    const io_t *pre_in;  // [I, J]: C is multiplied by the activation's slope there
    const io_t *add;     // [I, J]
    void *out;           // io, or float32 for the weights' gradient
    io_t *pre_out;
    float *dbias;        // [I]
    int accumulate;
    int tiled;           // the outputs' rows are whole 16-byte units: they leave by TMA
    int splits;          // CTAs of a cluster that share a tile and split the sum
};

struct Waits {
    int *status;
    unsigned long long ns;
};

constexpr int BM = 128, BK = 64;
constexpr int kLoaderWarps = 16;
constexpr uint32_t kPanel = BK * 128;  // an MN-major panel: 64 rows (of the sum) x 64 values

template <typename io_t, LinearOp OP, bool SOFT, int BN, bool PAIR>
struct Layout {
    static constexpr int PARTS = sizeof(io_t) == 4 ? 3 : 1;
    static constexpr bool GROUPED = PARTS == 3 || OP == LinearOp::weights;  // sums go on in registers
    static constexpr uint32_t A_PART = BM * 128, B_PART = ((PAIR ? BN / 2 : BN) + 63) / 64 * 64 * 128, STAGE = PARTS * (A_PART + B_PART);
    // the addends' pieces of a warp, two on their way
    static constexpr bool INCOMING = !SOFT && OP != LinearOp::weights;
    // SOFT: stages' halves are filled and freed one by one; float32 rows of whole units pass the second stage on their way, which has
    // room for three halves
    static constexpr int BLOCK = SOFT ? 32 : BK;
    static constexpr uint32_t RAW = 32768, OFF_RAW = STAGE;
    static_assert(!SOFT || PARTS == 1 || STAGE == 3 * RAW, "halves on their way");
    static constexpr int GROUP = PARTS == 3 ? 256 / BLOCK : 512 / BLOCK;  // blocks that share an accumulator where its sums go on in registers
    static constexpr int STAGES = SOFT ? (PARTS == 3 ? 4 : 8) : (INCOMING && STAGE <= 32768 ? 163840 : 196608) / STAGE - (INCOMING && STAGE > 32768 ? 1 : 0);
    // The warps that finish tiles: each element of an activation takes about 25 instructions one after the other, which two warps a
    // scheduler do not hide; where the sums go on in registers there is room for eight.
    static constexpr int FINISHERS = INCOMING ? 16 : 8, FINISHED = BN / (FINISHERS / 4);  // and a warp's columns
    static constexpr uint32_t OUT_WARP = 4096;  // a warp's staging: outputs of 32 x 32 values of 4 bytes, or two times 2 bytes, the second for addends
    static constexpr uint32_t OFF_OUT = SOFT ? STAGES / 2 * STAGE : STAGES * STAGE;
    static constexpr uint32_t SMEM = OFF_OUT + (OP == LinearOp::weights ? 2048 : FINISHERS * OUT_WARP) + 1024;  // + alignment slack
    static constexpr int THREADS = 128 + 32 * FINISHERS + (SOFT ? 32 * kLoaderWarps : 0);
    static constexpr int kColumns = 512;  // of tensor memory: two accumulators, and two for the small products or the sums over rows
    static constexpr int SUMS = OP == LinearOp::weights && !SOFT && 2 * BN + 32 <= kColumns ? 2 * BN : 0;
    // registers handed over to the warps that finish tiles, from the issuing ones
    static constexpr int kLaunchRegs = SOFT ? 72 : INCOMING ? 96 : 168, kIssueRegs = SOFT || INCOMING ? 40 : 56,
                         kEpilogueRegs = SOFT ? 136 : INCOMING ? 104 : 224, kLoaderRegs = 48;
    static_assert(128 * kIssueRegs + 32 * FINISHERS * kEpilogueRegs + (SOFT ? 32 * kLoaderWarps * kLoaderRegs : 0) <= THREADS * kLaunchRegs, "registers");
    static_assert(STAGES >= 2 && SMEM + (OP == LinearOp::weights && SOFT ? 9216 : 1024) <= 232448 && OFF_OUT % 1024 == 0, "layout");
};

// one look at a barrier's phase
__device__ __forceinline__ bool mbar_test(uint32_t mbar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(mbar), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return io::Unit<__nv_bfloat16, 8>::pack(a, b); }
// the leading halves of two floats, the first in the low half
__device__ __forceinline__ uint32_t leading(float a, float b)
{
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float without_leading(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); }

// ---- operands through registers ------------------------------------------------------------------------
// Half a stage of an operand: R rows x C values of a row-major matrix (128 x 32 along the sum, or 32 x 128 across it), cut to (rows, cols);
// what lies outside is zero.  A thread has eight of its values in registers and stores them, in the form that the tensor core reads, when
// their place is free.  Rows that are whole units of four values come four at a time.  Others come as segments, one value a lane and 32
// neighbours of a row at once, whatever their alignment; lanes then trade values with their neighbours so that each has two of one row.
// Either way the two rows that half a warp stores to at once are four apart (or lie across the sum), so that their swizzled halves fill
// all banks.
// float32 rows of whole units pass through shared memory of the thread's own, two halves ahead (cp.async of 16 bytes); others are loaded
// into the registers as soon as these are free.  Microseconds of 4096 x 4096 x 4096 (float32) and 4096 x 4095 x 4097 (float32, bfloat16),
// forward / dx / dW:
//   this                                                  1064 / 1138 / 1054    1320 / 1668 / 1087     872 / 921 / 818
//   all rows straight into registers                      1343 / 1335 / 994     1674 / 1587 / 1216
//   all by cp.async, of 4 bytes where rows are not whole  1063 / 1215 / 1142    1387 / 1557 / 1633    1282 / 1405 / 1365
// What bounds it is shared memory: of about 2300 cycles a half of float32, the products' operands take 770 and the values' ways 900.
template <typename io_t, bool MN>
struct SoftHalf {
    static constexpr int STEP = 32 * kLoaderWarps / (MN ? 32 : 8);  // rows between a thread's two groups of four
    const io_t *base;
    long long ld;
    int rows, cols, warp, lane;
    bool whole;
    __device__ __forceinline__ SoftHalf(const io_t *base_, long long ld_, int rows_, int cols_, int thread)
        : base(base_), ld(ld_), rows(rows_), cols(cols_), warp(thread >> 5), lane(thread & 31), whole(ld_ % 4 == 0)
    {
    }
    // the thread's first value in the half
    __device__ __forceinline__ int own_row() const
    {
        if (whole) return MN ? warp : (warp >> 1) * 8 + (lane >> 3 & 1) * 4 + (warp & 1) * 2 + (lane >> 4);
        return MN ? (warp & 3) + 8 * (warp >> 2) : 8 * warp;
    }
    __device__ __forceinline__ int own_column() const { return whole ? 4 * (MN ? lane : lane & 7) : lane; }
    // the half that is asked for or loaded next: its block of the sum, its tile, its first row and column in the matrix and the place of
    // the thread's first value
    int block, tile, row0, col0;
    const io_t *at;
    __device__ __forceinline__ void seek(int r0, int c0)
    {
        row0 = r0, col0 = c0;
        at = base + (long long)(r0 + own_row()) * ld + c0 + own_column();
    }
    __device__ __forceinline__ void advance()  // by a half along the sum
    {
        if constexpr (MN) row0 += 32, at += 32 * ld;
        else col0 += 32, at += 32;
    }
    __device__ __forceinline__ bool has(int r, int c) const { return row0 + own_row() + r < rows && col0 + own_column() + c < cols; }
    struct Words {
        uint32_t x[8];
    };
    // straight into registers
    __device__ __forceinline__ void load(Words &w) const
    {
        if (whole) {  // bfloat16
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint2 u = has(i * STEP, 0) ? *reinterpret_cast<const uint2 *>(at + i * STEP * ld) : make_uint2(0, 0);
                w.x[2 * i] = u.x, w.x[2 * i + 1] = u.y;
            }
        } else if (row0 + (MN ? 32 : 128) <= rows && col0 + (MN ? 128 : 32) <= cols) {
            single(w, [&](int, int) { return true; });
        } else {
            single(w, [&](int r, int c) { return has(r, c); });
        }
    }
    template <typename F>
    __device__ __forceinline__ void single(Words &w, F in) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = MN ? 4 * h : j + 4 * h, c = MN ? 32 * j : 0;
                const io_t *p = at + r * ld + c;
                uint32_t x = 0;
                if (in(r, c)) {
                    if constexpr (sizeof(io_t) == 4) x = *reinterpret_cast<const uint32_t *>(p);
                    else x = *reinterpret_cast<const uint16_t *>(p);
                }
                w.x[2 * j + h] = x;
            }
    }
    // float32 in whole units: into shared memory, a thread's values side by side, and from there into registers
    __device__ __forceinline__ uint32_t group_at(uint32_t raw, int i) const { return raw + (32 * kLoaderWarps * i + 32 * warp + lane) * 16; }
    __device__ __forceinline__ void ask(uint32_t raw) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = has(i * STEP, 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(group_at(raw, i)), "l"(in ? at + i * STEP * ld : base), "r"(in ? 16 : 0) : "memory");
        }
    }
    __device__ __forceinline__ void fetch(uint32_t raw, Words &w) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x[4 * i]), "=r"(w.x[4 * i + 1]), "=r"(w.x[4 * i + 2]), "=r"(w.x[4 * i + 3])
                         : "r"(group_at(raw, i)));
    }
    // N values of one row, or their parts, part_bytes apart
    template <int N>
    static __device__ __forceinline__ void store_parts(uint8_t *at, uint32_t part_bytes, float (&f)[N])
    {
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            if constexpr (N == 4) *reinterpret_cast<uint2 *>(at + part * part_bytes) = make_uint2(leading(f[0], f[1]), leading(f[2], f[3]));
            else *reinterpret_cast<uint32_t *>(at + part * part_bytes) = leading(f[0], f[1]);
            if (part < 2) {
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] = without_leading(f[e]);
            }
        }
    }
    static __device__ __forceinline__ uint8_t *place(uint8_t *to, int r, int c, int half)
    {
        return MN ? to + (c >> 6) * kPanel + sw128(r + 32 * half, c & 63) : to + sw128(r, c + 32 * half);
    }
    // into half `half` of panels of 64 values, 128-byte swizzled.  sums: of the thread's columns
    __device__ __forceinline__ void bring(uint8_t *to, uint32_t part_bytes, const Words &w, int half, bool add, float (&sums)[4]) const
    {
        const uint32_t(&x)[8] = w.x;
        if (whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint8_t *at = place(to, own_row() + i * STEP, own_column(), half);
                float f[4];
                if constexpr (sizeof(io_t) == 4) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(x[4 * i + e]);
                } else {
                    *reinterpret_cast<uint2 *>(at) = make_uint2(x[2 * i], x[2 * i + 1]);
                    io::Unit<__nv_bfloat16, 8>::two(x[2 * i], f[0], f[1]), io::Unit<__nv_bfloat16, 8>::two(x[2 * i + 1], f[2], f[3]);
                }
                if (add) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sums[e] += f[e];
                }
                if constexpr (sizeof(io_t) == 4) store_parts(at, part_bytes, f);
            }
            return;
        }
        const bool odd = lane & 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = x[2 * j], b = x[2 * j + 1];  // of two rows
            if (add) {
                if constexpr (sizeof(io_t) == 4) sums[j] += __uint_as_float(a) + __uint_as_float(b);
                else sums[j] += __uint_as_float(a << 16) + __uint_as_float(b << 16);
            }
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1), first = odd ? other : a, second = odd ? b : other;
            uint8_t *at = place(to, own_row() + (MN ? 0 : j) + (odd ? 4 : 0), (MN ? 32 * j : 0) + (lane & 30), half);
            if constexpr (sizeof(io_t) == 4) {
                float f[2] = {__uint_as_float(first), __uint_as_float(second)};
                store_parts(at, part_bytes, f);
            } else {
                *reinterpret_cast<uint32_t *>(at) = first | second << 16;
            }
        }
    }
    // the column of the half that sums[e] belong to
    __device__ __forceinline__ int column_of(int e) const { return whole ? own_column() + e : own_column() + 32 * e; }
};

// ---- outputs --------------------------------------------------------------------------------------------
// 32 lanes x 32 columns of an accumulator; the values may be used after ld_wait, which takes them as operands
__device__ __forceinline__ void ld_issue(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// waits for the loads so far and takes 16 values as operands
__device__ __forceinline__ void wait16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

template <typename F>
__device__ __forceinline__ void with_activation(prism_activation act, F f)
{
    if (act == PRISM_ACT_GELU) f(std::integral_constant<prism_activation, PRISM_ACT_GELU>());
    else if (act == PRISM_ACT_SILU) f(std::integral_constant<prism_activation, PRISM_ACT_SILU>());
    else f(std::integral_constant<prism_activation, PRISM_ACT_NONE>());
}

// N values of a row as they lie in memory, two at a time
template <typename T, int N = 32>
struct Held {
    uint32_t w[N * sizeof(T) / 4];
    __device__ __forceinline__ float2 pair(int i) const
    {
        float2 v;
        if constexpr (sizeof(T) == 2) io::Unit<__nv_bfloat16, 8>::two(w[i], v.x, v.y);
        else v = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        return v;
    }
    __device__ __forceinline__ void unit(int u, uint4 x) { w[4 * u] = x.x, w[4 * u + 1] = x.y, w[4 * u + 2] = x.z, w[4 * u + 3] = x.w; }
    __device__ __forceinline__ void set(const float (&f)[N])
    {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (sizeof(T) == 2) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
            else w[2 * i] = __float_as_uint(f[2 * i]), w[2 * i + 1] = __float_as_uint(f[2 * i + 1]);
        }
    }
    // of a row's values from `at` on; beyond `cols` zeros.  whole: rows are whole 16-byte units and at is one's start
    __device__ __forceinline__ void load(const T *p, int at, int cols, bool whole)
    {
        if (whole && at + N <= cols) {
#pragma unroll
            for (int u = 0; u < N * (int)sizeof(T) / 16; ++u) unit(u, reinterpret_cast<const uint4 *>(p + at)[u]);
            return;
        }
        float f[N];
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = at + e < cols ? io::ld(p + at + e) : 0.f;
        set(f);
    }
};
template <typename io_t, prism_activation ACT, typename T, int N>
__device__ __forceinline__ void times_slopes(float (&f)[N], const Held<T, N> &z)
{
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 x = z.pair(c / 2);
        if constexpr (sizeof(io_t) == 2) {
            const float2 v = io::mul2(make_float2(f[c], f[c + 1]), act_slope<ACT>(x));
            f[c] = v.x, f[c + 1] = v.y;
        } else {
            f[c] *= act_slope<ACT>(x.x), f[c + 1] *= act_slope<ACT>(x.y);
        }
    }
}
template <typename T, int N>
__device__ __forceinline__ void plus(float (&f)[N], const Held<T, N> &g)
{
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 v = io::add2(make_float2(f[c], f[c + 1]), g.pair(c / 2));
        f[c] = v.x, f[c + 1] = v.y;
    }
}

// A warp's 32 rows x 32 columns of an output or an addend: lane l holds row l.
template <typename T>
struct Patch {
    // rows that are not whole units come and go through shared memory, a row by all lanes
    static __device__ __forceinline__ void get(const T *p, int J, int rows, int j0, bool whole, float *t, int lane, Held<T> &held)
    {
        if (whole) {
            held.load(p + (size_t)min(lane, rows - 1) * J, j0, J, true);
            return;
        }
        __syncwarp();
#pragma unroll 8
        for (int r = 0; r < 32; ++r) t[r * 32 + (lane ^ r)] = r < rows && j0 + lane < J ? io::ld(p + (size_t)r * J + j0 + lane) : 0.f;
        __syncwarp();
        float f[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) f[c] = t[lane * 32 + (c ^ lane)];
        held.set(f);
    }
    static __device__ __forceinline__ void put_rows(T *p, int J, int rows, int j0, float *t, int lane, const float (&f)[32])
    {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c) t[lane * 32 + (c ^ lane)] = f[c];
        __syncwarp();
        if (j0 + lane >= J) return;
        T *to = p + j0 + lane;
        if (rows == 32) {  // eight rows' loads before their stores
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {
                float g[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) g[r] = t[(r0 + r) * 32 + (lane ^ (r0 + r))];
#pragma unroll
                for (int r = 0; r < 8; ++r, to += J) io::st(to, g[r]);
            }
        } else {
            for (int r = 0; r < rows; ++r, to += J) io::st(to, t[r * 32 + (lane ^ r)]);
        }
    }
    // 16 columns of this lane's row of a bf16 piece
    static __device__ __forceinline__ uint4 *unit_of(uint8_t *piece, int lane, int u) { return reinterpret_cast<uint4 *>(piece + lane * 64 + ((u ^ (lane >> 1 & 3)) << 4)); }
    static __device__ __forceinline__ void get_half(uint8_t *piece, int lane, int half, Held<T, 16> &held)
    {
        if constexpr (sizeof(T) == 2) held.unit(0, *unit_of(piece, lane, 2 * half)), held.unit(1, *unit_of(piece, lane, 2 * half + 1));
    }
    static __device__ __forceinline__ void put_half(uint8_t *piece, int lane, int half, const float (&f)[16])
    {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float g[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = f[8 * u + e];
                io::Unit<T, 8> x;
                x.set(g);
                *unit_of(piece, lane, 2 * half + u) = x.w;
            }
        }
    }
    // float32 by TMA: a piece of 32 rows x 32 columns, 128-byte swizzled
    static __device__ __forceinline__ void put_tiled(const CUtensorMap *tm, uint8_t *stage, int row0, int j0, int lane, const float (&f)[32])
    {
        if constexpr (sizeof(T) == 4) {
            bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u)
                *reinterpret_cast<float4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(tm, smem_u32(stage), j0, row0);
                bulk_commit();
            }
        }
    }
};

// one lane of a warp, the same each time
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// a shared-memory address of this CTA in another of the cluster
__device__ __forceinline__ uint32_t address_in(uint32_t addr, uint32_t cta)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
    return a;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void store_at(uint32_t remote, uint32_t v)
{
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}
__device__ __forceinline__ void store_at(uint32_t remote, unsigned long long v)
{
    asm volatile("st.relaxed.cluster.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t remote)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// ---- two CTAs at one tile ----
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
}
__device__ __forceinline__ void mma_commit_pair(uint32_t mbar, uint16_t ctas)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(mbar), "h"(ctas)
                 : "memory");
}
// into this CTA's shared memory, counted by a barrier of either CTA
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t mbar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(mbar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
template <typename V>
__device__ __forceinline__ V remote(uint32_t addr, int cta);
template <>
__device__ __forceinline__ float4 remote<float4>(uint32_t addr, int cta)
{
    uint32_t a;
    float4 x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
    return x;
}
template <>
__device__ __forceinline__ float remote<float>(uint32_t addr, int cta)
{
    uint32_t a;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
    return x;
}

// PAIR: two CTAs of neighbouring SMs share a tile of 256 rows (tcgen05 cta_group::2): each brings in and finishes its own 128 rows
// and brings in half of B, which both read, so that a block's operands are 32 KB an SM and not 48.  One thread of the first CTA issues the
// products of both; its barriers count the loads of both, and every completion of products arrives in both.
// SPLIT: one tile a cluster, whose CTAs (or pairs) split the sum (or one does it all).  Their sums meet in shared memory, where the operands
// were, and each CTA finishes a share of the rows, always adding in the cluster's order.
// Otherwise persistent: the next tile's products run into the other of two accumulators while this one is finished.
template <typename io_t, LinearOp OP, bool SOFT, int BN, bool SPLIT, bool PAIR>
__global__ void __launch_bounds__(Layout<io_t, OP, SOFT, BN, PAIR>::THREADS, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_out,
                const __grid_constant__ CUtensorMap tm_pre, const __grid_constant__ CUtensorMap tm_add, const Params<io_t> p, const Waits wt)
{
    using L = Layout<io_t, OP, SOFT, BN, PAIR>;
    using out_t = std::conditional_t<OP == LinearOp::weights, float, io_t>;
    constexpr int STAGES = L::STAGES, COLS = L::FINISHED, PARTS = L::PARTS;
    constexpr bool A_MN = OP == LinearOp::weights, B_MN = OP != LinearOp::forward, GROUPED = L::GROUPED;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint32_t tmem_base_s;
    __shared__ __align__(8) uint64_t full[STAGES], freed[STAGES], acc_full[2], acc_empty[2], incoming[L::FINISHERS];
    __shared__ int abort_s;
    __shared__ unsigned long long other_issued, products_s;  // after an expired wait: the loads of a pair's other CTA, the products issued
    __shared__ uint32_t accumulators_s;                       // ... and the accumulators that they have completed
    __shared__ __align__(16) float column_sums[OP == LinearOp::weights && SOFT ? kLoaderWarps : 1][OP == LinearOp::weights ? BM : 1];
    constexpr int CTAS = PAIR ? 2 : 1, TM = CTAS * BM;  // of a tile, and its rows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int in_tile = PAIR ? (int)(blockIdx.x & 1) : 0;  // the cluster's CTAs are numbered as the grid's
    const bool leads = in_tile == 0;
    const int tiles_i = (p.I + TM - 1) / TM, tiles_j = (p.J + BN - 1) / BN, blocks = (p.K + L::BLOCK - 1) / L::BLOCK;
    const long long tiles = (long long)tiles_i * tiles_j;
    const unsigned worker = blockIdx.x / CTAS, workers = gridDim.x / CTAS;
    const int my_tiles = SPLIT ? 1 : tiles > worker ? (int)((tiles - 1 - worker) / workers) + 1 : 0;
    const int rank = SPLIT ? (int)(worker % p.splits) : 0;
    const int b_from = SPLIT ? (int)((long long)rank * blocks / p.splits) : 0, b_to = SPLIT ? (int)((long long)(rank + 1) * blocks / p.splits) : blocks;
    const long long total = (long long)my_tiles * (b_to - b_from);
    const int groups = GROUPED ? (b_to - b_from + L::GROUP - 1) / L::GROUP : 1;  // of a tile's blocks, an accumulator each
    const int stages = SOFT && PARTS == 3 && (p.lda % 4 == 0 || p.ldb % 4 == 0) ? 2 : STAGES;
    const uint32_t sbase = smem_u32(sm), crank = PAIR ? cluster_rank() : 0;
    const uint32_t leader_full = PAIR ? address_in(smem_u32(&full[0]), crank & ~1) : smem_u32(&full[0]);

    // tiles of one column of tiles run at the same time on neighbouring CTAs and share B in L2
    auto tile_at = [&](int i, int &i0, int &j0) {
        const long long t = SPLIT ? (long long)(worker / p.splits) : (long long)worker + (long long)i * workers;
        i0 = (int)(t % tiles_i) * TM + in_tile * BM;
        j0 = (int)(t / tiles_i) * BN;
    };
    // the sums over dy's rows: products with ones, 16 columns beside a group's accumulator, or the loaders' registers
    bool sums = false;
    if constexpr (OP == LinearOp::weights) {
        int i0, j0;
        tile_at(0, i0, j0);
        sums = p.dbias && j0 == 0;
    }
    auto load_block = [&](int s, int b, int i0, int j0) {
        const uint32_t at = sbase + s * L::STAGE, mb = leader_full + 8 * s;
        if (leads) mbar_expect_tx(smem_u32(&full[s]), CTAS * L::STAGE);
        auto box = [&](uint32_t to, const CUtensorMap *map, int c0, int c1) {
            if constexpr (PAIR) tma_load_2d_pair(to, map, mb, c0, c1);
            else tma_load_2d(to, map, mb, c0, c1);
        };
        constexpr int OWN = BN / CTAS;  // B's rows (columns) that this CTA brings in
        j0 += in_tile * OWN;
        if constexpr (A_MN) {
#pragma unroll
            for (int h = 0; h < BM / 64; ++h) box(at + h * kPanel, &tm_a, i0 + 64 * h, b * BK);
        } else {
            box(at, &tm_a, b * BK, i0);
        }
        if constexpr (B_MN) {
#pragma unroll
            for (int h = 0; h < (OWN + 63) / 64; ++h) box(at + L::A_PART + h * kPanel, &tm_b, j0 + 64 * h, b * BK);
        } else {
#pragma unroll
            for (int h = 0; h < OWN / 128; ++h) box(at + L::A_PART + h * 16384, &tm_b, b * BK, j0 + 128 * h);
        }
    };
    // on their way while the tensor memory is allocated; a pair's barriers have to stand first
    const int early = !SOFT && !PAIR && my_tiles > 0 ? min(stages, b_to - b_from) : 0;
    if (tid == 32) {
        abort_s = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&full[s]), SOFT ? kLoaderWarps : 1);
            mbar_init(smem_u32(&freed[s]), 1);
        }
        for (int w = 0; w < L::FINISHERS; ++w) mbar_init(smem_u32(&incoming[w]), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&acc_full[s]), 1);
            mbar_init(smem_u32(&acc_empty[s]), CTAS * L::FINISHERS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        if constexpr (!SOFT && !PAIR) {
            int i0, j0;
            tile_at(0, i0, j0);
            for (int s = 0; s < early; ++s) load_block(s, b_from + s, i0, j0);
        }
        if (!SPLIT && p.tiled) prefetch_tmap(&tm_out);
    }
    if (L::SUMS > 0 && warp >= 4 && warp < 8) {  // 16 rows of ones (8 would do where two CTAs bring in half each)
        *reinterpret_cast<uint4 *>(sm + L::OFF_OUT + (tid - 128) * 16) = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        fence_async_smem();
    }
    if (warp == 0) {
        if constexpr (PAIR) tmem_alloc_pair(smem_u32(&tmem_base_s), L::kColumns);
        else tmem_alloc(smem_u32(&tmem_base_s), L::kColumns);
    }
    fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_barrier();
    fence_after_sync();
    const uint32_t tmem = tmem_base_s;

    auto give_up = [&] {
        atomicCAS(wt.status, 0, kDevTimeout);
        if constexpr (PAIR) {  // all of the cluster drain together
            for (uint32_t c = 0; c < cluster_size(); ++c) store_at(address_in(smem_u32(&abort_s), c), 1u);
        } else {
            *(volatile int *)&abort_s = 1;
        }
    };
    long long issued = 0;  // the issuing threads' counts of steps and of accumulators filled, also for the drain
    uint32_t accumulators = 0;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kIssueRegs));
        // Whole warps run these loops, so that their counters and descriptors stay in uniform registers, and one lane issues.  Each
        // looks at its next barrier while it issues: shared memory, busy with operands, takes some hundred cycles to answer
        // (4096 x 4096 x 4096 took 108 us with one thread a loop and two looks between a block's products and the next).
        if (!SOFT && warp == 1) {  // ---- operand loads ----
            const bool one = elect_one();
            int s = early % stages, i = b_from + early == b_to ? 1 : 0, b = i > 0 ? b_from : b_from + early, i0 = 0, j0 = 0;
            uint32_t round = early / stages;
            bool ready = false;
            issued = early;
            tile_at(0, i0, j0);
            for (long long g = early; g < total; ++g) {
                if (b == b_from) tile_at(i, i0, j0);
                if (round > 0 && !ready) {
                    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&freed[s]), (round - 1) & 1, wt.ns))) {
                        if (one) give_up();
                        break;
                    }
                }
                if (s == 0 && __any_sync(0xffffffffu, *(volatile int *)&abort_s)) break;
                const int next = s + 1 == stages ? 0 : s + 1;
                const uint32_t next_round = s + 1 == stages ? round + 1 : round;
                const bool seen = next_round > 0 && mbar_test(smem_u32(&freed[next]), (next_round - 1) & 1);
                if (one) load_block(s, b, i0, j0);
                __syncwarp();
                ready = __all_sync(0xffffffffu, seen);
                issued = g + 1;
                s = next, round = next_round;
                if (++b == b_to) b = b_from, ++i;
            }
        } else if (warp == 0 && leads) {  // ---- products ----
            const bool one = elect_one();
            int s = 0;
            uint32_t round = 0;
            auto product = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t more) {
                if constexpr (PAIR) mma_f16_pair(d, a, b, id, more);
                else mma_f16(d, a, b, id, more);
            };
            auto done = [&](uint64_t *barrier) {  // arrives once the products so far are complete, in both CTAs of a pair
                if constexpr (PAIR) mma_commit_pair(smem_u32(barrier), (uint16_t)(3u << (crank & ~1u)));
                else mma_commit(smem_u32(barrier));
            };
            bool ok = true, ready = false;
            for (int i = 0; i < my_tiles && ok; ++i) {
                for (int b = b_from; b < b_to; ++b) {
                    const int in_group = GROUPED ? (b - b_from) % L::GROUP : b - b_from;
                    const uint32_t buf = accumulators & 1;
                    if (in_group == 0 && accumulators >= 2) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_empty[buf]), ((accumulators - 2) >> 1) & 1, wt.ns));
                    if (ok && !ready) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), round & 1, wt.ns));
                    if (!ok) {
                        if (one) give_up();
                        break;
                    }
                    fence_after_sync();
                    const int next = s + 1 == stages ? 0 : s + 1;
                    const uint32_t next_round = s + 1 == stages ? round + 1 : round;
                    const bool seen = mbar_test(smem_u32(&full[next]), next_round & 1);
                    const uint32_t at = sbase + (SOFT ? s >> 1 : s) * L::STAGE, bt = at + PARTS * L::A_PART, d = tmem + buf * BN;
                    const uint64_t da = A_MN ? sdesc(at, kPanel, 1024) : sdesc(at, 16, 1024), db = B_MN ? sdesc(bt, kPanel, 1024) : sdesc(bt, 16, 1024);
                    constexpr uint64_t SA = (A_MN ? 2048 : 32) >> 4, SB = (B_MN ? 2048 : 32) >> 4;
                    constexpr uint32_t ID = idesc_bf16(TM, BN, A_MN, B_MN);
                    const uint32_t small = tmem + 2 * BN + (i & 1) * BN;  // the small products' accumulator, for the whole tile
                    const int from_k = SOFT ? (s & 1) * L::BLOCK / 16 : 0;  // the half of the stage
                    const bool last = b + 1 == b_to || (GROUPED && in_group + 1 == L::GROUP);
                    if (one) {
#pragma unroll
                        for (int pa = 0; pa < PARTS; ++pa)
#pragma unroll
                            for (int pb = 0; pa + pb < PARTS; ++pb)
#pragma unroll
                                for (int k = 0; k < L::BLOCK / 16; ++k)
                                    product(pa + pb == 0 ? d : small, da + (uint64_t)(pa * L::A_PART >> 4) + SA * (k + from_k),
                                            db + (uint64_t)(pb * L::B_PART >> 4) + SB * (k + from_k), ID, pa + pb == 0 ? in_group > 0 || k > 0 : b > b_from || pa > 0 || pb > 1 || k > 0);
                        if constexpr (OP == LinearOp::weights && !SOFT && L::SUMS > 0) {
                            if (sums) {
                                const uint64_t ones = sdesc(sbase + L::OFF_OUT, 16, 1024);
#pragma unroll
                                for (int k = 0; k < BK / 16; ++k)
                                    product(tmem + L::SUMS + 16 * buf, da + SA * k, ones + 2 * k, idesc_bf16(TM, 16, A_MN, 0), in_group > 0 || k > 0);
                            }
                        }
                        done(&freed[s]);
                        if (last) done(&acc_full[buf]);
                    }
                    __syncwarp();
                    ready = __all_sync(0xffffffffu, seen);
                    if (last) ++accumulators;
                    ++issued;
                    s = next, round = next_round;
                }
            }
        }
    } else if (SOFT && warp >= 4 + L::FINISHERS) {  // ---- operands through registers ----
        if constexpr (SOFT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLoaderRegs));
        const int thread = tid - 128 - 32 * L::FINISHERS;
        // rows and columns of the matrices in memory: the sum runs along a row (K-major) or from row to row
        SoftHalf<io_t, A_MN> ta(p.a, p.lda, A_MN ? p.K : p.I, A_MN ? p.I : p.K, thread);
        SoftHalf<io_t, B_MN> tb(p.b, p.ldb, B_MN ? p.K : p.J, B_MN ? p.J : p.K, thread);
        float column[4] = {}, unused[4];
        auto seek_a = [&] {
            int i0, j0;
            tile_at(ta.tile, i0, j0);
            ta.seek(A_MN ? ta.block * L::BLOCK : i0, A_MN ? i0 : ta.block * L::BLOCK);
        };
        auto seek_b = [&] {
            int i0, j0;
            tile_at(tb.tile, i0, j0);
            tb.seek(B_MN ? tb.block * L::BLOCK : j0, B_MN ? j0 : tb.block * L::BLOCK);
        };
        auto step = [&](auto &t, auto seek) {
            t.advance();
            if (++t.block == b_to) {
                t.block = b_from;
                if (++t.tile < my_tiles) seek();
            }
        };
        ta.block = tb.block = b_from, ta.tile = tb.tile = 0;
        seek_a(), seek_b();
        typename SoftHalf<io_t, A_MN>::Words wa;
        typename SoftHalf<io_t, B_MN>::Words wb;
        // float32 rows of whole units are asked for two halves ahead, others loaded when the registers are free
        const bool ask_a = PARTS == 3 && ta.whole, ask_b = PARTS == 3 && tb.whole;
        auto ask = [&](long long g) {
            if constexpr (PARTS == 3) {
                if (g < total) {
                    const uint32_t raw = sbase + L::OFF_RAW + (uint32_t)(g % 3) * L::RAW;
                    if (ask_a) ta.ask(raw), step(ta, seek_a);
                    if (ask_b) tb.ask(raw + L::RAW / 2), step(tb, seek_b);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        };
        if (ask_a || ask_b) ask(0), ask(1);
        if (total > 0 && !ask_a) ta.load(wa), step(ta, seek_a);
        if (total > 0 && !ask_b) tb.load(wb), step(tb, seek_b);
        int s = 0;
        uint32_t round = 0;
        for (long long g = 0; g < total; ++g) {
            if (ask_a || ask_b) {
                ask(g + 2);
                asm volatile("cp.async.wait_group 2;" ::: "memory");
                const uint32_t raw = sbase + L::OFF_RAW + (uint32_t)(g % 3) * L::RAW;
                if (ask_a) ta.fetch(raw, wa);  // on their way while the half is waited for
                if (ask_b) tb.fetch(raw + L::RAW / 2, wb);
            }
            const bool ok = round == 0 || mbar_wait(smem_u32(&freed[s]), (round - 1) & 1, wt.ns);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            uint8_t *to = sm + (s >> 1) * L::STAGE;
            ta.bring(to, L::A_PART, wa, s & 1, sums, column);
            if (!ask_a && g + 1 < total) ta.load(wa), step(ta, seek_a);
            tb.bring(to + PARTS * L::A_PART, L::B_PART, wb, s & 1, false, unused);
            if (!ask_b && g + 1 < total) tb.load(wb), step(tb, seek_b);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&full[s]));
            if (__any_sync(0xffffffffu, *(volatile int *)&abort_s)) break;
            if (++s == stages) s = 0, ++round;
        }
        if constexpr (PARTS == 3) asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (OP == LinearOp::weights) {
#pragma unroll
            for (int e = 0; e < 4; ++e) column_sums[thread / 32][ta.column_of(e)] = column[e];
        }
    } else {  // ---- what follows: lane quarter warp % 4, share (warp - 4) / 4 of the columns ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kEpilogueRegs));
        const int quarter = warp & 3, share = (warp - 4) >> 2;
        const uint32_t from = ((uint32_t)(quarter * 32) << 16) + share * COLS;
        uint8_t *stage = sm + L::OFF_OUT + (warp - 4) * L::OUT_WARP;
        float *flat = reinterpret_cast<float *>(stage);
        const bool whole = (long long)p.J * sizeof(io_t) % 16 == 0;
        uint32_t acc = 0;
        bool ok = true;
        auto hand_back = [&](uint32_t buf) {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_at(address_in(smem_u32(&acc_empty[buf]), crank & ~1));
                else mbar_arrive(smem_u32(&acc_empty[buf]));
            }
        };
        // An addend (pre_in if there is one, else add) comes by TMA where rows are whole units: a warp's pieces of 32 x 32 in the order in which
        // they are used, the next on its way while one is used, into the next tile too.  Its place is that of the second output.
        const bool has_pre = OP == LinearOp::backward && p.act != PRISM_ACT_NONE, has_add = p.add != nullptr;
        const bool by_tma = L::INCOMING && !SPLIT && p.tiled && (has_pre || has_add) && !p.pre_out;
        const CUtensorMap *tm_in = has_pre ? &tm_pre : &tm_add;
        uint32_t asked = 0, taken = 0;
        int ask_tile = 0, ask_piece = 0, ask_i0 = 0, ask_j = 0, ask_pieces = 0;
        auto pieces_of = [&](int i0, int j0) {  // of the warp's columns, those that the matrix has
            return i0 + quarter * 32 < p.I ? max(0, min(COLS / 32, (p.J - j0 - share * COLS + 31) / 32)) : 0;
        };
        auto look = [&] {  // the first tile from ask_tile on with pieces
            for (; ask_tile < my_tiles; ++ask_tile) {
                int j0;
                tile_at(ask_tile, ask_i0, j0);
                ask_j = j0 + share * COLS;
                ask_pieces = pieces_of(ask_i0, j0);
                if (ask_pieces > 0) return;
            }
        };
        auto ask = [&] {
            if (ask_tile >= my_tiles) return;
            if (lane == 0) {
                const uint32_t bar = smem_u32(&incoming[warp - 4]);
                mbar_expect_tx(bar, 2048);
                tma_load_2d(smem_u32(stage + 2048), tm_in, bar, ask_j + 32 * ask_piece, ask_i0 + quarter * 32);
            }
            ++asked;
            if (++ask_piece == ask_pieces) ask_piece = 0, ++ask_tile, look();
        };
        if (by_tma) look(), ask();
        for (int i = 0; i < my_tiles && ok; ++i) {
            int i0, j0;
            tile_at(i, i0, j0);
            float2 sum[GROUPED ? COLS / 2 : 1];
            float over_rows = 0.f;
            uint32_t buf = 0;
#pragma unroll 1
            for (int g = 0; g < groups; ++g, ++acc) {
                buf = acc & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[buf]), (acc >> 1) & 1, wt.ns));
                if (!ok) break;
                fence_after_sync();
                if constexpr (GROUPED) {
                    auto add = [&](uint32_t at, bool first) {
                        uint32_t r[2][16];
                        tmem_ld_nowait(at, r[0]);
#pragma unroll
                        for (int c = 0; c < COLS / 16; ++c) {  // the next columns load while these are added
                            wait16(r[c & 1]);
                            if (c + 1 < COLS / 16) tmem_ld_nowait(at + 16 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float2 x = make_float2(__uint_as_float(r[c & 1][2 * q]), __uint_as_float(r[c & 1][2 * q + 1]));
                                sum[8 * c + q] = first ? x : io::add2(sum[8 * c + q], x);
                            }
                        }
                    };
                    add(tmem + buf * BN + from, g == 0);
                    if constexpr (L::SUMS > 0) {
                        if (sums && share == 0) {
                            uint32_t x;
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(tmem + L::SUMS + 16 * buf + ((uint32_t)(quarter * 32) << 16)));
                            asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(x)::"memory");
                            over_rows += __uint_as_float(x);
                        }
                    }
                    if (PARTS == 3 && g + 1 == groups) add(tmem + 2 * BN + (i & 1) * BN + from, false);
                    hand_back(buf);
                }
            }
            if (!ok) {
                if (lane == 0) give_up();  // products may still be in flight: the drain below waits for them
                break;
            }
            // 32 columns of the sums, of which the last hand the accumulator back
            auto piece = [&](int ch, float (&f)[32]) {
                if constexpr (GROUPED) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) f[2 * q] = sum[16 * ch + q].x, f[2 * q + 1] = sum[16 * ch + q].y;
                } else {
                    uint32_t r[32];
                    ld_issue(tmem + buf * BN + from + 32 * ch, r);
                    ld_wait(r);
#pragma unroll
                    for (int c = 0; c < 32; ++c) f[c] = __uint_as_float(r[c]);
                    if (ch + 1 == COLS / 32) hand_back(buf);
                }
            };
            if constexpr (L::SUMS > 0) {
                if (share == 0) column_sums[0][quarter * 32 + lane] = over_rows;
            }
            if constexpr (SPLIT) {  // every load has landed and every product has read it: their shared memory is free
                const int row = quarter * 32 + lane;
#pragma unroll
                for (int ch = 0; ch < COLS / 32; ++ch) {
                    float f[32];
                    piece(ch, f);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<float4 *>(sm + row * BN * 4 + (((share * COLS / 4 + 8 * ch + q) ^ (row & 7)) << 4)) =
                            make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
                }
            } else {
                const int r0 = i0 + quarter * 32, rows = min(32, p.I - r0);
                with_activation(p.act, [&](auto act) {
                    constexpr prism_activation ACT = decltype(act)::value;
                    if constexpr (!GROUPED) {
                        if (p.tiled) {  // bf16 pieces of 32 columns through shared memory, 16 at a time through registers
                            const int row = min(r0 + lane, p.I - 1);
#pragma unroll 1
                            for (int ch = 0; ch < COLS / 32; ++ch) {
                                const int j = j0 + share * COLS + ch * 32;
                                const bool inside = rows > 0 && j < p.J;
                                if (inside) {
                                    // after an expired wait the piece stays asked for and no other is: the drain below waits for it
                                    if (by_tma && ok) {
                                        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&incoming[warp - 4]), taken & 1, wt.ns));
                                        if (ok) ++taken;
                                    }
                                    bulk_wait_read();  // the pieces before have left (two places for them in turn brought nothing)
                                    __syncwarp();
                                }
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t r[16];
                                    float f[16];
                                    tmem_ld_nowait(tmem + buf * BN + from + 32 * ch + 16 * h, r);
                                    const int at = j + 16 * h;
                                    Held<io_t, 16> g;
                                    if (OP == LinearOp::forward && p.bias && inside) g.load(p.bias, at, p.J, true);
                                    if (OP == LinearOp::backward && has_pre && inside) {
                                        if (by_tma) Patch<io_t>::get_half(stage + 2048, lane, h, g);
                                        else g.load(p.pre_in + (size_t)row * p.J, at, p.J, true);
                                    }
                                    wait16(r);
                                    if (h == 1 && ch + 1 == COLS / 32) hand_back(buf);
                                    if (!inside) continue;
#pragma unroll
                                    for (int c = 0; c < 16; ++c) f[c] = __uint_as_float(r[c]);
                                    if constexpr (OP == LinearOp::forward) {
                                        if (p.bias) plus(f, g);
                                        if (p.pre_out) Patch<io_t>::put_half(stage + 2048, lane, h, f);
                                        to_values<io_t, ACT>(f);
                                    } else if constexpr (ACT != PRISM_ACT_NONE) {
                                        times_slopes<io_t, ACT>(f, g);
                                    }
                                    if (has_add) {
                                        if (by_tma && !has_pre) Patch<io_t>::get_half(stage + 2048, lane, h, g);
                                        else g.load(p.add + (size_t)row * p.J, at, p.J, true);
                                        plus(f, g);
                                    }
                                    Patch<io_t>::put_half(stage, lane, h, f);
                                }
                                if (!inside) continue;
                                fence_async_smem();
                                __syncwarp();
                                if (lane == 0) {
                                    tma_store_2d(&tm_out, smem_u32(stage), j, r0);
                                    if (p.pre_out) tma_store_2d(&tm_pre, smem_u32(stage + 2048), j, r0);
                                    bulk_commit();
                                }
                                if (by_tma && ok) ask();
                            }
                            return;
                        }
                    }
#pragma unroll (GROUPED ? COLS / 32 : 1)
                    for (int ch = 0; ch < COLS / 32; ++ch) {
                        const int j = j0 + share * COLS + ch * 32;
                        const bool inside = rows > 0 && j < p.J;
                        float f[32];
                        Held<io_t> other;
                        if (!GROUPED && inside && has_pre) Patch<io_t>::get(p.pre_in + (size_t)r0 * p.J, p.J, rows, j, whole, flat, lane, other);
                        piece(ch, f);
                        if (!inside) continue;
                        if constexpr (OP == LinearOp::forward) {
                            if (p.bias) {
                                Held<io_t> bias;
                                bias.load(p.bias, j, p.J, true);
                                plus(f, bias);
                            }
                            if (p.pre_out) {
                                if (GROUPED && p.tiled) Patch<io_t>::put_tiled(&tm_pre, stage, r0, j, lane, f);
                                else Patch<io_t>::put_rows(p.pre_out + (size_t)r0 * p.J, p.J, rows, j, flat, lane, f);
                            }
                            to_values<io_t, ACT>(f);
                        } else if constexpr (OP == LinearOp::backward && ACT != PRISM_ACT_NONE) {
                            if (GROUPED) Patch<io_t>::get(p.pre_in + (size_t)r0 * p.J, p.J, rows, j, whole, flat, lane, other);  // the sums hold the registers
                            times_slopes<io_t, ACT>(f, other);
                        }
                        if (has_add) {
                            Patch<io_t>::get(p.add + (size_t)r0 * p.J, p.J, rows, j, whole, flat, lane, other);
                            plus(f, other);
                        }
                        if (GROUPED && p.tiled) Patch<out_t>::put_tiled(&tm_out, stage, r0, j, lane, f);
                        else Patch<out_t>::put_rows((out_t *)p.out + (size_t)r0 * p.J, p.J, rows, j, flat, lane, f);
                    }
                });
            }
        }
        if (!SPLIT && p.tiled) bulk_wait_read();  // before the staging goes
        if (by_tma && !ok) {  // the piece asked for lands before the CTA exits
            if (lane == 0) give_up();
            if (taken < asked) (void)mbar_wait(smem_u32(&incoming[warp - 4]), taken & 1, 1000000000ull);
        }
    }
    // drain: after an expired wait, the copies and products in flight land before the CTA exits, and what they signal
    auto landed = [&](uint64_t *ring, long long to) {  // the last round of steps before `to`
        for (long long g = to > stages ? to - stages : 0; g < to; ++g) (void)mbar_wait(smem_u32(&ring[g % stages]), (uint32_t)(g / stages) & 1, 1000000000ull);
    };
    auto products_landed = [&](long long steps, uint32_t accumulators) {
        landed(freed, steps);
        for (uint32_t a = accumulators > 2 ? accumulators - 2 : 0; a < accumulators; ++a) (void)mbar_wait(smem_u32(&acc_full[a & 1]), (a >> 1) & 1, 1000000000ull);
    };
    __syncthreads();
    if constexpr (!PAIR) {
        if (abort_s) {
            if (tid == 0) products_landed(issued, accumulators);
            if (!SOFT && tid == 32) landed(full, issued);
        }
    }
    fence_before_sync();
    __syncthreads();
    if constexpr (PAIR || SPLIT) cluster_barrier();  // the other CTA's products reach into this one until here; the sums stand in shared memory
    if constexpr (PAIR) {
        // The loads of both CTAs of a pair count in the first one's barriers, and the CTAs stopped where they were.  The one behind brings in
        // what it lacks (a stage that one of them loaded is free in both, and they are a ring apart at most), so that each barrier gets
        // all that it expects.  Then the first one waits for the loads, and both for the products, which signal both.  abort_s is the
        // same in all of the cluster here.
        if (abort_s) {
            if (tid == 32) store_at(address_in(smem_u32(&other_issued), crank ^ 1), (unsigned long long)issued);
            if (tid == 0 && leads)
                for (uint32_t c = crank; c <= crank + 1; ++c) {
                    store_at(address_in(smem_u32(&products_s), c), (unsigned long long)issued);
                    store_at(address_in(smem_u32(&accumulators_s), c), accumulators);
                }
            __syncthreads();
            cluster_barrier();
            if (tid == 32) {
                const int of_tile = b_to - b_from;
                for (const long long to = (long long)other_issued; issued < to; ++issued) {
                    int i0, j0;
                    tile_at((int)(issued / of_tile), i0, j0);
                    load_block((int)(issued % stages), b_from + (int)(issued % of_tile), i0, j0);
                }
                if (leads) landed(full, issued);
            }
            if (tid == 0) products_landed((long long)products_s, accumulators_s);
            __syncthreads();
            cluster_barrier();
        }
    }
    if (warp == 0) {
        if constexpr (PAIR) tmem_dealloc_pair(tmem, L::kColumns);
        else tmem_dealloc(tmem, L::kColumns);
    }
    if constexpr (SPLIT) {
        static_assert((uint32_t)BM * BN * 4 <= L::OFF_OUT, "the sums fit where the operands were");
        int i0, j0;
        tile_at(0, i0, j0);
        const int r_from = rank * BM / p.splits, r_to = min((rank + 1) * BM / p.splits, p.I - i0);
        const bool whole = (long long)p.J * sizeof(out_t) % 16 == 0;
        with_activation(p.act, [&](auto act) {
            constexpr prism_activation ACT = decltype(act)::value;
            for (int e = r_from * (BN / 4) + tid; e < r_to * (BN / 4); e += L::THREADS) {
                const int row = e / (BN / 4), unit = e % (BN / 4), j = j0 + 4 * unit;
                const uint32_t at = sbase + row * BN * 4 + ((unit ^ (row & 7)) << 4);
                float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int c = 0; c < p.splits; ++c) {
                    const float4 x = remote<float4>(at, CTAS * c + in_tile);
                    f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w;
                }
                if (j >= p.J) continue;
                const size_t line = (size_t)(i0 + row) * p.J;
                // four values of a row that is made of whole units, else one at a time
                auto four = [&](const auto *q, float (&g)[4]) {
                    using T = std::remove_cv_t<std::remove_pointer_t<decltype(q)>>;
                    if (whole) {
                        if constexpr (sizeof(T) == 4) {
                            io::load_unit<T, 4>(q + j).get(g);
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2 *>(q + j);
                            io::Unit<__nv_bfloat16, 8>::two(w.x, g[0], g[1]), io::Unit<__nv_bfloat16, 8>::two(w.y, g[2], g[3]);
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x) g[x] = j + x < p.J ? io::ld(q + j + x) : 0.f;
                    }
                };
                auto put = [&](auto *q) {
                    using T = std::remove_pointer_t<decltype(q)>;
                    if (whole) {
                        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(q + j) = make_float4(f[0], f[1], f[2], f[3]);
                        else *reinterpret_cast<uint2 *>(q + j) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (j + x < p.J) io::st(q + j + x, f[x]);
                    }
                };
                float g[4];
                if constexpr (OP == LinearOp::weights) {
                    float *to = (float *)p.out + line;
                    if (p.accumulate) {
                        four((const float *)to, g);
#pragma unroll
                        for (int x = 0; x < 4; ++x) f[x] += g[x];
                    }
                    put(to);
                } else {
                    if constexpr (OP == LinearOp::forward) {
                        if (p.bias) {
                            four(p.bias, g);
#pragma unroll
                            for (int x = 0; x < 4; ++x) f[x] += g[x];
                        }
                        if (p.pre_out) put(p.pre_out + line);
                        to_values<io_t, ACT>(f);
                    } else if constexpr (ACT != PRISM_ACT_NONE) {
                        four(p.pre_in + line, g);
                        times_slopes<io_t, ACT>(f, g);
                    }
                    if (p.add) {
                        four(p.add + line, g);
                        plus(f, g);
                    }
                    put((io_t *)p.out + line);
                }
            }
        });
        if (OP == LinearOp::weights && p.dbias && j0 == 0) {
            for (int row = r_from + tid; row < r_to; row += L::THREADS) {
                float v = 0.f;
                for (int c = 0; c < p.splits; ++c)
#pragma unroll
                    for (int w = 0; w < (SOFT ? kLoaderWarps : 1); ++w)
                        v += remote<float>(smem_u32(&column_sums[OP == LinearOp::weights ? w : 0][OP == LinearOp::weights ? row : 0]), CTAS * c + in_tile);
                p.dbias[i0 + row] = p.accumulate ? p.dbias[i0 + row] + v : v;
            }
        }
        cluster_barrier();  // the others may still read this CTA's sums
    }
}

// A row-major matrix as boxes of box_rows rows x box_cols columns, swizzled by the box's row of 128 or 64 bytes
inline bool encode(CUtensorMap *map, int size, const void *base, int cols, int rows, int box_cols, int box_rows)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)ptr;
    }();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)cols * size};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    return fn && fn(map, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides,
                    box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename io_t, LinearOp OP, bool SOFT, int BN, bool SPLIT, bool PAIR>
cudaError_t launch_tiles(Params<io_t> p, int splits, const TokenLaunch &l)
{
    using L = Layout<io_t, OP, SOFT, BN, PAIR>;
    constexpr bool A_MN = OP == LinearOp::weights, B_MN = OP != LinearOp::forward;
    constexpr int OUT = OP == LinearOp::weights ? 4 : (int)sizeof(io_t);
    CUtensorMap ma = {}, mb = {}, mo = {}, mp = {}, md = {};
    if (!SOFT) {  // bf16
        const bool a = A_MN ? encode(&ma, 2, p.a, p.I, p.K, 64, BK) : encode(&ma, 2, p.a, p.K, p.I, BK, BM);
        const bool b = B_MN ? encode(&mb, 2, p.b, p.J, p.K, 64, BK) : encode(&mb, 2, p.b, p.K, p.J, BK, 128);
        if (!a || !b) return cudaErrorInvalidValue;
    }
    p.tiled = (long long)p.J * OUT % 16 == 0;
    if (!SPLIT && p.tiled) {
        if (!encode(&mo, OUT, p.out, p.J, p.I, 32, 32)) return cudaErrorInvalidValue;
        const void *pre = p.pre_out ? (const void *)p.pre_out : p.pre_in;
        if (pre && !encode(&mp, OUT, pre, p.J, p.I, 32, 32)) return cudaErrorInvalidValue;
        if (p.add && !encode(&md, OUT, p.add, p.J, p.I, 32, 32)) return cudaErrorInvalidValue;
    }
    p.splits = splits;
    constexpr int CTAS = PAIR ? 2 : 1;
    const long long tiles = (long long)((p.I + CTAS * BM - 1) / (CTAS * BM)) * ((p.J + BN - 1) / BN), workers = l.sm_count / CTAS;
    const Waits wt{l.d_status, l.wait_ns > 0 ? (unsigned long long)l.wait_ns : 100000000ull};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CTAS * (SPLIT ? tiles * splits : tiles < workers ? tiles : workers)));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::SMEM;
    cfg.stream = l.timer->stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CTAS * splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = SPLIT || PAIR ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, tile_kernel<io_t, OP, SOFT, BN, SPLIT, PAIR>, ma, mb, mo, mp, md, p, wt);
}

template <typename io_t, LinearOp OP, bool SOFT, int BN, bool SPLIT, bool PAIR>
cudaError_t prepare_tiles()
{
    return cudaFuncSetAttribute(tile_kernel<io_t, OP, SOFT, BN, SPLIT, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<io_t, OP, SOFT, BN, PAIR>::SMEM);
}

// How the product at hand is cut, and the kernel for it (one translation unit each)
struct Cut {
    bool soft, split, pair;
    int bn, splits;
};
int clusters_at_once(int ctas);  // of so many CTAs, one an SM; after weights_prepare()
template <typename io_t>
cudaError_t forward_tiles(const Params<io_t> &p, const Cut &c, const TokenLaunch &l);
template <typename io_t>
cudaError_t backward_tiles(const Params<io_t> &p, const Cut &c, const TokenLaunch &l);
template <typename io_t>
cudaError_t weights_tiles(const Params<io_t> &p, const Cut &c, const TokenLaunch &l);
cudaError_t forward_prepare();
cudaError_t backward_prepare();
cudaError_t weights_prepare();

}  // namespace lin
}  // namespace prism
