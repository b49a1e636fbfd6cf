// From a projection's rows to the layer's queries, keys and values: the norm of each head, the position's rotation and the
// layout [B, heads, T, size], and the gradient of all three.
//
//   y_j = r x_j w_j,   r = 1, 1 / sqrt(sum x^2 + eps) or 1 / sqrt(mean x^2 + eps)
//   (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t) on pairs of y,   t = position inv_freq
//   backward: g = the cotangent turned by -t,  dx_j = r (w_j g_j - x_j r^2 c sum_i w_i g_i x_i),  dw_j = sum g_j r x_j
//
// A few operations per value read: HBM bounds both directions where rows are many, the launch where they are few.  A head's
// row is cut into units of 16 bytes (or single values where sizes or strides do not allow it), and a lane holds the two
// units whose values turn together, so that a rotation needs no exchange between lanes; the 1 to 32 lanes of a row share its sums
// by shuffles.  Such a group takes one token and several of its heads, for which the angles are the same.
#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

namespace prism {
namespace heads {

constexpr int kThreads = 256;
constexpr int kSlabs = 608;  // parts of each weight's gradient at most

struct Form {
    int n, T, d, dv, norm, rot, half;  // half: pairs (i, i + rot / 2)
    int H[3];                          // heads of each kind: queries, keys, values
    int chunks[3], chunk[3];           // the blocks' second coordinate: each kind's heads in chunks of so many
    float eps, amplitude;
    const float *inv_freq;
    const long long *positions;
    int lanes;  // per row, a power of two
};

// A block's kind of heads and its share of them
struct Share {
    int kind, h0, h1, index;  // index: of the chunk among its kind's
    __device__ __forceinline__ Share(const Form &f, int y) : kind(0)
    {
        while (kind < 2 && y >= f.chunks[kind]) y -= f.chunks[kind++];
        index = y, h0 = y * f.chunk[kind], h1 = min(h0 + f.chunk[kind], f.H[kind]);
    }
    // the first column of head h of this kind
    __device__ __forceinline__ long long column(const Form &f, int h) const
    {
        return kind == 2 ? (long long)(f.H[0] + f.H[1]) * f.d + (long long)h * f.dv : (long long)((kind ? f.H[0] : 0) + h) * f.d;
    }
};

// Turns per position as a fraction of 2^64, so that the product with a position, whole turns dropped, is one 64-bit multiplication
// of integers.  1 / (2 pi) in two parts: the result is within 2^-63 turns of the exact one.
__device__ __forceinline__ unsigned long long turns_of(float inv_freq)
{
    const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
    const double f = inv_freq, p = f * hi, rest = fma(f, hi, -p) + f * lo;
    const double frac = p - rint(p);
    return (unsigned long long)__double2ll_rn(frac * 18446744073709551616.0) + (unsigned long long)__double2ll_rn(rest * 18446744073709551616.0);
}

// cos and sin of a fraction of a turn: the nearest quarter by its top bits, and of the rest, at most an eighth, polynomials
// fitted with the least largest error (2^-28 of the sine, 2^-34)
__device__ __forceinline__ void cos_sin(unsigned long long turns, float &c, float &s)
{
    const uint32_t top = (uint32_t)(turns >> 32), quarter = top + (1u << 29);
    const float r = (float)(int)(top - (quarter & (3u << 30))) * 2.3283064365386963e-10f, r2 = r * r;
    const float sn = r * fmaf(r2, fmaf(r2, fmaf(r2, -75.39329528808594f, 81.59234619140625f), -41.34165954589844f), 6.2831854820251465f);
    const float cs = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, 59.2202033996582f, -85.4428482055664f), 64.93931579589844f), -19.739208221435547f), 1.f);
    const bool odd = quarter & (1u << 30);
    // the signs: cos is negative in quarters 1 and 2, sin in 2 and 3
    c = __uint_as_float(__float_as_uint(odd ? sn : cs) ^ ((quarter ^ (quarter << 1)) & 0x80000000u));
    s = __uint_as_float(__float_as_uint(odd ? cs : sn) ^ (quarter & 0x80000000u));
}

// The units of slot p.  Slots with p < half_units hold the pairs of the half layout, (p, p + rot / 2 / VEC); all others
// neighbouring units.
struct Units {
    int a, b;
    __device__ __forceinline__ Units(const Form &f, int p, int half_units) : a(2 * p), b(2 * p + 1)
    {
        if (f.half && p < half_units) a = p, b = p + half_units;
    }
};

// VEC values on their way: 16 or 32 bytes, or one value
template <typename T, int VEC>
struct Raw {
    static constexpr int N = sizeof(T) * VEC == 32 ? 2 : 1, EACH = VEC / N;
    io::Unit<T, EACH> u[N];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = io::load_unit<T, EACH>(p + i * EACH);
    }
    __device__ __forceinline__ void zero() { memset(u, 0, sizeof(u)); }
    __device__ __forceinline__ void get(float (&f)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float g[EACH];
            u[i].get(g);
#pragma unroll
            for (int e = 0; e < EACH; ++e) f[i * EACH + e] = g[e];
        }
    }
};

// Two at a time where there are two
template <int VEC, typename F2, typename F1>
__device__ __forceinline__ void by_two(F2 two, F1 one)
{
    if constexpr (VEC >= 2) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) two(e);
    } else {
        one(0);
    }
}
__device__ __forceinline__ float2 at2(const float *f) { return make_float2(f[0], f[1]); }
__device__ __forceinline__ void to2(float *f, float2 v) { f[0] = v.x, f[1] = v.y; }

template <int VEC>
__device__ __forceinline__ void scale(float (&a)[VEC], float s)
{
    by_two<VEC>([&](int e) { to2(a + e, io::mul2(at2(a + e), make_float2(s, s))); }, [&](int e) { a[e] *= s; });
}
template <int VEC>
__device__ __forceinline__ void times(float (&a)[VEC], const float *w)
{
    by_two<VEC>([&](int e) { to2(a + e, io::mul2(at2(a + e), at2(w + e))); }, [&](int e) { a[e] *= w[e]; });
}
// sum + a b, the sum in two halves
template <int VEC>
__device__ __forceinline__ float2 dot(const float (&a)[VEC], const float (&b)[VEC], float2 sum)
{
    by_two<VEC>([&](int e) { sum = io::fma2(at2(a + e), at2(b + e), sum); }, [&](int e) { sum.x = fmaf(a[e], b[e], sum.x); });
    return sum;
}

// The pairs' rotation by (c, sign s) on the units a and b: across the units, or within each (interleaved, VEC > 1).  `pairs` of the slot's VEC
// pairs are turned, of a slot across the units all or none.  The others are left as they are, which a rotation by no angle would not do to
// values that are not finite.
template <int VEC, bool WITHIN>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC], const float (&s)[VEC], int pairs)
{
    if constexpr (WITHIN) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1], u = b[2 * e], v = b[2 * e + 1];
            if (e < pairs) a[2 * e] = x * c[e] - y * s[e], a[2 * e + 1] = x * s[e] + y * c[e];
            if (VEC / 2 + e < pairs) b[2 * e] = u * c[VEC / 2 + e] - v * s[VEC / 2 + e], b[2 * e + 1] = u * s[VEC / 2 + e] + v * c[VEC / 2 + e];
        }
    } else if (pairs > 0) {
        by_two<VEC>(
            [&](int e) {
                const float2 x = at2(a + e), y = at2(b + e), c2 = at2(c + e), s2 = at2(s + e);
                to2(a + e, io::fma2(x, c2, io::mul2(y, make_float2(-s2.x, -s2.y))));
                to2(b + e, io::fma2(x, s2, io::mul2(y, c2)));
            },
            [&](int e) {
                const float x = a[e], y = b[e];
                a[e] = x * c[e] - y * s[e], b[e] = x * s[e] + y * c[e];
            });
    }
}

template <int VEC>
__device__ __forceinline__ void angles(const Form &f, const unsigned long long *table, long long position, int p, float sign, float (&c)[VEC], float (&s)[VEC])
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int i = p * VEC + e;
        c[e] = 1.f, s[e] = 0.f;
        if (i < f.rot / 2) {
            cos_sin(table[i] * (unsigned long long)position, c[e], s[e]);
            c[e] *= f.amplitude, s[e] *= f.amplitude * sign;
        }
    }
}

__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float scale_of(const Form &f, float inv_d, float squares)
{
    if (f.norm == PRISM_HEADS_PLAIN) return 1.f;
    return rsqrtf((f.norm == PRISM_HEADS_RMS ? squares * inv_d : squares) + f.eps);
}

// What the groups of a block share, and the way of a group through the tokens
struct Common {
    unsigned long long table[kMaxHeadSize / 2];
    __align__(16) float w[kMaxHeadSize];
    template <typename io_t>
    __device__ __forceinline__ void fill(const Form &f, const io_t *weight)
    {
        for (int i = threadIdx.x; i < f.rot / 2; i += kThreads) table[i] = turns_of(f.inv_freq[i]);
        if (weight)
            for (int i = threadIdx.x; i < f.d; i += kThreads) w[i] = io::ld(weight + i);
        __syncthreads();
    }
};

// Values are copied: rows [n][ld] (or heads) to heads (or rows), several of a token's heads at once
template <typename from_t, typename to_t, int VEC>
__device__ void copy_values(const Form &f, const Share &sh, const from_t *from, long long from_token, long long from_head, to_t *to, long long to_token, long long to_head,
                            bool from_heads)
{
    const int G = f.lanes, lane = threadIdx.x & (G - 1), units = f.dv / VEC, per_block = kThreads / G;
    for (int n = blockIdx.x * per_block + threadIdx.x / G; n < f.n; n += gridDim.x * per_block) {
        const int b = n / f.T, t = n - b * f.T;
        // the heads' layout: [b][head][t], the rows': [n][head]
        const from_t *src = from + (from_heads ? (size_t)b * f.H[2] * from_head + (size_t)t * from_token : (size_t)n * from_token) + sh.h0 * from_head;
        to_t *dst = to + (from_heads ? (size_t)n * to_token : (size_t)b * f.H[2] * to_head + (size_t)t * to_token) + sh.h0 * to_head;
        for (int u = lane; u < units; u += G) {
            constexpr int NB = 4;
            for (int h = sh.h0; h < sh.h1; h += NB) {
                Raw<from_t, VEC> x[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if (h + i < sh.h1) x[i].load(src + (h - sh.h0 + i) * from_head + u * VEC);
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if (h + i < sh.h1) {
                        float g[VEC];
                        x[i].get(g);
                        io::Unit<to_t, VEC> o;
                        o.set(g);
                        io::store_unit<to_t, VEC>(dst + (h - sh.h0 + i) * to_head + u * VEC, o);
                    }
            }
        }
    }
}

template <typename io_t>
struct Forward {
    Form f;
    const io_t *x, *weight[2];
    long long ld;
    io_t *out[3];
};

// NB heads of a token at once: their loads are in flight together.  16384 rows of 18 heads of 128 (bf16, 151 MB): 29.8 us, 5.1 TB/s, with
// two heads and four blocks an SM; three heads and three blocks 31.5 us.
template <typename io_t, int VEC, int PER, bool WITHIN, int NB>
__global__ void __launch_bounds__(kThreads, PER == 1 ? 4 : 1) forward_kernel(const Forward<io_t> p)
{
    __shared__ Common s;
    const Form &f = p.f;
    const Share sh(f, blockIdx.y);
    if (sh.kind == 2) {
        copy_values<io_t, io_t, VEC>(f, sh, p.x + sh.column(f, 0), p.ld, f.dv, p.out[2], f.dv, (long long)f.T * f.dv, false);
        return;
    }
    const io_t *weight = p.weight[sh.kind];
    s.fill(f, weight);
    const int G = f.lanes, lane = threadIdx.x & (G - 1), half_units = f.rot / 2 / VEC, units = f.d / VEC, per_block = kThreads / G;
    const float inv_d = 1.f / (float)f.d;
    const long long head = (long long)f.T * f.d;
    for (int base = blockIdx.x * per_block; base < f.n; base += gridDim.x * per_block) {  // all lanes take part in the sums
        const int n = min(base + (int)threadIdx.x / G, f.n - 1);
        const bool live = base + (int)threadIdx.x / G < f.n;
        const int b = n / f.T, t = n - b * f.T;
        const io_t *row = p.x + (size_t)n * p.ld + sh.column(f, sh.h0);
        io_t *to = p.out[sh.kind] + ((size_t)b * f.H[sh.kind] + sh.h0) * head + (size_t)t * f.d;
        const long long position = f.positions ? f.positions[n] : t;
        float c[PER][VEC], sn[PER][VEC];
        for (int h = sh.h0; h < sh.h1; h += NB, row += NB * f.d, to += NB * head) {
            Raw<io_t, VEC> raw[NB][PER][2];
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const Units u(f, lane + i * G, half_units);
                    raw[k][i][0].zero(), raw[k][i][1].zero();
                    if (h + k < sh.h1 && u.a < units) raw[k][i][0].load(row + k * f.d + u.a * VEC);
                    if (h + k < sh.h1 && u.b < units) raw[k][i][1].load(row + k * f.d + u.b * VEC);
                }
            if (h == sh.h0) {
#pragma unroll
                for (int i = 0; i < PER; ++i) angles<VEC>(f, s.table, position, lane + i * G, 1.f, c[i], sn[i]);
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                float a[PER][VEC], bb[PER][VEC];
                float2 squares = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    raw[k][i][0].get(a[i]), raw[k][i][1].get(bb[i]);
                    squares = dot<VEC>(bb[i], bb[i], dot<VEC>(a[i], a[i], squares));
                }
                const float r = scale_of(f, inv_d, group_sum(squares.x + squares.y, G));
                if (!live || h + k >= sh.h1) continue;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const Units u(f, lane + i * G, half_units);
                    scale<VEC>(a[i], r), scale<VEC>(bb[i], r);
                    if (weight) {
                        if (u.a < units) times<VEC>(a[i], s.w + u.a * VEC);
                        if (u.b < units) times<VEC>(bb[i], s.w + u.b * VEC);
                    }
                    turn<VEC, WITHIN>(a[i], bb[i], c[i], sn[i], f.rot / 2 - (lane + i * G) * VEC);
                    io::Unit<io_t, VEC> o;
                    if (u.a < units) o.set(a[i]), io::store_unit<io_t, VEC>(to + k * head + u.a * VEC, o);
                    if (u.b < units) o.set(bb[i]), io::store_unit<io_t, VEC>(to + k * head + u.b * VEC, o);
                }
            }
        }
    }
}

template <typename io_t, typename grad_t>
struct Backward {
    Form f;
    const io_t *x, *weight[2];
    long long ld, ld_dx;
    const grad_t *grad[3];
    io_t *dx;
    float *part[2];  // [blocks][chunks of the kind][d], or NULL where the weight's gradient is not wanted
};

// 16384 rows of 18 heads of 128 with float32 cotangents (277 MB): 62 us, 4.4 TB/s, 67.5 with the join behind it; 32768 rows of 12 heads of 64 in
// float32 (269 MB): 50 us, 5.4 TB/s.  The loads in flight bound it: two blocks an SM in bf16, where registers hold 96 bytes a lane on their way (three
// spill: 76 us), three in float32 (two: 62 us).
template <typename io_t, typename grad_t, int VEC, int PER, bool WITHIN, int NB>
__global__ void __launch_bounds__(kThreads, PER == 1 ? (VEC == 8 ? 2 : 3) : 1) backward_kernel(const Backward<io_t, grad_t> p)
{
    __shared__ Common s;
    __shared__ float dw_s[kThreads / 32][kMaxHeadSize];
    const Form &f = p.f;
    const Share sh(f, blockIdx.y);
    if (sh.kind == 2) {
        copy_values<grad_t, io_t, VEC>(f, sh, p.grad[2], f.dv, (long long)f.T * f.dv, p.dx + sh.column(f, 0), p.ld_dx, f.dv, true);
        return;
    }
    const io_t *weight = p.weight[sh.kind];
    float *part = p.part[sh.kind];
    s.fill(f, weight);
    const int G = f.lanes, lane = threadIdx.x & (G - 1), half_units = f.rot / 2 / VEC, units = f.d / VEC, per_block = kThreads / G;
    const float inv_d = 1.f / (float)f.d, along = f.norm == PRISM_HEADS_RMS ? inv_d : 1.f;
    const long long head = (long long)f.T * f.d;
    float dw[PER][2][VEC];  // this lane's share of the weight's gradient
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][0][e] = dw[i][1][e] = 0.f;
    for (int base = blockIdx.x * per_block; base < f.n; base += gridDim.x * per_block) {
        const int n = min(base + (int)threadIdx.x / G, f.n - 1);
        const bool live = base + (int)threadIdx.x / G < f.n;
        const int b = n / f.T, t = n - b * f.T;
        const io_t *row = p.x + (size_t)n * p.ld + sh.column(f, sh.h0);
        io_t *to = p.dx + (size_t)n * p.ld_dx + sh.column(f, sh.h0);
        const grad_t *from = p.grad[sh.kind] + ((size_t)b * f.H[sh.kind] + sh.h0) * head + (size_t)t * f.d;
        const long long position = f.positions ? f.positions[n] : t;
        float c[PER][VEC], sn[PER][VEC];
        for (int h = sh.h0; h < sh.h1; h += NB, row += NB * f.d, to += NB * f.d, from += NB * head) {
            Raw<io_t, VEC> raw[NB][PER][2];
            Raw<grad_t, VEC> grad[NB][PER][2];
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const Units u(f, lane + i * G, half_units);
                    raw[k][i][0].zero(), raw[k][i][1].zero(), grad[k][i][0].zero(), grad[k][i][1].zero();
                    const bool in = live && h + k < sh.h1;
                    if (in && u.a < units) raw[k][i][0].load(row + k * f.d + u.a * VEC), grad[k][i][0].load(from + k * head + u.a * VEC);
                    if (in && u.b < units) raw[k][i][1].load(row + k * f.d + u.b * VEC), grad[k][i][1].load(from + k * head + u.b * VEC);
                }
            if (h == sh.h0) {
#pragma unroll
                for (int i = 0; i < PER; ++i) angles<VEC>(f, s.table, position, lane + i * G, -1.f, c[i], sn[i]);
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                // g = the cotangent turned back; the sums of x^2 and w g x, from which r and the part along x come
                float ga[PER][VEC], gb[PER][VEC];
                float2 squares = make_float2(0.f, 0.f), wgx = squares;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const Units u(f, lane + i * G, half_units);
                    float a[VEC], bb[VEC];
                    raw[k][i][0].get(a), raw[k][i][1].get(bb);
                    grad[k][i][0].get(ga[i]), grad[k][i][1].get(gb[i]);
                    turn<VEC, WITHIN>(ga[i], gb[i], c[i], sn[i], f.rot / 2 - (lane + i * G) * VEC);
                    squares = dot<VEC>(bb, bb, dot<VEC>(a, a, squares));
                    float wa[VEC], wb[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) wa[e] = ga[i][e], wb[e] = gb[i][e];
                    if (weight) {
                        if (u.a < units) times<VEC>(wa, s.w + u.a * VEC);
                        if (u.b < units) times<VEC>(wb, s.w + u.b * VEC);
                    }
                    wgx = dot<VEC>(wb, bb, dot<VEC>(wa, a, wgx));
                }
                const float r = scale_of(f, inv_d, group_sum(squares.x + squares.y, G));
                float m = 0.f;  // of x: r^2 (times the mean's 1 / d) sum w g x
                if (f.norm != PRISM_HEADS_PLAIN) m = along * r * (r * group_sum(wgx.x + wgx.y, G));
                if (!live || h + k >= sh.h1) continue;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const Units u(f, lane + i * G, half_units);
                    float a[VEC], bb[VEC];
                    raw[k][i][0].get(a), raw[k][i][1].get(bb);
                    if (part) {
                        by_two<VEC>(
                            [&](int e) {
                                const float2 r2 = make_float2(r, r);
                                to2(dw[i][0] + e, io::fma2(io::mul2(at2(ga[i] + e), r2), at2(a + e), at2(dw[i][0] + e)));
                                to2(dw[i][1] + e, io::fma2(io::mul2(at2(gb[i] + e), r2), at2(bb + e), at2(dw[i][1] + e)));
                            },
                            [&](int e) {
                                dw[i][0][e] = fmaf(ga[i][e] * r, a[e], dw[i][0][e]);
                                dw[i][1][e] = fmaf(gb[i][e] * r, bb[e], dw[i][1][e]);
                            });
                    }
                    if (weight) {
                        if (u.a < units) times<VEC>(ga[i], s.w + u.a * VEC);
                        if (u.b < units) times<VEC>(gb[i], s.w + u.b * VEC);
                    }
                    if (f.norm != PRISM_HEADS_PLAIN) {  // without a norm the row's sums play no part, be they infinite
                        by_two<VEC>(
                            [&](int e) {
                                const float2 m2 = make_float2(-m, -m), r2 = make_float2(r, r);
                                to2(ga[i] + e, io::mul2(io::fma2(at2(a + e), m2, at2(ga[i] + e)), r2));
                                to2(gb[i] + e, io::mul2(io::fma2(at2(bb + e), m2, at2(gb[i] + e)), r2));
                            },
                            [&](int e) { ga[i][e] = r * fmaf(a[e], -m, ga[i][e]), gb[i][e] = r * fmaf(bb[e], -m, gb[i][e]); });
                    }
                    io::Unit<io_t, VEC> o;
                    if (u.a < units) o.set(ga[i]), io::store_unit<io_t, VEC>(to + k * f.d + u.a * VEC, o);
                    if (u.b < units) o.set(gb[i]), io::store_unit<io_t, VEC>(to + k * f.d + u.b * VEC, o);
                }
            }
        }
    }
    if (!part) return;
    // the block's part: over the groups of a warp by shuffles, over the warps in their order
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const Units u(f, lane + i * G, half_units);
#pragma unroll
        for (int side = 0; side < 2; ++side)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float v = dw[i][side][e];
                for (int o = 16; o >= G; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                const int unit = side ? u.b : u.a;
                if ((threadIdx.x & 31) < G && unit < units) dw_s[warp][unit * VEC + e] = v;
            }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < f.d; j += kThreads) {
        float v = 0.f;
        for (int k = 0; k < kThreads / 32; ++k) v += dw_s[k][j];
        part[((size_t)blockIdx.x * f.chunks[sh.kind] + sh.index) * f.d + j] = v;
    }
}

// A block per kind and 32 columns: eight warps add every eighth part, and then each other's sums, in a fixed order
__global__ void __launch_bounds__(256) join_kernel(const float *q_part, int q_parts, const float *k_part, int k_parts, int d, float *dq_weight, float *dk_weight)
{
    tc::grid_dependency_wait();
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    const float *part = blockIdx.y ? k_part : q_part;
    const int parts = blockIdx.y ? k_parts : q_parts;
    float *to = blockIdx.y ? dk_weight : dq_weight;
    if (!to) return;
    float v = 0.f;
    if (j < d) {
#pragma unroll 4
        for (int k = warp; k < parts; k += 8) v += part[(size_t)k * d + j];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || j >= d) return;
    for (int k = 1; k < 8; ++k) v += s[k][lane];
    to[j] = v;
}

int lanes_of(int slots)
{
    int g = 1;
    while (g < slots && g < 32) g *= 2;
    return g;
}

// Whether rows, their strides and the pairs of the half layout are made of whole units of vec values
bool whole_units(const prism_heads_form &f, int vec, long long ld)
{
    const bool rows = f.Hq + f.Hk > 0;
    return (!rows || f.d % vec == 0) && (f.Hv == 0 || f.dv % vec == 0) && ld % vec == 0 && (f.interleaved || f.rot / 2 % vec == 0);
}

// Blocks along the tokens and chunks along each kind's heads: all heads of a kind where tokens fill the machine, so that their
// angles are taken once, fewer where tokens are few
Form form_of(const prism_heads_form &f, int vec, int sm_count, int blocks_per_sm, int most, unsigned &blocks)
{
    Form o = {};
    const bool rows = f.Hq + f.Hk > 0;
    o.n = f.B * f.T, o.T = f.T, o.d = rows ? f.d : 0, o.dv = f.Hv > 0 ? f.dv : 0, o.norm = f.norm, o.rot = rows ? f.rot : 0;
    o.half = !f.interleaved;
    o.eps = f.eps, o.amplitude = f.amplitude, o.inv_freq = f.inv_freq, o.positions = f.positions;
    o.H[0] = f.Hq, o.H[1] = f.Hk, o.H[2] = f.Hv;
    const int widest = o.d > o.dv ? o.d : o.dv;
    o.lanes = lanes_of((widest / vec + 1) / 2);
    const int per_block = kThreads / o.lanes;
    const long long along = (o.n + per_block - 1) / per_block, room = (long long)blocks_per_sm * sm_count;
    const int total = f.Hq + f.Hk + f.Hv;
    int chunk = total;
    while (chunk > 1 && along * ((f.Hq + chunk - 1) / chunk + (f.Hk + chunk - 1) / chunk + (f.Hv + chunk - 1) / chunk) < room) chunk = (chunk + 1) / 2;
    while (most > 0 && ((f.Hq + chunk - 1) / chunk > most || (f.Hk + chunk - 1) / chunk > most)) chunk *= 2;
    int chunks = 0;
    for (int k = 0; k < 3; ++k) {
        o.chunk[k] = chunk;
        o.chunks[k] = (o.H[k] + chunk - 1) / chunk;
        chunks += o.chunks[k];
    }
    // where a kernel's blocks leave parts to be joined there are as many as run at once, and `most` parts of a kind
    long long x = along;
    if (most > 0) {
        x = (room + chunks - 1) / chunks < along ? (room + chunks - 1) / chunks : along;
        const int c = o.chunks[0] > o.chunks[1] ? o.chunks[0] : o.chunks[1];
        if (x * c > most) x = most / c > 0 ? most / c : 1;
    }
    blocks = (unsigned)(x < (1 << 30) ? x : (1 << 30));
    return o;
}

template <typename io_t, int VEC, int PER, bool WITHIN>
void launch_forward(const Forward<io_t> &p, unsigned blocks, const TokenLaunch &l)
{
    forward_kernel<io_t, VEC, PER, WITHIN, PER == 1 ? 2 : 1>
        <<<dim3(blocks, p.f.chunks[0] + p.f.chunks[1] + p.f.chunks[2]), kThreads, 0, l.timer->stream>>>(p);
}

template <typename io_t>
cudaError_t forward(const HeadsArgs &a, const TokenLaunch &l)
{
    constexpr int VEC = 16 / (int)sizeof(io_t);
    const bool whole = whole_units(a.form, VEC, a.ld_x);
    Forward<io_t> p = {};
    unsigned blocks;
    p.f = form_of(a.form, whole ? VEC : 1, l.sm_count, 6, 0, blocks);
    p.x = (const io_t *)a.x, p.weight[0] = (const io_t *)a.form.q_weight, p.weight[1] = (const io_t *)a.form.k_weight, p.ld = a.ld_x;
    p.out[0] = (io_t *)a.q, p.out[1] = (io_t *)a.k, p.out[2] = (io_t *)a.v;
    const int slots = ((whole ? p.f.d / VEC : p.f.d) + 1) / 2;
    l.timer->begin("heads");
    if (!whole) {
        if (slots <= p.f.lanes) launch_forward<io_t, 1, 1, false>(p, blocks, l);
        else launch_forward<io_t, 1, 8, false>(p, blocks, l);
    } else if (slots <= p.f.lanes) {
        if (a.form.interleaved) launch_forward<io_t, VEC, 1, true>(p, blocks, l);
        else launch_forward<io_t, VEC, 1, false>(p, blocks, l);
    } else if constexpr (VEC == 4) {
        if (a.form.interleaved) launch_forward<io_t, VEC, 2, true>(p, blocks, l);
        else launch_forward<io_t, VEC, 2, false>(p, blocks, l);
    }
    l.timer->end();
    return cudaGetLastError();
}

template <typename io_t, typename grad_t, int VEC, int PER, bool WITHIN>
void launch_backward(const Backward<io_t, grad_t> &p, unsigned blocks, const TokenLaunch &l)
{
    backward_kernel<io_t, grad_t, VEC, PER, WITHIN, 1>
        <<<dim3(blocks, p.f.chunks[0] + p.f.chunks[1] + p.f.chunks[2]), kThreads, 0, l.timer->stream>>>(p);
}

template <typename io_t, typename grad_t>
cudaError_t backward(const HeadsBackwardArgs &a, float *ws, const TokenLaunch &l)
{
    constexpr int VEC = 16 / (int)sizeof(io_t);
    const bool whole = whole_units(a.form, VEC, a.ld_x) && a.ld_dx % VEC == 0;
    const bool weights = a.dq_weight || a.dk_weight;
    Backward<io_t, grad_t> p = {};
    unsigned blocks;
    p.f = form_of(a.form, whole ? VEC : 1, l.sm_count, 4, weights ? kSlabs : 0, blocks);
    p.x = (const io_t *)a.x, p.weight[0] = (const io_t *)a.form.q_weight, p.weight[1] = (const io_t *)a.form.k_weight;
    p.ld = a.ld_x, p.ld_dx = a.ld_dx;
    p.grad[0] = (const grad_t *)a.dq, p.grad[1] = (const grad_t *)a.dk, p.grad[2] = (const grad_t *)a.dv, p.dx = (io_t *)a.dx;
    float *k_part = ws + (size_t)kSlabs * kMaxHeadSize;
    p.part[0] = a.dq_weight ? ws : nullptr, p.part[1] = a.dk_weight ? k_part : nullptr;
    const int slots = ((whole ? p.f.d / VEC : p.f.d) + 1) / 2;
    if (blocks > 0) {
        l.timer->begin("heads_backward");
        if (!whole) {
            if (slots <= p.f.lanes) launch_backward<io_t, grad_t, 1, 1, false>(p, blocks, l);
            else launch_backward<io_t, grad_t, 1, 8, false>(p, blocks, l);
        } else if (slots <= p.f.lanes) {
            if (a.form.interleaved) launch_backward<io_t, grad_t, VEC, 1, true>(p, blocks, l);
            else launch_backward<io_t, grad_t, VEC, 1, false>(p, blocks, l);
        } else if constexpr (VEC == 4) {
            if (a.form.interleaved) launch_backward<io_t, grad_t, VEC, 2, true>(p, blocks, l);
            else launch_backward<io_t, grad_t, VEC, 2, false>(p, blocks, l);
        }
        l.timer->end();
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!weights) return cudaSuccess;
    l.timer->begin("heads_join");
    const cudaError_t e = launch_behind(join_kernel, dim3((a.form.d + 31) / 32, 2), 256, l.timer->stream, (const float *)ws, (int)blocks * p.f.chunks[0],
                                        (const float *)k_part, (int)blocks * p.f.chunks[1], a.form.d, a.dq_weight, a.dk_weight);
    l.timer->end();
    return e;
}

}  // namespace heads

size_t heads_workspace_bytes() { return (size_t)heads::kSlabs * 2 * kMaxHeadSize * sizeof(float); }

cudaError_t heads_forward(prism_dtype io, const HeadsArgs &a, const TokenLaunch &l)
{
    return io == PRISM_BF16 ? heads::forward<__nv_bfloat16>(a, l) : heads::forward<float>(a, l);
}

cudaError_t heads_backward(prism_dtype io, const HeadsBackwardArgs &a, float *ws, const TokenLaunch &l)
{
    if (io == PRISM_F32) return heads::backward<float, float>(a, ws, l);
    return a.grads == PRISM_BF16 ? heads::backward<__nv_bfloat16, __nv_bfloat16>(a, ws, l) : heads::backward<__nv_bfloat16, float>(a, ws, l);
}

}  // namespace prism
