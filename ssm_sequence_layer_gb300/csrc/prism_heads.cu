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
constexpr int kSlabs = 608;  // blocks of the backward pass at most, each with a part of the weights' gradients

struct Form {
    int T, Hq, Hk, Hv, d, dv, norm, rot, half;  // half: pairs (i, i + rot / 2)
    long long n;                                // tokens
    float eps, amplitude;
    const float *inv_freq;
    const long long *positions;
    int lanes;   // per row, a power of two
    int chunk;   // heads that a group takes of one token
    int chunks;
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

// cos and sin of a fraction of a turn: the nearest quarter by its top bits, and the rest, at most an eighth, in float32
__device__ __forceinline__ void cos_sin(unsigned long long turns, float &c, float &s)
{
    const unsigned long long quarter = turns + (1ull << 61);
    const int rest = (int)((long long)(turns - (quarter & (3ull << 62))) >> 32);
    float sn, cs;
    sincospif((float)rest * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: pi times twice the turns
    const int q = (int)(quarter >> 62);
    c = q & 1 ? sn : cs;
    s = q & 1 ? cs : sn;
    if (q == 1 || q == 2) c = -c;
    if (q >= 2) s = -s;
}

// Values e of the units a and b of slot p: their columns, and the pairs' angle.  Slots with p < turned / VEC hold the pairs of
// the half layout, (p, p + rot / 2 / VEC); all others neighbouring units.
struct Units {
    int a, b;
    __device__ __forceinline__ Units(const Form &f, int p, int half_units) : a(2 * p), b(2 * p + 1)
    {
        if (f.half && p < half_units) a = p, b = p + half_units;
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void load(const T *p, float (&f)[VEC])
{
    if constexpr (sizeof(T) * VEC == 32) {
        float lo[4], hi[4];
        io::load_unit<T, 4>(p).get(lo);
        io::load_unit<T, 4>(p + 4).get(hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = lo[e], f[e + 4] = hi[e];
    } else {
        io::load_unit<T, VEC>(p).get(f);
    }
}

// The pairs' rotation by (c, s) on the units a and b: across the units, or within each (interleaved, VEC > 1)
template <int VEC, bool WITHIN>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC], const float (&s)[VEC], float sign)
{
    if constexpr (WITHIN) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1], u = b[2 * e], v = b[2 * e + 1], sa = sign * s[e], sb = sign * s[VEC / 2 + e];
            a[2 * e] = x * c[e] - y * sa, a[2 * e + 1] = x * sa + y * c[e];
            b[2 * e] = u * c[VEC / 2 + e] - v * sb, b[2 * e + 1] = u * sb + v * c[VEC / 2 + e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float x = a[e], y = b[e], se = sign * s[e];
            a[e] = x * c[e] - y * se, b[e] = x * se + y * c[e];
        }
    }
}

// A group's place: its token and first head, and the lane within the row
struct Place {
    long long n;
    int b, t, h0, h1;
    __device__ __forceinline__ Place(const Form &f, long long item)
    {
        n = item % f.n;
        b = (int)(n / f.T), t = (int)(n % f.T);
        h0 = (int)(item / f.n) * f.chunk;
        h1 = min(h0 + f.chunk, f.Hq + f.Hk + f.Hv);
    }
};

template <int VEC>
__device__ __forceinline__ void angles(const Form &f, const unsigned long long *table, long long position, int p, float (&c)[VEC], float (&s)[VEC])
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int i = p * VEC + e;
        c[e] = 1.f, s[e] = 0.f;
        if (i < f.rot / 2) {
            cos_sin(table[i] * (unsigned long long)position, c[e], s[e]);
            c[e] *= f.amplitude, s[e] *= f.amplitude;
        }
    }
}

__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float scale_of(const Form &f, float squares)
{
    if (f.norm == PRISM_HEADS_PLAIN) return 1.f;
    return rsqrtf((f.norm == PRISM_HEADS_RMS ? squares / (float)f.d : squares) + f.eps);
}

template <typename io_t>
struct Forward {
    Form f;
    const io_t *x, *q_weight, *k_weight;
    long long ld;
    io_t *q, *k, *v;
};

template <typename io_t, int VEC, int PER, bool WITHIN>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Forward<io_t> p)
{
    __shared__ unsigned long long table[kMaxHeadSize / 2];
    const Form &f = p.f;
    for (int i = threadIdx.x; i < f.rot / 2; i += kThreads) table[i] = turns_of(f.inv_freq[i]);
    __syncthreads();
    const int G = f.lanes, lane = threadIdx.x & (G - 1), half_units = f.rot / 2 / VEC;
    const int units = f.d / VEC, vunits = f.dv / VEC;
    const long long groups = (long long)gridDim.x * (kThreads / G), items = f.n * f.chunks;
    const long long first = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    for (long long base = first - (threadIdx.x & 31) / G; base < items; base += groups) {  // all lanes of a warp take part in the sums
        const long long item = base + (threadIdx.x & 31) / G;
        const bool live = item < items;
        const Place at(f, live ? item : items - 1);
        const io_t *row = p.x + at.n * p.ld;
        float c[PER][VEC], s[PER][VEC];
        const long long position = f.positions ? f.positions[at.n] : at.t;
#pragma unroll
        for (int i = 0; i < PER; ++i) angles<VEC>(f, table, position, lane + i * G, c[i], s[i]);
        for (int step = 0; step < f.chunk; ++step) {
            const int h = at.h0 + step;
            const bool mine = live && h < at.h1;
            if (mine && h >= f.Hq + f.Hk) {  // a value head: copied
                const int hv = h - f.Hq - f.Hk;
                const io_t *from = row + (size_t)(f.Hq + f.Hk) * f.d + (size_t)hv * f.dv;
                io_t *to = p.v + (((size_t)at.b * f.Hv + hv) * f.T + at.t) * f.dv;
                for (int u = lane; u < vunits; u += G) io::store_unit<io_t, VEC>(to + u * VEC, io::load_unit<io_t, VEC>(from + u * VEC));
            }
            const bool normed = mine && h < f.Hq + f.Hk;
            float a[PER][VEC], b[PER][VEC], squares = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const Units u(f, lane + i * G, half_units);
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[i][e] = b[i][e] = 0.f;
                if (normed && u.a < units) load(row + (size_t)h * f.d + u.a * VEC, a[i]);
                if (normed && u.b < units) load(row + (size_t)h * f.d + u.b * VEC, b[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) squares = fmaf(a[i][e], a[i][e], fmaf(b[i][e], b[i][e], squares));
            }
            const float r = scale_of(f, group_sum(squares, G));
            if (!normed) continue;
            const bool query = h < f.Hq;
            const io_t *w = query ? p.q_weight : p.k_weight;
            io_t *to = query ? p.q + (((size_t)at.b * f.Hq + h) * f.T + at.t) * f.d : p.k + (((size_t)at.b * f.Hk + h - f.Hq) * f.T + at.t) * f.d;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const Units u(f, lane + i * G, half_units);
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[i][e] *= r, b[i][e] *= r;
                if (w) {
                    float wa[VEC], wb[VEC];
                    if (u.a < units) {
                        load(w + u.a * VEC, wa);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) a[i][e] *= wa[e];
                    }
                    if (u.b < units) {
                        load(w + u.b * VEC, wb);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) b[i][e] *= wb[e];
                    }
                }
                turn<VEC, WITHIN>(a[i], b[i], c[i], s[i], 1.f);
                io::Unit<io_t, VEC> o;
                if (u.a < units) o.set(a[i]), io::store_unit<io_t, VEC>(to + u.a * VEC, o);
                if (u.b < units) o.set(b[i]), io::store_unit<io_t, VEC>(to + u.b * VEC, o);
            }
        }
    }
}

template <typename io_t, typename grad_t>
struct Backward {
    Form f;
    const io_t *x, *q_weight, *k_weight;
    long long ld, ld_dx;
    const grad_t *dq, *dk, *dv;
    io_t *dx;
    float *part;  // [gridDim.x][2][d], or NULL where no weight's gradient is wanted
};

template <typename io_t, typename grad_t, int VEC, int PER, bool WITHIN>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Backward<io_t, grad_t> p)
{
    __shared__ unsigned long long table[kMaxHeadSize / 2];
    __shared__ float dw_s[kThreads / 32][kMaxHeadSize];
    const Form &f = p.f;
    for (int i = threadIdx.x; i < f.rot / 2; i += kThreads) table[i] = turns_of(f.inv_freq[i]);
    __syncthreads();
    const int G = f.lanes, lane = threadIdx.x & (G - 1), half_units = f.rot / 2 / VEC;
    const int units = f.d / VEC, vunits = f.dv / VEC;
    const long long groups = (long long)gridDim.x * (kThreads / G), items = f.n * f.chunks;
    const long long first = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    const float along = f.norm == PRISM_HEADS_RMS ? 1.f / (float)f.d : f.norm == PRISM_HEADS_UNIT ? 1.f : 0.f;
    float dw[2][PER][2][VEC];  // this lane's share of the queries' and keys' weights' gradients
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) dw[z][i][0][e] = dw[z][i][1][e] = 0.f;
    for (long long base = first - (threadIdx.x & 31) / G; base < items; base += groups) {
        const long long item = base + (threadIdx.x & 31) / G;
        const bool live = item < items;
        const Place at(f, live ? item : items - 1);
        const io_t *row = p.x + at.n * p.ld;
        io_t *drow = p.dx + at.n * p.ld_dx;
        float c[PER][VEC], s[PER][VEC];
        const long long position = f.positions ? f.positions[at.n] : at.t;
#pragma unroll
        for (int i = 0; i < PER; ++i) angles<VEC>(f, table, position, lane + i * G, c[i], s[i]);
        for (int step = 0; step < f.chunk; ++step) {
            const int h = at.h0 + step;
            const bool mine = live && h < at.h1;
            if (mine && h >= f.Hq + f.Hk) {
                const int hv = h - f.Hq - f.Hk;
                const grad_t *from = p.dv + (((size_t)at.b * f.Hv + hv) * f.T + at.t) * f.dv;
                io_t *to = drow + (size_t)(f.Hq + f.Hk) * f.d + (size_t)hv * f.dv;
                for (int u = lane; u < vunits; u += G) {
                    float g[VEC];
                    load(from + u * VEC, g);
                    io::Unit<io_t, VEC> o;
                    o.set(g);
                    io::store_unit<io_t, VEC>(to + u * VEC, o);
                }
            }
            const bool normed = mine && h < f.Hq + f.Hk, query = h < f.Hq;
            const io_t *w = query ? p.q_weight : p.k_weight;
            const grad_t *from = query ? p.dq + (((size_t)at.b * f.Hq + h) * f.T + at.t) * f.d
                                       : p.dk + (((size_t)at.b * f.Hk + h - f.Hq) * f.T + at.t) * f.d;
            float a[PER][VEC], b[PER][VEC], ga[PER][VEC], gb[PER][VEC], squares = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const Units u(f, lane + i * G, half_units);
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[i][e] = b[i][e] = ga[i][e] = gb[i][e] = 0.f;
                if (normed && u.a < units) load(row + (size_t)h * f.d + u.a * VEC, a[i]), load(from + u.a * VEC, ga[i]);
                if (normed && u.b < units) load(row + (size_t)h * f.d + u.b * VEC, b[i]), load(from + u.b * VEC, gb[i]);
                turn<VEC, WITHIN>(ga[i], gb[i], c[i], s[i], -1.f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) squares = fmaf(a[i][e], a[i][e], fmaf(b[i][e], b[i][e], squares));
            }
            const float r = scale_of(f, group_sum(squares, G));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const Units u(f, lane + i * G, half_units);
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[i][e] *= r, b[i][e] *= r;  // the normalised values
                if (p.part && normed) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float da = ga[i][e] * a[i][e], db = gb[i][e] * b[i][e];
                        if (query) dw[0][i][0][e] += da, dw[0][i][1][e] += db;
                        else dw[1][i][0][e] += da, dw[1][i][1][e] += db;
                    }
                }
                if (w && normed) {
                    float wv[VEC];
                    if (u.a < units) {
                        load(w + u.a * VEC, wv);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) ga[i][e] *= wv[e];
                    }
                    if (u.b < units) {
                        load(w + u.b * VEC, wv);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) gb[i][e] *= wv[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) dot = fmaf(ga[i][e], a[i][e], fmaf(gb[i][e], b[i][e], dot));
            }
            const float m = along * group_sum(dot, G);
            if (!normed) continue;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const Units u(f, lane + i * G, half_units);
                // without a norm the row's sum plays no part, be it infinite
                if (f.norm != PRISM_HEADS_PLAIN) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ga[i][e] = r * (ga[i][e] - a[i][e] * m), gb[i][e] = r * (gb[i][e] - b[i][e] * m);
                }
                io::Unit<io_t, VEC> o;
                if (u.a < units) o.set(ga[i]), io::store_unit<io_t, VEC>(drow + (size_t)h * f.d + u.a * VEC, o);
                if (u.b < units) o.set(gb[i]), io::store_unit<io_t, VEC>(drow + (size_t)h * f.d + u.b * VEC, o);
            }
        }
    }
    if (!p.part) return;
    // the block's part: over the groups of a warp by shuffles, over the warps in their order
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const Units u(f, lane + i * G, half_units);
#pragma unroll
            for (int side = 0; side < 2; ++side)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float v = dw[z][i][side][e];
                    for (int o = 16; o >= G; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    const int unit = side ? u.b : u.a;
                    if ((threadIdx.x & 31) < G && unit < units) dw_s[warp][unit * VEC + e] = v;
                }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < f.d; j += kThreads) {
            float v = 0.f;
            for (int k = 0; k < kThreads / 32; ++k) v += dw_s[k][j];
            p.part[((size_t)blockIdx.x * 2 + z) * f.d + j] = v;
        }
        __syncthreads();
    }
}

// A block per weight of 32 columns: eight warps add every eighth part, and then each other's sums, in a fixed order
__global__ void __launch_bounds__(256) join_kernel(const float *part, int parts, int d, float *dq_weight, float *dk_weight)
{
    tc::grid_dependency_wait();
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane, z = blockIdx.y;
    float v = 0.f;
    if (j < d)
        for (int k = warp; k < parts; k += 8) v += part[((size_t)k * 2 + z) * d + j];
    s[warp][lane] = v;
    __syncthreads();
    float *to = z ? dk_weight : dq_weight;
    if (warp != 0 || j >= d || !to) return;
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

Form form_of(const prism_heads_form &f, int vec)
{
    Form o = {};
    o.T = f.T, o.Hq = f.Hq, o.Hk = f.Hk, o.Hv = f.Hv, o.d = f.Hq + f.Hk > 0 ? f.d : 0, o.dv = f.Hv > 0 ? f.dv : 0, o.norm = f.norm;
    o.rot = f.Hq + f.Hk > 0 ? f.rot : 0;
    o.half = !f.interleaved;
    o.n = (long long)f.B * f.T;
    o.eps = f.eps, o.amplitude = f.amplitude, o.inv_freq = f.inv_freq, o.positions = f.positions;
    const int widest = o.d > o.dv ? o.d : o.dv;
    o.lanes = lanes_of((widest / vec + 1) / 2);
    return o;
}

// Heads that a group takes of a token: all of them where tokens fill the machine, fewer where they are few
void split(Form &f, int sm_count)
{
    const int total = f.Hq + f.Hk + f.Hv;
    const long long want = (long long)sm_count * 2048 / f.lanes;
    long long chunks = f.n > 0 ? want / f.n : 1;
    if (chunks < 1) chunks = 1;
    if (chunks > total) chunks = total;
    f.chunk = (int)((total + chunks - 1) / chunks);
    f.chunks = (total + f.chunk - 1) / f.chunk;
}

unsigned blocks_of(const Form &f, int most)
{
    const long long blocks = (f.n * f.chunks * f.lanes + kThreads - 1) / kThreads;
    return (unsigned)(blocks < most ? blocks : most);
}

template <typename io_t, int VEC, int PER, bool WITHIN>
void launch_forward(const Forward<io_t> &p, const TokenLaunch &l)
{
    forward_kernel<io_t, VEC, PER, WITHIN><<<blocks_of(p.f, 64 * l.sm_count), kThreads, 0, l.timer->stream>>>(p);
}

template <typename io_t>
cudaError_t forward(const HeadsArgs &a, const TokenLaunch &l)
{
    constexpr int VEC = 16 / (int)sizeof(io_t);
    const bool whole = whole_units(a.form, VEC, a.ld_x);
    Forward<io_t> p = {};
    p.f = form_of(a.form, whole ? VEC : 1);
    split(p.f, l.sm_count);
    p.x = (const io_t *)a.x, p.q_weight = (const io_t *)a.form.q_weight, p.k_weight = (const io_t *)a.form.k_weight, p.ld = a.ld_x;
    p.q = (io_t *)a.q, p.k = (io_t *)a.k, p.v = (io_t *)a.v;
    const int slots = ((whole ? p.f.d / VEC : p.f.d) + 1) / 2;
    l.timer->begin("heads");
    if (!whole) {
        if (slots <= p.f.lanes) launch_forward<io_t, 1, 1, false>(p, l);
        else launch_forward<io_t, 1, 8, false>(p, l);
    } else if (slots <= p.f.lanes) {
        if (a.form.interleaved) launch_forward<io_t, VEC, 1, true>(p, l);
        else launch_forward<io_t, VEC, 1, false>(p, l);
    } else if constexpr (VEC == 4) {
        if (a.form.interleaved) launch_forward<io_t, VEC, 2, true>(p, l);
        else launch_forward<io_t, VEC, 2, false>(p, l);
    }
    l.timer->end();
    return cudaGetLastError();
}

template <typename io_t, typename grad_t, int VEC, int PER, bool WITHIN>
void launch_backward(const Backward<io_t, grad_t> &p, unsigned blocks, const TokenLaunch &l)
{
    backward_kernel<io_t, grad_t, VEC, PER, WITHIN><<<blocks, kThreads, 0, l.timer->stream>>>(p);
}

template <typename io_t, typename grad_t>
cudaError_t backward(const HeadsBackwardArgs &a, float *ws, const TokenLaunch &l)
{
    constexpr int VEC = 16 / (int)sizeof(io_t);
    const bool whole = whole_units(a.form, VEC, a.ld_x) && a.ld_dx % VEC == 0;
    const bool weights = a.dq_weight || a.dk_weight;
    Backward<io_t, grad_t> p = {};
    p.f = form_of(a.form, whole ? VEC : 1);
    split(p.f, l.sm_count);
    p.x = (const io_t *)a.x, p.q_weight = (const io_t *)a.form.q_weight, p.k_weight = (const io_t *)a.form.k_weight;
    p.ld = a.ld_x, p.ld_dx = a.ld_dx;
    p.dq = (const grad_t *)a.dq, p.dk = (const grad_t *)a.dk, p.dv = (const grad_t *)a.dv, p.dx = (io_t *)a.dx;
    p.part = weights ? ws : nullptr;
    const int slots = ((whole ? p.f.d / VEC : p.f.d) + 1) / 2;
    const unsigned blocks = blocks_of(p.f, weights ? kSlabs : 64 * l.sm_count);
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
    const cudaError_t e = launch_behind(join_kernel, dim3((p.f.d + 31) / 32, 2), 256, l.timer->stream, (const float *)ws, (int)blocks, p.f.d, a.dq_weight, a.dk_weight);
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
