// Drawing a token from logits under temperature, top-k, top-p and min-p, given a number u in [0, 1) for each row.
//
// With z = c logits, the tokens ordered by falling logit and then by rising id, the row keeps the shortest of three prefixes:
// the first k; the fewest whose mass sum e^(z - max) reaches p of that of the first k; those with e^(z - max) >= min_p.  The
// token is the first, by rising id, at which the kept tokens' running mass exceeds u times their mass.
//
// The choices are whole numbers, so the masses are whole numbers too: multiples of 2^-F of the first token's (F = 44, less
// for more than 2^19 tokens), whose sums have no rounding and no order.  Tokens among which a border may lie are sorted, with masses exact
// to two units; the many others' masses come from the machine's base-2 exponential first, whose sums are within 2^-19.6 of the exact
// ones.  If a border comes nearer to a token's edge than that, they are computed again within 2^-28.5 (a table of roots of 2, which
// takes about twice as long as the exponential), and if that is not near enough, to the last place (about 50 operations a token).
//
// Bound: not bandwidth (100 KB a row) but the way of one row through its steps, a barrier or two each, and operations per token in between.
// Cycles of a row of 50021 bf16, with top-k 50: copy into shared memory 2400, largest logit 2400, candidates by the threads' own largest
// 7000, sorting 2000, keeping and drawing 5000; counting tokens by their distance from the largest takes 10000 instead, with the places
// of top-p 20000.  Microseconds: 4 x 50021 bf16 with top-k 50 17, top-p 0.95 70 where it keeps 10000 tokens, 23 where it keeps five;
// 512 x 50021 float32 70, 193 and 99, without a rule 94.
#pragma once

#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

namespace prism {
namespace draw {

constexpr int kBuckets = 1024, kPerOctave = 32;  // of the distance from the row's largest logit, in 32nds of a halving
constexpr int kCounted = 256;                    // ... by counting
constexpr int kPlaceBits = 13;                   // of a place within a bucket
constexpr float kLowest = -3.3895313892515355e38f;  // bfloat16's: at or below it a token is masked

typedef unsigned long long u64;

// 2^(j / 64) in two parts
__device__ const float2 kRoots[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f}};

template <typename T>
struct Params {
    const T *logits;
    long long ld;
    const float *u, *inv_temperature;
    const int *top_k;
    const float *top_p, *min_p;
    long long *ids;
    float *logprob;
    int *kept;
    int n, V, fraction;
    int *status;
};

// The largest logit that counts as masked: bfloat16's lowest value, or the largest whose product with c overflows to -inf
__device__ __forceinline__ float mask_of(float c)
{
    float l = kLowest;
    if (c > 1.f) {
        l = fmaxf(l, -3.4028234663852886e38f / c);
        while (l * c == -INFINITY) l = __int_as_float(__float_as_int(l) - 1);  // up, to the first that does not overflow
        while (l * c != -INFINITY && l > kLowest) l = __int_as_float(__float_as_int(l) + 1);  // down, to the last that does
        l = fmaxf(l, kLowest);
    }
    return l;
}

// A whole number that orders as the logit does (both zeros alike)
__device__ __forceinline__ int order_of(float l)
{
    const int b = __float_as_int(l + 0.f);
    return b ^ ((b >> 31) & 0x7fffffff);
}

struct Mass {
    float top, mask, c, kh, kl;  // the row's largest logit, the largest masked one, c, c log2 e in two parts
    int fraction;
    float hi_scale, least;  // least: 2^-200 at this distance, beyond which products might overflow

    __device__ __forceinline__ Mass(float top_, float mask_, float c_, int fraction_) : top(top_), mask(mask_), c(c_), fraction(fraction_)
    {
        kh = c * 1.44269502162933349609375f;
        kl = fmaf(c, 1.44269502162933349609375f, -kh) + c * 1.925963033500011079e-8f;
        least = -200.f / kh;
        hi_scale = __int_as_float((127 + fraction - 22) << 23);
    }
    // log2 of a token's mass but for rounding errors: falls with the logit, never rises
    __device__ __forceinline__ float log_of(float l) const { return (l - top) * kh; }
    // falling logits, rising places: 32nds of a halving in 2^-13ths, but for rounding errors
    __device__ __forceinline__ uint32_t place(float l) const
    {
        return __float_as_uint(fmaf(fmaxf(log_of(l), -(float)(kBuckets - 1) / kPerOctave), -(float)kPerOctave, (float)kBuckets)) & 0x7fffffu;
    }
    __device__ __forceinline__ int bucket(float l) const { return (int)(place(l) >> kPlaceBits); }
    // l - top in two parts, the second its rounding error
    __device__ __forceinline__ void below(float l, float &dh, float &dl) const
    {
        dh = l - top;
        const float back = dh - l;
        dl = (l - (dh - back)) + (-top - back);
    }
    // the mass, within 2^-22 + 2^-25 |log2 of it| of itself
    __device__ __forceinline__ float rough(float l) const
    {
        const float d = fmaxf(l - top, least), y = d * kh;
        float e;
        asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(y));
        return fmaf(e, fmaf(d, kl, fmaf(d, kh, -y)) * 0.693147180559945f, e);
    }
    // a sum of few masses as a whole number
    __device__ __forceinline__ u64 whole(float e) const
    {
        e *= hi_scale;
        const uint32_t hi = __float2uint_rz(e);
        return ((u64)hi << 22) + __float2uint_rn((e - (float)hi) * 4194304.f);
    }
    __device__ __forceinline__ u64 quick(float l) const { return whole(rough(l)); }
    // the mass within 2^-29 of itself and two units: a root of 2 as a whole number, and what e^t - 1, |t| <= log 2 / 128, adds to it
    __device__ __forceinline__ u64 close(float l, const u64 *roots, float &rest) const
    {
        float dh, dl;
        below(l, dh, dl);
        const float y = dh * kh;
        rest = 0.f;
        if (!(y > -46.f)) return 0;
        const float yl = fmaf(dh, kh, -y) + fmaf(dh, kl, dl * kh);
        const float v = fmaf(y, 64.f, 12582912.f);  // 1.5 2^23: the whole number nearest to 64 y in the last bits
        const int n = __float_as_int(v) - 0x4b400000;
        const float t = fmaf(fmaf(v - 12582912.f, -1.f / 64, y), 0.69314718f, yl * 0.69314718f);
        const u64 root = roots[n & 63];
        const int down = -(n >> 6);
        rest = (float)(uint32_t)(root >> (fraction - 31)) * __int_as_float((96 - down) << 23) * (t * fmaf(t, fmaf(t, 1.f / 6, 0.5f), 1.f));
        return root >> down;
    }
    __device__ __forceinline__ u64 close_whole(u64 main, float rest) const
    {
        rest *= hi_scale;
        const int hi = __float2int_rd(rest);
        return main + (u64)((long long)hi << 22) + __float2uint_rn((rest - (float)hi) * 4194304.f);
    }
    __device__ __forceinline__ u64 close(float l, const u64 *roots) const
    {
        float rest;
        const u64 main = close(l, roots, rest);
        return close_whole(main, rest);
    }
    __device__ __forceinline__ u64 close_slack(u64 all, int V) const { return (all >> 28) + 4 * (u64)V; }
    // the logarithm of a token's share of a mass: (l - top) c - log of the mass's power of two, the parts of both kept, - log of its leading bits
    __device__ __forceinline__ float log_share(float l, u64 all) const
    {
        float dh, dl;
        below(l, dh, dl);
        const float xh = dh * c, xl = fmaf(dh, c, -xh) + dl * c;
        const int power = 63 - __clzll(all);
        const float n = (float)(power - fraction), f = (float)(all << (63 - power)) * 0x1p-63f;
        const float h = n * 0x1.62ep-1f, a = xh - h, back = a - xh;  // log 2 in two parts, the first product exact
        return a + (((xh - (a - back)) + (-h - back)) + (xl - fmaf(n, 3.194618495e-05f, logf(f))));
    }
    // How far sums of rough masses may be off, of tokens V of mass `all`: 2^-22 of the exponential, 2^-22.4 of adding up eight at a
    // time, and 2^-25 times the mean distance in halvings, which is log2 V at most
    __device__ __forceinline__ u64 slack(u64 all, int V) const { return (all >> 20) + (all >> 22) + V; }
    // within two units: e^x = 2^(n / 64) e^t, |t| <= log 2 / 128, with x, t and the result in two floats each; e^t - 1 by its
    // series, of which all but the first two terms are below 2^-24
    __device__ __noinline__ u64 exact(float l) const
    {
        float dh, dl;
        below(l, dh, dl);
        const float xh = dh * c;
        if (!(xh > -32.f)) return 0;
        const float xl = fmaf(dh, c, -xh) + dl * c;
        const float nf = rintf(xh * 92.332482616893656877f);
        const int n = (int)nf;
        const float r = fmaf(-nf, 0x1.62ep-7f, xh), r2 = nf * 0x1.0cp-21f;  // log 2 / 64 in three parts, the products exact
        const float s = r - r2, sb = s - r, rl = ((r - (s - sb)) + (-r2 - sb)) + fmaf(nf, 0x1.05c61p-35f, xl);
        const float th = s + rl, tb = th - s, tl = (s - (th - tb)) + (rl - tb);
        const float sq = th * th, sql = fmaf(th, th, -sq) + 2.f * th * tl;
        const float cube = th * sq * fmaf(th, fmaf(th, 1.f / 120, 1.f / 24), 1.f / 6);
        const float half = 0.5f * sq, ph = th + half, pb = ph - th, pl = ((th - (ph - pb)) + (half - pb)) + (tl + fmaf(0.5f, sql, cube));
        const float2 root = kRoots[n & 63];
        const float m = root.x * ph, eh = root.x + m;
        const float el = (m - (eh - root.x)) + (fmaf(root.x, ph, -m) + fmaf(root.y, ph, root.y) + root.x * pl);
        const float unit = __int_as_float((127 + fraction + (n >> 6)) << 23);
        return (u64)(__float2ll_rn(eh * unit) + __float2ll_rn(el * unit));
    }
    __device__ __forceinline__ u64 of(bool to_the_last, float l) const { return to_the_last ? exact(l) : quick(l); }
};

// A prefix of the order: the tokens above `order`, and those at it whose id is at most `id`
struct Cut {
    int order, id;
    u64 mass;  // of the prefix
    __device__ __forceinline__ bool keeps(int o, int i) const { return o > order || (o == order && i <= id); }
};

constexpr int kMostWarps = 32;
template <int CANDIDATES>  // tokens that are put in order directly
struct Shared {
    static constexpr int kCandidates = CANDIDATES;
    union {
        uint32_t count[kBuckets];
        int rank[CANDIDATES];
        struct {
            u64 masses[kCounted], below[kCounted];  // of a short list: a token's mass, and that of all up to its id
        };
    };
    union {
        struct {
            uint32_t lo[kBuckets], hi[kBuckets];  // a bucket's mass
        };
        u64 list[CANDIDATES];  // candidates, the order in the upper half and the id, reversed, in the lower one
    };
    u64 roots[64];  // 2^(j / 64) as masses
    u64 sums[kMostWarps], more[kMostWarps];
    uint32_t counts[kMostWarps];
    u64 mass, before;
    uint32_t number, number_before;
    int at, low, high, first, last;
    float top;
    int flag;
};
__device__ __forceinline__ u64 listed(int order, int id) { return (u64)((uint32_t)order ^ 0x80000000u) << 32 | (uint32_t)~id; }
__device__ __forceinline__ int order_in(u64 x) { return (int)((uint32_t)(x >> 32) ^ 0x80000000u); }
__device__ __forceinline__ int id_in(u64 x) { return (int)~(uint32_t)x; }
__device__ __forceinline__ float logit_of(int order) { return __int_as_float(order ^ ((order >> 31) & 0x7fffffff)); }

// A row and the block's way through it: units of 16 bytes from the last boundary at or before the row's start.  RESIDENT: a copy in
// shared memory, whose first and last units are filled up with -inf.
template <typename T, bool RESIDENT>
struct Row {
    static constexpr int VEC = 16 / (int)sizeof(T);
    const T *p;  // the row's first token, or its first unit in shared memory
    int V, skew, units;
    __device__ __forceinline__ Row(const T *row, int V_) : p(row), V(V_)
    {
        skew = (int)((uintptr_t)row % 16 / sizeof(T));
        units = (int)(((long long)skew + V + VEC - 1) / VEC);
    }
    template <int NT>
    __device__ __forceinline__ void copy_to(uint4 *to)
    {
        const uint32_t at = tc::smem_u32(to);
        for (int unit = threadIdx.x; unit < units; unit += NT) {
            const int id = first_id(unit);
            if (id >= 0 && id + VEC <= V) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + unit * 16), "l"(p + id) : "memory");
            } else {
                T *out = reinterpret_cast<T *>(to + unit);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (id + e >= 0 && id + e < V) out[e] = p[id + e];
                    else io::st(out + e, -INFINITY);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        p = reinterpret_cast<const T *>(to);
    }
    __device__ __forceinline__ int first_id(int unit) const { return unit * VEC - skew; }
    __device__ __forceinline__ io::Unit<T, VEC> get(int unit) const
    {
        if constexpr (RESIDENT) {
            io::Unit<T, VEC> u;
            asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.w.x), "=r"(u.w.y), "=r"(u.w.z), "=r"(u.w.w) : "r"(tc::smem_u32(p) + unit * 16));
            return u;
        } else {
            const int id = first_id(unit);
            if (id >= 0 && id + VEC <= V) return io::load_unit<T, VEC>(p + id);
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = id + e >= 0 && id + e < V ? io::ld(p + id + e) : -INFINITY;
            io::Unit<T, VEC> u;
            u.set(f);
            return u;
        }
    }
    __device__ __forceinline__ void get(int unit, float (&f)[VEC]) const { get(unit).get(f); }
    // f(logits, first id) for the units from, from + step, ... below `to`, several of them on their way at once; what the mask covers is
    // among them, as is -inf outside the row
    template <typename F>
    __device__ __forceinline__ void units_of(int from, int to, int step, F f) const
    {
        constexpr int AHEAD = RESIDENT ? 2 : 4;
#pragma unroll 1
        for (int unit = from; unit < to; unit += AHEAD * step) {
            io::Unit<T, VEC> u[AHEAD];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a)
                if (unit + a * step < to) u[a] = get(unit + a * step);
#pragma unroll
            for (int a = 0; a < AHEAD; ++a)
                if (unit + a * step < to) {
                    float l[VEC];
                    u[a].get(l);
                    f(l, first_id(unit + a * step));
                }
        }
    }
    // f(logit, id) for each token of theirs above the mask
    template <typename F>
    __device__ __forceinline__ void each_of(int from, int to, int step, float mask, F f) const
    {
        units_of(from, to, step, [&](const float (&l)[VEC], int id) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (l[e] > mask) f(l[e], id + e);
        });
    }
    // ... the block's threads side by side
    template <int NT, typename F>
    __device__ __forceinline__ void each(float mask, F f) const
    {
        each_of(threadIdx.x, units, NT, mask, f);
    }
    // the units of a warp: neighbouring ranges of ids
    __device__ __forceinline__ void range(int warp, int warps, int &from, int &to) const
    {
        const int each = (units + warps - 1) / warps;
        from = min(units, warp * each), to = min(units, from + each);
    }
};

// the sum of a unit's values, pairs first
template <int N>
__device__ __forceinline__ float sum_of(float (&e)[N])
{
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) e[i] += e[i + n];
    return e[0];
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }
// 27 bits at a time, of which 32 add up to 32 bits
__device__ __forceinline__ u64 warp_sum(u64 v)
{
    constexpr uint32_t M = (1u << 27) - 1;
    const uint32_t a = warp_sum((uint32_t)v & M), b = warp_sum((uint32_t)(v >> 27) & M), c = warp_sum((uint32_t)(v >> 54));
    return a + ((u64)b << 27) + ((u64)c << 54);
}
template <typename V>
__device__ __forceinline__ V warp_scan(V v)  // inclusive
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
    }
    return v;
}

// The block's sums of a mass and a number, to every thread
template <int NT, typename S>
__device__ __forceinline__ void block_sums(S &s, u64 &mass, uint32_t &number)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    mass = warp_sum(mass), number = warp_sum(number);
    __syncthreads();
    if (lane == 0) s.sums[warp] = mass, s.counts[warp] = number;
    __syncthreads();
    mass = warp_sum(lane < NT / 32 ? s.sums[lane] : (u64)0), number = warp_sum(lane < NT / 32 ? s.counts[lane] : 0u);
}
// A value's sum over the threads up to and with this one, given the warps' arrays
template <int NT, typename V>
__device__ __forceinline__ V block_scan(V v, V *of_warps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V up = warp_scan(v);
    __syncthreads();
    if (lane == 31) of_warps[warp] = up;
    __syncthreads();
    const V w = lane < NT / 32 ? of_warps[lane] : (V)0, before = warp_scan(w) - w;
    return up + __shfl_sync(0xffffffffu, before, warp);
}

// The first n of the list in falling order.  Few tokens count those before them, with all threads at work; more are compared and
// exchanged in pairs by a network, whose steps cost a barrier each (the whole draw of 4 rows of 50021 that keep 50: 23.5 us by counting,
// 26.3 by the network; that keep 1000: 54.5 and 40.3).
template <int NT, typename S>
__device__ __noinline__ void sort_list(S &s, int n)
{
    if (n > kCounted) {
        int size = 2 * kCounted;
        while (size < n) size *= 2;
        for (int i = n + threadIdx.x; i < size; i += NT) s.list[i] = 0;
        __syncthreads();
        for (int run = 2; run <= size; run *= 2)
            for (int d = run / 2; d > 0; d /= 2) {
                for (int t = threadIdx.x; t < size / 2; t += NT) {
                    const int i = 2 * t - (t & (d - 1)), j = i + d;
                    const u64 a = s.list[i], b = s.list[j];
                    if ((a < b) == ((i & run) == 0)) s.list[i] = b, s.list[j] = a;
                }
                __syncthreads();
            }
        return;
    }
    static_assert(kCounted <= NT, "a thread for each token");
    int across = 32;  // threads beside each other have tokens of their own; behind them others take further parts of the list
    while (across < n) across *= 2;
    const int i = threadIdx.x % across, per = (n + NT / across - 1) / (NT / across), from = threadIdx.x / across * per;
    if (threadIdx.x < n) s.rank[threadIdx.x] = 0;
    const u64 mine = i < n ? s.list[i] : ~0ull;
    __syncthreads();
    int rank = 0;
    for (int o = from; o < min(n, from + per); ++o) rank += s.list[o] > mine;
    if (i < n && rank > 0) atomicAdd(&s.rank[i], rank);
    __syncthreads();
    const int at = threadIdx.x < n ? s.rank[threadIdx.x] : 0;
    __syncthreads();
    if (threadIdx.x < n) s.list[at] = mine;  // the first part's token is this thread's own
    __syncthreads();
}

// The smallest prefix with at least `number` tokens (BY_MASS: of at least `mass`) of the tokens ordered, by cutting the range of the
// logits in which it ends into 1024 parts until that range holds few tokens, or equal ones only.
template <int NT, bool BY_MASS, typename S, typename R>
__device__ __noinline__ Cut find_cut(S &s, const R &row, const Mass &m, bool exact, uint32_t number, u64 mass)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t n_before = 0;  // of the tokens above the range at hand
    u64 m_before = 0;
    int low = INT_MIN, high = INT_MAX, shift = 0;  // the range, of order_of
    for (int level = 0;; ++level) {
        auto inside = [&](int o) { return o >= low && o <= high; };
        auto place = [&](float l, int o) { return level == 0 ? m.bucket(l) : (int)(((uint32_t)high - (uint32_t)o) >> shift); };
        for (int i = tid; i < kBuckets; i += NT) s.count[i] = s.lo[i] = s.hi[i] = 0;
        if (tid == 0) s.low = INT_MAX, s.high = INT_MIN, s.at = -1;
        __syncthreads();
        row.template each<NT>(m.mask, [&](float l, int) {
            const int o = order_of(l);
            if (!inside(o)) return;
            const int b = place(l, o);
            atomicAdd(&s.count[b], 1u);
            const u64 e = m.of(exact, l);
            const uint32_t add = (uint32_t)e, old = atomicAdd(&s.lo[b], add), up = (uint32_t)(e >> 32) + (old + add < old);
            if (up) atomicAdd(&s.hi[b], up);
        });
        __syncthreads();
        {  // the bucket at which the running number (mass) reaches what is asked for
            constexpr int EACH = kBuckets / NT;
            uint32_t n[EACH], nn = 0;
            u64 e[EACH], mm = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                n[i] = s.count[EACH * tid + i], e[i] = (u64)s.hi[EACH * tid + i] << 32 | s.lo[EACH * tid + i];
                nn += n[i], mm += e[i];
            }
            uint32_t at_n = n_before + block_scan<NT>(nn, s.counts) - nn;
            u64 at_m = m_before + block_scan<NT>(mm, s.sums) - mm;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const bool here = n[i] > 0 && (BY_MASS ? (at_m < mass || (mass == 0 && at_n == 0)) && at_m + e[i] >= mass : at_n < number && at_n + n[i] >= number);
                if (here) s.at = EACH * tid + i, s.number = n[i], s.number_before = at_n, s.before = at_m;
                at_n += n[i], at_m += e[i];
            }
            __syncthreads();
        }
        const int at = s.at;
        if (at < 0) return Cut{INT_MIN, INT_MAX, 0};  // not reached: everything is kept (the caller asks for no more than there is)
        const uint32_t held = s.number;
        n_before = s.number_before, m_before = s.before;
        __syncthreads();
        if (tid == 0) s.number = 0;
        __syncthreads();
        int my_low = INT_MAX, my_high = INT_MIN;
        row.template each<NT>(m.mask, [&](float l, int id) {
            const int o = order_of(l);
            if (!inside(o) || place(l, o) != at) return;
            my_low = min(my_low, o), my_high = max(my_high, o);
            if (held <= S::kCandidates) s.list[atomicAdd(&s.number, 1u)] = listed(o, id);
        });
        __syncthreads();
        if (held <= S::kCandidates) {
            sort_list<NT>(s, held);
            constexpr int EACH = S::kCandidates / NT;
            u64 e[EACH], mm = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                e[i] = EACH * tid + i < held ? m.of(exact, logit_of(order_in(s.list[EACH * tid + i]))) : 0;
                mm += e[i];
            }
            u64 at_m = m_before + block_scan<NT>(mm, s.sums) - mm;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const uint32_t nn = n_before + EACH * tid + i + 1;
                const bool reaches = EACH * tid + i < held &&
                                     (BY_MASS ? at_m + e[i] >= mass && (at_m < mass || (mass == 0 && nn == 1)) : nn == number);
                if (reaches) s.low = order_in(s.list[EACH * tid + i]), s.at = id_in(s.list[EACH * tid + i]), s.mass = at_m + e[i], s.before = at_m;
                at_m += e[i];
            }
            __syncthreads();
            return Cut{s.low, s.at, s.mass};
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            my_low = min(my_low, __shfl_xor_sync(0xffffffffu, my_low, d));
            my_high = max(my_high, __shfl_xor_sync(0xffffffffu, my_high, d));
        }
        if (lane == 0) atomicMin(&s.low, my_low), atomicMax(&s.high, my_high);
        __syncthreads();
        low = s.low, high = s.high;
        if (low == high) {  // equal logits: so many of them, by rising id
            const u64 e = m.of(exact, logit_of(low));
            uint32_t take = number - n_before;
            if (BY_MASS) take = e == 0 ? 1 : max((u64)1, (mass - m_before + e - 1) / e);
            // warps hold neighbouring ranges of ids; the one in which the last of them lies looks for it
            int u0, u1;
            row.range(warp, NT / 32, u0, u1);
            uint32_t mine = 0;
            row.each_of(u0 + lane, u1, 32, m.mask, [&](float l, int) { mine += order_of(l) == low; });
            mine = warp_sum(mine);
            __syncthreads();
            if (lane == 0) s.counts[warp] = mine;
            __syncthreads();
            const uint32_t w = lane < NT / 32 ? s.counts[lane] : 0;
            uint32_t past = __shfl_sync(0xffffffffu, warp_scan(w), warp) - mine;
            if (past < take && past + mine >= take) {
                for (int unit = u0; unit < u1; unit += 32) {
                    float l[R::VEC];
                    uint32_t n = 0;
                    if (unit + lane < u1) {
                        row.get(unit + lane, l);
#pragma unroll
                        for (int q = 0; q < R::VEC; ++q) n += l[q] > m.mask && order_of(l[q]) == low;
                    }
                    const uint32_t upto = past + warp_scan(n);
                    if (upto >= take && upto - n < take) {
                        uint32_t k = upto - n;
#pragma unroll
                        for (int q = 0; q < R::VEC; ++q)
                            if (l[q] > m.mask && order_of(l[q]) == low && ++k == take) s.at = row.first_id(unit + lane) + q;
                    }
                    past = __shfl_sync(0xffffffffu, upto, 31);
                }
            }
            if (tid == 0) s.mass = m_before + take * e, s.before = s.mass - e;
            __syncthreads();
            return Cut{low, s.at, s.mass};
        }
        shift = 0;
        while (((uint32_t)high - (uint32_t)low) >> shift >= kBuckets) ++shift;
        __syncthreads();
    }
}

// The part f, 0 <= f < 1, of a mass, cut off or rounded up to a whole number: f is a whole number of 24 bits times a power of two
__device__ __forceinline__ u64 share(float f, u64 all, bool up)
{
    const int b = __float_as_int(f), ex = b >> 23;
    if (f == 0.f) return 0;
    const u64 whole = ex ? (b & 0x7fffff) | 0x800000 : b & 0x7fffff;
    const int shift = 126 - max(ex, 1);  // f = whole 2^-24 2^-shift
    const u64 hi = __umul64hi(all, whole << 40), lo = all * (whole << 40);
    const u64 q = shift < 64 ? hi >> shift : 0;
    const bool rest = lo != 0 || (shift < 64 ? q << shift != hi : hi != 0);
    return q + (up && rest);
}

struct Rules {
    uint32_t k;  // 0: all
    float p, min_p, u;
    float log_min_p;
    // masses far enough from min_p are told by float32
    __device__ __forceinline__ bool reaches_min(const Mass &m, float l) const
    {
        if (l == m.top) return true;
        const float z = (l - m.top) * m.c;
        if (fabsf(z - log_min_p) > 1e-5f + 1e-5f * fabsf(log_min_p)) return z > log_min_p;
        return ((double)l - (double)m.top) * (double)m.c >= log((double)min_p);
    }
    __device__ __forceinline__ bool wants_last() const { return u >= 1.f; }  // the last kept id, whatever its mass
    __device__ __forceinline__ u64 target(u64 all) const { return share(u > 0.f ? u : 0.f, all, false); }  // u < 1
};

struct Drawn {
    int id;
    float logprob;
    uint32_t kept;
    bool sure;
};

// The token at which the running mass exceeds the target, given the warps' masses in s.sums and the number kept; mass(l, id) is a token's
// (0 where it is not kept), and the quick ones among them are off by `near` in all at most.
template <int NT, typename S, typename R, typename F>
__device__ Drawn draw_token(S &s, const R &row, const Mass &m, const Rules &rules, u64 near, F mass)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const u64 w = lane < NT / 32 ? s.sums[lane] : 0, incl = warp_scan(w), all = __shfl_sync(0xffffffffu, incl, 31);
    const u64 target = rules.target(all);
    if (tid == 0) s.flag = 0, s.at = -1;
    __syncthreads();
    // the range of the warp in which it lies, by all threads
    const uint32_t here = __ballot_sync(0xffffffffu, incl - w <= target && incl > target);
    const int owner = __ffs(here) - 1;
    u64 past = __shfl_sync(0xffffffffu, incl - w, max(owner, 0));
    int u0 = 0, u1 = 0;
    if (owner >= 0) row.range(owner, NT / 32, u0, u1);
#pragma unroll 1
    for (int unit = u0; unit < u1 && past <= target; unit += NT) {
        float l[R::VEC];
        u64 e[R::VEC], sum = 0;
        const bool in = unit + tid < u1;
        if (in) row.get(unit + tid, l);
#pragma unroll
        for (int q = 0; q < R::VEC; ++q) {
            e[q] = in && l[q] > m.mask ? mass(l[q], row.first_id(unit + tid) + q) : 0;
            sum += e[q];
        }
        const u64 upto = past + block_scan<NT>(sum, s.more);
        if (upto > target && upto - sum <= target) {
            u64 at = upto - sum;
            bool found = false;
#pragma unroll
            for (int q = 0; q < R::VEC; ++q) {
                if (!found && at + e[q] > target) {
                    found = true;
                    s.at = row.first_id(unit + tid) + q;
                    s.top = l[q];
                    s.flag = near == 0 || ((at == 0 || target > at + near) && at + e[q] > target + near);
                }
                at += e[q];
            }
        }
        if (tid == NT - 1) s.mass = upto;
        __syncthreads();
        past = s.mass;
    }
    __syncthreads();
    Drawn d;
    d.id = s.at, d.sure = s.flag, d.kept = 0;
    d.logprob = 0.f;
    if (tid == 0) d.logprob = m.log_share(s.top, all);
    __syncthreads();
    return d;
}

// Any rules and any number of tokens, in passes over the row for each of them; u >= 1 always comes this way (the window's ways would carry
// the search for the last kept id in their registers: 1 to 4 % of every draw).  The last id is taken on the way: with a pass of its own the
// kernel's frame passes 704 bytes, and the process's first plan takes 14 ms instead of 6.5 for more local memory.
template <int NT, typename S, typename R>
__device__ __noinline__ Drawn draw_row(S &s, const R &row, const Mass &m, const Rules &rules, uint32_t live, bool exact)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Cut cut{INT_MIN, INT_MAX, 0};
    const bool by_k = rules.k > 0 && rules.k < live;
    bool sure = true;
    if (by_k) cut = find_cut<NT, false>(s, row, m, exact, rules.k, 0);
    __syncthreads();
    if (rules.p < 1.f) {
        u64 all = cut.mass;
        if (!by_k) {
            uint32_t none = 0;
            all = 0;
            row.template each<NT>(m.mask, [&](float l, int) { all += m.of(exact, l); });
            block_sums<NT>(s, all, none);
        }
        const u64 target = share(fmaxf(rules.p, 0.f), all, true);
        __syncthreads();
        cut = find_cut<NT, true>(s, row, m, exact, 0, target);
        if (!exact) {
            const u64 near = m.slack(all, row.V);
            sure = cut.mass - target > near && (s.before == 0 || target > s.before + near);
        }
        __syncthreads();
    }
    const bool by_min = rules.min_p > 0.f;
    auto mass = [&](float l, int id) { return cut.keeps(order_of(l), id) && (!by_min || rules.reaches_min(m, l)) ? m.of(exact, l) : 0; };
    int u0, u1;
    row.range(warp, NT / 32, u0, u1);
    u64 mine = 0;
    uint32_t kept = 0;
    int last = -1;  // of the thread's own, which it meets by rising id
    float l_last = 0.f;
    row.each_of(u0 + lane, u1, 32, m.mask, [&](float l, int id) {
        if (cut.keeps(order_of(l), id) && (!by_min || rules.reaches_min(m, l))) mine += m.of(exact, l), ++kept, last = id, l_last = l;
    });
    u64 all = mine;
    block_sums<NT>(s, all, kept);  // leaves the warps' masses in s.sums
    if (rules.wants_last()) {
        if (threadIdx.x == 0) s.at = -1;
        __syncthreads();
        if (last >= 0) atomicMax(&s.at, last);
        __syncthreads();
        if (last == s.at) s.top = l_last;
        __syncthreads();
        Drawn d{s.at, 0.f, kept, sure};
        if (threadIdx.x == 0) d.logprob = m.log_share(s.top, all);
        return d;
    }
    Drawn d = draw_token<NT>(s, row, m, rules, exact ? 0 : m.slack(all, row.V), mass);
    d.kept = kept, d.sure = d.sure && sure;
    return d;
}

// The draw from a short list in order, all of whose first `keep` tokens are kept: each counts the mass up to its id, with all threads at work
template <int NT, typename S, typename R, int PER>
__device__ Drawn draw_listed(S &s, const R &row, const Mass &m, const Rules &rules, uint32_t keep, uint32_t per, const u64 (&e)[PER], u64 list_before)
{
    const int tid = threadIdx.x;
    u64 at = list_before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        at += e[i];
        const uint32_t j = per * tid + i;
        if (i < per && j < keep) s.masses[j] = e[i], s.below[j] = 0;
        if (i < per && j + 1 == keep) s.mass = at;
    }
    __syncthreads();
    const u64 all = s.mass, target = rules.target(all);
    int across = 32;
    while (across < (int)keep) across *= 2;
    const int i = tid % across, others = ((int)keep + NT / across - 1) / (NT / across), from = tid / across * others;
    if (i < (int)keep) {
        const int id = id_in(s.list[i]);
        u64 sum = 0;
        for (int o = from; o < min((int)keep, from + others); ++o) sum += id_in(s.list[o]) <= id ? s.masses[o] : 0;
        if (sum > 0) atomicAdd(&s.below[i], sum);
    }
    __syncthreads();
    if (tid < (int)keep && s.below[tid] > target && s.below[tid] - s.masses[tid] <= target) s.at = id_in(s.list[tid]), s.top = logit_of(order_in(s.list[tid]));
    __syncthreads();
    Drawn d;
    d.id = s.at, d.kept = keep, d.sure = true, d.logprob = 0.f;
    if (tid == 0) d.logprob = m.log_share(s.top, all);
    return d;
}

// The row in three passes where that is enough: its largest logit (the caller); numbers of tokens by distance from it, and the
// masses' sum if top-p asks for it; the masses of those that are kept for certain, while those among which the borders lie
// (the window, all candidates where they are few) are listed, to be put in order.
template <int NT, typename S, typename R>
__device__ Drawn draw_window(S &s, const R &row, const Mass &m, Rules rules, float own, uint32_t &live, bool &done)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool by_p = rules.p < 1.f, by_min = rules.min_p > 0.f;
    bool by_k = rules.k > 0;
    constexpr int EACH = kBuckets / NT;
    int first = kBuckets, last = kBuckets - 1;  // the window's buckets: empty
    u64 total = 0;                              // of all masses, quick ones
    uint32_t sure_n = 0, listed_n = 0;
    bool min_ends = by_min;  // the window ends where min_p does, not top-p
    constexpr int VEC = R::VEC;
    auto rough_sum = [&](const float (&l)[VEC]) {
        float e[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) e[q] = l[q] > m.mask ? m.rough(l[q]) : 0.f;
        return m.whole(sum_of<VEC>(e));
    };
    // Candidates by a bound where the rules give one: k of the threads' own largest logits that lie above it, so many of these that they
    // have top-p's mass, or min_p.  (Counting all tokens' buckets takes 10000 cycles of a row of 50021, the threads' largest 1500.)
    const bool by_mass = by_p && !by_k;
    bool few = false;
    if ((by_k && rules.k <= NT * 3 / 4) || by_mass || (by_min && !by_k)) {
        float low = -INFINITY;
        bool found = true;
        if (tid == 0) s.number = 0, s.at = -1;
        if (by_mass) {
            row.units_of(tid, row.units, NT, [&](const float (&l)[VEC], int) { total += rough_sum(l); });
            uint32_t none = 0;
            block_sums<NT>(s, total, none);
        }
        if (by_k || by_mass) {
            for (int i = tid; i < kBuckets; i += NT) s.count[i] = 0;
            __syncthreads();
            // their number, or their mass in 2^-21ths, rounded down
            if (own > m.mask) atomicAdd(&s.count[m.bucket(own)], by_k ? 1u : __float2uint_rz(m.rough(own) * 2097152.f));
            __syncthreads();
            if (by_k) {
                uint32_t n[EACH], nn = 0;
#pragma unroll
                for (int i = 0; i < EACH; ++i) n[i] = s.count[EACH * tid + i], nn += n[i];
                uint32_t at_n = block_scan<NT>(nn, s.counts) - nn;
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    if (at_n < rules.k && at_n + n[i] >= rules.k) s.at = EACH * tid + i;
                    at_n += n[i];
                }
            } else {
                const float part = fmaxf(rules.p * (float)total * __int_as_float((127 - m.fraction) << 23), 1e-30f) * 1.0001f;
                float d[EACH], dd = 0.f;
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    d[i] = (float)s.count[EACH * tid + i] * (1.f / 2097152.f), dd += d[i];
                }
                float at_d = block_scan<NT>(dd, reinterpret_cast<float *>(s.sums)) - dd;
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    if (at_d < part && at_d + d[i] >= part) s.at = EACH * tid + i;
                    at_d += d[i];
                }
            }
            __syncthreads();
            found = s.at >= 0 && s.at + 1 < kBuckets;  // the last bucket has no lower end
            if (found) low = -((float)s.at + 1.05f) / kPerOctave;
        }
        if (by_min && !(by_k && by_p)) {  // the first k are needed for their mass
            low = fmaxf(low, rules.log_min_p * 1.442695f * 1.0001f - 1e-4f);
            found |= by_mass;
        }
        if (found) {
            __syncthreads();
            bool room = true;  // too many are not counted to the end
            row.units_of(tid, row.units, NT, [&](const float (&l)[VEC], int id) {
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    if (m.log_of(l[q]) >= low && l[q] > m.mask && room) {
                        const uint32_t to = atomicAdd(&s.number, 1u);
                        if (to < S::kCandidates) s.list[to] = listed(order_of(l[q]), id + q);
                        else room = false;
                    }
            });
            __syncthreads();
            listed_n = s.number;
            few = listed_n <= S::kCandidates;
            if (few) first = 0, live = row.V + 1;  // k of them at least are live
            else listed_n = 0;
            __syncthreads();
        }
    }
    if (!few && (by_p || by_k || by_min)) {
        for (int i = tid; i < kBuckets; i += NT) s.count[i] = s.lo[i] = 0;
        if (tid == 0) s.first = s.last = kBuckets - 1, s.number = 0;
        __syncthreads();
        // with top-p the places within the buckets are added up too, which brings the masses' bounds together
        auto count_places = [&](const float (&l)[VEC]) {
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                if (l[q] > m.mask) {
                    const uint32_t x = m.place(l[q]);
                    atomicAdd(&s.count[x >> kPlaceBits], 1u), atomicAdd(&s.lo[x >> kPlaceBits], x & ((1 << kPlaceBits) - 1));
                }
        };
        auto add_places = [&](const float (&l)[VEC]) {
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                if (l[q] > m.mask) {
                    const uint32_t x = m.place(l[q]);
                    atomicAdd(&s.lo[x >> kPlaceBits], x & ((1 << kPlaceBits) - 1));
                }
        };
        auto count = [&](const float (&l)[VEC]) {
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                if (l[q] > m.mask) atomicAdd(&s.count[m.bucket(l[q])], 1u);
        };
        if (by_mass) row.units_of(tid, row.units, NT, [&](const float (&l)[VEC], int) { count_places(l); });
        else row.units_of(tid, row.units, NT, [&](const float (&l)[VEC], int) { count(l); });
        uint32_t none = 0, n[EACH], nn = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) n[i] = s.count[EACH * tid + i], nn += n[i];
        uint32_t at_n = block_scan<NT>(nn, s.counts) - nn;
        if (tid == NT - 1) s.number_before = at_n + nn;
        __syncthreads();
        live = s.number_before;
        // Whether k is a rule has to stand before anything is made for the others: one that reaches all tokens leaves top-p to find its end as
        // if it were alone, by the mass of all of them, their places and both bounds' running sums.
        if (by_k && rules.k >= live) {
            by_k = false;
            if (by_p) {
                total = 0;
                row.units_of(tid, row.units, NT, [&](const float (&l)[VEC], int) { total += rough_sum(l), add_places(l); });
                block_sums<NT>(s, total, none);
            }
        }
        // Running numbers, and bounds of the running masses: with t = log 2 / 32 times the tokens' mean place in their bucket b, their mean mass
        // is between (1 - t) and (1 - t + t^2 / 2) 2^(-b / 32) where t may be any in 0 .. log 2 / 32; the last bucket's tokens lie anywhere
        // beyond.  (A sum of places stays below 2^32 for 2^19 tokens of a bucket; longer rows do without.)
        float up[EACH], down[EACH], uu = 0.f, dd = 0.f;
        const bool places = by_p && !by_k && row.V <= (1 << 19);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = EACH * tid + i;
            const float whole = (float)n[i] * exp2f(-(float)b / kPerOctave), t = places && n[i] > 0 ? 0.02166085f * (float)s.lo[b] / ((float)(1 << kPlaceBits) * (float)n[i]) : 0.f;
            up[i] = whole * (1.f - t + (places ? 2.4e-4f : 0.f)), uu += up[i];
            down[i] = b + 1 == kBuckets ? 0.f : whole * (places ? 1.f - t : 0.97857f), dd += down[i];
        }
        float at_u = 0.f, at_d = 0.f;
        if (by_p && !by_k) {
            at_u = block_scan<NT>(uu, reinterpret_cast<float *>(s.sums)) - uu;
            at_d = block_scan<NT>(dd, reinterpret_cast<float *>(s.more)) - dd;
        }
        // Each rule ends the prefix in a bucket that is known (k) or known to a few (p, min_p); the window reaches from the first of these to
        // the first by which one of them has ended.  k and p together need the first k's mass: all of them are candidates.
        const float part = by_k ? 0.f : fmaxf(rules.p * (float)total * __int_as_float((127 - m.fraction) << 23), 1e-30f);
        const float at_min = by_min ? fmaxf(-rules.log_min_p, 0.f) * (1.442695f * kPerOctave) : 0.f;
        const int b_min = by_min ? (int)fminf((float)(kBuckets - 1), at_min * 1.00001f + 1.5f) : kBuckets - 1;
        if (tid == 0) {
            if (by_k && by_p) s.first = 0;
            else if (by_min) atomicMin(&s.first, (int)fminf((float)(kBuckets - 1), fmaxf(at_min * 0.99999f - 1.5f, 0.f)));
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = EACH * tid + i;
            if (by_k && at_n < rules.k && at_n + n[i] >= rules.k) atomicMin(&s.last, b), atomicMin(&s.first, b);
            if (by_p && !by_k) {
                // the first bucket by whose end the mass may, and the first by whose end it must have been reached.  Two threads' sums up to the
                // buckets between them differ in their last bits: what a bucket starts from is told with room for that, so that none is left
                // out between them, and the first of those told apart by their ends counts.
                if (at_u * 0.9999f < part && (at_u + up[i]) * 1.00002f >= part) atomicMin(&s.first, b);
                if (at_d * 0.9999f < part && (at_d + down[i]) * 0.99998f >= part) atomicMin(&s.last, b);
            }
            if (by_min && b == b_min && !(by_k && by_p)) atomicMin(&s.last, b);  // the first k are needed for their mass
            at_n += n[i], at_u += up[i], at_d += down[i];
        }
        __syncthreads();
        first = s.first, last = s.last;
        min_ends = by_min && last == b_min;
        __syncthreads();
        // the tokens before and in the window; where all candidates are few, the window begins at the first
        uint32_t before = 0, upto = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = EACH * tid + i;
            if (b < first) before += n[i];
            if (b <= last) upto += n[i];
        }
        u64 both = (u64)before << 32 | upto;
        block_sums<NT>(s, both, none);
        before = (uint32_t)(both >> 32), upto = (uint32_t)both;
        if (!by_p && !by_k && !by_min) first = kBuckets;  // top_k reaches all of them
        else if (upto <= (first == 0 ? S::kCandidates : 1024)) first = 0;  // sorting more takes longer than adding up what is before the window
        else if (first == 0 || upto - before > S::kCandidates) {
            done = false;
            return Drawn{};
        }
        sure_n = first == kBuckets ? live : first == 0 ? 0 : before;
        listed_n = first == kBuckets ? 0 : upto - sure_n;
        if (by_p && first > 0 && listed_n == 0 && !min_ends) {  // top-p ends somewhere: without a window that is for the passes to find
            done = false;
            return Drawn{};
        }
    }
    // the masses that are kept for certain, and the window's list
    int u0, u1;
    row.range(warp, NT / 32, u0, u1);
    u64 mine = 0;
    uint32_t passed = 0;
    auto list_up = [&](float l, int id) {
        if (l > m.mask) s.list[atomicAdd(&s.number, 1u)] = listed(order_of(l), id);
    };
    if (first == kBuckets) {
        row.units_of(u0 + lane, u1, 32, [&](const float (&l)[VEC], int) {
            float e[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const bool in = l[q] > m.mask;
                e[q] = in ? m.rough(l[q]) : 0.f, passed += in;
            }
            mine += m.whole(sum_of<VEC>(e));
        });
    } else if (few) {
    } else if (first == 0) {
        row.units_of(tid, row.units, NT, [&](const float (&l)[VEC], int id) {
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                if (m.bucket(l[q]) <= last) list_up(l[q], id + q);
        });
    } else {
        row.units_of(u0 + lane, u1, 32, [&](const float (&l)[VEC], int id) {
            float e[VEC];
            bool some = false;
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const int b = m.bucket(l[q]);
                e[q] = 0.f;
                if (b < first) e[q] = m.rough(l[q]), some = true;  // above the mask, as the window is
                else if (b <= last) list_up(l[q], id + q);
            }
            if (some) mine += m.whole(sum_of<VEC>(e));
        });
    }
    if (first == kBuckets && !(by_p || by_k || by_min)) {
        u64 none = 0;
        block_sums<NT>(s, none, passed);
        live = sure_n = passed;
    }
    __syncthreads();
    if (listed_n > 0) sort_list<NT>(s, listed_n);
    constexpr int PER = S::kCandidates / NT;
    const uint32_t per = listed_n <= NT ? 1 : PER;  // neighbouring tokens a thread
    auto place = [&](int i) { return i < (int)per ? (int)per * tid + i : INT_MAX - 1; };
    u64 e[PER], of_list = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        e[i] = place(i) < (int)listed_n ? m.exact(logit_of(order_in(s.list[place(i)]))) : 0;
        of_list += e[i];
    }
    const u64 list_before = listed_n > 0 ? block_scan<NT>(of_list, s.sums) - of_list : 0;
    for (int again = 0; again < 3; ++again) {  // with rough masses, if a border is too near with close ones, and then with exact ones
        if (again) {
            if (tid < 64) s.roots[tid] = (u64)(kRoots[tid].x * 2147483648.f) << (m.fraction - 31);
            __syncthreads();
            if (tid < 64) s.roots[tid] += (u64)(long long)rintf(ldexpf(kRoots[tid].y, m.fraction));
            __syncthreads();
            mine = total = 0;
            const bool others = by_p && !by_k;
            row.units_of(u0 + lane, u1, 32, [&](const float (&l)[VEC], int) {
                u64 of_sure = 0, of_others = 0;
                float rest_sure = 0.f, rest_others = 0.f;
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    const bool sure = first == kBuckets ? l[q] > m.mask : m.bucket(l[q]) < first;
                    if (!sure && !(others && l[q] > m.mask)) continue;
                    float rest = 0.f;
                    const u64 x = again == 2 ? m.exact(l[q]) : m.close(l[q], s.roots, rest);
                    if (sure) of_sure += x, rest_sure += rest;
                    else of_others += x, rest_others += rest;
                }
                const u64 x = m.close_whole(of_sure, rest_sure);
                mine += x, total += x + m.close_whole(of_others, rest_others);
            });
            uint32_t none = 0;
            block_sums<NT>(s, total, none);
        }
        u64 sure_mass = 0, warp_mass = 0;
        if (first > 0) {
            uint32_t none = 0;
            sure_mass = mine;
            block_sums<NT>(s, sure_mass, none);
            warp_mass = s.sums[warp];
            __syncthreads();
        }
        // the number of the list's tokens that are kept
        uint32_t keep = listed_n;
        if (listed_n > 0) {
            if (tid == 0) s.number = listed_n, s.mass = 0;
            __syncthreads();
            if (by_k) keep = min(keep, rules.k - sure_n);
            if (by_min) {  // those before the window reach it all
                uint32_t reach = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) reach += place(i) < (int)listed_n && rules.reaches_min(m, logit_of(order_in(s.list[place(i)])));
                u64 zero = 0;
                block_sums<NT>(s, zero, reach);
                keep = min(keep, reach);
            }
            if (by_p) {
                if (by_k) {  // the mass of the first k, all of them in the list
                    u64 at = list_before;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        at += e[i];
                        if (place(i) + 1 == (int)min(rules.k, listed_n)) s.mass = at;
                    }
                    __syncthreads();
                    total = s.mass;
                }
                const u64 target = share(fmaxf(rules.p, 0.f), total, true), near = by_k || again == 2 ? 0 : again ? m.close_slack(total, row.V) : m.slack(total, row.V);
                if (tid == 0) s.flag = 1;
                __syncthreads();
                u64 at = sure_mass + list_before;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int j = place(i);
                    if (j < (int)listed_n && at + e[i] >= target && (at < target || j == 0)) {
                        s.number = j + 1;
                        if (near && (at + e[i] - target <= near || (at != 0 && target <= at + near))) s.flag = 0;
                        if (j == 0 && at >= target && at != 0) s.flag = 0;  // reached before the window: only for quick masses' errors
                    }
                    // or behind it: where min_p ends the window that is as it should be, if it is certain
                    if (j + 1 == (int)listed_n && at + e[i] < target && !by_k && (!min_ends || target - (at + e[i]) <= near)) s.flag = 0;
                    at += e[i];
                }
                __syncthreads();
                const bool ok = s.flag;
                keep = min(keep, s.number);
                __syncthreads();
                if (!ok) continue;
            }
            if (sure_n == 0) keep = max(keep, 1u);
        }
        if (first == 0 && keep <= kCounted) return draw_listed<NT>(s, row, m, rules, keep, per, e, list_before);
        // the warps' masses with the list's share
        Cut cut{INT_MAX, -1, 0};  // of the window's tokens
        if (keep > 0 && listed_n > 0) cut = Cut{order_in(s.list[keep - 1]), id_in(s.list[keep - 1]), 0};
        if (lane == 0) s.sums[warp] = warp_mass;
        __syncthreads();
        const int each = (row.units + NT / 32 - 1) / (NT / 32);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (place(i) < (int)keep) atomicAdd(&s.sums[(id_in(s.list[place(i)]) + row.skew) / R::VEC / each], e[i]);
        __syncthreads();
        const u64 near = first == 0 || again == 2 ? 0 : again ? m.close_slack(sure_mass, row.V) : m.slack(sure_mass, row.V);
        auto mass = [&](float l, int id) -> u64 {
            if (first > 0 && (first == kBuckets || m.bucket(l) < first)) return again == 2 ? m.exact(l) : again ? m.close(l, s.roots) : m.quick(l);
            return cut.keeps(order_of(l), id) ? m.exact(l) : 0;
        };
        Drawn d = draw_token<NT>(s, row, m, rules, near, mass);
        if (d.sure) {
            d.kept = sure_n + keep;
            return d;
        }
    }
    done = false;
    return Drawn{};
}

template <typename T, int NT, bool RESIDENT>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_kernel(const Params<T> p)
{
    using R = Row<T, RESIDENT>;
    extern __shared__ uint4 copy[];
    __shared__ Shared<RESIDENT && NT < 1024 ? 1024 : 2048> s;  // the window of a longer row holds more
    const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    R row(p.logits + (size_t)i * p.ld, p.V);
    if constexpr (RESIDENT) row.template copy_to<NT>(copy);
    const float c = p.inv_temperature ? p.inv_temperature[i] : 1.f;
    const bool usable = c >= 0x1p-60f && c <= 0x1p126f;
    float top = -INFINITY;  // NaN if there is one
    row.units_of(tid, row.units, NT, [&](const float (&l)[R::VEC], int) {
#pragma unroll
        for (int e = 0; e < R::VEC; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(l[e]));
    });
    const float own = top;
    // as whole numbers, of which the one NaN that max.NaN gives is the largest
    const int warp_top = __reduce_max_sync(0xffffffffu, order_of(top));
    if (lane == 0) s.counts[warp] = warp_top;
    __syncthreads();
    top = logit_of(__reduce_max_sync(0xffffffffu, lane < NT / 32 ? (int)s.counts[lane] : INT_MIN));
    __syncthreads();
    const bool bad = !(top < INFINITY);  // NaN or +inf
    const float mask = usable ? mask_of(c) : 0.f;
    if (!usable || bad || !(top > mask)) {
        if (tid == 0) {
            if (!usable) atomicCAS(p.status, 0, kDevTemperature);
            p.ids[i] = -1;
            if (p.logprob) p.logprob[i] = usable && !bad ? -INFINITY : NAN;
            if (p.kept) p.kept[i] = 0;
        }
        return;
    }
    const Mass m(top + 0.f, mask, c, p.fraction);
    Rules rules;
    rules.u = p.u[i];
    rules.k = p.top_k ? (uint32_t)max(p.top_k[i], 0) : 0;
    rules.p = p.top_p ? p.top_p[i] : 1.f;
    if (rules.p != rules.p) rules.p = 1.f;
    rules.min_p = p.min_p ? p.min_p[i] : 0.f;
    if (rules.min_p != rules.min_p) rules.min_p = 0.f;
    rules.log_min_p = rules.min_p > 0.f ? logf(rules.min_p) : 0.f;
    if (rules.k >= (uint32_t)p.V) rules.k = 0;  // all of them: no rule
    if (rules.min_p > 1.f) rules.k = 1, rules.p = 1.f, rules.min_p = 0.f;  // nothing reaches it: the first token alone
    uint32_t live = 0;
    bool done = !rules.wants_last();
    Drawn d;
    if (done) {
        d = draw_window<NT>(s, row, m, rules, own, live, done);
    } else {
        row.template each<NT>(mask, [&](float, int) { ++live; });
        u64 none = 0;
        block_sums<NT>(s, none, live);
    }
    if (!done) {
        __syncthreads();
        d = draw_row<NT>(s, row, m, rules, live, false);
        __syncthreads();
        if (!d.sure) d = draw_row<NT>(s, row, m, rules, live, true);
    }
    if (tid == 0) {
        p.ids[i] = d.id;
        if (p.logprob) p.logprob[i] = d.logprob;
        if (p.kept) p.kept[i] = (int)d.kept;
    }
}

// Shared memory for a row where one or two blocks share an SM, beside what the kernel has of its own and the system's 1024 bytes
constexpr size_t room(int blocks) { return (233472 / blocks - (blocks > 1 ? sizeof(Shared<1024>) : sizeof(Shared<2048>)) - 1024) / 16 * 16; }

template <typename T>
cudaError_t prepare()
{
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, 512, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)room(2));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T, 1024, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)room(1));
    return e;
}

template <typename T>
cudaError_t run(const SampleArgs &a, const TokenLaunch &l)
{
    int bits = 0;
    while ((1ll << bits) < a.V) ++bits;
    const Params<T> p{(const T *)a.logits, a.ld, a.u, a.inv_temperature, a.top_k, a.top_p, a.min_p, a.ids, a.logprob, a.kept, a.n, a.V,
                      bits <= 19 ? 44 : 63 - bits, l.d_status};  // the masses' sum fits 64 bits
    l.timer->begin("sample");
    // Short rows take few threads, whose barriers cost less (16 x 1000 float32: 8).  Many rows: two on an SM, so that one computes while the
    // other waits, as long as two fit its shared memory (512 x 50021 with top-k 50: 39 in bf16, which fits, 68 in float32).  Rows that do
    // not fit are read again from L2.
    const size_t bytes = ((size_t)a.V * sizeof(T) + 30) / 16 * 16;
    if (bytes <= 16384) sample_kernel<T, 256, true><<<a.n, 256, bytes, l.timer->stream>>>(p);
    else if (a.n > l.sm_count && bytes <= room(2)) sample_kernel<T, 512, true><<<a.n, 512, bytes, l.timer->stream>>>(p);
    else if (bytes <= room(1)) sample_kernel<T, 1024, true><<<a.n, 1024, bytes, l.timer->stream>>>(p);
    else sample_kernel<T, 1024, false><<<a.n, 1024, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace draw
}  // namespace prism
