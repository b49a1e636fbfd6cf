// Drawing a token from logits under temperature, top-k, top-p and min-p, given a number u in [0, 1) for each row.
//
// With z = c logits, the tokens ordered by falling logit and then by rising id, the row keeps the shortest of three prefixes:
// the first k; the fewest whose mass sum e^(z - max) reaches p of that of the first k; those with e^(z - max) >= min_p.  The
// token is the first, by rising id, at which the kept tokens' running mass exceeds u times their mass.
//
// The choices are whole numbers, so the masses are whole numbers too: multiples of 2^-F of the first token's (F = 44, less
// for more than 2^19 tokens), whose sums have no rounding and no order.  They are computed twice.  First from the
// machine's base-2 exponential, within 2^-21 of the exact ones; if a border comes nearer to a token's edge than these
// errors reach, the row is done again with masses exact to the last place (about 50 operations a token).
#include "io_util.h"
#include "prism_tokens.h"

namespace prism {
namespace draw {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBuckets = 2048, kPerOctave = 64;  // of the first cut by distance from the row's largest logit
constexpr int kList = 1024;                      // tokens that a border's bucket may hold to be put in order directly
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

__device__ __forceinline__ bool masked(float l, float c) { return !(l > kLowest) || l * c == -INFINITY; }

// A whole number that orders as the logit does (both zeros alike)
__device__ __forceinline__ int order_of(float l)
{
    const int b = __float_as_int(l + 0.f);
    return b ^ ((b >> 31) & 0x7fffffff);
}

struct Mass {
    float top, c, kh, kl;  // the row's largest logit, c and c log2 e in two parts
    int fraction;
    float hi_scale, lo_scale;

    __device__ __forceinline__ Mass(float top_, float c_, int fraction_) : top(top_), c(c_), fraction(fraction_)
    {
        kh = c * 1.44269502162933349609375f;
        kl = fmaf(c, 1.44269502162933349609375f, -kh) + c * 1.925963033500011079e-8f;
        hi_scale = __int_as_float((127 + fraction - 22) << 23), lo_scale = 4194304.f;
    }
    // l - top in two parts, the second its rounding error
    __device__ __forceinline__ void below(float l, float &dh, float &dl) const
    {
        dh = l - top;
        const float back = dh - l;
        dl = (l - (dh - back)) + (-top - back);
    }
    // within 2^-21 of itself and half a unit
    __device__ __forceinline__ u64 quick(float l) const
    {
        float dh, dl;
        below(l, dh, dl);
        const float y = dh * kh;
        if (!(y > -46.f)) return 0;
        const float yl = fmaf(dh, kh, -y) + fmaf(dh, kl, dl * kh);
        float e;
        asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(y));
        e = fmaf(e, yl * 0.693147180559945f, e) * hi_scale;
        const uint32_t hi = __float2uint_rz(e);
        return ((u64)hi << 22) + __float2uint_rn((e - (float)hi) * lo_scale);
    }
    // within two units: e^x = 2^(n / 64) e^t, |t| <= log 2 / 128, with x, t and the result in two floats each; e^t - 1 by its
    // series, of which all but the first two terms are below 2^-24
    __device__ __forceinline__ u64 exact(float l) const
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
    template <bool EXACT>
    __device__ __forceinline__ u64 of(float l) const { return EXACT ? exact(l) : quick(l); }
};

// A prefix of the order: the tokens above `order`, and those at it whose id is at most `id`
struct Cut {
    int order, id;
    u64 mass;  // of the prefix
    __device__ __forceinline__ bool keeps(int o, int i) const { return o > order || (o == order && i <= id); }
};

struct Shared {
    uint32_t count[kBuckets], lo[kBuckets], hi[kBuckets];
    int list_order[kList], list_id[kList];
    u64 sums[kWarps];
    uint32_t counts[kWarps];
    u64 mass, before;
    uint32_t number, number_before;
    int at, low, high;
    float top;
    int flag;
};

// A row and the block's way through it: units of 16 bytes from the last boundary at or before the row's start
template <typename T>
struct Row {
    static constexpr int VEC = 16 / (int)sizeof(T);
    const T *p;
    int V, skew, units;
    __device__ __forceinline__ Row(const T *row, int V_) : p(row), V(V_)
    {
        skew = (int)((uintptr_t)row % 16 / sizeof(T));
        units = (int)(((long long)skew + V + VEC - 1) / VEC);
    }
    __device__ __forceinline__ int first_id(int unit) const { return unit * VEC - skew; }
    __device__ __forceinline__ void get(int unit, float (&f)[VEC]) const
    {
        const int id = first_id(unit);
        if (id >= 0 && id + VEC <= V) {
            io::load_unit<T, VEC>(p + id).get(f);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = id + e >= 0 && id + e < V ? io::ld(p + id + e) : -INFINITY;
        }
    }
    // f(logit, id) for each unmasked token, the block's threads side by side
    template <typename F>
    __device__ __forceinline__ void each(float c, F f) const
    {
        for (int unit = threadIdx.x; unit < units; unit += kThreads) {
            float l[VEC];
            get(unit, l);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (!masked(l[e], c)) f(l[e], first_id(unit) + e);
        }
    }
};

template <typename V>
__device__ __forceinline__ V warp_sum(V v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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
__device__ __forceinline__ void block_sums(Shared &s, u64 &mass, uint32_t &number)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    mass = warp_sum(mass), number = warp_sum(number);
    __syncthreads();
    if (lane == 0) s.sums[warp] = mass, s.counts[warp] = number;
    __syncthreads();
    mass = warp_sum(s.sums[lane]), number = warp_sum(s.counts[lane]);
}

// The smallest prefix with at least `number` tokens (BY_MASS: of at least `mass`) of the tokens ordered.
template <bool EXACT, bool BY_MASS, typename T>
__device__ Cut find_cut(Shared &s, const Row<T> &row, const Mass &m, uint32_t number, u64 mass)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float scale = m.kh * kPerOctave;
    auto bucket_of = [&](float l) { return min(kBuckets - 1, __float2int_rz((m.top - l) * scale)); };
    uint32_t n_before = 0;  // of the tokens above the range at hand
    u64 m_before = 0;
    int low = INT_MIN, high = INT_MAX, shift = 0;  // the range, of order_of
    for (int level = 0;; ++level) {
        auto inside = [&](int o) { return o >= low && o <= high; };
        auto place = [&](float l, int o) { return level == 0 ? bucket_of(l) : (int)(((uint32_t)high - (uint32_t)o) >> shift); };
        for (int i = tid; i < kBuckets; i += kThreads) s.count[i] = s.lo[i] = s.hi[i] = 0;
        if (tid == 0) s.low = INT_MAX, s.high = INT_MIN, s.at = -1, s.number = 0;
        __syncthreads();
        row.each(m.c, [&](float l, int) {
            const int o = order_of(l);
            if (!inside(o)) return;
            const int b = place(l, o);
            atomicAdd(&s.count[b], 1u);
            const u64 e = m.of<EXACT>(l);
            const uint32_t add = (uint32_t)e, old = atomicAdd(&s.lo[b], add), up = (uint32_t)(e >> 32) + (old + add < old);
            if (up) atomicAdd(&s.hi[b], up);
        });
        __syncthreads();
        {  // the bucket at which the running number (mass) reaches what is asked for
            const int b = 2 * tid;
            const uint32_t n0 = s.count[b], n1 = s.count[b + 1];
            const u64 m0 = (u64)s.hi[b] << 32 | s.lo[b], m1 = (u64)s.hi[b + 1] << 32 | s.lo[b + 1];
            uint32_t nn = warp_scan(n0 + n1);
            u64 mm = warp_scan(m0 + m1);
            if (lane == 31) s.counts[warp] = nn, s.sums[warp] = mm;
            __syncthreads();
            const uint32_t nw = warp_scan(s.counts[lane]) - s.counts[lane];
            const u64 mw = warp_scan(s.sums[lane]) - s.sums[lane];
            nn += n_before + __shfl_sync(0xffffffffu, nw, warp), mm += m_before + __shfl_sync(0xffffffffu, mw, warp);
            const uint32_t na = nn - n1, nb = na - n0;  // after the first bucket, before it
            const u64 ma = mm - m1, mb = ma - m0;
            auto here = [&](uint32_t nb_, u64 mb_, uint32_t na_, u64 ma_) {
                return na_ > nb_ && (BY_MASS ? (mb_ < mass || (mass == 0 && nb_ == 0)) && ma_ >= mass : nb_ < number && na_ >= number);
            };
            __syncthreads();
            if (here(nb, mb, na, ma)) s.at = b, s.number = n0, s.number_before = nb, s.before = mb;
            if (here(na, ma, nn, mm)) s.at = b + 1, s.number = n1, s.number_before = na, s.before = ma;
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
        row.each(m.c, [&](float l, int id) {
            const int o = order_of(l);
            if (!inside(o) || place(l, o) != at) return;
            my_low = min(my_low, o), my_high = max(my_high, o);
            if (held <= kList) {
                const uint32_t to = atomicAdd(&s.number, 1u);
                s.list_order[to] = o, s.list_id[to] = id;
            }
        });
        if (held <= kList) {  // put in order by counting who comes before
            __syncthreads();
            int o = 0, id = 0;
            uint32_t rank = 0;
            if (tid < held) {
                o = s.list_order[tid], id = s.list_id[tid];
                for (uint32_t i = 0; i < held; ++i) {
                    const int oi = s.list_order[i];
                    rank += oi > o || (oi == o && s.list_id[i] < id);
                }
            }
            __syncthreads();
            if (tid < held) s.list_order[rank] = o, s.list_id[rank] = id;
            __syncthreads();
            u64 e = 0;
            if (tid < held) {
                o = s.list_order[tid], id = s.list_id[tid];
                e = m.of<EXACT>(__int_as_float(o ^ ((o >> 31) & 0x7fffffff)));
            }
            u64 mm = warp_scan(e);
            if (lane == 31) s.sums[warp] = mm;
            __syncthreads();
            const u64 mw = warp_scan(s.sums[lane]) - s.sums[lane];
            mm += m_before + __shfl_sync(0xffffffffu, mw, warp);
            const uint32_t nn = n_before + tid + 1;
            const bool reaches = tid < held && (BY_MASS ? mm >= mass && (mm - e < mass || (mass == 0 && nn == 1)) : nn == number);
            if (reaches) s.low = o, s.at = id, s.mass = mm, s.before = mm - e;
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
            const u64 e = m.of<EXACT>(__int_as_float(low ^ ((low >> 31) & 0x7fffffff)));
            uint32_t take = number - n_before;
            if (BY_MASS) take = e == 0 ? 1 : max((u64)1, (mass - m_before + e - 1) / e);
            // warps hold neighbouring ranges of ids; the one in which the last of them lies looks for it
            const int each = (row.units + kWarps - 1) / kWarps, u0 = min(row.units, warp * each), u1 = min(row.units, u0 + each);
            uint32_t mine = 0;
            for (int unit = u0 + lane; unit < u1; unit += 32) {
                float l[Row<T>::VEC];
                row.get(unit, l);
#pragma unroll
                for (int q = 0; q < Row<T>::VEC; ++q) mine += !masked(l[q], m.c) && order_of(l[q]) == low;
            }
            mine = warp_sum(mine);
            if (lane == 0) s.counts[warp] = mine;
            __syncthreads();
            const uint32_t incl = warp_scan(s.counts[lane]);
            uint32_t past = __shfl_sync(0xffffffffu, incl, warp) - mine;
            if (past < take && past + mine >= take) {
                for (int unit = u0; unit < u1; unit += 32) {
                    float l[Row<T>::VEC];
                    uint32_t n = 0;
                    if (unit + lane < u1) {
                        row.get(unit + lane, l);
#pragma unroll
                        for (int q = 0; q < Row<T>::VEC; ++q) n += !masked(l[q], m.c) && order_of(l[q]) == low;
                    }
                    const uint32_t upto = past + warp_scan(n);
                    if (upto >= take && upto - n < take) {
                        uint32_t k = upto - n;
#pragma unroll
                        for (int q = 0; q < Row<T>::VEC; ++q)
                            if (!masked(l[q], m.c) && order_of(l[q]) == low && ++k == take) s.at = row.first_id(unit + lane) + q;
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

struct Rules {
    uint32_t k;  // 0: all
    float p, min_p;
    double log_min_p;
};

struct Drawn {
    int id;
    float logprob;
    uint32_t kept;
    bool sure;
};

template <bool EXACT, typename T>
__device__ Drawn draw_row(Shared &s, const Row<T> &row, const Mass &m, const Rules &rules, uint32_t live, float u, int V)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Cut cut{INT_MIN, INT_MAX, 0};
    const bool by_k = rules.k > 0 && rules.k < live;
    bool sure = true;
    if (by_k) cut = find_cut<EXACT, false>(s, row, m, rules.k, 0);
    if (rules.p < 1.f) {
        u64 all = cut.mass;
        if (!by_k) {
            uint32_t none = 0;
            all = 0;
            row.each(m.c, [&](float l, int) { all += m.of<EXACT>(l); });
            block_sums(s, all, none);
        }
        const double part = fmax((double)rules.p, 0.0) * (double)all;
        const u64 target = (u64)ceil(part);
        __syncthreads();
        cut = find_cut<EXACT, true>(s, row, m, 0, target);
        if (!EXACT) {
            const u64 near = (all >> 20) + V;
            sure = cut.mass - target > near && (s.before == 0 || target > s.before + near);
        }
        __syncthreads();
    }
    // masses far enough from min_p are told by float32
    const bool by_min = rules.min_p > 0.f;
    const float lm = (float)rules.log_min_p, slack = 1e-5f + 1e-5f * fabsf(lm);
    auto member = [&](float l, int id) {
        if (!cut.keeps(order_of(l), id)) return false;
        if (!by_min || l == m.top) return !by_min || rules.min_p <= 1.f;
        const float z = (l - m.top) * m.c;
        if (fabsf(z - lm) > slack) return z > lm;
        return ((double)l - (double)m.top) * (double)m.c >= rules.log_min_p;
    };
    // warps hold neighbouring ranges of ids
    const int each = (row.units + kWarps - 1) / kWarps, u0 = min(row.units, warp * each), u1 = min(row.units, u0 + each);
    u64 mine = 0;
    uint32_t count = 0;
    for (int unit = u0 + lane; unit < u1; unit += 32) {
        float l[Row<T>::VEC];
        row.get(unit, l);
#pragma unroll
        for (int q = 0; q < Row<T>::VEC; ++q)
            if (!masked(l[q], m.c) && member(l[q], row.first_id(unit) + q)) mine += m.of<EXACT>(l[q]), ++count;
    }
    mine = warp_sum(mine), count = warp_sum(count);
    __syncthreads();
    if (lane == 0) s.sums[warp] = mine, s.counts[warp] = count;
    if (tid == 0) s.at = -1, s.flag = 1;
    __syncthreads();
    const u64 incl = warp_scan(s.sums[lane]), all = __shfl_sync(0xffffffffu, incl, 31);
    const uint32_t kept = warp_sum(s.counts[lane]);
    const u64 target = u >= 1.f ? all - 1 : min(all - 1, (u64)((double)(u > 0.f ? u : 0.f) * (double)all));
    u64 past = __shfl_sync(0xffffffffu, incl, warp) - mine;
    if (past <= target && past + mine > target) {  // this warp's range
        for (int unit = u0; unit < u1; unit += 32) {
            float l[Row<T>::VEC];
            u64 e[Row<T>::VEC], sum = 0;
            const bool in = unit + lane < u1;
            if (in) row.get(unit + lane, l);
#pragma unroll
            for (int q = 0; q < Row<T>::VEC; ++q) {
                e[q] = in && !masked(l[q], m.c) && member(l[q], row.first_id(unit + lane) + q) ? m.of<EXACT>(l[q]) : 0;
                sum += e[q];
            }
            const u64 upto = past + warp_scan(sum);
            const bool here = upto > target && upto - sum <= target;
            if (here) {
                u64 at = upto - sum;
                bool found = false;
#pragma unroll
                for (int q = 0; q < Row<T>::VEC; ++q) {
                    if (!found && at + e[q] > target) {
                        found = true;
                        s.at = row.first_id(unit + lane) + q;
                        s.top = l[q];
                        s.mass = e[q];
                        if (!EXACT && u < 1.f) {
                            const u64 near = (all >> 20) + V;
                            s.flag = (at == 0 || target > at + near) && (at + e[q] == all || at + e[q] > target + near);
                        }
                    }
                    at += e[q];
                }
            }
            if (__any_sync(0xffffffffu, here)) break;
            past = __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    __syncthreads();
    Drawn d;
    d.id = s.at, d.kept = kept, d.sure = sure && s.flag;
    d.logprob = 0.f;
    if (tid == 0) d.logprob = (float)(((double)s.top - (double)m.top) * (double)m.c - log(ldexp((double)all, -m.fraction)));
    __syncthreads();
    return d;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const Params<T> p)
{
    __shared__ Shared s;
    const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row<T> row(p.logits + (size_t)i * p.ld, p.V);
    const float c = p.inv_temperature ? p.inv_temperature[i] : 1.f;
    const bool usable = c >= 0x1p-60f && c <= 0x1p126f;
    float top = -INFINITY;
    uint32_t live = 0;
    bool bad = false;  // NaN or +inf
    for (int unit = tid; unit < row.units; unit += kThreads) {
        float l[Row<T>::VEC];
        row.get(unit, l);
#pragma unroll
        for (int e = 0; e < Row<T>::VEC; ++e) {
            bad |= !(l[e] < INFINITY);
            if (!masked(l[e], c)) top = fmaxf(top, l[e]), ++live;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s.sums[warp] = (u64)__float_as_uint(top);
    const bool any_bad = __syncthreads_or(bad);
    top = __uint_as_float((uint32_t)s.sums[lane]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    u64 none = 0;
    block_sums(s, none, live);
    if (!usable || any_bad || live == 0) {
        if (tid == 0) {
            if (!usable) atomicCAS(p.status, 0, kDevTemperature);
            p.ids[i] = -1;
            if (p.logprob) p.logprob[i] = usable && !any_bad ? -INFINITY : NAN;
            if (p.kept) p.kept[i] = 0;
        }
        return;
    }
    const Mass m(top + 0.f, c, p.fraction);
    Rules rules;
    rules.k = p.top_k ? (uint32_t)max(p.top_k[i], 0) : 0;
    rules.p = p.top_p ? p.top_p[i] : 1.f;
    if (rules.p != rules.p) rules.p = 1.f;
    rules.min_p = p.min_p ? p.min_p[i] : 0.f;
    if (rules.min_p != rules.min_p) rules.min_p = 0.f;
    rules.log_min_p = rules.min_p > 0.f ? log((double)rules.min_p) : 0.0;
    if (rules.min_p > 1.f) rules.k = 1, rules.p = 1.f, rules.min_p = 0.f;  // nothing reaches it: the first token alone
    Drawn d = draw_row<false>(s, row, m, rules, live, p.u[i], p.V);
    if (!d.sure) d = draw_row<true>(s, row, m, rules, live, p.u[i], p.V);
    if (tid == 0) {
        p.ids[i] = d.id;
        if (p.logprob) p.logprob[i] = d.logprob;
        if (p.kept) p.kept[i] = (int)d.kept;
    }
}

template <typename T>
cudaError_t run(const SampleArgs &a, const TokenLaunch &l)
{
    int bits = 0;
    while ((1ll << bits) < a.V) ++bits;
    const Params<T> p{(const T *)a.logits, a.ld, a.u, a.inv_temperature, a.top_k, a.top_p, a.min_p, a.ids, a.logprob, a.kept, a.n, a.V,
                      bits <= 19 ? 44 : 63 - bits, l.d_status};  // the masses' sum fits 64 bits
    l.timer->begin("sample");
    sample_kernel<T><<<a.n, kThreads, 0, l.timer->stream>>>(p);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace draw

cudaError_t sample_prepare() { return cudaSuccess; }

cudaError_t sample(prism_dtype logits, const SampleArgs &a, const TokenLaunch &l)
{
    return logits == PRISM_BF16 ? draw::run<__nv_bfloat16>(a, l) : draw::run<float>(a, l);
}

}  // namespace prism
