// Log probabilities of given tokens with entropy and top alternatives, and the gradient.
//
// With z = inv_temperature logits, m = max_j z_j, s = sum_j exp(z_j - m), t = sum_j exp(z_j - m) (z_j - m):
//   lse = m + log s,   logprob = (z_target - m) - log s,   entropy = log s - t / s
//   dlogits_j = inv_temperature (dlogprob (1_{j = target} - p_j) - dentropy p_j (log p_j + entropy))
// One pass over the row with a running maximum; two parts of a row join as
//   m = max(m1, m2),  f_i = exp(m_i - m),  s = sum f_i s_i,  t = sum f_i (t_i + s_i (m_i - m))
// The differences are taken between logits (exact where they are near, and no finite logit overflows)
// and scaled by c2 = inv_temperature log2 e, so that an exponential is one ex2; t is kept in base 2.
// A few operations and one exponential per value: HBM bounds both directions (4096 x 50021 bf16: 69 us, 5.9 TB/s, without
// alternatives; 81 us, 5.0 TB/s, with 8; the gradient 131 us, 6.2 TB/s), and the steps after the last load where rows are
// few (4 x 50021 with 20 alternatives: 10.3 us).
//
// A logit of -inf or of the lowest value (of bfloat16, or below) marks a masked token, and so does a
// product that overflows to -inf: z = -inf there.
#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

namespace prism {
namespace logp {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAhead = 4;             // 16-byte units in flight per thread: a batch
constexpr int kBatch = kAhead * kThreads;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.38953139e38f;  // the lowest bfloat16 value
constexpr float kFar = -1e4f;         // 2^kFar = 0, and kFar times anything in range is finite
constexpr int kLogClusterMax = 3, kTopMax = 32;
constexpr int kCandidates = 1024, kFew = 160, kQueue = 1024;
constexpr int kBatchesMax = 96;       // batches of a slice whose largest logits are kept

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b)  // NaN if either is
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

using io::add2;
using io::fma2;
using io::mul2;
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

template <typename logit_t>
struct Row;
template <>
struct Row<__nv_bfloat16> {
    static constexpr int VEC = 8;
    using U = io::Unit<__nv_bfloat16, 8>;
    static __device__ __forceinline__ U nothing()
    {
        U u;
        u.w = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
        return u;
    }
    // the largest number
    static __device__ __forceinline__ float largest(const U &u)
    {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u.w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    // ... or NaN if there is one
    static __device__ __forceinline__ float largest_nan(const U &u)
    {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u.w);
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        return max_nan(__low2float(m), __high2float(m));
    }
};
template <>
struct Row<float> {
    static constexpr int VEC = 4;
    using U = io::Unit<float, 4>;
    static __device__ __forceinline__ U nothing()
    {
        U u;
        u.w = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
        return u;
    }
    static __device__ __forceinline__ float largest(const U &u)
    {
        float f[4];
        u.get(f);
        return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
    }
    static __device__ __forceinline__ float largest_nan(const U &u)
    {
        float f[4];
        u.get(f);
        return max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3]));
    }
};

// Is it a masked token's logit?  (NaN is none.)
__device__ __forceinline__ bool masked(float x, float c) { return x <= kLowest || x * c == -INFINITY; }

// A part of a row: its largest logit (-inf: no live token), s and t relative to it
struct Part {
    float top, s, t;
};
__device__ __forceinline__ Part join(const Part a, const Part b, float c2)
{
    Part r;
    r.top = fmaxf(a.top, b.top);
    const float da = a.top == r.top ? 0.f : (a.top - r.top) * c2, db = b.top == r.top ? 0.f : (b.top - r.top) * c2;
    const float fa = ex2(da), fb = ex2(db);
    r.s = a.s * fa + b.s * fb;
    r.t = (fa > 0.f ? fa * (a.t + a.s * da) : 0.f) + (fb > 0.f ? fb * (b.t + b.s * db) : 0.f);
    return r;
}

// A thread's share of a row; top = kLowest: no live token so far (then s = t = 0, or NaN)
struct Share {
    float top = kLowest;
    float2 s = {0.f, 0.f}, t = {0.f, 0.f};  // even and odd values

    // returns the units' largest logit
    template <typename R, int N>
    __device__ __forceinline__ float add(const typename R::U (&x)[N], float c2)
    {
        float most = R::largest(x[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) most = fmaxf(most, R::largest(x[i]));
        const float now = fmaxf(top, most);
        const float2 d = both(fmaxf((top - now) * c2, kFar)), f = both(ex2(d.x));
        t = mul2(f, fma2(s, d, t));
        s = mul2(f, s);
        top = now;
        const float2 minus_from = both(now > kLowest ? -now : 0.f), cc = both(c2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[R::VEC];
            x[i].get(v);
#pragma unroll
            for (int e = 0; e < R::VEC; e += 2) {
                // masked tokens end at kFar, where p = 0; NaN (and +inf against itself) goes into the sums
                float2 z = mul2(add2(make_float2(v[e], v[e + 1]), minus_from), cc);
                z.x = max_nan(z.x, kFar), z.y = max_nan(z.y, kFar);
                const float2 p = make_float2(ex2(z.x), ex2(z.y));
                s = add2(s, p);
                t = fma2(p, z, t);
            }
        }
        return most;
    }
    // the share relative to a larger logit (kLowest: nobody has a live token)
    __device__ __forceinline__ Part part(float onto, float c2) const
    {
        const float d = fmaxf((top - onto) * c2, kFar), f = ex2(d), sum = s.x + s.y;
        return {onto > kLowest ? onto : -INFINITY, f * sum, f * fmaf(sum, d, t.x + t.y)};
    }
};

// A logit's place in the order of the top: by value (NaN first), then by lowest id.  Larger keys come
// first; 0 stands for nothing (masked tokens never become keys).
__device__ __forceinline__ unsigned long long key_of(float x, int id)
{
    uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // -0 = +0
    b = x != x ? 0xffffffffu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((unsigned long long)b << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float value_of(unsigned long long key)
{
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);  // 0xffffffff gives a NaN
}
__device__ __forceinline__ int id_of(unsigned long long key) { return (int)~(uint32_t)key; }

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

// A row's slice for one CTA of its cluster: single values up to the first 16-byte boundary (first CTA),
// units, single values behind the last unit (last CTA).
template <typename logit_t>
struct Slice {
    const logit_t *x;
    int head, u0, u1, tail0, tail1;  // singles [0, head), units [u0, u1) behind them, singles [tail0, tail1)
    __device__ Slice(const logit_t *row, int V, int rank, int log_size)
    {
        constexpr int VEC = Row<logit_t>::VEC;
        x = row;
        const int off = (int)(((uintptr_t)row & 15) / sizeof(logit_t)), before = min(V, off ? VEC - off : 0);
        const int units = (V - before) / VEC;
        u0 = (int)((long long)units * rank >> log_size);
        u1 = (int)((long long)units * (rank + 1) >> log_size);
        tail0 = before + units * VEC;
        tail1 = rank + 1 == 1 << log_size ? V : tail0;
        first = before;
        head = rank == 0 ? before : 0;
    }
    int first;  // id of unit 0's first value
    // the single value that thread tid holds: its id, or -1
    __device__ __forceinline__ int single(int tid) const
    {
        if (tid < head) return tid;
        if (tid >= 32 && tail0 + tid - 32 < tail1) return tail0 + tid - 32;
        return -1;
    }
    __device__ __forceinline__ const uint4 *units() const { return reinterpret_cast<const uint4 *>(x + first); }
};

// A CTA, or a cluster of up to eight where rows are few, per row: four units of 16 bytes per thread in flight, the
// running maximum and sums in registers, the parts joined in a fixed order.
template <typename logit_t, bool TOP>
__global__ void __launch_bounds__(kThreads, 6) forward_kernel(const ForwardParams<logit_t> p, int log_cluster, int kept)
{
    using R = Row<logit_t>;
    using U = typename R::U;
    extern __shared__ float batch_top[];                     // [kept][kThreads] the largest logit of each thread's batches
    __shared__ Part parts[kWarps];
    __shared__ Part mine;                                    // this CTA's part
    __shared__ unsigned long long best[TOP ? kTopMax : 1];   // its first k keys
    __shared__ unsigned long long cand[TOP ? kCandidates : 1];
    __shared__ float thread_top[TOP ? kWarps : 1][32];
    __shared__ unsigned long long group_key[TOP ? kWarps : 1][32];
    __shared__ int queue[TOP ? kQueue : 1];                   // batches to be looked at again
    __shared__ int found, queued;
    __shared__ float threshold;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cluster = 1 << log_cluster, rank = blockIdx.x & (cluster - 1);
    const long long row = blockIdx.x >> log_cluster;
    const Slice<logit_t> sl(p.logits + row * p.ld, p.V, rank, log_cluster);
    const float c2 = p.inv_temperature * kLog2e;
    const uint4 *units = sl.units();

    Share sh;
    int u = sl.u0, batch = 0;
    for (; u + kBatch <= sl.u1; u += kBatch, ++batch) {
        U x[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) x[a].w = __ldg(units + u + a * kThreads + tid);
        const float most = sh.template add<R, kAhead>(x, c2);
        if (TOP && batch < kept) batch_top[batch * kThreads + tid] = most;
    }
    {  // the last batch is not full
        U x[kAhead];
        float most = kLowest;
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            x[a] = R::nothing();
            if (u + a * kThreads + tid < sl.u1) x[a].w = __ldg(units + u + a * kThreads + tid);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (u + a * kThreads >= sl.u1) break;
            const U one[1] = {x[a]};
            most = fmaxf(most, sh.template add<R, 1>(one, c2));
        }
        if (TOP && batch < kept) batch_top[batch * kThreads + tid] = most;
    }
    const int single = sl.single(tid);
    if (single >= 0) {
        U x[1] = {R::nothing()};
        *reinterpret_cast<logit_t *>(&x[0].w) = sl.x[single];
        sh.template add<R, 1>(x, c2);
    }
    // the warp's largest logit, the thread's sums brought onto it, and the warp's sums
    float warp_top = sh.top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) warp_top = fmaxf(warp_top, __shfl_xor_sync(0xffffffffu, warp_top, o));
    if constexpr (TOP) {
        thread_top[warp][lane] = sh.top;
        if (tid == 0) found = queued = 0;
    }
    Part r = sh.part(warp_top, c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
        r.t += __shfl_xor_sync(0xffffffffu, r.t, o);
    }
    if (lane == 0) parts[warp] = r;
    __syncthreads();
    if (warp == 0) {
        r = lane < kWarps ? parts[lane] : Part{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            const Part other{__shfl_xor_sync(0xffffffffu, r.top, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                            __shfl_xor_sync(0xffffffffu, r.t, o)};
            r = lane & o ? join(other, r, c2) : join(r, other, c2);
        }
        if (lane == 0) mine = r;
    }
    if constexpr (TOP) {
        // A lane's threads are a group, which holds every 32nd unit.  The k-th largest of the 32 groups' largest
        // logits: at least k of the slice's logits reach it, and few more (about 130 of any number at k = 32).
        // Those are collected and ordered by counting.
        if (warp == 1) {
            float g = thread_top[0][lane];
            for (int w = 1; w < kWarps; ++w) g = fmaxf(g, thread_top[w][lane]);
            int above = 0;
            for (int o = 0; o < 32; ++o) {
                const float other = __shfl_sync(0xffffffffu, g, o);
                above += other > g || (other == g && o < lane);
            }
            if (above == p.k - 1) threshold = g;
        }
        __syncthreads();
        const float least = threshold;
        auto offer = [&](float v, int id) {
            if (v < least || masked(v, p.inv_temperature)) return;  // NaN passes
            const int at = atomicAdd(&found, 1);
            if (at < kCandidates) cand[at] = key_of(v, id);
        };
        // Only batches that reach the threshold are looked at again (from L2), all of them at once: they are
        // queued, and four threads take one.  A thread whose sum is NaN queues all of its own.
        const bool all = sh.s.x + sh.s.y != sh.s.x + sh.s.y;
        batch = 0;
        for (u = sl.u0; u < sl.u1; u += kBatch, ++batch) {
            if (!all && batch < kept && batch_top[batch * kThreads + tid] < least) continue;
            const int at = atomicAdd(&queued, 1);
            if (at < kQueue) queue[at] = batch * kThreads + tid;
        }
        __syncthreads();
        auto look_at = [&](int at) {
            if (at >= sl.u1) return;
            U x;
            x.w = __ldg(units + at);
            if (R::largest_nan(x) < least) return;
            float v[R::VEC];
            x.get(v);
#pragma unroll
            for (int e = 0; e < R::VEC; ++e) offer(v[e], sl.first + at * R::VEC + e);
        };
        const int waiting = queued;
        if (waiting <= kQueue) {
            static_assert(kAhead == 4, "four threads a batch");
            for (int i = tid; i < 4 * waiting; i += kThreads) {
                const int item = queue[i >> 2];
                look_at(sl.u0 + item / kThreads * kBatch + (i & 3) * kThreads + item % kThreads);
            }
        } else {
            for (int at = sl.u0 + tid; at < sl.u1; at += kThreads) look_at(at);
        }
        if (single >= 0) offer(io::ld(sl.x + single), single);
        if (tid < kTopMax) best[tid] = 0;
        __syncthreads();
        int count = found;
        // The k-th largest of the groups' largest keys, for keys that a thread offers by `mine`; ends with a
        // barrier.  Keys differ, so at least k of them reach it, however many logits are equal.
        auto key_threshold = [&](unsigned long long mine) {
            group_key[warp][lane] = mine;
            __syncthreads();
            unsigned long long g = group_key[0][lane];
            for (int w = 1; w < kWarps; ++w) g = max(g, group_key[w][lane]);
            int above = 0;
            for (int o = 0; o < 32; ++o) above += __shfl_sync(0xffffffffu, g, o) > g;
            // the group that has k - 1 above it; with fewer than k groups that hold a key, 0
            unsigned long long at = above == p.k - 1 ? g : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) at = max(at, __shfl_xor_sync(0xffffffffu, at, o));
            if (tid == 0) found = 0;
            __syncthreads();
            return at;
        };
        auto for_each = [&](auto look) {  // this thread's live logits once more
            for (int at = sl.u0 + tid; at < sl.u1; at += kThreads) {
                U x;
                x.w = __ldg(units + at);
                float v[R::VEC];
                x.get(v);
#pragma unroll
                for (int e = 0; e < R::VEC; ++e)
                    if (!masked(v[e], p.inv_temperature)) look(key_of(v[e], sl.first + at * R::VEC + e));
            }
            if (single >= 0) {
                const float v = io::ld(sl.x + single);
                if (!masked(v, p.inv_temperature)) look(key_of(v, single));
            }
        };
        if (count > kCandidates) {  // many equal logits: by keys instead of by values
            unsigned long long mine_best = 0;
            for_each([&](unsigned long long key) { mine_best = max(mine_best, key); });
            const unsigned long long at = key_threshold(mine_best);
            for_each([&](unsigned long long key) {
                if (key < at) return;
                const int to = atomicAdd(&found, 1);
                if (to < kCandidates) cand[to] = key;
            });
            __syncthreads();
            count = found;
        } else if (count > kFew) {  // many candidates: the same choice among them
            unsigned long long held[kCandidates / kThreads], mine_best = 0;
#pragma unroll
            for (int i = 0; i < kCandidates / kThreads; ++i) {
                held[i] = tid + i * kThreads < count ? cand[tid + i * kThreads] : 0;
                mine_best = max(mine_best, held[i]);
            }
            const unsigned long long at = key_threshold(mine_best);
#pragma unroll
            for (int i = 0; i < kCandidates / kThreads; ++i)
                if (held[i] && held[i] >= at) cand[atomicAdd(&found, 1)] = held[i];
            __syncthreads();
            count = found;
        }
        if (count <= kCandidates) {
            // order by counting; few candidates need one warp only
            if (count > 32 || warp == 0)
                for (int i = tid; i < count; i += kThreads) {
                    const unsigned long long key = cand[i];
                    int above = 0;
                    for (int o = 0; o < count; ++o) above += cand[o] > key;
                    if (above < p.k) best[above] = key;
                }
            if (count > 32) __syncthreads();
            __syncwarp();
        } else {
            // an order that the groups miss: the largest key below the last one, k times
            unsigned long long last = ~0ull;
            for (int i = 0; i < p.k; ++i) {
                unsigned long long b = 0;
                for_each([&](unsigned long long key) {
                    if (key < last && key > b) b = key;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
                __syncthreads();  // cand is free: the round before has been read
                if (lane == 0) cand[warp] = b;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w) b = max(b, cand[w]);
                last = b;
                if (tid == 0) best[i] = b;
                if (b == 0) break;
            }
            __syncwarp();
        }
    }
    // The cluster's parts and keys join in its first CTA; without a cluster the rest is one warp's work
    // (warp 0 wrote mine and, but for the barriers above, best).
    if (cluster > 1)
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
    else if (warp > 0)
        return;
    __syncwarp();
    if (rank == 0) {
        auto remote = [&](const void *local, int cta) {
            uint32_t a;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(local)), "r"(cta));
            return a;
        };
        auto far_float = [&](const float *local, int cta) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(local, cta)) : "memory");
            return v;
        };
        Part all = mine;
        for (int o = 1; o < cluster; ++o)  // every thread joins them: the top needs the row's sum as well
            all = join(all, {far_float(&mine.top, o), far_float(&mine.s, o), far_float(&mine.t, o)}, c2);
        const float c = p.inv_temperature;
        const bool none = all.s == all.s && all.top * c == -INFINITY;
        const float top = none ? 0.f : all.top, logs = none ? -INFINITY : logf(all.s);
        if (tid == 0) {
            if (p.lse) p.lse[row] = fmaf(top, c, logs);
            if (p.entropy) p.entropy[row] = none ? 0.f : logs - all.t / all.s * kLn2;
            if (p.logprob) {
                const long long t = p.targets[row];
                if (t >= p.V) atomicCAS(p.status, 0, kDevBounds);
                float v = 0.f;
                if (t >= 0 && t < p.V) {
                    const float x = io::ld(sl.x + t);
                    v = none || masked(x, c) ? -INFINITY : (x - top) * c - logs;
                    if (all.s != all.s) v = all.s;
                }
                p.logprob[row] = v;
            }
        }
        if constexpr (TOP) {
            unsigned long long key = 0;
            int place = tid;
            if (cluster > 1) {
                const int total = cluster * p.k;
                __syncthreads();  // cand is free
                if (tid < total) {
                    unsigned long long v;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(&best[tid % p.k], tid / p.k)) : "memory");
                    cand[tid] = v;
                }
                __syncthreads();
                place = p.k;
                if (tid < total) {
                    key = cand[tid];
                    place = 0;  // empty places (key 0) keep their order behind the keys
                    for (int o = 0; o < total; ++o) place += cand[o] > key || (cand[o] == key && o < tid);
                }
            } else if (tid < p.k) {
                key = best[tid];
            }
            if (place < p.k && (cluster > 1 ? tid < cluster * p.k : tid < p.k)) {
                const float x = value_of(key);
                if (p.top_ids) p.top_ids[row * p.k + place] = key ? id_of(key) : -1;
                if (p.top_logprob) p.top_logprob[row * p.k + place] = key ? (x - top) * c - logs : -INFINITY;
            }
        }
    }
    // the other CTAs' shared memory stays until the first one has read it
    if (cluster > 1) asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

// Many short rows: a warp per row and no barriers.  The same steps as in forward_kernel, the lanes being the
// groups: the k-th largest of their largest logits is the threshold, and only batches whose largest logit
// reaches it are looked at again.
constexpr int kShortUnits = 2048, kShortCandidates = 256, kShortBatches = kShortUnits / (32 * kAhead) + 1;

template <typename logit_t, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) short_kernel(const ForwardParams<logit_t> p)
{
    using R = Row<logit_t>;
    using U = typename R::U;
    // the batches' largest logits, then the candidates
    __shared__ union {
        float tops[kShortBatches][32];
        unsigned long long cand[kShortCandidates];
    } sh_s[TOP ? kWarps : 1];
    __shared__ unsigned long long best_s[TOP ? kWarps : 1][TOP ? kTopMax : 1];
    __shared__ int found_s[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = (long long)blockIdx.x * kWarps + warp;
    if (row >= p.n) return;
    const Slice<logit_t> sl(p.logits + row * p.ld, p.V, 0, 0);
    const float c = p.inv_temperature, c2 = c * kLog2e;
    const uint4 *units = sl.units();
    // single values: the head's on the first lanes, the tail's from lane 16 on (fewer than 8 each)
    const int single = lane < sl.head ? lane : lane >= 16 && sl.tail0 + lane - 16 < sl.tail1 ? sl.tail0 + lane - 16 : -1;

    Share sh;
    int u = lane, batches = 0;
    auto keep_top = [&](float most) {  // u < kShortUnits, so that batches < kShortBatches
        if constexpr (TOP) sh_s[warp].tops[batches++][lane] = most;
    };
    for (; u + 32 * (kAhead - 1) < sl.u1; u += 32 * kAhead) {
        U x[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) x[a].w = __ldg(units + u + 32 * a);
        keep_top(sh.template add<R, kAhead>(x, c2));
    }
    {
        U x[kAhead];  // what is left, and the single value in the last place
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            x[a] = R::nothing();
            if (a < kAhead - 1 && u + 32 * a < sl.u1) x[a].w = __ldg(units + u + 32 * a);
        }
        if (single >= 0) *reinterpret_cast<logit_t *>(&x[kAhead - 1].w) = sl.x[single];
        keep_top(sh.template add<R, kAhead>(x, c2));
    }
    float top = sh.top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    Part all = sh.part(top, c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all.s += __shfl_xor_sync(0xffffffffu, all.s, o);
        all.t += __shfl_xor_sync(0xffffffffu, all.t, o);
    }
    const bool none = all.s == all.s && all.top * c == -INFINITY;
    const float m = none ? 0.f : all.top, logs = none ? -INFINITY : logf(all.s);
    if (lane == 0) {
        if (p.lse) p.lse[row] = fmaf(m, c, logs);
        if (p.entropy) p.entropy[row] = none ? 0.f : logs - all.t / all.s * kLn2;
        if (p.logprob) {
            const long long t = p.targets[row];
            if (t >= p.V) atomicCAS(p.status, 0, kDevBounds);
            float v = 0.f;
            if (t >= 0 && t < p.V) {
                const float x = io::ld(sl.x + t);
                v = none || masked(x, c) ? -INFINITY : (x - m) * c - logs;
                if (all.s != all.s) v = all.s;
            }
            p.logprob[row] = v;
        }
    }
    if constexpr (TOP) {
        unsigned long long *cand = sh_s[warp].cand, *best = best_s[warp];
        int &found = found_s[warp];
        auto keep = [&](unsigned long long key) {
            const int at = atomicAdd(&found, 1);
            if (at < kShortCandidates) cand[at] = key;
        };
        auto kth = [&](auto g) {  // the k-th largest of the lanes' values (ties by lane)
            int above = 0;
            for (int o = 0; o < 32; ++o) {
                const auto other = __shfl_sync(0xffffffffu, g, o);
                above += other > g || (other == g && o < lane);
            }
            return __shfl_sync(0xffffffffu, g, __ffs(__ballot_sync(0xffffffffu, above == p.k - 1)) - 1);
        };
        const float least = kth(sh.top);
        uint32_t reach = 0;  // the lane's batches that reach `least`; all where a NaN may hide one
        for (int b = 0; b < batches; ++b) reach |= (uint32_t)(sh_s[warp].tops[b][lane] >= least || !(sh.s.x + sh.s.y < INFINITY)) << b;
        auto for_each = [&](auto look) {  // this lane's live logits that reach `least`, and NaN
            for (uint32_t left = reach; left; left &= left - 1) {
                const int at = lane + 32 * kAhead * (__ffs(left) - 1);
                uint32_t in = 0;  // the batch's units that do
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    U x = R::nothing();
                    if (at + 32 * a < sl.u1) x.w = __ldg(units + at + 32 * a);
                    in |= (uint32_t)!(R::largest_nan(x) < least) << a;
                }
                for (; in; in &= in - 1) {
                    const int unit = at + 32 * (__ffs(in) - 1);
                    if (unit >= sl.u1) break;  // nothing is no less than the lowest value
                    U x;
                    x.w = __ldg(units + unit);
                    float v[R::VEC];
                    x.get(v);
#pragma unroll
                    for (int e = 0; e < R::VEC; ++e)
                        if (!(v[e] < least || masked(v[e], c))) look(key_of(v[e], sl.first + unit * R::VEC + e));
                }
            }
            if (single >= 0) {
                const float v = io::ld(sl.x + single);
                if (!(v < least || masked(v, c))) look(key_of(v, single));
            }
        };
        best[lane] = 0;
        if (lane == 0) found = 0;
        __syncwarp();
        for_each(keep);
        __syncwarp();
        int count = found;
        __syncwarp();
        if (count > kShortCandidates) {  // many equal logits: by keys instead of by values
            unsigned long long mine = 0;
            for_each([&](unsigned long long key) { mine = max(mine, key); });
            const unsigned long long at = kth(mine);
            if (lane == 0) found = 0;
            __syncwarp();
            for_each([&](unsigned long long key) {
                if (key >= at) keep(key);
            });
            __syncwarp();
            count = found;
        }
        if (count <= kShortCandidates) {
            for (int i = lane; i < count; i += 32) {
                const unsigned long long key = cand[i];
                int above = 0;
                for (int o = 0; o < count; ++o) above += cand[o] > key;
                if (above < p.k) best[above] = key;
            }
        } else {  // an order that the lanes miss: the largest key below the last one, k times
            unsigned long long last = ~0ull;
            for (int i = 0; i < p.k && last; ++i) {
                unsigned long long b = 0;
                for_each([&](unsigned long long key) {
                    if (key < last && key > b) b = key;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
                last = b;
                if (lane == 0) best[i] = b;
            }
        }
        __syncwarp();
        if (lane < p.k) {
            const unsigned long long key = best[lane];
            if (p.top_ids) p.top_ids[row * p.k + lane] = key ? id_of(key) : -1;
            if (p.top_logprob) p.top_logprob[row * p.k + lane] = key ? (value_of(key) - m) * c - logs : -INFINITY;
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

// A CTA takes kAhead units per thread of one row, or 256 / GROUP whole short rows, GROUP threads each (6437 x 850 fp32:
// 18.4 us with 256 threads a row, 8.8 with 64).  dlogits_j = p_j (B - dentropy log p_j), plus dlogprob at the
// target, with inv_temperature in dlogprob and dentropy, and B = -dlogprob - dentropy entropy.  Every thread loads all that
// it takes before it computes and stores, which keeps HBM busy: 4096 x 50021 bf16 131 us, 6.2 TB/s.
template <typename logit_t, int GROUP>
__global__ void __launch_bounds__(kThreads, 6) backward_kernel(const BackwardParams<logit_t> p, int chunks)
{
    static_assert(GROUP >= 64, "Slice::single takes two warps");
    using R = Row<logit_t>;
    using U = typename R::U;
    const int tid = threadIdx.x % GROUP;
    const long long row = (long long)(blockIdx.x / chunks) * (kThreads / GROUP) + threadIdx.x / GROUP;
    const int chunk = (int)(blockIdx.x % chunks);
    if (row >= p.n) return;
    const Slice<logit_t> sl(p.logits + row * p.ld, p.V, 0, 0);
    logit_t *out = p.dlogits + row * p.ld_d;
    const uint4 *units = sl.units();
    const int per = (sl.u1 + chunks - 1) / chunks, u0 = chunk * per + tid, u1 = min(sl.u1, chunk * per + per);
    U x[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
        if (u0 + a * GROUP < u1) x[a].w = units[u0 + a * GROUP];
    const float lse = p.lse[row], c = p.inv_temperature;
    long long t = p.dlogprob ? p.targets[row] : -1;
    if (t >= p.V) {
        if (tid == 0) atomicCAS(p.status, 0, kDevBounds);
        t = -1;
    }
    const bool none = lse == -INFINITY;
    const float dlp = t >= 0 && !none ? p.dlogprob[row] * c : 0.f;
    const float dh = p.dentropy && !none ? p.dentropy[row] * c : 0.f, h = p.dentropy && !none ? p.entropy[row] : 0.f;
    const float minus_lse = none ? 0.f : -lse, Bc = fmaf(-dh, h, -dlp);
    auto grad = [&](float2 v) {
        float2 z = fma2(v, both(c), both(minus_lse));
        z.x = max_nan(z.x, kFar), z.y = max_nan(z.y, kFar);
        const float2 y = mul2(z, both(kLog2e));
        return mul2(make_float2(ex2(y.x), ex2(y.y)), fma2(both(-dh), z, both(Bc)));
    };
    auto at_target = [&](float v) { return masked(v, c) ? 0.f : dlp; };  // a masked target has no gradient
    const bool aligned = (((uintptr_t)(out + sl.first)) & 15) == 0;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
        const int u = u0 + a * GROUP;
        if (u >= u1) break;
        const int id = sl.first + u * R::VEC;
        float v[R::VEC], logit = 0.f;  // at the target
        x[a].get(v);
        const int hit = t >= id && t < id + R::VEC ? (int)t - id : -1;
#pragma unroll
        for (int e = 0; e < R::VEC; e += 2) {
            const float2 x2 = make_float2(v[e], v[e + 1]), g = grad(x2);
            if (e == hit) logit = x2.x;
            if (e + 1 == hit) logit = x2.y;
            v[e] = g.x, v[e + 1] = g.y;
        }
        if (hit >= 0) {
            const float more = at_target(logit);
#pragma unroll
            for (int e = 0; e < R::VEC; ++e)
                if (e == hit) v[e] += more;
        }
        if (aligned) {
            x[a].set(v);
            *reinterpret_cast<uint4 *>(out + id) = x[a].w;
        } else {
#pragma unroll
            for (int e = 0; e < R::VEC; ++e) io::st(out + id + e, v[e]);
        }
    }
    const int single = chunk == 0 ? sl.single(tid) : -1;
    if (single >= 0) {
        const float v = io::ld(sl.x + single), g = grad(both(v)).x;
        io::st(out + single, single == t ? g + at_target(v) : g);
    }
}

template <typename logit_t, bool TOP>
cudaError_t launch_forward(const ForwardParams<logit_t> &p, int log_cluster, int kept, cudaStream_t s)
{
    const int cluster = 1 << log_cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)kept * kThreads * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, forward_kernel<logit_t, TOP>, p, log_cluster, kept);
}

template <typename logit_t>
cudaError_t forward(const LogprobArgs &a, const TokenLaunch &l)
{
    const ForwardParams<logit_t> p{(const logit_t *)a.logits, a.targets, a.lse, a.logprob, a.entropy, a.top_logprob, a.top_ids,
                                   a.ld, a.inv_temperature, a.n, a.V, a.k, l.d_status};
    const long long units = a.V / Row<logit_t>::VEC + 1;
    // A warp per row where its lanes have one batch at most, and up to 2048 units where there are rows enough for
    // eight warps an SM: 2979 x 8892 with 5 alternatives takes 19.2 us so and 27.2 with 256 threads a row, 4096 x
    // 16000 with 8 33.3 and 41.4, without 27.0 and 29.2; 700 x 8000 with 8 would take 17 us so, 8.7 in clusters.
    if (units <= 32 * (kAhead - 1) || (units <= kShortUnits && a.n >= 8 * l.sm_count)) {
        l.timer->begin("token_logprobs");
        const unsigned grid = (unsigned)((a.n + kWarps - 1) / kWarps);
        if (a.k == 0) short_kernel<logit_t, false><<<grid, kThreads, 0, l.timer->stream>>>(p);
        else short_kernel<logit_t, true><<<grid, kThreads, 0, l.timer->stream>>>(p);
        l.timer->end();
        return cudaGetLastError();
    }
    // Few rows are split over a cluster, down to one unit per thread.
    int log_cluster = 0;
    while (log_cluster < kLogClusterMax && ((long long)a.n << log_cluster) < 2 * l.sm_count && units >> log_cluster > kThreads) ++log_cluster;
    const long long batches = (units >> log_cluster) / kBatch + 1;
    l.timer->begin("token_logprobs");
    const cudaError_t e =
        a.k == 0 ? launch_forward<logit_t, false>(p, log_cluster, 0, l.timer->stream)
                 : launch_forward<logit_t, true>(p, log_cluster, (int)(batches < kBatchesMax ? batches : kBatchesMax), l.timer->stream);
    l.timer->end();
    return e;
}

template <typename logit_t>
cudaError_t backward(const LogprobBackwardArgs &a, const TokenLaunch &l)
{
    const BackwardParams<logit_t> p{(const logit_t *)a.logits, a.targets, a.lse, a.entropy, a.dlogprob, a.dentropy,
                                    (logit_t *)a.dlogits, a.ld, a.ld_d, a.inv_temperature, a.n, a.V, l.d_status};
    const int units = a.V / Row<logit_t>::VEC, per = kAhead * kThreads, chunks = units > per ? (units + per - 1) / per : 1;
    l.timer->begin("token_logprobs_backward");
    // n chunks: below 2^31 for any logits that fit the device's memory
    cudaStream_t s = l.timer->stream;
    if (units <= kAhead * 64)
        backward_kernel<logit_t, 64><<<(unsigned)(((long long)a.n + 3) / 4), kThreads, 0, s>>>(p, 1);
    else if (units <= kAhead * 128)
        backward_kernel<logit_t, 128><<<(unsigned)(((long long)a.n + 1) / 2), kThreads, 0, s>>>(p, 1);
    else
        backward_kernel<logit_t, kThreads><<<(unsigned)((long long)a.n * chunks), kThreads, 0, s>>>(p, chunks);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace logp

cudaError_t logprobs_prepare()
{
    const int smem = logp::kBatchesMax * logp::kThreads * 4;
    cudaError_t e = cudaFuncSetAttribute(logp::forward_kernel<float, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(logp::forward_kernel<__nv_bfloat16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e;
}

cudaError_t logprobs_forward(prism_dtype logits, const LogprobArgs &a, const TokenLaunch &l)
{
    return logits == PRISM_BF16 ? logp::forward<__nv_bfloat16>(a, l) : logp::forward<float>(a, l);
}

cudaError_t logprobs_backward(prism_dtype logits, const LogprobBackwardArgs &a, const TokenLaunch &l)
{
    return logits == PRISM_BF16 ? logp::backward<__nv_bfloat16>(a, l) : logp::backward<float>(a, l);
}

}  // namespace prism
