// Embedding lookup and its gradient.
//
//   out_i     = scale table[ids_i]                           (zeros where there is no token)
//   dtable[v] = scale sum_{i : ids_i = v} dout_i             (every row written, or added to)
//
// Both only move data: the lookup reads one table row and writes one output row per token; the
// gradient reads dout once and writes the whole fp32 table once, so HBM bounds both.
//
// The gradient's sum over equal ids must not depend on the order in which blocks run, so the tokens
// are first sorted by id, stably: up to 512 by counting, up to 65536 in one cluster of eight CTAs, more in
// a kernel per digit; least significant digit first, digits of at most 9 bits (two passes for vocabularies
// below 2^18).  A pass ranks keys inside a warp by votes, so a digit that half of the tokens share costs no more
// than any other.  Then a warp walks a tile of consecutive sorted tokens and adds their rows up in
// registers, writing a sum whenever the id changes.  Runs that cross a tile's edge leave their part
// in the workspace; a last kernel adds those parts in order (a token that fills many tiles, as the
// most frequent ones of a text do, is spread over eight warps there).  The sort keeps few SMs busy, so the
// table's zeros are written beside it.
//
// 16384 x 768 bf16 of 50021: 40 us in a graph for 179 MB (4.5 TB/s); timed one by one the sort with 96 MB of zeros takes 22, the sums
// with the other zeros 20 and the join 10 (onto a table that is not cleared: 15, 16 and 10, 33 in all).  14309 x 648
// of 130295: 71 us for 356 MB (5.0 TB/s).
#include <type_traits>

#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

namespace prism {
namespace embed {

constexpr int kBins = 512;       // digits of up to 9 bits
constexpr int kPassesMax = 4;    // ids below 2^30 and the "no token" key: at most 31 bits
constexpr int kBlocksMax = 128;  // blocks of one sort pass
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32, kSteps = 8;
constexpr int kSub = kSortThreads * kSteps;  // keys that a block ranks at a time

constexpr int kThreads = 256;
// Bytes of the table that one sort kernel clears: what the L2 takes while the sort runs.  Measured for 16384 x
// 768 of 50021 (bf16) and 32768 x 256 of 200003 (fp32): 16 MB 51 and 73 us, 48 MB 48 and 65 us, 80 MB 48 and
// 57 us, 112 MB 52 and 53 us, all of it 53 and 56 us.
constexpr long long kBesideSort = 96 << 20;
constexpr int kTile = 8;  // sorted tokens per warp, at least (tile_of)

// ---------------------------------------------------------------------------------------------
// lookup: a warp takes 32 UPL units of one row, loads them all and then stores them.  HBM bounds it where tokens are many
// (16384 x 768 bf16 of 50021 different rows: 12.5 us, 4.0 TB/s), the launch where they are few (16 tokens: 5 us).
template <typename io_t, int VEC, int UPL>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const long long *__restrict__ ids, const io_t *__restrict__ table,
                                                         long long ld_table, float scale, io_t *__restrict__ out, int n,
                                                         int D, int V, int chunks, int *status)
{
    const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const long long row = w / chunks;
    if (row >= n) return;
    const int u0 = (int)(w % chunks) * 32 * UPL + lane, units = D / VEC;
    const long long id = ids[row];
    if (id >= V && lane == 0) atomicCAS(status, 0, kDevBounds);
    const bool live = id >= 0 && id < V;
    const io_t *src = table + (live ? id : 0) * ld_table;
    io_t *dst = out + row * D;
    io::Unit<io_t, VEC> x[UPL];
#pragma unroll
    for (int j = 0; j < UPL; ++j)
        if (live && u0 + 32 * j < units) x[j] = io::load_unit<io_t, VEC>(src + (size_t)(u0 + 32 * j) * VEC);
#pragma unroll
    for (int j = 0; j < UPL; ++j)
        if (u0 + 32 * j < units) {
            float f[VEC];
            if (live)
                x[j].get(f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = live ? f[e] * scale : 0.f;
            x[j].set(f);
            io::store_unit<io_t, VEC>(dst + (size_t)(u0 + 32 * j) * VEC, x[j]);
        }
}

// ---------------------------------------------------------------------------------------------
// sort
__device__ __forceinline__ int key_of(long long id, int V) { return id >= 0 && id < V ? (int)id : V; }

// Ranks of a tile's keys: warp w holds keys w 32 STEPS + 32 s + lane.  count[w][d] is the number of
// the warp's keys with digit d so far; rank[s] the number of them before this lane's key.
// The lanes that share a digit are found with one vote per bit: match_any took about 360 cycles a step
// here (it goes through the distinct values), the votes take a tenth of that.
__device__ __forceinline__ uint32_t peers_of(int d, int width)
{
    uint32_t peers = 0xffffffffu;
    for (int b = 0; b < width; ++b) {
        const bool bit = (d >> b) & 1;
        const uint32_t set = __ballot_sync(0xffffffffu, bit);
        peers &= bit ? set : ~set;
    }
    return peers;
}

template <int STEPS>
__device__ __forceinline__ void rank_in_warp(const int (&key)[STEPS], int shift, int width, uint16_t *count, int (&rank)[STEPS])
{
    const int mask = (1 << width) - 1;
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int d = (key[s] >> shift) & mask;
        const uint32_t peers = peers_of(d, width);
        const int before = count[d];
        rank[s] = before + __popc(peers & below);
        __syncwarp();
        if ((peers & below) == 0) count[d] = (uint16_t)(before + __popc(peers));
        __syncwarp();
    }
}

// Exclusive prefix over the kBins values of the block's threads (thread t holds bins 2 t and 2 t + 1;
// kSortThreads threads).
__device__ __forceinline__ void scan_bins(int &a, int &b, int *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mine = a + b;
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
    }
    if (lane == 31) warp_sums[warp] = run;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sums[w];
    const int first = base + run - mine;
    b = first + a;
    a = first;
}
static_assert(kBins == 2 * kSortThreads, "scan_bins");

// Counts per warp and digit to each warp's first place among its digit's keys; sum: the digits' counts
// (thread t: digits 2 t and 2 t + 1).
__device__ __forceinline__ void prefix_over_warps(uint16_t (&count)[kSortWarps][kBins], int (&sum)[2])
{
    sum[0] = sum[1] = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = count[w][2 * threadIdx.x + e];
            count[w][2 * threadIdx.x + e] = (uint16_t)sum[e];
            sum[e] += c;
        }
}

// The sort leaves most SMs and all of HBM idle, so the blocks behind a sort kernel's own clear a share of
// the table meanwhile (rows that have tokens are written again by the sums, which run after the sort).
// What the sort's few microseconds cannot hide is cleared beside the sums (clear_absent).
struct Fill {
    float *dtable;
    size_t from, to;  // floats, multiples of 4 except the table's end
};
__device__ __forceinline__ void fill_share(const Fill &f, int block, int blocks)
{
    float4 *d = reinterpret_cast<float4 *>(f.dtable);
    const size_t end = f.to / 4, step = (size_t)blocks * blockDim.x;
    for (size_t i = f.from / 4 + (size_t)block * blockDim.x + threadIdx.x; i < end; i += step)
        d[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (block == 0 && threadIdx.x < f.to % 4) f.dtable[end * 4 + threadIdx.x] = 0.f;
}

// Digit counts of each block's chunk of the tokens, for the first pass; clears the later passes' counts.
__global__ void __launch_bounds__(kSortThreads) count_kernel(const long long *__restrict__ ids, int n, int V, int chunk,
                                                            int mask, int passes, int nb, int *hist, uint32_t *present, int *status,
                                                            const Fill f)
{
    __shared__ int bins[kBins];
    tc::allow_dependent_launch();
    if ((int)blockIdx.x >= nb) return fill_share(f, blockIdx.x - nb, gridDim.x - nb);
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) bins[d] = 0;
    __syncthreads();
    for (int i = blockIdx.x * kSortThreads + threadIdx.x; i <= V / 32; i += nb * kSortThreads) present[i] = 0;
    const int i1 = min((long long)n, ((long long)blockIdx.x + 1) * chunk);
    bool bad = false;
    for (int i = blockIdx.x * chunk + threadIdx.x; i < i1; i += kSortThreads) {
        const long long id = ids[i];
        bad |= id >= V;
        atomicAdd(&bins[key_of(id, V) & mask], 1);  // counts: the order of the additions does not matter
    }
    if (bad) atomicCAS(status, 0, kDevBounds);
    __syncthreads();
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) {
        hist[(size_t)blockIdx.x * kBins + d] = bins[d];
        for (int p = 1; p < passes; ++p) hist[((size_t)p * kBlocksMax + blockIdx.x) * kBins + d] = 0;
    }
}

// One pass: block b places the keys of its chunk; hist holds the counts per block and digit.  The
// next pass's counts are taken here (hist_next): where a key lands decides which block will read it.
struct Pass {
    const long long *ids;       // the first pass reads these ...
    const int *key_in, *pos_in;  // ... the later ones these
    int *key_out, *pos_out;
    const int *hist;
    int *hist_next;
    uint32_t *present;  // set by the first pass
    int n, V, chunk, nb, shift, width, mask, next_shift;
};

template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) scatter_kernel(const Pass p, const Fill f)
{
    __shared__ uint16_t count[kSortWarps][kBins];
    __shared__ int base[kBins];
    __shared__ int warp_sums[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
    tc::allow_dependent_launch();
    if (b >= p.nb) return fill_share(f, b - p.nb, gridDim.x - p.nb);
    tc::grid_dependency_wait();
    int total[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll 8
    for (int o = 0; o < p.nb; ++o) {
        const int2 h = *reinterpret_cast<const int2 *>(p.hist + (size_t)o * kBins + 2 * tid);
        total[0] += h.x, total[1] += h.y;
        if (o < b) before[0] += h.x, before[1] += h.y;
    }
    scan_bins(total[0], total[1], warp_sums);
    base[2 * tid] = total[0] + before[0];
    base[2 * tid + 1] = total[1] + before[1];
    const int i1 = min((long long)p.n, ((long long)b + 1) * p.chunk);
    for (int i0 = b * p.chunk; i0 < i1; i0 += kSub) {
        for (int d = lane; d < kBins; d += 32) count[warp][d] = 0;
        __syncwarp();
        int key[kSteps], pos[kSteps], rank[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = i0 + warp * 32 * kSteps + 32 * s + lane;
            key[s] = -1;  // no token: the last digit in every pass, behind that digit's keys; not stored
            pos[s] = i;
            if (i < i1) {
                key[s] = FIRST ? key_of(p.ids[i], p.V) : p.key_in[i];
                if (!FIRST) pos[s] = p.pos_in[i];
            }
        }
        rank_in_warp<kSteps>(key, p.shift, p.width, count[warp], rank);
        __syncthreads();
        int sum[2];  // of this tile, for the next one's base
        prefix_over_warps(count, sum);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = i0 + warp * 32 * kSteps + 32 * s + lane;
            const bool live = i < i1;
            const int d = (key[s] >> p.shift) & p.mask;
            const int to = base[d] + count[warp][d] + rank[s];
            if (live) {
                p.key_out[to] = key[s];
                p.pos_out[to] = pos[s];
                const uint32_t bit = 1u << (key[s] & 31);  // frequent ids find it set
                if (FIRST && !(*(volatile uint32_t *)&p.present[key[s] >> 5] & bit)) atomicOr(&p.present[key[s] >> 5], bit);
            }
            if (p.hist_next) {  // one addition per warp and counter: frequent tokens share theirs
                const int at = live ? to / p.chunk * kBins + ((key[s] >> p.next_shift) & p.mask) : -1;
                const uint32_t peers = __match_any_sync(0xffffffffu, at);
                if (live && (peers & ((1u << lane) - 1u)) == 0) atomicAdd(&p.hist_next[at], __popc(peers));
            }
        }
        __syncthreads();
        base[2 * tid] += sum[0];
        base[2 * tid + 1] += sum[1];
        __syncthreads();
    }
}

// All passes in one cluster of CS CTAs (one CTA for few tokens), the keys in registers and in shared
// memory: CTA c holds the sorted places [c per, (c + 1) per) of a pass, reads the other CTAs' digit
// counts and writes each key straight to the shared memory of the CTA that holds its place.  A pass
// costs two cluster barriers instead of two launches.  At most CS kClusterThreads STEPS tokens.  The chain of
// barriers and shared-memory trips bounds it: 15 us for 16384 keys in two passes, 21 for 32768.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32, kCluster = 8, kClusterSteps = 8;

struct ClusterShared {
    uint16_t count[kClusterWarps][kBins];
    int total[kBins];  // this CTA's keys by digit; read by the others
    int base[kBins];
    int warp_sums[16];
    int2 sorted[1];    // [STEPS kClusterThreads] key and position
};

template <int CS>
__device__ __forceinline__ void cluster_sync()
{
    if constexpr (CS > 1)
        asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
    else
        __syncthreads();
}

// A few tokens: a token's place is the number of tokens before it in the order, which its thread counts (205
// tokens of 1697 take 11 us in all, 16.6 with the cluster's passes).
constexpr int kCounted = 512;
__global__ void __launch_bounds__(kCounted) counted_sort_kernel(const long long *__restrict__ ids, int n, int V, int *__restrict__ key_out,
                                                               int *__restrict__ pos_out, uint32_t *present, int *status, const Fill f)
{
    __shared__ __align__(16) int keys[kCounted];
    const int tid = threadIdx.x;
    tc::allow_dependent_launch();
    if (blockIdx.x > 0) return fill_share(f, blockIdx.x - 1, gridDim.x - 1);
    const long long id = tid < n ? ids[tid] : -1;
    if (id >= V) atomicCAS(status, 0, kDevBounds);
    const int key = tid < n ? key_of(id, V) : 0x7fffffff;
    keys[tid] = key;
    for (int i = tid; i <= V / 32; i += kCounted) present[i] = 0;
    __syncthreads();
    if (tid >= n) return;
    int place = 0;
    for (int o = 0; o < n; o += 4) {  // the padding is larger than every key
        const int4 k = *reinterpret_cast<const int4 *>(keys + o);
        place += (k.x < key || (k.x == key && o < tid)) + (k.y < key || (k.y == key && o + 1 < tid)) +
                 (k.z < key || (k.z == key && o + 2 < tid)) + (k.w < key || (k.w == key && o + 3 < tid));
    }
    key_out[place] = key;
    pos_out[place] = tid;
    atomicOr(&present[key >> 5], 1u << (key & 31));
}

template <int CS, int STEPS>
__global__ void __launch_bounds__(kClusterThreads) cluster_sort_kernel(const long long *__restrict__ ids, int n, int per, int V,
                                                                      int width, int passes, int *__restrict__ key_out,
                                                                      int *__restrict__ pos_out, uint32_t *present, int *status,
                                                                      const Fill f)
{
    extern __shared__ __align__(16) uint8_t raw[];
    ClusterShared &sh = *reinterpret_cast<ClusterShared *>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, mask = (1 << width) - 1;
    tc::allow_dependent_launch();
    if (blockIdx.x >= CS) return fill_share(f, blockIdx.x - CS, gridDim.x - CS);
    const int rank = blockIdx.x, i0 = rank * per, mine = max(0, min(n - i0, per));
    int key[STEPS], pos[STEPS], place[STEPS];
    bool bad = false;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int i = warp * 32 * STEPS + 32 * s + lane;
        key[s] = -1;  // no token: the last digit in every pass, behind that digit's keys; not stored
        pos[s] = i0 + i;
        if (i < mine) {
            const long long id = ids[i0 + i];
            bad |= id >= V;
            key[s] = key_of(id, V);
        }
    }
    if (bad) atomicCAS(status, 0, kDevBounds);
    for (int i = rank * kClusterThreads + tid; i <= V / 32; i += CS * kClusterThreads) present[i] = 0;
    for (int p = 0; p < passes; ++p) {
        for (int d = lane; d < kBins; d += 32) sh.count[warp][d] = 0;
        __syncwarp();
        rank_in_warp<STEPS>(key, p * width, width, sh.count[warp], place);
        __syncthreads();
        if (tid < kBins) {  // to each warp's first place among its digit's keys; the padding has the last digit
            int sum = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const int c = sh.count[w][tid];
                sh.count[w][tid] = (uint16_t)sum;
                sum += c;
            }
            sh.total[tid] = sum - (tid == mask ? STEPS * kClusterThreads - mine : 0);
        }
        cluster_sync<CS>();
        int all = 0, before = 0;
        if (tid < kBins) {
            if constexpr (CS > 1) {
#pragma unroll
                for (int c = 0; c < CS; ++c) {
                    uint32_t a;
                    int v;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(&sh.total[tid])), "r"(c));
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
                    all += v;
                    if (c < rank) before += v;
                }
            } else {
                all = sh.total[tid];
            }
            int run = all;  // exclusive sum over the digits
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += x;
            }
            if (lane == 31) sh.warp_sums[warp] = run;
            all = run - all;
        }
        __syncthreads();
        if (tid < kBins) {
            for (int w = 0; w < warp; ++w) all += sh.warp_sums[w];
            sh.base[tid] = all + before;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int i = warp * 32 * STEPS + 32 * s + lane;
            if (i >= mine) continue;
            const int d = (key[s] >> (p * width)) & mask, to = sh.base[d] + sh.count[warp][d] + place[s];
            if constexpr (CS > 1) {
                uint32_t a;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(&sh.sorted[to % per])), "r"(to / per));
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(key[s]), "r"(pos[s]) : "memory");
            } else {
                sh.sorted[to] = make_int2(key[s], pos[s]);
            }
        }
        cluster_sync<CS>();
        if (p == passes - 1) break;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int i = warp * 32 * STEPS + 32 * s + lane;
            key[s] = -1;
            if (i < mine) {
                const int2 v = sh.sorted[i];
                key[s] = v.x;
                pos[s] = v.y;
            }
        }
        __syncthreads();
    }
    // (the last barrier also keeps every CTA until the others have read its counts)
    for (int i = tid; i < mine; i += kClusterThreads) {
        const int2 v = sh.sorted[i];
        key_out[i0 + i] = v.x;
        pos_out[i0 + i] = v.y;
        if (i == 0 || sh.sorted[i - 1].x != v.x) atomicOr(&present[v.x >> 5], 1u << (v.x & 31));
    }
}
static_assert(kBins <= 16 * 32, "warp_sums");

// ---------------------------------------------------------------------------------------------
// sums: a warp adds up the rows of one tile of sorted tokens, 32 UPL units of the columns, eight rows in flight: HBM
// bounds it together with the zeros that the blocks behind write.  Sums are fp32, scaled once at their end.
struct SumParams {
    const int *key, *pos;
    float *dtable, *part;
    float scale;
    int n, D, Dp, V, tile, tiles, accumulate;
    int cleared;  // rows [0, cleared) are zero already; V when there is nothing to clear
    const uint32_t *present;  // a bit for each id that has a token
};

// Clears the rows without a token among those that the sort's kernels left.  The warps of all clearing
// blocks sweep over the table side by side; a lane reads the presence bit of one of its warp's next 32 rows.
__device__ __forceinline__ void clear_absent(const SumParams &p, int block, int blocks)
{
    const int lane = threadIdx.x & 31, warps = blocks * (kThreads / 32);
    for (long long r0 = p.cleared + block * (kThreads / 32) + (threadIdx.x >> 5); r0 < p.V; r0 += 32LL * warps) {
        const long long mine = r0 + (long long)lane * warps;
        const bool absent = mine < p.V && !(p.present[mine >> 5] >> (mine & 31) & 1);
        for (uint32_t left = __ballot_sync(0xffffffffu, absent); left; left &= left - 1) {
            float *d = p.dtable + (size_t)(r0 + (long long)(__ffs(left) - 1) * warps) * p.D;
            // single values up to a 16-byte boundary, units, and what is left behind them
            const int head = min(p.D, (int)(-((uintptr_t)d >> 2) & 3)), quads = (p.D - head) >> 2, tail = head + 4 * quads;
            for (int c = lane; c < quads; c += 32) reinterpret_cast<float4 *>(d + head)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < head) d[lane] = 0.f;
            if (lane < p.D - tail) d[tail + lane] = 0.f;
        }
    }
}

// Adds onto the table without waiting for its old value.  Each element gets one addition in a call, so
// the order of these operations cannot change a result.  They take subnormal numbers for zeros; a load, a fused
// multiply-add and a store in their place take 40 us for 33 (16384 x 768 bf16 of 50021), with the loads beside those of the rows 36.
__device__ __forceinline__ void add_onto(float *p, const float4 v)
{
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

template <typename io_t, int VEC, int UPL>
__global__ void __launch_bounds__(kThreads, 3) sum_kernel(const io_t *__restrict__ dout, const SumParams p, int chunks)
{
    constexpr int AHEAD = 8 / UPL;
    const int lane = threadIdx.x & 31;
    const int sums = (p.tiles + kThreads / 32 - 1) / (kThreads / 32) * chunks;  // blocks that add; the others clear
    tc::allow_dependent_launch();
    tc::grid_dependency_wait();
    if ((int)blockIdx.x >= sums) return clear_absent(p, blockIdx.x - sums, gridDim.x - sums);
    const int tile = blockIdx.x / chunks * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile >= p.tiles) return;
    const int s0 = tile * p.tile, s1 = min(p.n, s0 + p.tile), units = p.D / VEC;
    const int u0 = blockIdx.x % chunks * 32 * UPL + lane;
    const int before = s0 > 0 ? p.key[s0 - 1] : -1, behind = s1 < p.n ? p.key[s1] : -1;
    const int first = p.key[s0];
    const bool from_before = before == first;
    float acc[UPL][VEC];
#pragma unroll
    for (int j = 0; j < UPL; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    bool in_first = true;
    int cur = first;
    auto flush = [&](bool in_last) {
        if (cur != p.V) {
            float *to;
            const bool partial = (in_first && from_before) || (in_last && behind == cur);
            if (partial)
                to = p.part + ((size_t)tile * 2 + (in_first && from_before ? 0 : 1)) * p.Dp;
            else
                to = p.dtable + (size_t)cur * p.D;
#pragma unroll
            for (int j = 0; j < UPL; ++j)
                if (u0 + 32 * j < units) {
                    float *q = to + (size_t)(u0 + 32 * j) * VEC;
#pragma unroll
                    for (int e = 0; e < VEC; e += (VEC >= 4 ? 4 : 1)) {
                        if constexpr (VEC >= 4) {
                            float4 v = make_float4(acc[j][e], acc[j][e + 1], acc[j][e + 2], acc[j][e + 3]);
                            if (!partial) v.x *= p.scale, v.y *= p.scale, v.z *= p.scale, v.w *= p.scale;
                            if (!partial && p.accumulate)
                                add_onto(q + e, v);
                            else
                                *reinterpret_cast<float4 *>(q + e) = v;
                        } else {
                            const float v = partial ? acc[j][e] : acc[j][e] * p.scale;
                            if (!partial && p.accumulate)
                                atomicAdd(q + e, v);
                            else
                                q[e] = v;
                        }
                    }
                }
        }
#pragma unroll
        for (int j = 0; j < UPL; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
        in_first = false;
    };
    for (int c0 = s0; c0 < s1; c0 += 32) {  // 32 tokens: their keys and positions in one load each
        const int key32 = c0 + lane < s1 ? p.key[c0 + lane] : p.V, pos32 = c0 + lane < s1 ? p.pos[c0 + lane] : 0;
        const int here = min(32, s1 - c0);
        for (int s = 0; s < here; s += AHEAD) {
            io::Unit<io_t, VEC> x[AHEAD][UPL];
            int key[AHEAD];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                key[a] = __shfl_sync(0xffffffffu, key32, s + a);  // AHEAD divides 32; p.V behind the tile's end
                const int pos = __shfl_sync(0xffffffffu, pos32, s + a);
                if (key[a] != p.V) {
                    const io_t *src = dout + (size_t)pos * p.D;
#pragma unroll
                    for (int j = 0; j < UPL; ++j)
                        if (u0 + 32 * j < units) x[a][j] = io::load_unit<io_t, VEC>(src + (size_t)(u0 + 32 * j) * VEC);
                }
            }
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                if (s + a >= here) break;
                if (key[a] != cur) {
                    flush(false);
                    cur = key[a];
                }
                if (cur == p.V) continue;
#pragma unroll
                for (int j = 0; j < UPL; ++j)
                    if (u0 + 32 * j < units) {
                        float f[VEC];
                        x[a][j].get(f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) acc[j][e] += f[e];
                    }
            }
        }
    }
    flush(true);
}

// A run that crosses tile edges starts in tile a (its part is the tile's last), fills tiles a + 1 ..
// b - 1 and ends in tile b (their first parts).  A block looks at eight tiles and joins the runs that
// start there, 128 columns of them: the parts are split over the warps, whose sums are added in order.
__global__ void __launch_bounds__(kThreads) join_kernel(const SumParams p)
{
    __shared__ float4 sums[kThreads / 32][32];
    __shared__ int long_key[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = blockIdx.y * 128 + lane * 4;
    tc::grid_dependency_wait();
    // part 0: the last one of tile a; part i: the first one of tile a + i
    auto add_parts = [&](int a, int i0, int i1) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < p.Dp) {
#pragma unroll 8
            for (int i = i0; i < i1; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(p.part + ((size_t)(a + i) * 2 + (i == 0 ? 1 : 0)) * p.Dp + col);
                acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
            }
        }
        return acc;
    };
    auto finish = [&](int key, const float4 acc) {
        const float f[4] = {acc.x, acc.y, acc.z, acc.w};
        float *to = p.dtable + (size_t)key * p.D + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < p.D) to[i] = p.accumulate ? fmaf(f[i], p.scale, to[i]) : f[i] * p.scale;
    };
    // A warp takes the edge behind one tile: does a run cross it that did not start before tile a?
    const int a = blockIdx.x * (kThreads / 32) + warp;
    int key = -1, more = 0;
    if (a < p.tiles - 1) {
        const int e = (a + 1) * p.tile;  // the first token of the next tile
        const int last = p.key[e - 1], next = p.key[e], earlier = a > 0 ? p.key[e - p.tile - 1] : -1;
        // keys are sorted, so the tiles that begin with the key follow each other
        const int i = a + 1 + lane;
        const bool same = i < p.tiles && p.key[(size_t)i * p.tile] == next;
        more = __popc(__ballot_sync(0xffffffffu, same));
        if (next != p.V && last == next && earlier != next) key = next;
    }
    // One warp adds a few parts; more of them are worth the block's eight warps (16384 x 768 of 50021 in a graph: up to 32
    // parts by one warp 41.1 us, up to 8 39.8).
    const bool fits = more < 8;
    if (key >= 0 && fits) finish(key, add_parts(a, 0, more + 1));
    if (lane == 0) long_key[warp] = fits ? -1 : key;
    __syncthreads();
    for (int t = 0; t < kThreads / 32; ++t) {  // runs of more tiles: the whole block
        const int from = blockIdx.x * (kThreads / 32) + t, k = long_key[t];
        if (k < 0) continue;
        int b = from + 1;  // the first tile that does not begin with the key
        for (;;) {
            const int i = b + tid;
            const int same = __syncthreads_count(i < p.tiles && p.key[(size_t)i * p.tile] == k);
            b += same;
            if (same < kThreads) break;
        }
        const int parts = b - from, per = (parts + kThreads / 32 - 1) / (kThreads / 32);
        float4 acc = add_parts(from, min(parts, warp * per), min(parts, warp * per + per));
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kThreads / 32; ++w) {
                const float4 v = sums[w][lane];
                acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
            }
            finish(k, acc);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------
// Tokens per tile: 8, the rows that a warp has in flight, up to 1024 tiles; then up to 32, which leaves fewer
// runs to join (32768 tokens: 8 62 us, 32 54 us); longer ones for more tokens than 8192 tiles hold,
// which bounds the workspace.
constexpr int kTilesMax = 8193;
int tile_of(int n)
{
    int t = kTile;
    while (t < 32 && n / t > 1024) t *= 2;
    while (n / t >= kTilesMax) t *= 2;
    return t;
}

constexpr int kSmall = 2048;  // tokens that one CTA sorts

constexpr size_t cluster_smem(int steps) { return sizeof(ClusterShared) + (size_t)steps * kClusterThreads * sizeof(int2); }

// Columns are split over warps (32 units each, 64 for the narrow units of unaligned rows): tiles are few
// when tokens are, and a warp with one unit per lane keeps eight rows in flight.
template <typename io_t, int VEC>
cudaError_t launch_sum(const void *dout, const SumParams &p, int clear_blocks, cudaStream_t s)
{
    constexpr int UPL = VEC > 1 ? 1 : 2;
    const unsigned gx = (p.tiles + kThreads / 32 - 1) / (kThreads / 32), gy = (p.D / VEC + 32 * UPL - 1) / (32 * UPL);
    return launch_behind(sum_kernel<io_t, VEC, UPL>, dim3(gx * gy + clear_blocks), kThreads, s, (const io_t *)dout, p, (int)gy);
}

template <typename io_t, int VEC>
cudaError_t launch_lookup(const EmbedArgs &a, const TokenLaunch &l)
{
    const int units = a.D / VEC, upl = units > 64 ? 4 : units > 32 ? 2 : 1, chunks = (units + 32 * upl - 1) / (32 * upl);
    const long long warps = (long long)a.n * chunks;
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    cudaStream_t s = l.timer->stream;
    l.timer->begin("embed");
    if (upl == 4)
        lookup_kernel<io_t, VEC, 4><<<grid, kThreads, 0, s>>>(a.ids, (const io_t *)a.table, a.ld_table, a.scale, (io_t *)a.out,
                                                             a.n, a.D, a.V, chunks, l.d_status);
    else if (upl == 2)
        lookup_kernel<io_t, VEC, 2><<<grid, kThreads, 0, s>>>(a.ids, (const io_t *)a.table, a.ld_table, a.scale, (io_t *)a.out,
                                                             a.n, a.D, a.V, chunks, l.d_status);
    else
        lookup_kernel<io_t, VEC, 1><<<grid, kThreads, 0, s>>>(a.ids, (const io_t *)a.table, a.ld_table, a.scale, (io_t *)a.out,
                                                             a.n, a.D, a.V, chunks, l.d_status);
    l.timer->end();
    return cudaGetLastError();
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
int padded(int D) { return (D + 3) & ~3; }

}  // namespace embed

using namespace embed;

template <int CS, int STEPS>
static cudaError_t prepare_sort()
{
    return cudaFuncSetAttribute(cluster_sort_kernel<CS, STEPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cluster_smem(STEPS));
}

cudaError_t embed_prepare()
{
    cudaError_t e = prepare_sort<1, 2>();
    if (e == cudaSuccess) e = prepare_sort<kCluster, 1>();
    if (e == cudaSuccess) e = prepare_sort<kCluster, 2>();
    if (e == cudaSuccess) e = prepare_sort<kCluster, 4>();
    if (e == cudaSuccess) e = prepare_sort<kCluster, kClusterSteps>();
    return e;
}

cudaError_t embed_forward(prism_dtype io, const EmbedArgs &a, const TokenLaunch &l)
{
    // 16-byte units where every row of both tensors starts on a 16-byte boundary
    const int vec = io == PRISM_BF16 ? 8 : 4;
    const bool units = a.D % vec == 0 && a.ld_table % vec == 0;
    if (io == PRISM_BF16)
        return units ? launch_lookup<__nv_bfloat16, 8>(a, l) : launch_lookup<__nv_bfloat16, 1>(a, l);
    return units ? launch_lookup<float, 4>(a, l) : launch_lookup<float, 1>(a, l);
}

size_t embed_workspace_bytes(int max_rows, int D, int V)
{
    const size_t all = ((size_t)max_rows + kTile - 1) / kTile, tiles = all < kTilesMax ? all : kTilesMax;
    return 4 * up256((size_t)max_rows * 4) + up256((size_t)kPassesMax * kBlocksMax * kBins * 4) +
           up256(((size_t)V / 32 + 1) * 4) +
           up256(tiles * 2 * padded(D) * 4);
}

void embed_carve(int max_rows, int V, void *base, EmbedWorkspace *w)
{
    char *p = (char *)base;
    auto take = [&](size_t bytes) {
        char *q = p;
        p += up256(bytes);
        return q;
    };
    for (int i = 0; i < 2; ++i) {
        w->key[i] = (int *)take((size_t)max_rows * 4);
        w->pos[i] = (int *)take((size_t)max_rows * 4);
    }
    w->hist = (int *)take((size_t)kPassesMax * kBlocksMax * kBins * 4);
    w->present = (uint32_t *)take(((size_t)V / 32 + 1) * 4);
    w->part = (float *)take(0);
}

cudaError_t embed_backward(prism_dtype io, const EmbedBackwardArgs &a, const EmbedWorkspace &w, const TokenLaunch &l)
{
    cudaStream_t s = l.timer->stream;
    cudaError_t e;
    int bits = 1;
    while ((1LL << bits) <= a.V) ++bits;  // keys 0 .. V
    const int passes = (bits + 8) / 9, width = (bits + passes - 1) / passes, mask = (1 << width) - 1;
    // The sort's kernels clear the table's first rows in equal shares, as many as fit beside them (without
    // tokens there are no sums, and they clear everything).
    const bool in_cluster = a.n <= kCluster * kClusterThreads * kClusterSteps;
    const int kernels = in_cluster ? 1 : passes + 1, fill_blocks = a.accumulate ? 0 : (in_cluster && a.n > kCounted ? 2 : 4) * l.sm_count;
    const long long beside = kernels * kBesideSort / ((long long)a.D * 4);
    const int cleared = a.accumulate || a.n == 0 || beside >= a.V ? a.V : (int)beside;
    const size_t floats = (size_t)cleared * a.D;
    auto share = [&](int i) {
        const size_t quads = floats / 4;
        return Fill{a.dtable, quads * i / kernels * 4, i == kernels - 1 ? floats : quads * (i + 1) / kernels * 4};
    };
    int result = 0;  // which of the two buffers holds the sorted tokens
    if (a.n <= kCounted) {
        l.timer->begin("embed_sort");
        counted_sort_kernel<<<1 + fill_blocks, kCounted, 0, s>>>(a.ids, a.n, a.V, w.key[0], w.pos[0], w.present, l.d_status, share(0));
        l.timer->end();
    } else if (in_cluster) {
        l.timer->begin("embed_sort");
        const int per = a.n <= kSmall ? a.n : (a.n + kCluster - 1) / kCluster;
        auto go = [&](auto cs, auto steps) {
            constexpr int CS = decltype(cs)::value, STEPS = decltype(steps)::value;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(CS + fill_blocks / kCluster * kCluster);
            cfg.blockDim = dim3(kClusterThreads);
            cfg.dynamicSmemBytes = cluster_smem(STEPS);
            cfg.stream = s;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = CS;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = CS > 1 ? 1 : 0;
            e = cudaLaunchKernelEx(&cfg, cluster_sort_kernel<CS, STEPS>, a.ids, a.n, per, a.V, width, passes, w.key[0], w.pos[0],
                                   w.present, l.d_status, share(0));
        };
        if (a.n <= kSmall) go(std::integral_constant<int, 1>(), std::integral_constant<int, 2>());
        else if (per <= kClusterThreads) go(std::integral_constant<int, kCluster>(), std::integral_constant<int, 1>());
        else if (per <= 2 * kClusterThreads) go(std::integral_constant<int, kCluster>(), std::integral_constant<int, 2>());
        else if (per <= 4 * kClusterThreads) go(std::integral_constant<int, kCluster>(), std::integral_constant<int, 4>());
        else go(std::integral_constant<int, kCluster>(), std::integral_constant<int, kClusterSteps>());
        l.timer->end();
        if (e != cudaSuccess) return e;
    } else {
        // at most kBlocksMax blocks, of whole tiles of kSub keys
        const int chunk = (int)((((long long)a.n + kBlocksMax - 1) / kBlocksMax + kSub - 1) / kSub * kSub);
        const int nb = (a.n + chunk - 1) / chunk;
        auto hist = [&](int pass) { return w.hist + (size_t)pass * kBlocksMax * kBins; };
        l.timer->begin("embed_count");
        count_kernel<<<nb + fill_blocks, kSortThreads, 0, s>>>(a.ids, a.n, a.V, chunk, mask, passes, nb, w.hist, w.present, l.d_status, share(0));
        l.timer->end();
        for (int p = 0; p < passes; ++p) {
            const int to = p & 1, from = to ^ 1;
            const Pass ps{a.ids, w.key[from], w.pos[from], w.key[to], w.pos[to], hist(p), p + 1 < passes ? hist(p + 1) : nullptr, w.present,
                          a.n, a.V, chunk, nb, p * width, width, mask, (p + 1) * width};
            l.timer->begin("embed_scatter");
            e = launch_behind(p == 0 ? scatter_kernel<true> : scatter_kernel<false>, dim3(nb + fill_blocks), kSortThreads, s, ps, share(p + 1));
            l.timer->end();
            if (e != cudaSuccess) return e;
            result = to;
        }
    }
    if ((e = cudaGetLastError()) != cudaSuccess || a.n == 0) return e;
    SumParams sp;
    sp.key = w.key[result];
    sp.pos = w.pos[result];
    sp.dtable = a.dtable;
    sp.part = w.part;
    sp.scale = a.scale;
    sp.n = a.n;
    sp.D = a.D;
    sp.Dp = padded(a.D);
    sp.V = a.V;
    sp.tile = tile_of(a.n);
    sp.tiles = (a.n + sp.tile - 1) / sp.tile;
    sp.accumulate = a.accumulate;
    sp.cleared = cleared;
    sp.present = w.present;
    // Blocks that clear, behind those that add: many small shares even out (14309 x 648 of 130295: 2 a SM 83 us, 4 76 us, 8
    // 72 us, 16 71 us, 32 72 us; 16384 x 768 of 50021 46, 43.6, 43.4, 43.8 and 45.5 us).
    const int clear_blocks = cleared < a.V ? 16 * l.sm_count : 0;
    l.timer->begin("embed_sum");
    if (io == PRISM_BF16)
        e = a.D % 8 == 0 ? launch_sum<__nv_bfloat16, 8>(a.dout, sp, clear_blocks, s) : launch_sum<__nv_bfloat16, 1>(a.dout, sp, clear_blocks, s);
    else
        e = a.D % 4 == 0 ? launch_sum<float, 4>(a.dout, sp, clear_blocks, s) : launch_sum<float, 1>(a.dout, sp, clear_blocks, s);
    l.timer->end();
    if (e != cudaSuccess || sp.tiles < 2) return e;
    l.timer->begin("embed_join");
    e = launch_behind(join_kernel, dim3((sp.tiles + kThreads / 32 - 1) / (kThreads / 32), (a.D + 127) / 128), kThreads, s, sp);
    l.timer->end();
    return e;
}

}  // namespace prism
