// Embedding lookup and its gradient.
//
//   out_i     = scale table[ids_i]                           (zeros where there is no token)
//   dtable[v] = scale sum_{i : ids_i = v} dout_i             (every row written, or added to)
//
// Both only move data: the lookup reads one table row and writes one output row per token; the
// gradient reads dout once and writes the whole fp32 table once, so HBM bounds both.
//
// The gradient's sum over equal ids must not depend on the order in which blocks run, so the tokens
// are first sorted by id, stably (least significant digit first, digits of at most 9 bits: two
// passes for vocabularies below 2^18).  A pass ranks keys inside a warp with match_any (the lanes
// that hold the same digit), so a digit that half of the tokens share costs no more than any other;
// the offsets of a block come from the digit counts of the blocks before it, which every block adds
// up for itself.  Then a warp walks a tile of consecutive sorted tokens and adds their rows up in
// registers, writing a sum whenever the id changes.  Runs that cross a tile's edge leave their part
// in the workspace; a last kernel adds those parts in order (a token that fills many tiles, as the
// most frequent ones of a text do, is spread over eight warps there).
#include "io_util.h"
#include "prism_tokens.h"

namespace prism {
namespace embed {

constexpr int kBins = 512;       // digits of up to 9 bits
constexpr int kPassesMax = 4;    // ids below 2^30 and the "no token" key: at most 31 bits
constexpr int kBlocksMax = 128;  // blocks of one sort pass
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32, kSteps = 8;
constexpr int kSub = kSortThreads * kSteps;  // keys that a block ranks at a time

constexpr int kThreads = 256;
constexpr int kTile = 16;  // sorted tokens per warp, at least (tile_of)

// ---------------------------------------------------------------------------------------------
// lookup: a warp takes 32 UPL units of one row
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
template <int STEPS>
__device__ __forceinline__ void rank_in_warp(const int (&key)[STEPS], int shift, int mask, uint16_t *count, int (&rank)[STEPS])
{
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int d = (key[s] >> shift) & mask;
        const uint32_t peers = __match_any_sync(0xffffffffu, d);
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

// Digit counts of each block's chunk of the tokens, for the first pass; clears the later passes' counts.
__global__ void __launch_bounds__(kSortThreads) count_kernel(const long long *__restrict__ ids, int n, int V, int chunk,
                                                            int mask, int passes, int *hist, int *status)
{
    __shared__ int bins[kBins];
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) bins[d] = 0;
    __syncthreads();
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
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) scatter_kernel(const long long *__restrict__ ids, const int *__restrict__ key_in,
                                                              const int *__restrict__ pos_in, int *__restrict__ key_out,
                                                              int *__restrict__ pos_out, int n, int V, int chunk, int shift,
                                                              int mask, int next_shift, int next_mask,
                                                              const int *__restrict__ hist, int *hist_next)
{
    __shared__ uint16_t count[kSortWarps][kBins];
    __shared__ int base[kBins];
    __shared__ int warp_sums[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x, nb = gridDim.x;
    int total[2] = {0, 0}, before[2] = {0, 0};
    for (int o = 0; o < nb; ++o) {
        const int2 h = *reinterpret_cast<const int2 *>(hist + (size_t)o * kBins + 2 * tid);
        total[0] += h.x, total[1] += h.y;
        if (o < b) before[0] += h.x, before[1] += h.y;
    }
    scan_bins(total[0], total[1], warp_sums);
    base[2 * tid] = total[0] + before[0];
    base[2 * tid + 1] = total[1] + before[1];
    const int i1 = min((long long)n, ((long long)b + 1) * chunk);
    for (int i0 = b * chunk; i0 < i1; i0 += kSub) {
        for (int d = lane; d < kBins; d += 32) count[warp][d] = 0;
        __syncwarp();
        int key[kSteps], pos[kSteps], rank[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = i0 + warp * 32 * kSteps + 32 * s + lane;
            key[s] = 0x7fffffff;  // behind every key of its digit, and not stored
            pos[s] = i;
            if (i < i1) {
                key[s] = FIRST ? key_of(ids[i], V) : key_in[i];
                if (!FIRST) pos[s] = pos_in[i];
            }
        }
        rank_in_warp<kSteps>(key, shift, mask, count[warp], rank);
        __syncthreads();
        int sum[2] = {0, 0};  // of this tile, for the next one's base
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = count[w][2 * tid + e];
                count[w][2 * tid + e] = (uint16_t)sum[e];
                sum[e] += c;
            }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = i0 + warp * 32 * kSteps + 32 * s + lane;
            if (i >= i1) continue;
            const int d = (key[s] >> shift) & mask;
            const int to = base[d] + count[warp][d] + rank[s];
            key_out[to] = key[s];
            pos_out[to] = pos[s];
            if (hist_next) atomicAdd(&hist_next[(size_t)(to / chunk) * kBins + ((key[s] >> next_shift) & next_mask)], 1);
        }
        __syncthreads();
        base[2 * tid] += sum[0];
        base[2 * tid + 1] += sum[1];
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------
// sums: a warp adds up the rows of one tile of sorted tokens, 32 UPL units of the columns
struct SumParams {
    const int *key, *pos;
    float *dtable, *part;
    float scale;
    int n, D, Dp, V, tile, tiles, accumulate;
};

template <typename io_t, int VEC, int UPL>
__global__ void __launch_bounds__(kThreads) sum_kernel(const io_t *__restrict__ dout, const SumParams p)
{
    constexpr int AHEAD = 4;
    const int lane = threadIdx.x & 31;
    const int tile = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile >= p.tiles) return;
    const int s0 = tile * p.tile, s1 = min(p.n, s0 + p.tile), units = p.D / VEC;
    const int u0 = blockIdx.y * 32 * UPL + lane;
    const int first = p.key[s0], last = p.key[s1 - 1];
    const bool from_before = s0 > 0 && p.key[s0 - 1] == first, goes_on = s1 < p.n && p.key[s1] == last;
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
            const bool partial = (in_first && from_before) || (in_last && goes_on);
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
                            if (!partial) {
                                v.x *= p.scale, v.y *= p.scale, v.z *= p.scale, v.w *= p.scale;
                                if (p.accumulate) {
                                    const float4 o = *reinterpret_cast<const float4 *>(q + e);
                                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                                }
                            }
                            *reinterpret_cast<float4 *>(q + e) = v;
                        } else {
                            float v = acc[j][e];
                            if (!partial) v = p.accumulate ? fmaf(v, p.scale, q[e]) : v * p.scale;
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
    for (int s = s0; s < s1; s += AHEAD) {
        io::Unit<io_t, VEC> x[AHEAD][UPL];
        int key[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            key[a] = s + a < s1 ? p.key[s + a] : p.V;
            if (key[a] != p.V) {
                const io_t *src = dout + (size_t)p.pos[s + a] * p.D;
#pragma unroll
                for (int j = 0; j < UPL; ++j)
                    if (u0 + 32 * j < units) x[a][j] = io::load_unit<io_t, VEC>(src + (size_t)(u0 + 32 * j) * VEC);
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (s + a >= s1) break;
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
    flush(true);
}

// A run that crosses tile edges starts in tile a (its part is the tile's last), fills tiles a + 1 ..
// b - 1 and ends in tile b (their first parts).  A block looks at eight tiles and joins the runs that
// start there, 128 columns of them: the parts are split over the warps, whose sums are added in order.
__global__ void __launch_bounds__(kThreads) join_kernel(const SumParams p)
{
    __shared__ float4 sums[kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.y * 128 + lane * 4;
    for (int t = 0; t < 8; ++t) {
        const int a = blockIdx.x * 8 + t;
        if (a >= p.tiles - 1) break;
        const int e = (a + 1) * p.tile;  // the first token of the next tile (a is not the last tile)
        const int key = p.key[e];
        if (key == p.V || p.key[e - 1] != key) continue;               // no run crosses this edge
        if (a > 0 && p.key[e - p.tile - 1] == key) continue;           // ... or it started before tile a
        int b0 = a + 1, b1 = p.tiles;                                  // the first tile that does not begin with the key
        while (b0 < b1) {
            const int m = (b0 + b1) >> 1;
            if (p.key[m * p.tile] == key) b0 = m + 1;
            else b1 = m;
        }
        const int parts = b0 - a;  // part 0: the last one of tile a; part i: the first one of tile a + i
        const int per = (parts + kThreads / 32 - 1) / (kThreads / 32);
        const int i0 = min(parts, warp * per), i1 = min(parts, i0 + per);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < p.Dp) {
#pragma unroll 8
            for (int i = i0; i < i1; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(p.part + ((size_t)(a + i) * 2 + (i == 0 ? 1 : 0)) * p.Dp + col);
                acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
            }
        }
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp == 0 && col < p.D) {
            const int used = (parts + per - 1) / per;
            for (int w = 1; w < used; ++w) {
                const float4 v = sums[w][lane];
                acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
            }
            const float f[4] = {acc.x, acc.y, acc.z, acc.w};
            float *to = p.dtable + (size_t)key * p.D + col;
            for (int i = 0; i < 4; ++i)
                if (col + i < p.D) to[i] = p.accumulate ? fmaf(f[i], p.scale, to[i]) : f[i] * p.scale;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------
// Tokens per tile: 16, so that 16K tokens make 1024 warps; longer ones for more tokens than 8192
// tiles hold, which bounds the workspace.
constexpr int kTilesMax = 8193;
int tile_of(int n)
{
    int t = kTile;
    while (n / t >= kTilesMax) t *= 2;
    return t;
}

template <typename io_t, int VEC>
cudaError_t launch_sum(const io_t *dout, const SumParams &p, cudaStream_t s)
{
    const int units = p.D / VEC;
    const unsigned gx = (p.tiles + kThreads / 32 - 1) / (kThreads / 32);
    if (units > 64)
        sum_kernel<io_t, VEC, 4><<<dim3(gx, (units + 127) / 128), kThreads, 0, s>>>(dout, p);
    else if (units > 32)
        sum_kernel<io_t, VEC, 2><<<dim3(gx, 1), kThreads, 0, s>>>(dout, p);
    else
        sum_kernel<io_t, VEC, 1><<<dim3(gx, 1), kThreads, 0, s>>>(dout, p);
    return cudaGetLastError();
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

cudaError_t embed_forward(prism_dtype io, const EmbedArgs &a, const TokenLaunch &l)
{
    // 16-byte units where every row of both tensors starts on a 16-byte boundary
    const int vec = io == PRISM_BF16 ? 8 : 4;
    const bool units = a.D % vec == 0 && a.ld_table % vec == 0;
    if (io == PRISM_BF16)
        return units ? launch_lookup<__nv_bfloat16, 8>(a, l) : launch_lookup<__nv_bfloat16, 1>(a, l);
    return units ? launch_lookup<float, 4>(a, l) : launch_lookup<float, 1>(a, l);
}

size_t embed_workspace_bytes(int max_rows, int D)
{
    const size_t all = ((size_t)max_rows + kTile - 1) / kTile, tiles = all < kTilesMax ? all : kTilesMax;
    return 4 * up256((size_t)max_rows * 4) + up256((size_t)kPassesMax * kBlocksMax * kBins * 4) +
           up256(tiles * 2 * padded(D) * 4);
}

void embed_carve(int max_rows, int D, void *base, EmbedWorkspace *w)
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
    w->part = (float *)take(0);
}

cudaError_t embed_backward(prism_dtype io, const EmbedBackwardArgs &a, const EmbedWorkspace &w, const TokenLaunch &l)
{
    cudaStream_t s = l.timer->stream;
    cudaError_t e;
    if (!a.accumulate && (e = cudaMemsetAsync(a.dtable, 0, (size_t)a.V * a.D * 4, s)) != cudaSuccess) return e;
    if (a.n == 0) return cudaSuccess;
    int bits = 1;
    while ((1LL << bits) <= a.V) ++bits;  // keys 0 .. V
    const int passes = (bits + 8) / 9, width = (bits + passes - 1) / passes, mask = (1 << width) - 1;
    // at most kBlocksMax blocks, of whole tiles of kSub keys
    const int chunk = (int)((((long long)a.n + kBlocksMax - 1) / kBlocksMax + kSub - 1) / kSub * kSub);
    const int nb = (a.n + chunk - 1) / chunk;
    auto hist = [&](int pass) { return w.hist + (size_t)pass * kBlocksMax * kBins; };
    l.timer->begin("embed_count");
    count_kernel<<<nb, kSortThreads, 0, s>>>(a.ids, a.n, a.V, chunk, mask, passes, w.hist, l.d_status);
    l.timer->end();
    for (int p = 0; p < passes; ++p) {
        const int to = p & 1, from = to ^ 1;
        l.timer->begin("embed_scatter");
        int *next = p + 1 < passes ? hist(p + 1) : nullptr;
        if (p == 0)
            scatter_kernel<true><<<nb, kSortThreads, 0, s>>>(a.ids, nullptr, nullptr, w.key[to], w.pos[to], a.n, a.V, chunk, 0,
                                                             mask, width, mask, hist(0), next);
        else
            scatter_kernel<false><<<nb, kSortThreads, 0, s>>>(nullptr, w.key[from], w.pos[from], w.key[to], w.pos[to], a.n, a.V,
                                                              chunk, p * width, mask, (p + 1) * width, mask, hist(p), next);
        l.timer->end();
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    SumParams sp;
    sp.key = w.key[(passes - 1) & 1];
    sp.pos = w.pos[(passes - 1) & 1];
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
    l.timer->begin("embed_sum");
    if (io == PRISM_BF16)
        e = a.D % 8 == 0 ? launch_sum<__nv_bfloat16, 8>((const __nv_bfloat16 *)a.dout, sp, s)
                         : launch_sum<__nv_bfloat16, 1>((const __nv_bfloat16 *)a.dout, sp, s);
    else
        e = a.D % 4 == 0 ? launch_sum<float, 4>((const float *)a.dout, sp, s) : launch_sum<float, 1>((const float *)a.dout, sp, s);
    l.timer->end();
    if (e != cudaSuccess || sp.tiles < 2) return e;
    l.timer->begin("embed_join");
    join_kernel<<<dim3((sp.tiles + 7) / 8, (a.D + 127) / 128), kThreads, 0, s>>>(sp);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace prism
