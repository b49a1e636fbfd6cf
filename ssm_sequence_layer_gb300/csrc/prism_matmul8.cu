// Matrix product of e4m3 operands with a scale for each block of 128, and the weights' layout.
//
//   out[m, j] = sum_b a_scale[m, b] w_scale[j / 128, b] c_b[m, j],   c_b[m, j] = sum_{k in block b} a8[m, k] w8[j, k]
//
// Products of e4m3 values are exact in fp32; the sum over a block is scaled and added in fp32 once per
// block.  Few rows are bound by the weights' bytes (skinny_kernel), many by the tensor cores and by the
// output's bytes (product_kernel).
#include <cudaTypedefs.h>

#include "io_util.h"
#include "prism_tokens.h"
#include "tc_ptx.h"

namespace prism {
namespace mm8 {

constexpr int kBlock = 128;
constexpr float kMaxE4M3 = 448.f, kMinScale = 1.17549435e-38f;

template <typename out_t>
struct Params {
    const uint8_t *a, *w;
    const float *a_scale, *w_scale;
    out_t *out;
    int M, N, K, KB;
};

// ---------------------------------------------------------------------------------------------
// Few rows (M <= 16): the weights' bytes bound the product, every weight is used M times at most.  A
// warp takes RPW tiles of 16 rows of w8 as A operands of m16n8k32 products straight from global memory to
// registers (16 bytes of a row per lane and load, four loads for a block of 16 x 128), and 8 NT rows
// of a8 as B operands.  The products' k order is a free choice as long as both operands share it: the
// four words of a lane's 16 bytes serve as the k slots (lane % 4) 4 .. + 3 and 16 + (lane % 4) 4 .. + 3 of
// two products.  KS warps of a CTA share their tiles and split the blocks of 128 among them, so that
// narrow products still fill the machine; their sums are added in a fixed order.  8 x 50048 x 768 takes 10.0 us
// (3.9 TB/s) and 8 x 32768 x 4096 24.8 us (5.4 TB/s) among calls of a graph: the loads in flight bound it, but three or
// four blocks ahead (14 us, against 12 by single calls), whole lines of one row per load (14.8), rings of bulk copies (16.4)
// and the weights as the tcgen05 operand (14.1) are all slower.
constexpr int kSkinnyWarps = 8;

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename out_t, int NT, int KS, int RPW>  // RPW: tiles of 16 rows of a warp, which share a8
__global__ void __launch_bounds__(32 * kSkinnyWarps) skinny_kernel(const Params<out_t> p)
{
    constexpr int RT = kSkinnyWarps / KS;  // warps of a CTA with rows of their own
    constexpr int AHEAD = 2;               // blocks of 128 in flight
    __shared__ float parts[KS > 1 ? kSkinnyWarps : 1][16 * RPW][8 * NT + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int ks = warp % KS, n0 = (blockIdx.x * RT + warp / KS) * 16 * RPW;
    float total[RPW][NT][4];
#pragma unroll
    for (int r = 0; r < RPW; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[r][t][i] = 0.f;
    if (n0 < p.N) {
        // rows beyond the operands' last are read as the last and not stored
        const uint8_t *wr[2 * RPW];
#pragma unroll
        for (int r = 0; r < 2 * RPW; ++r) wr[r] = p.w + (size_t)min(n0 + g + 8 * r, p.N - 1) * p.K;
        const float *ws = p.w_scale + (size_t)(n0 / kBlock) * p.KB;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        uint4 w[AHEAD][2 * RPW][2];
        auto load = [&](int slot, int b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = b * kBlock + h * 64 + q * 16;
#pragma unroll
                for (int r = 0; r < 2 * RPW; ++r)
                    w[slot][r][h] = k < p.K ? __ldcs(reinterpret_cast<const uint4 *>(wr[r] + k)) : zero;
            }
        };
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) load(s, ks + s * KS);
        for (int b0 = ks; b0 < p.KB; b0 += AHEAD * KS) {
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) {
                const int b = b0 + s * KS;
                if (b >= p.KB) break;
                uint4 a[NT][2];
                float sa[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint8_t *ar = p.a + (size_t)min(8 * t + g, p.M - 1) * p.K;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = b * kBlock + h * 64 + q * 16;
                        a[t][h] = k < p.K ? __ldg(reinterpret_cast<const uint4 *>(ar + k)) : zero;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) sa[t][i] = p.a_scale[(size_t)min(8 * t + 2 * q + i, p.M - 1) * p.KB + b];
                }
                const float sw = ws[b];
#pragma unroll
                for (int r = 0; r < RPW; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 lo = w[s][2 * r][h], hi = w[s][2 * r + 1][h];
                            mma_e4m3(c, lo.x, hi.x, lo.y, hi.y, a[t][h].x, a[t][h].y);
                            mma_e4m3(c, lo.z, hi.z, lo.w, hi.w, a[t][h].z, a[t][h].w);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[r][t][i] = fmaf(c[i], sa[t][i & 1] * sw, total[r][t][i]);
                    }
                load(s, b + AHEAD * KS);
            }
        }
    }
    if constexpr (KS > 1) {
#pragma unroll
        for (int r = 0; r < RPW; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) parts[warp][16 * r + g + 8 * (i >> 1)][8 * t + 2 * q + (i & 1)] = total[r][t][i];
        __syncthreads();
        if (ks != 0) return;
#pragma unroll
        for (int r = 0; r < RPW; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    for (int o = 1; o < KS; ++o) total[r][t][i] += parts[warp + o][16 * r + g + 8 * (i >> 1)][8 * t + 2 * q + (i & 1)];
    }
#pragma unroll
    for (int r = 0; r < RPW; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = 8 * t + 2 * q + (i & 1), n = n0 + 16 * r + g + 8 * (i >> 1);
                if (m < p.M && n < p.N) io::st(p.out + (size_t)m * p.N + n, total[r][t][i]);
            }
}

template <typename out_t, int NT>
void launch_skinny(const Params<out_t> &p, int sm_count, cudaStream_t s)
{
    // Two tiles of 16 rows per warp share the reads of a8 and keep twice the bytes in flight, where that leaves enough warps:
    // 8 x 8192 x 8192 takes 21.2 us with one and 14.9 with two, 8 x 32768 x 4096 31.6 and 24.8, 16 x 8192 x 768 5.4 and 4.4, but
    // 8 x 6144 x 1024 3.4 and 3.7, 8 x 2304 x 768 2.2 and 2.4, 16 x 2304 x 768 2.8 and 3.0 (calls of a graph).
    const int pairs = (p.N + 31) / 32;
    constexpr int T = 32 * kSkinnyWarps;
    if (pairs * 8LL < (NT == 1 ? 12 : 6) * sm_count) {  // few: all warps of a CTA on one tile
        skinny_kernel<out_t, NT, 8, 1><<<(p.N + 15) / 16, T, 0, s>>>(p);
        return;
    }
    // As many warps as keep each SM's loads in flight, as far as the blocks of 128 reach: 4, 8 or 16 a SM give 30.3, 24.8 and
    // 26.7 us for 8 x 32768 x 4096, 10.0, 10.0 and 11.5 for 8 x 50048 x 768; 16 x 8192 x 8192 20.2, 22.3 and 22.2, 16 x 16384 x 768
    // 6.2, 7.7 and 10.5.
    int ks = 1;
    while (ks < 8 && ks < p.KB && (long long)pairs * ks < (NT == 1 ? 8 : 4) * sm_count) ks *= 2;
    const int rt = kSkinnyWarps / ks;
    const unsigned grid = (pairs + rt - 1) / rt;
    if (ks == 1) skinny_kernel<out_t, NT, 1, 2><<<grid, T, 0, s>>>(p);
    else if (ks == 2) skinny_kernel<out_t, NT, 2, 2><<<grid, T, 0, s>>>(p);
    else if (ks == 4) skinny_kernel<out_t, NT, 4, 2><<<grid, T, 0, s>>>(p);
    else skinny_kernel<out_t, NT, 8, 2><<<grid, T, 0, s>>>(p);
}

// ---------------------------------------------------------------------------------------------
// More rows: tcgen05 (kind::f8f6f4), persistent.  A tile of 128 rows x BN columns per CTA; each block
// of 128 in k is one stage of the operand ring (TMA, 128-byte swizzle: a row of a stage is 128 e4m3
// values) and four tcgen05.mma (K = 32) into one of two accumulators of BN columns in tensor memory.
// The accumulator holds c_b of one block only: the eight epilogue warps read it, scale it by
// a_scale[m, b] w_scale[j / 128, b] and add it to the sums in their registers (one row and BN / 2
// columns per thread, two columns per instruction) while the next block's products run into the other
// accumulator.  The sums take more registers than an even share, so the four warps of the issuing group hand
// theirs over.
//
// 4096 x 50048 x 768 takes 172 us among a graph's calls, 1.83 PFLOP/s.  The turn-around of the two accumulators bounds it: from the
// arrival that frees one to the moment its next sums can be read, the wake-ups of two threads, the products' latency and the
// reading take a time that neither the bytes nor the other CTAs change, and each block pays half of it.  Tiles of 128
// columns take 0.39 us a block on 8 CTAs and 0.41 on 80, of which the products are 0.13 and the operands' way into the SM, 64 bytes
// a cycle, is 0.26; tiles of 256 columns 0.52 us a block (4096 x 8192 x 4096: 116 us) for 0.26 and 0.39.  Without sums and stores
// 119 us are left.  Other forms: CTAs in pairs that read a shared operand once take 174 us (there, without sums and stores 117, with the
// sums 133, with the stores 161, and with one product of a block's four and neither 94, so that the other three, 384 cycles, cost half
// of that); tiles of two SMs, whose accumulators change hands over a longer way, 301.
using namespace prism::tc;

constexpr int BM = 128, STAGE_ROWS = 128;
constexpr int kEpilogueWarps = 8, kThreads = 128 + 32 * kEpilogueWarps;  // three warpgroups
// 384 threads launch with 168 registers each; 128 x 56 + 256 x 224 is the same number
constexpr int kIssueRegs = 56, kEpilogueRegs = 224;
static_assert(128 * kIssueRegs + 256 * kEpilogueRegs <= kThreads * 168, "registers handed over");

template <int BN>
struct Layout {
    static constexpr int STAGES = BN == 256 ? 3 : 5;
    static constexpr uint32_t A_BYTES = BM * kBlock, B_BYTES = BN * kBlock, STAGE = A_BYTES + B_BYTES;
    static constexpr uint32_t PIECE = 4096, OUT_WARP = 2 * PIECE;  // a warp's staging: pieces of 32 rows x 128 bytes of output
    static constexpr uint32_t OFF_OUT = STAGES * STAGE;
    static constexpr uint32_t SMEM = OFF_OUT + kEpilogueWarps * OUT_WARP + 1024;  // + alignment slack
    static_assert(SMEM <= 232448 && OFF_OUT % 1024 == 0, "layout");
};

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
}

// K-major 128B-swizzled operand: 16-byte core-matrix rows, 1024-byte groups of 8 rows
__device__ __forceinline__ uint64_t operand(uint32_t addr) { return sdesc(addr, 16, 1024); }

// instruction descriptor: e4m3 A and B (format 0), fp32 accumulator
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct Waits {
    int *status;
    unsigned long long ns;
};

// Lanes x 32 columns of an accumulator; the values may be used after ld_wait, which takes them as
// operands so that no use moves in front of it.
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

// acc += c s for the 32 values, two at a time
__device__ __forceinline__ void add_scaled(float2 *acc, const uint32_t (&r)[32], float s)
{
    const float2 s2 = make_float2(s, s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 c = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        acc[i] = io::fma2(c, s2, acc[i]);
    }
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

// The float4 at a shared-memory address of another CTA of the cluster
__device__ __forceinline__ float4 remote_float4(uint32_t addr, int cta)
{
    uint32_t a;
    float4 x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
    return x;
}

// Few tiles: the CTAs of a cluster share a tile and split its blocks of 128 (SPLIT).  Their sums meet in shared
// memory, where the operands were, and each CTA adds a share of the rows, always in the cluster's order.
template <typename out_t, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_out, const Params<out_t> p, const Waits wt, int tiled_out, int splits)
{
    using L = Layout<BN>;
    constexpr int STAGES = L::STAGES, HALF = BN / 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint32_t tmem_base_s;
    __shared__ __align__(8) uint64_t full[STAGES], freed[STAGES], acc_full[2], acc_empty[2];
    __shared__ int abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    const long long tiles = (long long)tiles_m * tiles_n;
    const int my_tiles = SPLIT ? 1 : tiles > blockIdx.x ? (int)((tiles - 1 - blockIdx.x) / gridDim.x) + 1 : 0;
    const int rank = SPLIT ? (int)(blockIdx.x % splits) : 0;
    const int b_from = SPLIT ? rank * p.KB / splits : 0, b_to = SPLIT ? (rank + 1) * p.KB / splits : p.KB;
    const long long total = (long long)my_tiles * (b_to - b_from);
    const uint32_t sbase = smem_u32(sm);

    // tiles of one column of tiles run at the same time on neighbouring CTAs and share w8 in L2
    auto tile_at = [&](int i, int &m0, int &n0) {
        const long long t = SPLIT ? (long long)(blockIdx.x / splits) : (long long)blockIdx.x + (long long)i * gridDim.x;
        m0 = (int)(t % tiles_m) * BM;
        n0 = (int)(t / tiles_m) * BN;
    };
    auto load_block = [&](int s, int b, int m0, int n0) {
        const uint32_t mb = smem_u32(&full[s]), at = sbase + s * L::STAGE;
        mbar_expect_tx(mb, L::STAGE);
        tma_load_2d(at, &tm_a, mb, b * kBlock, m0);
#pragma unroll
        for (int h = 0; h < BN / STAGE_ROWS; ++h)
            tma_load_2d(at + L::A_BYTES + h * STAGE_ROWS * kBlock, &tm_w, mb, b * kBlock, n0 + h * STAGE_ROWS);
    };
    // The narrow tiles' first blocks are on their way while the tensor memory is allocated (128 x 4096 x 4096: 11.65 us
    // without, 11.3 with); in the wide ones the registers are better used otherwise (4096 x 50048 x 768: 172 and 192 us).
    constexpr bool EARLY = BN == 128;
    const int early = EARLY && my_tiles > 0 ? min(STAGES, b_to - b_from) : 0;
    if (tid == 32) {
        abort_s = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&freed[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&acc_full[s]), 1);
            mbar_init(smem_u32(&acc_empty[s]), kEpilogueWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        if constexpr (EARLY) {
            int m0, n0;
            tile_at(0, m0, n0);
            for (int s = 0; s < early; ++s) load_block(s, b_from + s, m0, n0);
        } else {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_w);
        }
        if (tiled_out) prefetch_tmap(&tm_out);
    }
    if (warp == 0) tmem_alloc(smem_u32(&tmem_base_s), 2 * BN);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tmem_base_s;

    auto give_up = [&] {
        atomicCAS(wt.status, 0, kDevTimeout);
        *(volatile int *)&abort_s = 1;
    };
    long long issued = 0;  // the issuing threads' counts of steps, for the drain
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (tid == 32) {  // ---- operand loads ----
        int s = early % STAGES, i = EARLY && b_from + early == b_to ? 1 : 0, b = i > 0 ? b_from : b_from + early, m0 = 0, n0 = 0;
        uint32_t round = early / STAGES;
        issued = early;
        if (EARLY) tile_at(0, m0, n0);
        for (long long g = early; g < total; ++g) {
            if (b == b_from) tile_at(i, m0, n0);
            if (round > 0 && !mbar_wait(smem_u32(&freed[s]), (round - 1) & 1, wt.ns)) {
                give_up();
                break;
            }
            if (*(volatile int *)&abort_s) break;
            load_block(s, b, m0, n0);
            issued = g + 1;
            if (++s == STAGES) s = 0, ++round;
            if (++b == b_to) b = b_from, ++i;
        }
    } else if (tid == 0) {  // ---- products ----
        int s = 0;
        uint32_t round = 0;
        for (long long g = 0; g < total; ++g) {
            const int buf = (int)(g & 1);
            bool ok = g < 2 || mbar_wait(smem_u32(&acc_empty[buf]), (uint32_t)((g - 2) >> 1) & 1, wt.ns);
            ok = ok && mbar_wait(smem_u32(&full[s]), round & 1, wt.ns);
            if (!ok) {
                give_up();
                break;
            }
            if (*(volatile int *)&abort_s) break;
            fence_after_sync();
            const uint64_t da = operand(sbase + s * L::STAGE), db = operand(sbase + s * L::STAGE + L::A_BYTES);
#pragma unroll
            for (int j = 0; j < kBlock / 32; ++j)
                mma_f8(tmem + buf * BN, da + 2 * j, db + 2 * j, idesc_e4m3(BM, BN), j > 0);
            mma_commit(smem_u32(&freed[s]));
            mma_commit(smem_u32(&acc_full[buf]));
            issued = g + 1;
            if (++s == STAGES) s = 0, ++round;
        }
    }
    } else {  // ---- scaled sums: lane quarter warp % 4, columns of half (warp - 4) / 4 ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t from = ((uint32_t)(quarter * 32) << 16) + half * HALF;
        uint8_t *stage = sm + L::OFF_OUT + (warp - 4) * L::OUT_WARP;
        const uint32_t stage_u32 = smem_u32(stage);
        long long g = 0;
        bool ok = true;
        for (int i = 0; i < my_tiles && ok; ++i) {
            int m0, n0;
            tile_at(i, m0, n0);
            n0 += half * HALF;
            const int m = m0 + quarter * 32 + lane;
            const float *sa = p.a_scale + (size_t)min(m, p.M - 1) * p.KB;
            const float *sw = p.w_scale + (size_t)(min(n0, p.N - 1) / kBlock) * p.KB;
            float2 acc[HALF / 2];
#pragma unroll
            for (int c = 0; c < HALF / 2; ++c) acc[c] = make_float2(0.f, 0.f);
            float scale = sa[b_from] * sw[b_from];
            for (int b = b_from; b < b_to; ++b, ++g) {
                const int buf = (int)(g & 1);
                const float next = b + 1 < b_to ? sa[b + 1] * sw[b + 1] : 0.f;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[buf]), (uint32_t)(g >> 1) & 1, wt.ns));
                if (!ok) break;
                fence_after_sync();
                const uint32_t at = tmem + buf * BN + from;
                uint32_t r[2][32];
                ld_issue(at, r[0]);
#pragma unroll
                for (int ch = 0; ch < HALF / 32; ++ch) {  // the next columns load while these are added
                    ld_wait(r[ch & 1]);
                    if (ch + 1 < HALF / 32) ld_issue(at + 32 * (ch + 1), r[(ch + 1) & 1]);
                    if (ch + 1 == HALF / 32) {
                        fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
                    }
                    add_scaled(acc + 16 * ch, r[ch & 1], scale);
                }
                scale = next;
            }
            if (!ok) {
                if (lane == 0) give_up();  // products may still be in flight: the drain below waits for them
                break;
            }
            if constexpr (SPLIT) {  // every load has landed and every product has read it: their shared memory is free
                const int row = quarter * 32 + lane;
#pragma unroll
                for (int c = 0; c < HALF / 4; ++c)
                    *reinterpret_cast<float4 *>(sm + row * BN * 4 + (((half * HALF / 4 + c) ^ (row & 7)) << 4)) =
                        make_float4(acc[2 * c].x, acc[2 * c].y, acc[2 * c + 1].x, acc[2 * c + 1].y);
            } else if (tiled_out) {
                // The sums go to shared memory and leave by TMA while the next tile is added up: a piece is 32 rows x
                // 128 bytes, and the staging holds two, all of the warp's bf16 columns.
                constexpr int COLS = 128 / (int)sizeof(out_t), PER = 16 / (int)sizeof(out_t);
#pragma unroll
                for (int c0 = 0; c0 < HALF; c0 += COLS) {
                    const int piece = c0 / COLS & 1;
                    if (piece == 0) bulk_wait_read();  // the pieces before have left the staging (lane 0's own copies)
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        float f[PER];
#pragma unroll
                        for (int e = 0; e < PER; e += 2)
                            f[e] = acc[(c0 + PER * u + e) / 2].x, f[e + 1] = acc[(c0 + PER * u + e) / 2].y;
                        io::Unit<out_t, PER> x;
                        x.set(f);
                        *reinterpret_cast<uint4 *>(stage + piece * L::PIECE + lane * 128 + ((u ^ (lane & 7)) << 4)) = x.w;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && m0 + quarter * 32 < p.M && n0 + c0 < p.N) {
                        tma_store_2d(&tm_out, stage_u32 + piece * L::PIECE, n0 + c0, m0 + quarter * 32);
                        bulk_commit();
                    }
                }
            } else {
                // Rows that are not aligned: 32 x 32 sums at a time, transposed through shared memory; eight rows' loads before
                // their stores (1003 x 4626 x 1040: 13.6 us, with a plain loop over the rows 15.5, 16 rows 13.8; whole lines of 128 bytes
                // in place of the tile's columns take 16.6).
                float *t = reinterpret_cast<float *>(stage);
#pragma unroll
                for (int q = 0; q < HALF; q += 32) {
                    if (n0 + q >= p.N) break;
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 32; ++c) t[lane * 32 + (c ^ lane)] = c & 1 ? acc[(q + c) / 2].y : acc[(q + c) / 2].x;
                    __syncwarp();
                    const int n = n0 + q + lane, rows = min(32, p.M - m0 - quarter * 32);
                    out_t *to = p.out + (size_t)(m0 + quarter * 32) * p.N + n;
                    if (n < p.N) {
                        if (rows == 32) {
#pragma unroll
                            for (int r0 = 0; r0 < 32; r0 += 8) {
                                float f[8];
#pragma unroll
                                for (int r = 0; r < 8; ++r) f[r] = t[(r0 + r) * 32 + (lane ^ (r0 + r))];
#pragma unroll
                                for (int r = 0; r < 8; ++r, to += p.N) io::st(to, f[r]);
                            }
                        } else {
                            for (int r = 0; r < rows; ++r, to += p.N) io::st(to, t[r * 32 + (lane ^ r)]);
                        }
                    }
                }
            }
        }
        if (!SPLIT && tiled_out) bulk_wait_read();  // before the staging goes
    }
    // drain: after an expired wait, the copies and products in flight land before the CTA exits
    __syncthreads();
    if (abort_s && issued > 0) {
        const long long last = issued - 1;
        if (tid == 0)  // products complete in order
            (void)mbar_wait(smem_u32(&freed[last % STAGES]), (uint32_t)(last / STAGES) & 1, 1000000000ull);
        if (tid == 32)
            for (long long g = last >= STAGES ? last - STAGES + 1 : 0; g <= last; ++g)
                (void)mbar_wait(smem_u32(&full[g % STAGES]), (uint32_t)(g / STAGES) & 1, 1000000000ull);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 2 * BN);
    if constexpr (SPLIT) {
        static_assert(BN == 128 && (uint32_t)BM * BN * 4 <= L::OFF_OUT, "a row of sums is one float4 per lane");
        cluster_barrier();
        int m0, n0;
        tile_at(0, m0, n0);
        const int n = n0 + 4 * lane, each = BM / splits, rows = min(each, p.M - m0 - rank * each);
        for (int r = warp; r < rows; r += kThreads / 32) {
            const int row = rank * each + r;
            const uint32_t at = sbase + row * BN * 4 + ((lane ^ (row & 7)) << 4);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < splits; ++c) {
                const float4 x = remote_float4(at, c);
                sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
            }
            out_t *to = p.out + (size_t)(m0 + row) * p.N + n;
            if (tiled_out && n + 4 <= p.N) {
                if constexpr (sizeof(out_t) == 4) {
                    *reinterpret_cast<float4 *>(to) = sum;
                } else {
                    using U = io::Unit<out_t, 8>;
                    *reinterpret_cast<uint2 *>(to) = make_uint2(U::pack(sum.x, sum.y), U::pack(sum.z, sum.w));
                }
            } else {
                const float f[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) io::st(to + e, f[e]);
            }
        }
        cluster_barrier();  // the others may still read this CTA's sums
    }
}

// A row-major matrix as boxes of box_rows rows x 128 bytes, 128-byte swizzled in shared memory
bool encode(CUtensorMap *map, CUtensorMapDataType type, int size, const void *base, int cols, int rows, int box_rows)
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
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows}, steps[2] = {1, 1};
    return fn && fn(map, type, 2, const_cast<void *>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename out_t, int BN, bool SPLIT>
cudaError_t launch_product(const Params<out_t> &p, const TokenLaunch &l, int splits)
{
    CUtensorMap ma, mw, mo;
    if (!encode(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.a, p.K, p.M, BM) ||
        !encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.w, p.K, p.N, STAGE_ROWS))
        return cudaErrorInvalidValue;
    const bool tiled = (long long)p.N * sizeof(out_t) % 16 == 0;  // TMA takes rows whose stride is a multiple of 16 bytes
    if (!tiled)
        mo = ma;  // not used
    else if (!encode(&mo, sizeof(out_t) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, sizeof(out_t), p.out,
                     p.N, p.M, 32))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
    const Waits wt{l.d_status, l.wait_ns > 0 ? (unsigned long long)l.wait_ns : 100000000ull};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * splits : tiles < l.sm_count ? tiles : l.sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<BN>::SMEM;
    cfg.stream = l.timer->stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = SPLIT ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, product_kernel<out_t, BN, SPLIT>, ma, mw, mo, p, wt, tiled ? 1 : 0, splits);
}

// ---------------------------------------------------------------------------------------------
// A CTA lays out 128 rows of one block of 128 columns, which it holds in registers between the search for their
// largest magnitude and the division (50048 x 768 bf16: 35 us, 3.3 TB/s; one value at a time, read twice, 68 us).  K is a multiple of 16, so
// rows are made of whole units.
template <typename io_t>
__global__ void __launch_bounds__(256) weights_kernel(const io_t *__restrict__ W, uint8_t *__restrict__ w8,
                                                     float *__restrict__ w_scale, int N, int K, int KB)
{
    constexpr int VEC = 16 / (int)sizeof(io_t), PER_ROW = kBlock / VEC, ROWS = 256 / PER_ROW, STEPS = kBlock / ROWS;
    __shared__ float peaks[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n0 = blockIdx.x * kBlock + tid / PER_ROW, k = blockIdx.y * kBlock + tid % PER_ROW * VEC;
    io::Unit<io_t, VEC> x[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int n = n0 + i * ROWS;
        x[i].w = make_uint4(0, 0, 0, 0);
        if (n < N && k < K) x[i] = io::load_unit<io_t, VEC>(W + (size_t)n * K + k);
    }
    float peak = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        float f[VEC];
        x[i].get(f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) peak = fmaxf(peak, fabsf(f[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
    if (lane == 0) peaks[warp] = peak;
    __syncthreads();
    for (int w = 0; w < 8; ++w) peak = fmaxf(peak, peaks[w]);
    const float scale = fmaxf(peak / kMaxE4M3, kMinScale);
    if (tid == 0) w_scale[(size_t)blockIdx.x * KB + blockIdx.y] = scale;
    // The quotient by way of the reciprocal, corrected once by its remainder with fused operations (P. W. Markstein,
    // "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990), which gives
    // the values of a division; a division per value takes 39 us.
    // Beside the range in which reciprocal and remainder are exact enough (and for infinite scales) it is divided.
    const bool near = scale >= 1e-30f && scale <= 1e30f;
    const float inverse = 1.f / scale;
    auto quotient = [&](float v) {
        if (!near) return v / scale;
        const float q = v * inverse;
        return fmaf(fmaf(-q, scale, v), inverse, q);
    };
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int n = n0 + i * ROWS;
        if (n >= N || k >= K) continue;
        float f[VEC];
        x[i].get(f);
        uint32_t out[VEC / 4];
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(quotient(f[e + 1])), "f"(quotient(f[e])));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(quotient(f[e + 3])), "f"(quotient(f[e + 2])));
            out[e / 4] = lo | (uint32_t)hi << 16;
        }
        uint8_t *to = w8 + (size_t)n * K + k;
        if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(out[0], out[1]);
        else *reinterpret_cast<uint32_t *>(to) = out[0];
    }
}

template <typename out_t>
cudaError_t product(const Matmul8Args &a, const TokenLaunch &l)
{
    const Params<out_t> p{(const uint8_t *)a.a8, (const uint8_t *)a.w8, a.a_scale, a.w_scale, (out_t *)a.out, a.M, a.N, a.K,
                          (a.K + kBlock - 1) / kBlock};
    cudaError_t e;
    l.timer->begin("matmul8");
    // Few rows, among calls of a graph: 16 of N x K = 50048 x 768 take 14.9 us here and 17 13.9 in tiles, of 8192 x 8192
    // 20.1 and 20.1, of 4096 x 4096 7.8 and 10.7; 8 take 10.0, 14.9 and 6.4.  With four operands of 8 rows the loads wait
    // for registers (32 rows of 50048 x 768 22.8 by single calls, in tiles 16.3).
    if (a.M <= 16) {
        if (a.M <= 8) launch_skinny<out_t, 1>(p, l.sm_count, l.timer->stream);
        else launch_skinny<out_t, 2>(p, l.sm_count, l.timer->stream);
        e = cudaGetLastError();
    } else {
        // The width of tiles that takes less time: turns of the SMs times the rows that a block brings in.
        const long long rows = (a.M + BM - 1) / BM;
        auto time = [&](long long bn) { return (rows * ((a.N + bn - 1) / bn) + l.sm_count - 1) / l.sm_count * (bn + BM); };
        // Few tiles: the CTAs of a cluster split the blocks of 128, as many as the machine holds at once.  Meeting costs
        // about 2 us and a block about 0.4, so there have to be some: 64 x 6144 x 1024 (8 blocks) takes 8.5 us
        // whole and 10.6 split, 17 x 768 x 2304 (18) 12.4 and 10.0, 128 x 4096 x 4096 (32) 18.7 and 12.5,
        // 64 x 8192 x 8192 31.3 and 23.1, 64 x 1024 x 16384 55.7 and 14.6.
        const long long tiles = rows * ((a.N + 127) / 128);
        int splits = 1;
        while (p.KB >= 12 && splits < 8 && 2 * splits <= p.KB && tiles * 2 * splits <= l.sm_count) splits *= 2;
        e = splits > 1 ? launch_product<out_t, 128, true>(p, l, splits)
            : time(256) <= time(128) ? launch_product<out_t, 256, false>(p, l, 1) : launch_product<out_t, 128, false>(p, l, 1);
    }
    l.timer->end();
    return e;
}

template <typename out_t, int BN, bool SPLIT>
cudaError_t prepare()
{
    return cudaFuncSetAttribute(product_kernel<out_t, BN, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<BN>::SMEM);
}

}  // namespace mm8

cudaError_t matmul8_prepare()
{
    cudaError_t e = mm8::prepare<float, 128, false>();
    if (e == cudaSuccess) e = mm8::prepare<float, 128, true>();
    if (e == cudaSuccess) e = mm8::prepare<float, 256, false>();
    if (e == cudaSuccess) e = mm8::prepare<__nv_bfloat16, 128, false>();
    if (e == cudaSuccess) e = mm8::prepare<__nv_bfloat16, 128, true>();
    if (e == cudaSuccess) e = mm8::prepare<__nv_bfloat16, 256, false>();
    return e;
}

cudaError_t matmul8(prism_dtype out, const Matmul8Args &a, const TokenLaunch &l)
{
    return out == PRISM_BF16 ? mm8::product<__nv_bfloat16>(a, l) : mm8::product<float>(a, l);
}

cudaError_t matmul8_weights(prism_dtype io, int N, int K, const void *W, void *w8, float *w_scale, const TokenLaunch &l)
{
    const int KB = (K + mm8::kBlock - 1) / mm8::kBlock, NB = (N + mm8::kBlock - 1) / mm8::kBlock;
    l.timer->begin("matmul8_weights");
    if (io == PRISM_BF16)
        mm8::weights_kernel<__nv_bfloat16><<<dim3(NB, KB), 256, 0, l.timer->stream>>>((const __nv_bfloat16 *)W, (uint8_t *)w8, w_scale, N, K, KB);
    else
        mm8::weights_kernel<float><<<dim3(NB, KB), 256, 0, l.timer->stream>>>((const float *)W, (uint8_t *)w8, w_scale, N, K, KB);
    l.timer->end();
    return cudaGetLastError();
}

}  // namespace prism
