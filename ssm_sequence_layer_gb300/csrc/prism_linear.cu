// Matrix product with bias, activation and residual in its epilogue, and its gradients: how a call is cut, and the product of
// few rows.
//
//   forward   pre = x W^T + bias,  y = act(pre) + residual
//   backward  dx = (dy W) act'(pre) + dsum
//   weights   dW (+)= dy^T x,  dbias (+)= sum over rows of dy
#include "prism_linear.h"

namespace prism {
namespace lin {

// ---- few rows ---------------------------------------------------------------------------------------------
// Few rows of bf16, as a served token of each of some sequences has them: the weights' bytes bound the product, each weight
// is used M times at most, and tiles of 128 rows would be empty for the most part.  (16 x 2304 x 768: 3.2 us, 1.1 TB/s of weights from a
// graph's launch to the next one's; 16 x 8192 x 8192: 24, 5.5 TB/s.)  A warp takes RPW tiles of 16 rows of W as A operands
// of m16n8k16 products straight from global memory to registers (16 bytes of a row per lane and load), and 8 NT rows of x as B
// operands.  The products' k order is a free choice as long as both operands share it: the four words of a lane's 16 bytes serve as
// the k slots of two products.  KS warps of a CTA share their tiles and split the sum, so that narrow products still fill the
// machine; their sums are added in a fixed order.
constexpr int kFewWarps = 8, kFewBlock = 64;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT, int KS, int RPW>
__global__ void __launch_bounds__(32 * kFewWarps) few_kernel(const Params<__nv_bfloat16> p)
{
    constexpr int RT = kFewWarps / KS;  // warps of a CTA with rows of their own
    constexpr int AHEAD = 2;            // blocks of 64 in flight
    __shared__ float parts[KS > 1 ? kFewWarps : 1][16 * RPW][8 * NT + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int ks = warp % KS, n0 = (blockIdx.x * RT + warp / KS) * 16 * RPW, blocks = (p.K + kFewBlock - 1) / kFewBlock;
    float c[RPW][NT][4] = {};
    if (n0 < p.J) {
        // rows beyond the operands' last are read as the last and not stored
        const __nv_bfloat16 *wr[2 * RPW], *xr[NT];
#pragma unroll
        for (int r = 0; r < 2 * RPW; ++r) wr[r] = p.b + (size_t)min(n0 + g + 8 * r, p.J - 1) * p.K;
#pragma unroll
        for (int t = 0; t < NT; ++t) xr[t] = p.a + (size_t)min(8 * t + g, p.I - 1) * p.K;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        uint4 w[AHEAD][2 * RPW][2];
        auto load = [&](int slot, int b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = b * kFewBlock + h * 32 + q * 8;
#pragma unroll
                for (int r = 0; r < 2 * RPW; ++r) w[slot][r][h] = k < p.K ? __ldcs(reinterpret_cast<const uint4 *>(wr[r] + k)) : zero;
            }
        };
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) load(s, ks + s * KS);
        for (int b0 = ks; b0 < blocks; b0 += AHEAD * KS) {
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) {
                const int b = b0 + s * KS;
                if (b >= blocks) break;
                uint4 x[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = b * kFewBlock + h * 32 + q * 8;
                        x[t][h] = k < p.K ? __ldg(reinterpret_cast<const uint4 *>(xr[t] + k)) : zero;
                    }
#pragma unroll
                for (int r = 0; r < RPW; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 lo = w[s][2 * r][h], hi = w[s][2 * r + 1][h];
                            mma_bf16(c[r][t], lo.x, hi.x, lo.y, hi.y, x[t][h].x, x[t][h].y);
                            mma_bf16(c[r][t], lo.z, hi.z, lo.w, hi.w, x[t][h].z, x[t][h].w);
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
                for (int i = 0; i < 4; ++i) parts[warp][16 * r + g + 8 * (i >> 1)][8 * t + 2 * q + (i & 1)] = c[r][t][i];
        __syncthreads();
    }
    // A warp finishes the rows of W that it took (with KS warps a share of them each), a column of its tiles per lane and m: the
    // stores of neighbouring lanes are neighbours
    with_activation(p.act, [&](auto act) {
        constexpr prism_activation ACT = decltype(act)::value;
        auto finish = [&](int m, int n, float v) {
            if (m >= p.I || n >= p.J) return;
            const size_t at = (size_t)m * p.J + n;
            if (p.bias) v += io::ld(p.bias + n);
            if (p.pre_out) io::st(p.pre_out + at, v);
            v = act_value<ACT>(v);
            if (p.add) v += io::ld(p.add + at);
            io::st((__nv_bfloat16 *)p.out + at, v);
        };
        if constexpr (KS > 1) {
            for (int e = ks * 32 + lane; e < 16 * RPW * 8 * NT; e += 32 * KS) {
                const int n = e % (16 * RPW), m = e / (16 * RPW);
                float v = 0.f;
#pragma unroll
                for (int o = 0; o < KS; ++o) v += parts[warp - ks + o][n][m];
                finish(m, n0 + n, v);
            }
        } else {
#pragma unroll
            for (int r = 0; r < RPW; ++r)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) finish(8 * t + 2 * q + (i & 1), n0 + 16 * r + g + 8 * (i >> 1), c[r][t][i]);
        }
    });
}

bool few_weights(int J, const TokenLaunch &l) { return (J + 31) / 32 * 8LL < 12 * l.sm_count; }

template <int NT>
cudaError_t launch_few(const Params<__nv_bfloat16> &p, const TokenLaunch &l)
{
    constexpr int T = 32 * kFewWarps;
    const int blocks = (p.K + kFewBlock - 1) / kFewBlock, pairs = (p.J + 31) / 32;
    cudaStream_t s = l.timer->stream;
    if (NT > 2 || few_weights(p.J, l)) {  // all warps of a CTA on one tile
        few_kernel<NT, 8, 1><<<(p.J + 15) / 16, T, 0, s>>>(p);
        return cudaGetLastError();
    }
    if constexpr (NT <= 2) {
        // as many warps as keep each SM's loads in flight, as far as the blocks of 64 reach
        int ks = 1;
        while (ks < 8 && ks < blocks && (long long)pairs * ks < 8 * l.sm_count) ks *= 2;
        const unsigned grid = (unsigned)((pairs + kFewWarps / ks - 1) / (kFewWarps / ks));
        if (ks == 1) few_kernel<NT, 1, 2><<<grid, T, 0, s>>>(p);
        else if (ks == 2) few_kernel<NT, 2, 2><<<grid, T, 0, s>>>(p);
        else if (ks == 4) few_kernel<NT, 4, 2><<<grid, T, 0, s>>>(p);
        else few_kernel<NT, 8, 2><<<grid, T, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// Whether M rows are few: up to 16 always (17 rows of 2304 x 768 in tiles: 6.8 us, 16 here 3.2).  More rows only where the weights are small, since
// each CTA reads all rows again.  Microseconds here / in tiles: 32 rows of 2304 x 768 3.4 / 7.4, of 3584 x 2048 7.5 / 8.6, of 768 x 8192 10.3 / 10.5,
// of 4096 x 4096 13.6 / 10.9; 64 rows of 2304 x 768 4.7 / 7.2, of 2048 x 2048 6.2 / 8.5, of 768 x 2304 6.9 / 7.9, of 7168 x 768 10.4 / 8.8,
// of 768 x 8192 14.9 / 10.9.
bool few_rows(const Params<__nv_bfloat16> &p, const TokenLaunch &l)
{
    if (p.K % 8 != 0) return false;
    const long long weights = (long long)p.J * p.K;
    return p.I <= 16 || (few_weights(p.J, l) && ((p.I <= 32 && weights <= 1 << 23 && p.K <= 8192) || (p.I <= 64 && weights <= 1 << 22 && p.K <= 2304)));
}

template <typename io_t>
cudaError_t run(const LinearArgs &a, const TokenLaunch &l)
{
    Params<io_t> p = {};
    p.a = (const io_t *)a.a, p.b = (const io_t *)a.b;
    p.act = a.act, p.bias = (const io_t *)a.bias, p.add = (const io_t *)a.add, p.out = a.out, p.pre_out = (io_t *)a.pre_out;
    p.pre_in = (const io_t *)a.pre_in, p.dbias = a.dbias, p.accumulate = a.accumulate;
    const bool weights = a.op == LinearOp::weights;
    const char *name = "linear";
    if (a.op == LinearOp::forward) {
        p.I = a.M, p.J = a.N, p.K = a.K, p.lda = a.K, p.ldb = a.K;
    } else if (a.op == LinearOp::backward) {
        name = "linear_backward";
        p.I = a.M, p.J = a.K, p.K = a.N, p.lda = a.N, p.ldb = a.K;
    } else {
        name = "linear_weights";
        p.I = a.N, p.J = a.K, p.K = a.M, p.lda = a.N, p.ldb = a.K;
    }
    if constexpr (sizeof(io_t) == 2) {
        if (a.op == LinearOp::forward && few_rows(p, l)) {
            l.timer->begin(name);
            const cudaError_t e = a.M <= 8 ? launch_few<1>(p, l) : a.M <= 16 ? launch_few<2>(p, l) : a.M <= 32 ? launch_few<4>(p, l) : launch_few<8>(p, l);
            l.timer->end();
            return e;
        }
    }
    Cut c = {};
    // TMA takes rows whose stride is a multiple of 16 bytes
    c.soft = sizeof(io_t) == 4 || p.lda % 8 != 0 || p.ldb % 8 != 0;
    const long long blocks = (p.K + BK - 1) / BK;
    auto tiles = [&](long long bm, long long bn) { return (p.I + bm - 1) / bm * ((p.J + bn - 1) / bn); };
    auto turns = [&](long long n, int ctas) { return (n + clusters_at_once(ctas) - 1) / clusters_at_once(ctas); };
    c.bn = 128, c.splits = 1;
    if (weights) {
        // The tile, and the CTAs or pairs that split its sum, of least cycles: turns of the clusters that run at once (clusters of six
        // leave 14 SMs without work, of eight 32) times a share of the blocks, at what a block costs, and about 7000 until the first
        // products and for the join.
        c.split = true;
        long long best = 0;
        auto consider = [&](bool pair, int bn, long long block) {
            const int ctas = pair ? 2 : 1;
            for (int s = 1; s * ctas <= 8 && s <= blocks; ++s) {
                const long long time = turns(tiles(ctas * BM, bn), s * ctas) * ((blocks + s - 1) / s * block + 7000);
                if (best == 0 || time < best) best = time, c.pair = pair, c.bn = bn, c.splits = s;
            }
        };
        consider(false, 128, sizeof(io_t) == 4 ? 4700 : c.soft ? 3600 : 540);
        // the sums over rows need tensor memory beside the accumulators, which tiles of 256 columns leave none of
        if (!c.soft) consider(true, 192, 430);
        if (!c.soft && !p.dbias) consider(false, 256, 800), consider(true, 256, 560);
    } else {
        // Few tiles split their sum over a cluster as long as all clusters run at once: 32 x 2304 x 768 backward 13.9 us in one piece, 8.6 in four, 7.3
        // in eight; 256 rows 14.2, 9.3, 9.0; of 1024 rows, which fit in two parts only, 14.3, 11.6 in two, 17.8 in four.  Below eight blocks it is a
        // draw (7.4 to 8.4).  Many tiles: of 256 columns where that takes no more turns for its width (4096 x 768 x 768: 10.0, of 128 11.7; 2048 rows
        // 9.8, of 128 8.1), in pairs of SMs where there are as many (8192 x 2304 x 768: 23.3, 26.0 by single SMs; 4096 rows 15.4 and 15.5; 2048 x 768 x 768
        // 10.6 and 9.8).
        while (c.splits < 8 && 2 * c.splits <= blocks && blocks >= 8 && tiles(BM, 128) <= clusters_at_once(2 * c.splits)) c.splits *= 2;
        c.split = c.splits > 1;
        c.pair = !c.split && !c.soft && tiles(256, 256) * 2 > l.sm_count;
        if (!c.split && !c.soft && turns(tiles(BM, 256), 1) * (256 + BM) <= turns(tiles(BM, 128), 1) * (128 + BM)) c.bn = 256;
    }
    l.timer->begin(name);
    const cudaError_t e = weights ? weights_tiles<io_t>(p, c, l) : a.op == LinearOp::forward ? forward_tiles<io_t>(p, c, l) : backward_tiles<io_t>(p, c, l);
    l.timer->end();
    return e;
}

}  // namespace lin

cudaError_t linear_prepare()
{
    cudaError_t e = lin::forward_prepare();
    if (e == cudaSuccess) e = lin::backward_prepare();
    if (e == cudaSuccess) e = lin::weights_prepare();
    return e;
}

cudaError_t linear(prism_dtype io, const LinearArgs &a, const TokenLaunch &l)
{
    return io == PRISM_BF16 ? lin::run<__nv_bfloat16>(a, l) : lin::run<float>(a, l);
}

}  // namespace prism
