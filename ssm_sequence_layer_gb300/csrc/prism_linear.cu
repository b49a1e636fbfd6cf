// Matrix product with bias, activation and residual in its epilogue, and its gradients: how a call is cut, and the product of
// few rows.
//
//   forward   pre = x W^T + bias,  y = act(pre) + residual
//   backward  dx = (dy W) act'(pre) + dsum
//   weights   dW (+)= dy^T x,  dbias (+)= sum over rows of dy
#include "prism_linear.h"

namespace prism {
namespace lin {

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
        consider(false, 128, sizeof(io_t) == 4 ? 3000 : c.soft ? 1500 : 540);
        // the sums over rows need tensor memory beside the accumulators, which tiles of 256 columns leave none of
        if (!c.soft) consider(true, 192, 430);
        if (!c.soft && !p.dbias) consider(false, 256, 800), consider(true, 256, 560);
    } else {
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
