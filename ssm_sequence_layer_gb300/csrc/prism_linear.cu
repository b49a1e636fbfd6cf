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
    const long long rows = (p.I + BM - 1) / BM, blocks = (p.K + BK - 1) / BK;
    auto tiles = [&](long long bn) { return rows * ((p.J + bn - 1) / bn); };
    auto turns = [&](long long n) { return (n + l.sm_count - 1) / l.sm_count; };
    c.bn = 128, c.splits = 1;
    if (weights) {
        if (!c.soft && p.J > 128) c.bn = 256;
        long long best = 0;
        for (int s = 1; s <= 8 && s <= blocks; ++s) {
            const long long time = turns(tiles(c.bn) * s) * ((blocks + s - 1) / s + 12);
            if (s == 1 || time < best) best = time, c.splits = s;
        }
        c.split = true;
        // two CTAs a tile of 256 x 256: clusters of up to eight CTAs
        if (c.bn == 256 && p.I > BM) {
            c.pair = true, best = 0;
            const long long pairs = (p.I + 255) / 256 * ((p.J + 255) / 256);
            for (int s = 1; s <= 4 && s <= blocks; ++s) {
                const long long time = (pairs * s + l.sm_count / 2 - 1) / (l.sm_count / 2) * ((blocks + s - 1) / s + 12);
                if (s == 1 || time < best) best = time, c.splits = s;
            }
        }
    } else {
        while (c.splits < 8 && 2 * c.splits <= blocks && blocks >= 8 && tiles(128) * 2 * c.splits <= l.sm_count) c.splits *= 2;
        c.split = c.splits > 1;
        c.pair = !c.split && !c.soft && (p.I + 255) / 256 * ((p.J + 255) / 256) * 2 > l.sm_count;
        if (!c.split && !c.soft && turns(tiles(256)) * (256 + BM) <= turns(tiles(128)) * (128 + BM)) c.bn = 256;
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
