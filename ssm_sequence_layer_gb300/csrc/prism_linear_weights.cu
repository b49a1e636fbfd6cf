// The tile kernels of dW = dy^T x and the sums over dy's rows (prism_linear.h).
#include "prism_linear.h"

namespace prism {
namespace lin {

template <>
cudaError_t weights_tiles<__nv_bfloat16>(const Params<__nv_bfloat16> &p, const Cut &c, const TokenLaunch &l)
{
    if (c.soft) return launch_tiles<__nv_bfloat16, LinearOp::weights, true, 128, true, false>(p, c.splits, l);
    if (c.pair) return launch_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, true>(p, c.splits, l);
    return c.bn == 256 ? launch_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, false>(p, c.splits, l)
                       : launch_tiles<__nv_bfloat16, LinearOp::weights, false, 128, true, false>(p, c.splits, l);
}

template <>
cudaError_t weights_tiles<float>(const Params<float> &p, const Cut &c, const TokenLaunch &l)
{
    return launch_tiles<float, LinearOp::weights, true, 128, true, false>(p, c.splits, l);
}

cudaError_t weights_prepare()
{
    cudaError_t e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, true>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 128, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, true, 128, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<float, LinearOp::weights, true, 128, true, false>();
    return e;
}

}  // namespace lin
}  // namespace prism
