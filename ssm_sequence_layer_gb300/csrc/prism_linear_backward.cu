// The tile kernels of dx = (dy W) act'(pre) + dsum (prism_linear.h).
#include "prism_linear.h"

namespace prism {
namespace lin {

template <>
cudaError_t backward_tiles<__nv_bfloat16>(const Params<__nv_bfloat16> &p, const Cut &c, const TokenLaunch &l)
{
    if (c.soft)
        return c.split ? launch_tiles<__nv_bfloat16, LinearOp::backward, true, 128, true, false>(p, c.splits, l)
                       : launch_tiles<__nv_bfloat16, LinearOp::backward, true, 128, false, false>(p, 1, l);
    if (c.split) return launch_tiles<__nv_bfloat16, LinearOp::backward, false, 128, true, false>(p, c.splits, l);
    if (c.pair) return launch_tiles<__nv_bfloat16, LinearOp::backward, false, 256, false, true>(p, 1, l);
    return c.bn == 256 ? launch_tiles<__nv_bfloat16, LinearOp::backward, false, 256, false, false>(p, 1, l)
                       : launch_tiles<__nv_bfloat16, LinearOp::backward, false, 128, false, false>(p, 1, l);
}

template <>
cudaError_t backward_tiles<float>(const Params<float> &p, const Cut &c, const TokenLaunch &l)
{
    return c.split ? launch_tiles<float, LinearOp::backward, true, 128, true, false>(p, c.splits, l)
                   : launch_tiles<float, LinearOp::backward, true, 128, false, false>(p, 1, l);
}

cudaError_t backward_prepare()
{
    cudaError_t e = prepare_tiles<__nv_bfloat16, LinearOp::backward, false, 256, false, true>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::backward, false, 256, false, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::backward, false, 128, false, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::backward, false, 128, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::backward, true, 128, false, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::backward, true, 128, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<float, LinearOp::backward, true, 128, false, false>();
    if (e == cudaSuccess) e = prepare_tiles<float, LinearOp::backward, true, 128, true, false>();
    return e;
}

}  // namespace lin
}  // namespace prism
