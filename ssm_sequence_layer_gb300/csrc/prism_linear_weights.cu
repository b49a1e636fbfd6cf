// The tile kernels of dW = dy^T x and the sums over dy's rows (prism_linear.h).
#include "prism_linear.h"

#include <mutex>

namespace prism {
namespace lin {

template <>
cudaError_t weights_tiles<__nv_bfloat16>(const Params<__nv_bfloat16> &p, const Cut &c, const TokenLaunch &l)
{
    if (c.soft) return launch_tiles<__nv_bfloat16, LinearOp::weights, true, 128, true, false>(p, c.splits, l);
    if (c.pair)
        return c.bn == 256 ? launch_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, true>(p, c.splits, l)
                           : launch_tiles<__nv_bfloat16, LinearOp::weights, false, 192, true, true>(p, c.splits, l);
    return c.bn == 256 ? launch_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, false>(p, c.splits, l)
                       : launch_tiles<__nv_bfloat16, LinearOp::weights, false, 128, true, false>(p, c.splits, l);
}

template <>
cudaError_t weights_tiles<float>(const Params<float> &p, const Cut &c, const TokenLaunch &l)
{
    return launch_tiles<float, LinearOp::weights, true, 128, true, false>(p, c.splits, l);
}

namespace {
// The same on every device that the library runs on.  Written once, under the lock that every plan passes before its handle is used
int at_once[9];
std::mutex at_once_lock;
}  // namespace

int clusters_at_once(int ctas) { return at_once[ctas]; }

cudaError_t weights_prepare()
{
    cudaError_t e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, true>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 192, true, true>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 256, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, false, 128, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<__nv_bfloat16, LinearOp::weights, true, 128, true, false>();
    if (e == cudaSuccess) e = prepare_tiles<float, LinearOp::weights, true, 128, true, false>();
    using L = Layout<__nv_bfloat16, LinearOp::weights, false, 256, false>;
    const std::lock_guard<std::mutex> hold(at_once_lock);
    if (at_once[8] != 0) return e;
    int counts[9] = {};
    for (int ctas = 1; ctas <= 8 && e == cudaSuccess; ++ctas) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas), cfg.blockDim = dim3(L::THREADS), cfg.dynamicSmemBytes = L::SMEM;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = ctas, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at, cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, tile_kernel<__nv_bfloat16, LinearOp::weights, false, 256, true, false>, &cfg);
        counts[ctas] = n > 0 ? n : 1;
    }
    if (e == cudaSuccess) memcpy(at_once, counts, sizeof(at_once));
    return e;
}

}  // namespace lin
}  // namespace prism
