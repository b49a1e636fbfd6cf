// Drawing a token: the kernels for bfloat16 logits (prism_sample.h) and the entry.
#include "prism_sample.h"

namespace prism {
namespace draw {

cudaError_t prepare_float();
cudaError_t run_float(const SampleArgs &a, const TokenLaunch &l);

}  // namespace draw

cudaError_t sample_prepare()
{
    const cudaError_t e = draw::prepare_float();
    return e == cudaSuccess ? draw::prepare<__nv_bfloat16>() : e;
}

cudaError_t sample(prism_dtype logits, const SampleArgs &a, const TokenLaunch &l)
{
    return logits == PRISM_BF16 ? draw::run<__nv_bfloat16>(a, l) : draw::run_float(a, l);
}

}  // namespace prism
