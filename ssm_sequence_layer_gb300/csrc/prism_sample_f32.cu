// Drawing a token: the kernels for float32 logits (prism_sample.h).
#include "prism_sample.h"

namespace prism {
namespace draw {

cudaError_t prepare_float() { return prepare<float>(); }
cudaError_t run_float(const SampleArgs &a, const TokenLaunch &l) { return run<float>(a, l); }

}  // namespace draw
}  // namespace prism
