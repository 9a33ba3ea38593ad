// gemm_gated_grad_large.hip -- gemm_gated_large.h, backward, E4M3 gradients.
#include "gemm_gated_large.h"

namespace fp8lin {

hipError_t launch_gated_grad_large(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  return p.d_fp8 ? launch_gated_grad_as<0, true>(p, e, s) : launch_gated_grad_as<0, false>(p, e, s);
}

}  // namespace fp8lin
