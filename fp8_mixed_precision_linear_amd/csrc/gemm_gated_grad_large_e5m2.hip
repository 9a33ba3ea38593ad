// gemm_gated_grad_large_e5m2.hip -- gemm_gated_large.h, backward, E5M2 gradients.
#include "gemm_gated_large.h"

namespace fp8lin {

hipError_t launch_gated_grad_large_e5m2(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  return p.d_fp8 ? launch_gated_grad_as<1, true>(p, e, s) : launch_gated_grad_as<1, false>(p, e, s);
}

}  // namespace fp8lin
