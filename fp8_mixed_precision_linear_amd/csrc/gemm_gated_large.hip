// gemm_gated_large.hip -- gemm_gated_large.h, forward.
#include "gemm_gated_large.h"

namespace fp8lin {

hipError_t launch_gated_large(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  return p.d_fp8 ? launch_gated_large_as<0, true, GatedEp, GatedStripEp>(p, e, s) : launch_gated_large_as<0, false, GatedEp, GatedStripEp>(p, e, s);
}

}  // namespace fp8lin
