// gemm_gated_tile.hip -- gemm_gated_tile.h, forward, no promotion.
#include "gemm_gated_tile.h"

namespace fp8lin {

hipError_t launch_gated_tile(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s) {
  return p.d_fp8 ? launch_gated_sum<GatedOp, true>(p, e, plan, s) : launch_gated_sum<GatedOp, false>(p, e, plan, s);
}

}  // namespace fp8lin
