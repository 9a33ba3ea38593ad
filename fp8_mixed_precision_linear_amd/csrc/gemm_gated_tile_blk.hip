// gemm_gated_tile_blk.hip -- gemm_gated_tile.h, forward, promoted block scales.
#include "gemm_gated_tile.h"

namespace fp8lin {

hipError_t launch_gated_tile_blk(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s) {
  return p.d_fp8 ? launch_gated_blk<GatedOp, true>(p, e, plan, s) : launch_gated_blk<GatedOp, false>(p, e, plan, s);
}

}  // namespace fp8lin
