// gemm_ep_tile_fp8out.hip -- the tile kernels with the linear's epilogue, FP8
// output
// (a translation unit of its own, compiled beside the others).
#include "gemm_ep_tile.h"

namespace fp8lin {

hipError_t launch_gemm_ep_tile_fp8out(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  return launch_tile_sum<true>(p, e, plan, s);
}

}  // namespace fp8lin
