// gemm_ep_large_fp8out.hip -- the large-tile kernels with the linear's epilogue,
// FP8 output (a translation unit of its own, compiled beside the others).
#include "gemm_ep_large.h"

namespace fp8lin {

hipError_t launch_gemm_ep_large_fp8out(const GemmParams& p, const EpParams& e, hipStream_t s) {
  return launch_large_out<true>(p, e, s);
}

}  // namespace fp8lin
