// gemm_ep_large.hip -- the large-tile kernels with the linear's epilogue, BF16 /
// FP32 output.
#include "gemm_ep_large.h"

namespace fp8lin {

hipError_t launch_gemm_ep_large(const GemmParams& p, const EpParams& e, hipStream_t s) {
  return launch_large_out<false>(p, e, s);
}

}  // namespace fp8lin
