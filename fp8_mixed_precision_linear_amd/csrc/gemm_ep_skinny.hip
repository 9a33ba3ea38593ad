// gemm_ep_skinny.hip -- the few-row product with the linear's epilogue, BF16 / FP32 output.
#include "gemm_ep_skinny.h"

namespace fp8lin {

hipError_t launch_gemm_ep_skinny(const GemmParams& p, const EpParams& e, hipStream_t s) {
  return launch_skinny_out<false>(p, e, s);
}

}  // namespace fp8lin
