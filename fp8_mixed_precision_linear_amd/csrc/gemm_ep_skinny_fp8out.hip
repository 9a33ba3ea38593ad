// gemm_ep_skinny_fp8out.hip -- the few-row product with the linear's epilogue, FP8 output.
#include "gemm_ep_skinny.h"

namespace fp8lin {

hipError_t launch_gemm_ep_skinny_fp8out(const GemmParams& p, const EpParams& e, hipStream_t s) {
  return launch_skinny_out<true>(p, e, s);
}

}  // namespace fp8lin
