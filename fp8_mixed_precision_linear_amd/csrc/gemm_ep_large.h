// gemm_ep_large.h -- the large-tile kernels (k_gemm_w4, k_gemm_big) with the
// linear's epilogue, for the operands a layer's forward and dgrad products have:
// B (the weights) in E4M3, A in E4M3 forward and E5M2 backward; per-tensor, per-row,
// or block scales with A in 1x128 segments and B in 128x128 blocks.  Everything else
// runs on the tile kernels (gemm_ep_tile.h), which take any combination.
//
// Bound: the matrix units, as without the epilogue.  Measured on an MI355X: 8192 x
// 28672 x 8192, GELU, stored pre-activation, FP8 out with transposed copy, 1.60 ms,
// 2.40 PFLOP/s (fp8_scaled_gemm at 8192^3: 2.52); backward 8192 x 14336 x 4096 with 1x128
// scales and bias gradient 516 us, 1.86 PFLOP/s, where the promotion bounds it.
#pragma once

#include "gemm_w4_kernel.h"
#include "gemm_ep.h"

namespace fp8lin {

namespace {

template <int AF, bool OUT8>
hipError_t launch_large_f(const GemmParams& p, const EpParams& e, hipStream_t s) {
  const int tm = (int)((p.M + BM - 1) / BM), tn = (int)((p.N + BN - 1) / BN);
  const dim3 grid((unsigned)(tm * tn));
  using Ep = LinearEp<AF == 0 ? EP_FWD : EP_BWD>;
  const Ep ep{e};
  if (p.a_scaling == 1)
    hipLaunchKernelGGL((k_gemm_big<AF, 0, true, true, false, false, OUT8, Ep>), grid, dim3(THREADS), 0, s, p, tm,
                       tn, ep);
  else if (p.a_scaling == 3)
    hipLaunchKernelGGL((k_gemm_w4<AF, 0, false, OUT8, W4_MX + 1, Ep>), grid, dim3(W4_THREADS), 0, s, p, tm, tn, ep);
  else if (p.a_scaling == 5 || p.b_scaling == 5) {
    if (p.K % BK == 0)
      hipLaunchKernelGGL((k_gemm_w4<AF, 0, false, OUT8, W4_ROWS, Ep>), grid, dim3(W4_THREADS), 0, s, p, tm, tn, ep);
    else
      hipLaunchKernelGGL((k_gemm_w4<AF, 0, true, OUT8, W4_ROWS, Ep>), grid, dim3(W4_THREADS), 0, s, p, tm, tn, ep);
  } else {
    if (p.K % BK == 0)
      hipLaunchKernelGGL((k_gemm_w4<AF, 0, false, OUT8, W4_TENSOR, Ep>), grid, dim3(W4_THREADS), 0, s, p, tm, tn, ep);
    else
      hipLaunchKernelGGL((k_gemm_w4<AF, 0, true, OUT8, W4_TENSOR, Ep>), grid, dim3(W4_THREADS), 0, s, p, tm, tn, ep);
  }
  return hipGetLastError();
}

template <bool OUT8>
hipError_t launch_large_out(const GemmParams& p, const EpParams& e, hipStream_t s) {
  return p.a_fmt == 0 ? launch_large_f<0, OUT8>(p, e, s) : launch_large_f<1, OUT8>(p, e, s);
}

}  // namespace

}  // namespace fp8lin
