// gemm_ep_large.h -- the large-tile kernels (k_gemm_w4, k_gemm_big) with the
// linear's epilogue, for the operands a layer's forward and dgrad products have:
// B (the weights) in E4M3, A in E4M3 forward and E5M2 backward; per-tensor, per-row,
// or block scales with A in 1x128 segments and B in 128x128 blocks; N a multiple of 8.
// Everything else runs on the tile kernels (gemm_ep_tile.h), which take any combination,
// at a third more time: 8192 x 14336 x 4096 backward with E4M3 gradients 704 us (1x128),
// 668 (power of two), 641 (per tensor), with E5M2 ones 524, 485 and 468 here.
//
// Bound: the matrix units, as without the epilogue, then the epilogue, whose inputs are
// fetched strip by strip when the sums are done.  Measured on an MI355X: 8192 x 28672 x
// 8192, GELU, stored pre-activation, FP8 out with transposed copy, 1.60 .. 1.63 ms, 2.4
// PFLOP/s (fp8_scaled_gemm: 2.52 at 8192^3, up to 2.80 at 8192 x 8192 x 10240); backward
// 8192 x 14336 x 4096 with 1x128 scales 512 us, 1.88 PFLOP/s: 454 for the product, which the
// promotion bounds, about 55 for the pre-activation (235 MB, 47 us at 5 TB/s, with the
// matrix units idle) and 5 for the bias gradient's join.
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
