// gemm_gated_large.h -- the large-tile kernels (k_gemm_w4, k_gemm_big) with the gated
// pair's epilogue; instantiated by gemm_gated_large.hip (forward) and
// gemm_gated_grad_large.hip, gemm_gated_grad_large_e5m2.hip (backward, by the gradient's
// format).  Per-tensor, per-row, or block scales with A in 1x128 segments and B in
// 128x128 blocks; F a multiple of 32 (of 128 forward with block scales, so that a tile has
// one scale of each factor); rows that start on a dword.  Everything else runs on tiles.
#pragma once

#include "gemm_w4_kernel.h"
#include "gemm_gated_direct.h"

namespace fp8lin {

namespace {

// Per-tensor and per-row scales.  TI: 32 TI rows a tile (8 or 5).
template <int AF, bool OUT8, typename Ep, int TI>
hipError_t launch_gated_plain_as(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  const int tm = (int)((p.M + 32 * TI - 1) / (32 * TI));
  const int tn = (int)(((Ep::PAIRED ? paired_columns(p.N) : p.N) + BN - 1) / BN);
  const dim3 grid((unsigned)(tm * tn)), block(W4_THREADS);
  const Ep ep{e};
  if (p.a_scaling == 5 || p.b_scaling == 5) {
    if (p.K % BK == 0) hipLaunchKernelGGL((k_gemm_w4<AF, 0, false, OUT8, W4_ROWS, Ep, TI>), grid, block, 0, s, p, tm, tn, ep);
    else hipLaunchKernelGGL((k_gemm_w4<AF, 0, true, OUT8, W4_ROWS, Ep, TI>), grid, block, 0, s, p, tm, tn, ep);
  } else {
    if (p.K % BK == 0) hipLaunchKernelGGL((k_gemm_w4<AF, 0, false, OUT8, W4_TENSOR, Ep, TI>), grid, block, 0, s, p, tm, tn, ep);
    else hipLaunchKernelGGL((k_gemm_w4<AF, 0, true, OUT8, W4_TENSOR, Ep, TI>), grid, block, 0, s, p, tm, tn, ep);
  }
  return hipGetLastError();
}

// Every scaling, on 256 rows.
template <int AF, bool OUT8, typename Ep, typename StripEp>
hipError_t launch_gated_large_as(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  if (p.a_scaling != 1 && p.a_scaling != 3) return launch_gated_plain_as<AF, OUT8, Ep, 8>(p, e, s);
  const int tm = (int)((p.M + BM - 1) / BM);
  const int tn = (int)(((Ep::PAIRED ? paired_columns(p.N) : p.N) + BN - 1) / BN);
  const dim3 grid((unsigned)(tm * tn));
  if (p.a_scaling == 1)
    hipLaunchKernelGGL((k_gemm_big<AF, 0, true, true, false, false, OUT8, StripEp>), grid, dim3(THREADS), 0, s, p, tm, tn,
                       StripEp{e});
  else
    hipLaunchKernelGGL((k_gemm_w4<AF, 0, false, OUT8, W4_MX + 1, Ep>), grid, dim3(W4_THREADS), 0, s, p, tm, tn, Ep{e});
  return hipGetLastError();
}

template <int AF, bool OUT8>
hipError_t launch_gated_grad_as(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  return e.ck ? launch_gated_large_as<AF, OUT8, GatedGradEp<1>, GatedGradStripEp<1>>(p, e, s)
              : launch_gated_large_as<AF, OUT8, GatedGradEp<0>, GatedGradStripEp<0>>(p, e, s);
}

}  // namespace

}  // namespace fp8lin
