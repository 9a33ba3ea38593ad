// gemm_gated_tile.h -- the tile kernels (gemm_ep_tile.h) with the gated pair's epilogue;
// instantiated by gemm_gated_tile.hip, gemm_gated_grad_tile.hip and, for promoted block
// scales, their _blk twins.  Forward both operands are E4M3; backward the gradient may be
// E5M2 or E4M3, the weights are E4M3.  777 x 1999 x 2304 with power-of-two scales takes 22.3 us
// forward, 1037 rows 27.6 backward: a step of K 0.59, the rest launch, first loads and
// epilogue.
#pragma once

#include "gemm_ep_tile.h"
#include "gemm_gated.h"

namespace fp8lin {

namespace {

template <typename OP, int MODE, bool OUT8>
hipError_t launch_gated_mode(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s) {
  if constexpr (!OP::PAIRED) {
    if (p.a_fmt == 1) return launch_tile<1, 0, MODE, OUT8, OP>(p, e, plan, s);
  }
  return launch_tile<0, 0, MODE, OUT8, OP>(p, e, plan, s);
}
// Per-tensor, per-row and power-of-two block scales: no promotion.
template <typename OP, bool OUT8>
hipError_t launch_gated_sum(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s) {
  const bool per_a = p.a_scaling == 0 || p.a_scaling == 5, per_b = p.b_scaling == 0 || p.b_scaling == 5;
  return per_a && per_b ? launch_gated_mode<OP, EP_SUM, OUT8>(p, e, plan, s)
                        : launch_gated_mode<OP, EP_MX, OUT8>(p, e, plan, s);
}
// Other block scales.  A tile's 64 rows of the second factor lie in one 128 x 128 block
// only if that factor starts at a multiple of 64.
template <typename OP, bool OUT8>
hipError_t launch_gated_blk(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s) {
  const bool by_column = p.b_scaling == 1 || (OP::PAIRED && p.b_scaling == 2 && p.N % 64 != 0);
  return by_column ? launch_gated_mode<OP, EP_BLKCOL, OUT8>(p, e, plan, s)
                   : launch_gated_mode<OP, EP_BLK, OUT8>(p, e, plan, s);
}

}  // namespace

}  // namespace fp8lin
