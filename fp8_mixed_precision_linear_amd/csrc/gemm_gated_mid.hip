// gemm_gated_mid.hip -- gemm_gated_large.h, forward with per-tensor and per-row scales, on
// tiles of 160 x 256.  Where rows fall short of a whole 256-row tile, fewer of them are
// computed in vain, and 160 rows leave the LDS a third stage: a step then waits for loads
// that were issued two steps before, and it is these loads' way, not the products, that
// takes longest (300 x 14336 x 4096: 52.1 us on 256-row tiles, 48.4 on 160 with two stages,
// 43.7 with three; 117 MB of weights alone take 24; a step's 53 KB take 1.1 us to arrive, its
// products 0.6).  Over sixteen products of 160 to 1500
// rows that the times per step (ep_plan) give to them: 4% slower to 55% faster, 22% faster
// on average.
#include "gemm_gated_large.h"

namespace fp8lin {

hipError_t launch_gated_mid(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  return p.d_fp8 ? launch_gated_plain_as<0, true, GatedStripEp, 5>(p, e, s)
                 : launch_gated_plain_as<0, false, GatedStripEp, 5>(p, e, s);
}

}  // namespace fp8lin
