// abi_gated.hip -- extern "C" entry points of the gated feed-forward pair and of 8-bit
// checkpoints: host-side argument validation, then the launchers.  Nothing is enqueued
// when validation fails; a rejected launch maps to FP8_ERR_LAUNCH.
#include "../../include/fp8lin.h"
#include "launch.h"

using namespace fp8lin;

namespace {

constexpr int64_t kMost = (int64_t)1 << 26;   // outputs per token; columns of a checkpoint are 2^28

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline unsigned size_of(int dt) { return dt == FP8_DT_F32 ? 4u : 2u; }
inline bool dtype_ok(int d) { return d == FP8_DT_BF16 || d == FP8_DT_F32; }
inline fp8_status launched(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_LAUNCH; }
inline int64_t blocks(int64_t cols) { return (cols + 31) / 32; }

// Checks everything but the workspace and, if it is right, fills p and e.
fp8_status gated_params(const fp8_gemm_args* a, const fp8_gated_args* g, GemmParams& p, GatedParams& e) {
  if (a == nullptr || g == nullptr) return FP8_ERR_NULL;
  const fp8_status st = gemm_params(a, p);
  if (st != FP8_OK) return st;
  if (g->backward != 0 && g->backward != 1) return FP8_ERR_ARG;
  if (g->act < FP8_ACT_NONE || g->act > FP8_ACT_SILU || !dtype_ok(g->param_dtype)) return FP8_ERR_ARG;
  if (g->backward ? g->bias != nullptr : g->dbias != nullptr) return FP8_ERR_ARG;
  if ((g->ck != nullptr) != (g->ck_exp != nullptr)) return FP8_ERR_NULL;
  if (g->backward && g->aux != nullptr && g->ck != nullptr) return FP8_ERR_ARG;   // one of them, not both
  if (a->accumulate) return FP8_ERR_UNSUPPORTED;
  if (a->b_fmt != FP8_E4M3 || (!g->backward && a->a_fmt != FP8_E4M3)) return FP8_ERR_UNSUPPORTED;
  const int64_t M = a->M, F = a->N;
  if (F > kMost) return FP8_ERR_UNSUPPORTED;
  if (M > 0 && F > 0) {
    if (g->backward && g->aux == nullptr && g->ck == nullptr) return FP8_ERR_NULL;
    if (g->backward && a->ldd < 2 * F) return FP8_ERR_SHAPE;
    if (g->aux != nullptr && g->ldaux < 2 * F) return FP8_ERR_SHAPE;
    if (g->ck != nullptr && (g->ldck < 2 * F || g->ldexp < 2 * blocks(F))) return FP8_ERR_SHAPE;
    if (a->K > 0 && !gemm_big_supported(p)) return FP8_ERR_UNSUPPORTED;
    // a launch's threads are counted in 32 bits: tiles of 128 x 128 columns of B's rows
    if ((M + 127) / 128 > ((int64_t)1 << 23) / ((2 * F + 127) / 128)) return FP8_ERR_UNSUPPORTED;
  }
  const unsigned ps = size_of(g->param_dtype);
  if (!aligned(g->bias, ps) || !aligned(g->dbias, ps) || !aligned(g->aux, 2) || !aligned(g->workspace, 16))
    return FP8_ERR_ALIGN;
  e = {};
  e.backward = g->backward; e.act = g->act; e.bias_f32 = g->param_dtype; e.bias = g->bias;
  e.aux = g->aux; e.ldaux = g->ldaux; e.ck = g->ck; e.ldck = g->ldck; e.ck_exp = g->ck_exp; e.ldexp = g->ldexp;
  e.dbias = g->dbias;
  return FP8_OK;
}

}  // namespace

extern "C" {

int64_t fp8_gated_linear_workspace(int64_t M, int64_t F, int64_t K, fp8_scaling a_scaling, fp8_scaling b_scaling,
                                   int backward) {
  if (M < 0 || F < 0 || K < 0 || F > kMost) return 0;   // (the call refuses them)
  GemmParams p = {};
  p.M = M; p.N = F; p.K = K;
  p.a_scaling = a_scaling; p.b_scaling = b_scaling;
  const EpPlan plan = gated_plan(p, backward != 0);
  return plan.part_bytes + plan.sums_bytes;
}

fp8_status fp8_gated_linear(const fp8_gemm_args* gemm, const fp8_gated_args* gated, hipStream_t stream) {
  GemmParams p;
  GatedParams e;
  const fp8_status st = gated_params(gemm, gated, p, e);
  if (st != FP8_OK) return st;
  const int64_t need =
      fp8_gated_linear_workspace(gemm->M, gemm->N, gemm->K, gemm->a_scaling, gemm->b_scaling, gated->backward);
  if (need > 0 && gated->workspace == nullptr) return FP8_ERR_NULL;
  if (gated->workspace_bytes < need) return FP8_ERR_SHAPE;
  return launched(launch_gated(p, e, static_cast<uint8_t*>(gated->workspace), stream));
}

fp8_status fp8_gated_linear_plan(const fp8_gemm_args* gemm, const fp8_gated_args* gated, fp8_ep_plan* plan) {
  GemmParams p;
  GatedParams e;
  const fp8_status st = gated_params(gemm, gated, p, e);
  if (st != FP8_OK) return st;
  if (plan == nullptr) return FP8_ERR_NULL;
  const EpPlan t = gated_plan(p, e);
  plan->kernel = t.large || t.mid ? FP8_EP_LARGE : (t.skinny ? FP8_EP_FEW_ROWS : FP8_EP_TILES);
  plan->tile_rows = t.large ? 256 : t.mid ? 160 : (t.skinny ? 16 : t.bm);
  plan->k_parts = t.splits;
  return FP8_OK;
}

namespace {

fp8_status checkpoint_args(const void* x, fp8_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, const uint8_t* ck,
                           int64_t ldck, const uint8_t* ck_exp, int64_t ldexp) {
  if (rows < 0 || cols < 0) return FP8_ERR_SHAPE;
  if (!dtype_ok(dtype)) return FP8_ERR_ARG;
  if (cols > 4 * kMost) return FP8_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return FP8_OK;
  if (x == nullptr || ck == nullptr || ck_exp == nullptr) return FP8_ERR_NULL;
  if (ldx < cols || ldck < cols || ldexp < blocks(cols)) return FP8_ERR_SHAPE;
  return aligned(x, size_of(dtype)) ? FP8_OK : FP8_ERR_ALIGN;
}

}  // namespace

fp8_status fp8_checkpoint_save(const void* x, fp8_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* ck,
                               int64_t ldck, uint8_t* ck_exp, int64_t ldexp, hipStream_t stream) {
  const fp8_status st = checkpoint_args(x, dtype, rows, cols, ldx, ck, ldck, ck_exp, ldexp);
  if (st != FP8_OK || rows == 0 || cols == 0) return st;
  return launched(launch_checkpoint_save(x, dtype, rows, cols, ldx, ck, ldck, ck_exp, ldexp, stream));
}

fp8_status fp8_checkpoint_load(const uint8_t* ck, int64_t ldck, const uint8_t* ck_exp, int64_t ldexp, int64_t rows,
                               int64_t cols, void* y, fp8_dtype dtype, int64_t ldy, hipStream_t stream) {
  const fp8_status st = checkpoint_args(y, dtype, rows, cols, ldy, ck, ldck, ck_exp, ldexp);
  if (st != FP8_OK || rows == 0 || cols == 0) return st;
  return launched(launch_checkpoint_load(ck, ldck, ck_exp, ldexp, rows, cols, y, dtype, ldy, stream));
}

}  // extern "C"
