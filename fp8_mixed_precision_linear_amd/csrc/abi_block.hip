// abi_block.hip -- extern "C" entry points of the operators around the
// linears: host-side argument validation, then the launchers.  Nothing is
// enqueued when validation fails; a rejected launch maps to FP8_ERR_LAUNCH.
#include "../../include/fp8lin.h"
#include "launch.h"

#include <cmath>

using namespace fp8lin;

namespace {

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline unsigned size_of(int dt) { return dt == FP8_DT_F32 ? 4u : 2u; }
inline bool dtype_ok(int d) { return d == FP8_DT_BF16 || d == FP8_DT_F32; }
inline bool flag_ok(int f) { return f == 0 || f == 1; }
inline fp8_status launched(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_LAUNCH; }

// What the norm's two directions have in common.
template <typename A>
fp8_status norm_common(const A& a) {
  if (a.rows < 0 || a.cols < 0) return FP8_ERR_SHAPE;
  if (a.kind != FP8_NORM_RMS && a.kind != FP8_NORM_LAYER) return FP8_ERR_ARG;
  if (!dtype_ok(a.stream_dtype) || !dtype_ok(a.param_dtype)) return FP8_ERR_ARG;
  if (a.gate_kind < FP8_GATE_NONE || a.gate_kind > FP8_GATE_FULL) return FP8_ERR_ARG;
  if (a.gate_act < FP8_GATE_LINEAR || a.gate_act > FP8_GATE_TANH) return FP8_ERR_ARG;
  if ((a.gate != nullptr) != (a.gate_kind != FP8_GATE_NONE) && a.rows > 0 && a.cols > 0) return FP8_ERR_ARG;
  if (a.gate != nullptr && a.z == nullptr && a.rows > 0 && a.cols > 0) return FP8_ERR_ARG;
  if (a.kind == FP8_NORM_RMS && a.b_post != nullptr) return FP8_ERR_ARG;
  if (a.cols > norm_max_cols()) return FP8_ERR_UNSUPPORTED;
  if (a.gate_kind == FP8_GATE_FULL && a.ldg < a.cols) return FP8_ERR_SHAPE;
  const unsigned ps = size_of(a.param_dtype);
  const unsigned gs = a.gate_kind == FP8_GATE_TOKEN ? 4u : (a.gate_kind == FP8_GATE_FULL ? 2u : ps);
  if (!aligned(a.w_post, ps) || !aligned(a.b_post, ps) || !aligned(a.w_pre, ps) || !aligned(a.gate, gs))
    return FP8_ERR_ALIGN;
  if (!aligned(a.z, 2) || !aligned(a.stats_z, 4) || !aligned(a.stats_h, 4)) return FP8_ERR_ALIGN;
  if (a.z != nullptr && a.ldz < a.cols) return FP8_ERR_SHAPE;
  return FP8_OK;
}

// Checks a product's and its epilogue's arguments, all but the workspace, and, if
// they are right, fills p and e.
fp8_status ep_params(const fp8_gemm_args* a, const fp8_epilogue_args* ep, GemmParams& p, EpParams& e) {
  if (a == nullptr || ep == nullptr) return FP8_ERR_NULL;
  const fp8_status st = gemm_params(a, p);
  if (st != FP8_OK) return st;
  if (!flag_ok(ep->backward) || ep->act < FP8_ACT_NONE || ep->act > FP8_ACT_SILU) return FP8_ERR_ARG;
  if (!dtype_ok(ep->param_dtype) || !dtype_ok(ep->residual_dtype)) return FP8_ERR_ARG;
  if (ep->backward ? (ep->bias != nullptr || ep->residual != nullptr) : ep->dbias != nullptr) return FP8_ERR_ARG;
  if (a->accumulate) return FP8_ERR_UNSUPPORTED;
  if (p.d_fp8 && ep->residual != nullptr && ep->residual_dtype == FP8_DT_F32) return FP8_ERR_UNSUPPORTED;
  if (a->M > 0 && a->N > 0) {
    if (ep->backward && ep->act != FP8_ACT_NONE && ep->aux == nullptr) return FP8_ERR_NULL;
    if (ep->aux != nullptr && ep->ldaux < a->N) return FP8_ERR_SHAPE;
    if (ep->residual != nullptr && ep->ldres < a->N) return FP8_ERR_SHAPE;
    if (a->K > 0 && !gemm_big_supported(p)) return FP8_ERR_UNSUPPORTED;
    // the grids' threads are counted in 32 bits: tiles of 128 x 128, the few-row
    // kernel's 16 per column, the bias gradient's 16 per column
    if ((a->M + 127) / 128 > ((int64_t)1 << 23) / ((a->N + 127) / 128)) return FP8_ERR_UNSUPPORTED;
    if (a->N > ((int64_t)1 << 28) - 64 && (a->M <= 16 || ep->dbias != nullptr)) return FP8_ERR_UNSUPPORTED;
  }
  const unsigned ps = size_of(ep->param_dtype);
  if (!aligned(ep->bias, ps) || !aligned(ep->dbias, ps) || !aligned(ep->aux, 2) ||
      !aligned(ep->residual, size_of(ep->residual_dtype)) || !aligned(ep->workspace, 16))
    return FP8_ERR_ALIGN;
  e = {};
  e.backward = ep->backward; e.act = ep->act; e.bias_f32 = ep->param_dtype; e.res_f32 = ep->residual_dtype;
  e.bias = ep->bias; e.residual = ep->residual; e.ldres = ep->ldres; e.res_scale = ep->res_scale;
  e.aux = ep->aux; e.ldaux = ep->ldaux; e.dbias = ep->dbias;
  return FP8_OK;
}

}  // namespace

extern "C" {

fp8_status fp8_block_norm(const fp8_norm_args* args, hipStream_t stream) {
  if (args == nullptr) return FP8_ERR_NULL;
  const fp8_norm_args& a = *args;
  const fp8_status st = norm_common(a);
  if (st != FP8_OK) return st;
  if (!(a.eps >= 0.0f)) return FP8_ERR_ARG;
  if (a.kind == FP8_NORM_RMS && a.b_pre != nullptr) return FP8_ERR_ARG;
  if (a.y8 != nullptr) {
    if (a.y8_format != FP8_E4M3 && a.y8_format != FP8_E5M2) return FP8_ERR_ARG;
    if (a.y8_scaling != FP8_SCALE_TENSOR && a.y8_scaling != FP8_SCALE_ROW && a.y8_scaling != FP8_SCALE_1x128)
      return FP8_ERR_UNSUPPORTED;
  }
  if (a.rows == 0 || a.cols == 0) return FP8_OK;   // no row to normalise
  if (a.x == nullptr || (a.z != nullptr && a.h == nullptr)) return FP8_ERR_NULL;
  if (a.z == nullptr && a.h != nullptr) return FP8_ERR_ARG;
  if (a.z == nullptr && a.y == nullptr && a.y8 == nullptr) return FP8_ERR_ARG;
  if (a.ldx < a.cols || (a.h && a.ldh < a.cols) || (a.y && a.ldy < a.cols) || (a.y8 && a.ldy8 < a.cols))
    return FP8_ERR_SHAPE;
  if (a.y8 != nullptr) {
    if (a.y8_scaling == FP8_SCALE_TENSOR ? a.y8_scale == nullptr : a.y8_scale_inv == nullptr) return FP8_ERR_NULL;
    if (!aligned(a.y8_scale, 4) || !aligned(a.y8_scale_inv, 4) || !aligned(a.y8_amax, 4)) return FP8_ERR_ALIGN;
  }
  const unsigned ss = size_of(a.stream_dtype), ps = size_of(a.param_dtype);
  if (!aligned(a.x, ss) || !aligned(a.h, ss) || !aligned(a.y, 2) || !aligned(a.b_pre, ps)) return FP8_ERR_ALIGN;
  NormParams p = {};
  p.rows = a.rows; p.cols = a.cols;
  p.x = a.x; p.ldx = a.ldx; p.x_f32 = a.stream_dtype; p.p_f32 = a.param_dtype;
  p.layer = a.kind == FP8_NORM_LAYER; p.gate_kind = a.gate_kind; p.gate_act = a.gate_act;
  p.z = a.z; p.ldz = a.ldz;
  p.w_post = a.w_post; p.b_post = a.b_post; p.w_pre = a.w_pre; p.b_pre = a.b_pre;
  p.gate = a.gate; p.ldg = a.ldg;
  p.res_scale = a.res_scale; p.branch_scale = a.branch_scale; p.eps = a.eps;
  p.h = a.h; p.ldh = a.ldh; p.stats_z = a.z ? a.stats_z : nullptr; p.stats_h = a.stats_h;
  p.y = a.y; p.ldy = a.ldy; p.y8 = a.y8; p.ldy8 = a.ldy8;
  p.y8_fmt = a.y8_format; p.y8_scaling = a.y8_scaling;
  p.y8_scale = a.y8_scale; p.y8_sinv = a.y8_scale_inv;
  p.y8_amax = a.y8 && a.y8_scaling == FP8_SCALE_TENSOR ? a.y8_amax : nullptr;
  return launched(launch_norm_fwd(p, stream));
}

int64_t fp8_block_norm_bwd_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols > norm_max_cols()) return 0;   // (the call refuses wider rows)
  return 4 * norm_parts(rows, cols) * cols * (int64_t)sizeof(float);
}

fp8_status fp8_block_norm_bwd(const fp8_norm_bwd_args* args, hipStream_t stream) {
  if (args == nullptr) return FP8_ERR_NULL;
  const fp8_norm_bwd_args& a = *args;
  const fp8_status st = norm_common(a);
  if (st != FP8_OK) return st;
  if (a.kind == FP8_NORM_RMS && (a.db_pre != nullptr || a.db_post != nullptr)) return FP8_ERR_ARG;
  if (a.cols == 0) {   // a gate of each token is summed over no columns; every other output is empty
    if (a.dgate == nullptr || a.gate_kind != FP8_GATE_TOKEN) return FP8_OK;
    if (!aligned(a.dgate, 4)) return FP8_ERR_ALIGN;
    return launched(launch_fill_u32(static_cast<uint32_t*>(a.dgate), a.rows, 0u, stream));
  }
  const bool rows = a.rows > 0;
  // an output needs its input; without rows only the column sums are set, to 0
  if (rows) {
    if (a.dy != nullptr && (a.h == nullptr || a.stats_h == nullptr)) return FP8_ERR_NULL;
    if (a.z != nullptr && a.stats_z == nullptr) return FP8_ERR_NULL;
    if (a.dy == nullptr && (a.dw_pre != nullptr || a.db_pre != nullptr)) return FP8_ERR_ARG;
    if (a.z == nullptr && (a.dz != nullptr || a.dw_post != nullptr || a.db_post != nullptr)) return FP8_ERR_ARG;
    if (a.dgate != nullptr && a.gate == nullptr) return FP8_ERR_ARG;
    if (a.dy == nullptr && a.dh == nullptr) return FP8_ERR_NULL;
  }
  if ((a.dy && a.lddy < a.cols) || (a.dh && a.lddh < a.cols) || (a.dy && a.ldh < a.cols) ||
      (a.dx && a.lddx < a.cols) || (a.dz && a.lddz < a.cols) ||
      (a.dgate && a.gate_kind == FP8_GATE_FULL && a.lddg < a.cols))
    return FP8_ERR_SHAPE;
  const unsigned ss = size_of(a.stream_dtype), ps = size_of(a.param_dtype);
  const unsigned gs = a.gate_kind == FP8_GATE_TOKEN ? 4u : (a.gate_kind == FP8_GATE_FULL ? 2u : ps);
  if (!aligned(a.dy, 2) || !aligned(a.dh, ss) || !aligned(a.h, ss) || !aligned(a.dx, ss) || !aligned(a.dz, 2) ||
      !aligned(a.dgate, gs) || !aligned(a.dw_pre, ps) || !aligned(a.db_pre, ps) || !aligned(a.dw_post, ps) ||
      !aligned(a.db_post, ps) || !aligned(a.workspace, 16))
    return FP8_ERR_ALIGN;
  if (a.workspace == nullptr) return FP8_ERR_NULL;
  if (a.workspace_bytes < fp8_block_norm_bwd_workspace(a.rows, a.cols)) return FP8_ERR_SHAPE;
  NormGradParams p = {};
  p.rows = a.rows; p.cols = a.cols;
  p.dy = a.dy; p.lddy = a.lddy; p.dh = a.dh; p.lddh = a.lddh;
  p.h = a.h; p.ldh = a.ldh; p.stats_h = a.stats_h;
  p.z = a.z; p.ldz = a.ldz; p.stats_z = a.stats_z;
  p.x_f32 = a.stream_dtype; p.p_f32 = a.param_dtype;
  p.layer = a.kind == FP8_NORM_LAYER; p.gate_kind = a.gate_kind; p.gate_act = a.gate_act;
  p.w_post = a.w_post; p.b_post = a.b_post; p.w_pre = a.w_pre; p.gate = a.gate; p.ldg = a.ldg;
  p.res_scale = a.res_scale; p.branch_scale = a.branch_scale;
  p.dx = a.dx; p.lddx = a.lddx; p.dz = a.dz; p.lddz = a.lddz; p.dgate = a.dgate; p.lddg = a.lddg;
  p.dw_pre = a.dw_pre; p.db_pre = a.db_pre; p.dw_post = a.dw_post; p.db_post = a.db_post;
  p.part = static_cast<float*>(a.workspace);
  return launched(launch_norm_bwd(p, stream));
}

int64_t fp8_scaled_gemm_ep_workspace(int64_t M, int64_t N, int64_t K, fp8_scaling a_scaling, fp8_scaling b_scaling) {
  if (M < 0 || N < 0 || K < 0) return 0;
  GemmParams p = {};
  p.M = M; p.N = N; p.K = K;
  p.a_scaling = a_scaling; p.b_scaling = b_scaling;
  const EpPlan plan = ep_plan(p);
  return plan.part_bytes + plan.sums_bytes;
}

fp8_status fp8_scaled_gemm_ep(const fp8_gemm_args* gemm, const fp8_epilogue_args* ep, hipStream_t stream) {
  GemmParams p;
  EpParams e;
  const fp8_status st = ep_params(gemm, ep, p, e);
  if (st != FP8_OK) return st;
  const int64_t need = fp8_scaled_gemm_ep_workspace(gemm->M, gemm->N, gemm->K, gemm->a_scaling, gemm->b_scaling);
  if (need > 0 && ep->workspace == nullptr) return FP8_ERR_NULL;
  if (ep->workspace_bytes < need) return FP8_ERR_SHAPE;
  return launched(launch_gemm_ep(p, e, static_cast<uint8_t*>(ep->workspace), stream));
}

fp8_status fp8_scaled_gemm_ep_plan(const fp8_gemm_args* gemm, const fp8_epilogue_args* ep, fp8_ep_plan* plan) {
  GemmParams p;
  EpParams e;
  const fp8_status st = ep_params(gemm, ep, p, e);
  if (st != FP8_OK) return st;
  if (plan == nullptr) return FP8_ERR_NULL;
  const EpPlan t = ep_plan(p, e);
  plan->kernel = t.large ? FP8_EP_LARGE : (t.skinny ? FP8_EP_FEW_ROWS : FP8_EP_TILES);
  plan->tile_rows = t.large ? 256 : (t.skinny ? 16 : t.bm);
  plan->k_parts = t.splits;
  return FP8_OK;
}

fp8_status fp8_rope(const fp8_rope_args* args, hipStream_t stream) {
  if (args == nullptr) return FP8_ERR_NULL;
  const fp8_rope_args& a = *args;
  if (a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0 || a.dim < 0 || a.pairs < 0 || a.pairs > a.dim / 2)
    return FP8_ERR_SHAPE;
  if (!dtype_ok(a.dtype) || (a.layout != FP8_ROPE_HALF && a.layout != FP8_ROPE_INTERLEAVED)) return FP8_ERR_ARG;
  if (!flag_ok(a.inverse) || !flag_ok(a.positions_i64)) return FP8_ERR_ARG;
  const int64_t k_heads = a.k != nullptr ? a.k_heads : 0;
  // the grid and a workgroup's units are counted in 32 bits
  if (a.pairs > rope_max_pairs() || a.dim > 65535 || a.q_heads > 65535 || k_heads > 65535 - a.q_heads ||
      a.tokens > (int64_t)1 << 23)
    return FP8_ERR_UNSUPPORTED;
  if (a.tokens == 0 || a.dim == 0 || a.q_heads + k_heads == 0) return FP8_OK;
  if ((a.q_heads > 0 && (a.q == nullptr || a.q_out == nullptr)) || (k_heads > 0 && a.k_out == nullptr))
    return FP8_ERR_NULL;
  if (a.pairs > 0 && a.freqs == nullptr) return FP8_ERR_NULL;
  const unsigned s = size_of(a.dtype);
  if (!aligned(a.q, s) || !aligned(a.k, s) || !aligned(a.q_out, s) || !aligned(a.k_out, s) || !aligned(a.freqs, 8) ||
      !aligned(a.positions, a.positions_i64 ? 8 : 4))
    return FP8_ERR_ALIGN;
  RopeParams p = {};
  p.tokens = a.tokens; p.q_heads = a.q_heads; p.k_heads = k_heads; p.dim = a.dim; p.pairs = a.pairs;
  p.freqs = a.freqs; p.pos = a.positions; p.offset = a.offset; p.pos_i64 = a.positions_i64;
  p.f32 = a.dtype; p.interleaved = a.layout == FP8_ROPE_INTERLEAVED; p.inverse = a.inverse; p.scale = a.scale;
  p.q = a.q; p.q_st = a.q_token_stride; p.q_sh = a.q_head_stride;
  p.k = a.k; p.k_st = a.k_token_stride; p.k_sh = a.k_head_stride;
  p.q_out = a.q_out; p.qo_st = a.q_out_token_stride; p.qo_sh = a.q_out_head_stride;
  p.k_out = a.k_out; p.ko_st = a.k_out_token_stride; p.ko_sh = a.k_out_head_stride;
  p.copy_rest = (a.q_heads > 0 && a.q != a.q_out) || (k_heads > 0 && a.k != a.k_out);
  return launched(launch_rope(p, stream));
}

fp8_status fp8_rope_freqs(double* freqs, int64_t pairs, double base, fp8_rope_scaling scaling, double factor,
                          double trained, double low, double high, hipStream_t stream) {
  if (pairs < 0 || pairs >= (int64_t)1 << 24) return FP8_ERR_SHAPE;
  if (scaling < FP8_ROPE_PLAIN || scaling > FP8_ROPE_PARTS) return FP8_ERR_ARG;
  if (!(base > 0.0) || !std::isfinite(base)) return FP8_ERR_ARG;
  if (scaling != FP8_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return FP8_ERR_ARG;
  if (scaling == FP8_ROPE_PARTS &&
      (!(trained > 0.0) || !std::isfinite(trained) || !std::isfinite(low) || !std::isfinite(high) || high <= low))
    return FP8_ERR_ARG;
  if (pairs > 0 && freqs == nullptr) return FP8_ERR_NULL;
  if (!aligned(freqs, 8)) return FP8_ERR_ALIGN;
  return launched(launch_rope_freqs(freqs, pairs, base, scaling, factor, trained, low, high, stream));
}

}  // extern "C"
