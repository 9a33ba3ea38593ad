// launch.h -- host-side launchers behind the C ABI (internal to the library).
// Each launcher assumes its arguments were validated by the entry point in
// abi.hip and returns the hipError_t of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8lin.h"

namespace fp8lin {

// Compute units of the current device (queried once per device).
int64_t device_cu_count();

// Fill n dwords at p with v (a kernel, so it is safe inside graph capture).
hipError_t launch_fill_u32(uint32_t* p, int64_t n, uint32_t v, hipStream_t s);

// amax over n bf16 values (x 16-byte aligned) into *amax: overwritten
// (acc = 0, a fill kernel runs first) or max-accumulated (acc = 1).
hipError_t launch_amax(const uint16_t* x, int64_t n, float* amax, int acc, hipStream_t s);
// the same over [rows][cols] bf16 with row stride ld >= cols (x 16-byte aligned).
hipError_t launch_amax_rows(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, float* amax,
                            int acc, hipStream_t s);

// Saturated / underflowed element counts of the per-tensor cast of n bf16
// values (x 16-byte aligned), added to counts[0] / counts[1].
hipError_t launch_cast_stats(const uint16_t* x, int64_t n, const float* scale, int fmt,
                             uint64_t* counts, hipStream_t s);

// pow2 != 0: power-of-two (exponent-bias) scales instead of fmax / amax.
hipError_t launch_compute_scale(const float* amax, int64_t n, int fmt, int margin, int pow2,
                                float* scale, float* scale_inv, hipStream_t s);

// reset != 0: amax_new[i] is set to 0 once consumed.
hipError_t launch_history_update(float* history, int64_t n, int64_t len, float* amax_new,
                                 int fmt, int margin, int algo, int pow2, int reset, float* scale,
                                 float* scale_inv, hipStream_t s);

// Exponentially weighted amax and its scale, n tensors.
hipError_t launch_ewma_update(float* ewma, int64_t n, const float* amax_new, float beta, int fmt,
                              int margin, float* scale, float* scale_inv, hipStream_t s);

// Per-tensor cast with optional transpose and amax (zeroed here first when
// given, unless amax_acc: then max-accumulated into its current value);
// sr != 0: stochastic rounding with Philox words from (seed, offset), or,
// when rng is given, from (rng[0], rng[1]) read on the device, after which
// rng[1] is advanced by `advance`.
hipError_t launch_cast(const uint16_t* x, int64_t rows, int64_t cols, const float* scale, int fmt,
                       uint8_t* y, uint8_t* y_t, float* amax, int amax_acc, int sr, uint64_t seed,
                       uint64_t offset, uint64_t* rng, uint64_t advance, hipStream_t s);

// Block-wise cast (tile: 1 = 1x128, 2 = 128x128; pow2: power-of-two scales).
hipError_t launch_cast_block(const uint16_t* x, int64_t rows, int64_t cols, int fmt, int tile,
                             int pow2, uint8_t* y, float* sinv, uint8_t* y_t, float* sinv_t,
                             hipStream_t s);

// Row-wise cast: per-row scales for y, per-column scales for y_t (either
// output pair may be absent).
hipError_t launch_cast_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int fmt, uint8_t* y,
                               float* sinv, uint8_t* y_t, float* sinv_t, hipStream_t s);

struct GemmParams {
  int64_t M, N, K, lda, ldb, ldd;
  const uint8_t* A;
  int a_fmt, a_scaling;
  const float* a_sinv;
  const uint8_t* B;
  int b_fmt, b_scaling;
  const float* b_sinv;
  void* D;
  int d_f32;
  float* d_amax;  // max |output| is atomically max-ed into it
  int accumulate;
  int amax_acc;             // 0: launch_gemm zeroes *d_amax first; 1: it does not
  int d_fp8;                // 0: BF16/FP32 output; 1: E4M3 codes; 2: E5M2 codes
  const float* d_scale;     // FP8 output: quantisation scale (1 float)
  uint8_t* D_t;             // FP8 output: optional transposed codes [N][ldt]
  int64_t ldt;
};

// Checks a GEMM's arguments (abi.hip) and, if they are right, fills p.
fp8_status gemm_params(const fp8_gemm_args* a, GemmParams& p);

hipError_t launch_gemm(const GemmParams& p, hipStream_t s);

// Large-tile GEMM (gemm_big.hip): used when supported (32-bit buffer offsets
// cover a 256-row panel of each operand).
bool gemm_big_supported(const GemmParams& p);
hipError_t launch_gemm_big(const GemmParams& p, hipStream_t s);
hipError_t launch_gemm_big_fp8out(const GemmParams& p, hipStream_t s);   // p.d_fp8 != 0
// Per-tensor or per-row scales on both operands: the four-wavefront kernel
// (gemm_w4.hip, gemm_w4_fp8out.hip), under the same size limits.
hipError_t launch_gemm_w4(const GemmParams& p, hipStream_t s);
hipError_t launch_gemm_w4_fp8out(const GemmParams& p, hipStream_t s);   // p.d_fp8 != 0
// Power-of-two block scales (codes 3 / 4, the other operand possibly per
// tensor): the same kernel with the scales in the matrix instruction
// (gemm_w4_mx.hip, gemm_w4_mx_fp8out.hip).
hipError_t launch_gemm_w4_mx(const GemmParams& p, hipStream_t s);
hipError_t launch_gemm_w4_mx_fp8out(const GemmParams& p, hipStream_t s);   // p.d_fp8 != 0

// ---- operators around the linears (arguments validated by abi_block.hip)

// Norms before and after a block with its gate and residual scale
// (norm_kernels.hip).  x_f32: type of x and h; p_f32: of the weights, biases
// and a channel gate; gate_kind: 0 none, 1 per channel, 2 per token (FP32),
// 3 per element (BF16); gate_act: 0 none, 1 sigmoid, 2 tanh; layer: layer
// norm, else RMS norm; y8_scaling: 0 per tensor, 5 per row, 1 per 128 columns.
struct NormParams {
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  int x_f32, p_f32, layer, gate_kind, gate_act;
  const void* z;
  int64_t ldz;
  const void *w_post, *b_post, *w_pre, *b_pre, *gate;
  int64_t ldg;
  float res_scale, branch_scale, eps;
  void* h;
  int64_t ldh;
  float *stats_z, *stats_h;
  void* y;
  int64_t ldy;
  uint8_t* y8;
  int64_t ldy8;
  int y8_fmt, y8_scaling;
  const float* y8_scale;
  float *y8_sinv, *y8_amax;
};
struct NormGradParams {
  int64_t rows, cols;
  const void* dy;
  int64_t lddy;
  const void* dh;
  int64_t lddh;
  const void* h;
  int64_t ldh;
  const float* stats_h;
  const void* z;
  int64_t ldz;
  const float* stats_z;
  int x_f32, p_f32, layer, gate_kind, gate_act;
  const void *w_post, *b_post, *w_pre, *gate;
  int64_t ldg;
  float res_scale, branch_scale;
  void* dx;
  int64_t lddx;
  void* dz;
  int64_t lddz;
  void *dgate;
  int64_t lddg;
  void *dw_pre, *db_pre, *dw_post, *db_post;
  float* part;   // workspace: 4 * norm_parts(rows, cols) * cols floats
};
int64_t norm_max_cols();
int64_t norm_parts(int64_t rows, int64_t cols);
hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s);
hipError_t launch_norm_bwd(const NormGradParams& p, hipStream_t s);

// Rotary positions (rope_kernels.hip): strides in elements, of tokens (st) and
// heads (sh).
struct RopeParams {
  int64_t tokens, q_heads, k_heads, dim, pairs;
  const double* freqs;
  const void* pos;   // NULL: offset + token
  int64_t offset;
  int pos_i64, f32, interleaved, inverse, copy_rest;
  float scale;
  const void* q;
  int64_t q_st, q_sh;
  const void* k;
  int64_t k_st, k_sh;
  void* q_out;
  int64_t qo_st, qo_sh;
  void* k_out;
  int64_t ko_st, ko_sh;
  int tokens_wg, heads_wg;   // set by the launcher
};
int64_t rope_max_pairs();
hipError_t launch_rope(RopeParams p, hipStream_t s);
hipError_t launch_rope_freqs(double* f, int64_t pairs, double base, int scaling, double factor, double trained,
                             double low, double high, hipStream_t s);

// The FP8 product with the linear's epilogue (gemm_ep*.hip).
struct EpParams {
  int backward, act, bias_f32, res_f32, splits;
  const void* bias;      // forward
  const void* residual;  // forward
  int64_t ldres;
  float res_scale;
  const void* aux;       // forward: written (bf16(u)) or NULL; backward: read
  int64_t ldaux;
  void* dbias;           // backward; type bias_f32
  float* part;           // workspace: column sums
  float* sums;           // workspace: [splits][M][ldw]
  int64_t ldw;
};
// How a product is cut: tile, parts of K, rows of column sums, workspace.
struct EpPlan {
  int bm, bn, splits;
  bool large;   // 256 x 256 tiles of the large kernels
  bool mid;     // 160 x 256 tiles would be faster (the gated pair has them)
  bool skinny;  // few rows: weights streamed to registers
  int64_t parts, large_parts;   // rows of column sums; on the large kernels
  int64_t ldw, part_bytes, sums_bytes;
};
EpPlan ep_plan(const GemmParams& p);                      // what the workspace has to allow for
EpPlan ep_plan(const GemmParams& p, const EpParams& e);   // what a call takes
// Power-of-two scalings keep their codes in launch_gemm_ep_large*, are block
// scales like any others in the tile kernels.
hipError_t launch_gemm_ep_large(const GemmParams& p, const EpParams& e, hipStream_t s);
hipError_t launch_gemm_ep_large_fp8out(const GemmParams& p, const EpParams& e, hipStream_t s);
hipError_t launch_gemm_ep_tile(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gemm_ep_tile_fp8out(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gemm_ep_tile_blk(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gemm_ep_tile_blk_fp8out(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gemm_ep_skinny(const GemmParams& p, const EpParams& e, hipStream_t s);
hipError_t launch_gemm_ep_skinny_fp8out(const GemmParams& p, const EpParams& e, hipStream_t s);
hipError_t launch_gemm_ep(const GemmParams& p, EpParams e, uint8_t* ws, hipStream_t s);
// dbias[n] = sum over `parts` rows of column sums part[parts][N], in a fixed order.
hipError_t launch_ep_dbias(const float* part, int64_t parts, int64_t N, void* dbias, int f32, hipStream_t s);

// The gated pair of a feed-forward block (gemm_gated*.hip).  p.N = F, the outputs per
// token; forward, B has 2 F rows; backward, D has 2 F columns.
struct GatedParams {
  int backward, act, bias_f32, splits;
  const void* bias;   // forward: [2 F]
  void* aux;          // [M][2 F] bf16: forward written, backward read
  int64_t ldaux;
  uint8_t* ck;        // the same as a checkpoint (checkpoint.h), each half by itself
  int64_t ldck;
  uint8_t* ck_exp;    // [M][2 ceil(F / 32)]
  int64_t ldexp;
  void* dbias;        // backward: [2 F]
  float* part;        // workspace: column sums (one row of them: dbias itself, in its type)
  float* sums;        // workspace: [splits][M][ldw]
  int64_t ldw;
  int part_f32;
  uint32_t* keys;     // forward with FP8 output and an amax (workspace): see k_gated_amax
  uint2* key_at;
  int key_waves;      // wavefronts of a workgroup that write one
};
// What the workspace has to allow for, and what a call takes.
EpPlan gated_plan(const GemmParams& p, int backward);
EpPlan gated_plan(const GemmParams& p, const GatedParams& e);
hipError_t launch_gated(const GemmParams& p, GatedParams e, uint8_t* ws, hipStream_t s);
hipError_t launch_gated_tile(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gated_tile_blk(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gated_grad_tile(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s);
hipError_t launch_gated_grad_tile_blk(const GemmParams& p, const GatedParams& e, const EpPlan& plan, hipStream_t s);
// (power-of-two scalings keep their codes, as in launch_gemm_ep_large)
hipError_t launch_gated_large(const GemmParams& p, const GatedParams& e, hipStream_t s);
hipError_t launch_gated_mid(const GemmParams& p, const GatedParams& e, hipStream_t s);
hipError_t launch_gated_grad_large(const GemmParams& p, const GatedParams& e, hipStream_t s);
hipError_t launch_gated_grad_large_e5m2(const GemmParams& p, const GatedParams& e, hipStream_t s);
hipError_t launch_gated_skinny(const GemmParams& p, const GatedParams& e, hipStream_t s);

// 8-bit checkpoints (checkpoint_kernels.hip).
hipError_t launch_checkpoint_save(const void* x, int f32, int64_t rows, int64_t cols, int64_t ldx, uint8_t* ck,
                                  int64_t ldck, uint8_t* ck_exp, int64_t ldexp, hipStream_t s);
hipError_t launch_checkpoint_load(const uint8_t* ck, int64_t ldck, const uint8_t* ck_exp, int64_t ldexp, int64_t rows,
                                  int64_t cols, void* y, int f32, int64_t ldy, hipStream_t s);

}  // namespace fp8lin
