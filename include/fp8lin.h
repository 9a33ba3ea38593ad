/*
 * fp8lin.h -- C ABI of the FP8 scaled linear layer for AMD gfx950 (CDNA4).
 *
 * The layer: an amax reduction, a scale (current per-tensor, delayed from an
 * amax history, or block-wise), a saturating round-to-nearest-even cast to
 * FP8 (E4M3 for activations and weights, E5M2 for gradients), and the
 * forward / dgrad / wgrad GEMMs with FP32 accumulation and the inverse
 * scales applied in the epilogue (per-tensor) or per 128-wide K block
 * (block-wise).
 *
 * Sources, cited by page title and section:
 *   [MPG]  "Mixed Precision LLM Training: The Complete Guide"
 *   [TALK] PyData Amsterdam 2026, "FP8 for pretraining" (talk abstract)
 *   [P3]   "Training and inference of large language models using 8-bit
 *          floating point" (arXiv 2309.17224 library entry: abstract and
 *          reviews)
 *
 * Conventions for every entry point:
 *   - Pointers are caller-owned DEVICE memory on the current HIP device,
 *     unless stated otherwise.  The library never allocates, frees or keeps
 *     a pointer after the call returns.
 *   - Every call only enqueues work on `stream` (0 = the null stream) and
 *     returns; nothing is read back to the host, so a sequence of calls can
 *     run without host synchronisation.
 *   - Arguments are validated on the host before anything is enqueued; on
 *     any error code other than FP8_ERR_LAUNCH nothing was enqueued.
 *   - bf16 tensors are row-major [rows][cols] arrays of 16-bit patterns.
 *   - Outputs named *amax* are overwritten (not max-accumulated).
 *   - No global mutable state: calls on different streams may interleave.
 *   - FP8 codes are OCP E4M3 (max 448, no Inf, NaN = 0x7F/0xFF) and OCP E5M2
 *     (max 57344); the cast saturates finite overflow and +-Inf to +-max,
 *     maps NaN to 0x7F|sign, keeps the sign of zero, and rounds to nearest
 *     even after a binary32 multiply by the scale.
 */
#ifndef FP8LIN_H
#define FP8LIN_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8LIN_ABI_VERSION 10

/* [MPG] "The precision formats", "FP8 E4M3", "FP8 E5M2": E4M3 = 4 exponent
 * and 3 mantissa bits, range about 2^-9..448; E5M2 = 5 and 2, range about
 * 2^-16..57344.  "The HYBRID recipe": E4M3 forward, E5M2 for gradients. */
typedef enum { FP8_E4M3 = 0, FP8_E5M2 = 1 } fp8_format;

typedef enum {
  FP8_OK = 0,
  FP8_ERR_NULL = 1,         /* a required pointer is NULL */
  FP8_ERR_SHAPE = 2,        /* negative size, or a shape rule is broken */
  FP8_ERR_ALIGN = 3,        /* pointer or leading dimension misaligned */
  FP8_ERR_UNSUPPORTED = 4,  /* valid request the library does not implement */
  FP8_ERR_LAUNCH = 5,       /* the HIP runtime rejected a kernel launch */
  FP8_ERR_ARG = 6           /* an enum or scalar argument is out of range */
} fp8_status;

/* [MPG] "Calibration deep dive > Dynamic calibration (delayed scaling)":
 * amax_compute_algo "max" (over the history) or "most_recent". */
typedef enum { FP8_AMAX_MAX = 0, FP8_AMAX_MOST_RECENT = 1 } fp8_amax_algo;

/* [MPG] "Per-row vs per-tensor scaling" and "DeepSeek FP8 training recipe
 * in detail > Block-wise scaling at 128 granularity": one scale per tensor,
 * per 128-element segment of a row (1x128), or per 128x128 block.
 * The *_POW2 codes (GEMM operands only) are the same block layouts whose
 * inverse scales are exact powers of two 2^e, |e| <= 126, as produced by
 * fp8_cast_block_pow2 ([P3] exponent-bias scaling).
 * FP8_SCALE_ROW (GEMM operands only): one scale per row of a K-contiguous
 * operand, i.e. per token or per output channel, as produced by
 * fp8_cast_rowwise ("Per-row vs per-tensor scaling"). */
typedef enum {
  FP8_SCALE_TENSOR = 0,
  FP8_SCALE_1x128 = 1,
  FP8_SCALE_128x128 = 2,
  FP8_SCALE_1x128_POW2 = 3,
  FP8_SCALE_128x128_POW2 = 4,
  FP8_SCALE_ROW = 5
} fp8_scaling;

/* GEMM output: BF16, FP32, or FP8 codes quantised in the epilogue (the
 * next layer's cast fused into this GEMM). */
typedef enum { FP8_OUT_BF16 = 0, FP8_OUT_F32 = 1, FP8_OUT_E4M3 = 2, FP8_OUT_E5M2 = 3 } fp8_out_dtype;

/* ABI version (FP8LIN_ABI_VERSION of the built library). */
int fp8_abi_version(void);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* fp8_status_string(fp8_status status);

/* ------------------------------------------------------------------------
 * fp8_amax -- amax = max |x| over a bf16 tensor.
 * [MPG] "Transformer Engine internals > Per-tensor scaling": the scale is
 * set from the tensor's maximum absolute value.
 *   x_bf16  [rows][ld] bf16 (the first cols of each row are read),
 *           16-byte aligned; ld >= cols, in elements (ld == cols: a
 *           contiguous tensor).
 *   amax    1 float, overwritten.  The maximum is exact (no rounding is
 *           involved); a NaN element makes the result NaN; an empty tensor
 *           gives 0.
 * Errors: FP8_ERR_NULL (x with rows*cols > 0, or amax NULL), FP8_ERR_SHAPE
 * (negative size, ld < cols), FP8_ERR_ALIGN (x not 16-byte aligned).
 * ---------------------------------------------------------------------- */
fp8_status fp8_amax(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld, float* amax,
                    hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_stats -- saturation and underflow counts of the per-tensor cast
 * (fp8_cast_e4m3 / e5m2 with the same scale), for the diagnostic
 * dashboard's overflow and underflow ratios per layer.
 * [MPG] "Numerical-failure taxonomy > A diagnostic dashboard".
 * With v = fl32(x * scale[0]) as the cast computes it:
 *   counts[0] += number of elements with |v| beyond the format's largest
 *                finite value (448 / 57344; +-Inf included, NaN not);
 *   counts[1] += number of nonzero elements x whose code is +-0 (|v| at
 *                most half the smallest subnormal step: 2^-10 / 2^-17).
 *   x_bf16  [rows][cols] bf16, contiguous, 16-byte aligned.
 *   scale   1 float (device).
 *   counts  2 uint64 (device), 8-byte aligned; added to, never cleared.
 * Reads x once (2 B/elem); writes nothing else.
 * Errors: FP8_ERR_NULL (counts; x or scale with rows*cols > 0),
 * FP8_ERR_SHAPE, FP8_ERR_ALIGN, FP8_ERR_ARG (fmt).
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_stats(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                          const float* scale, uint64_t* counts, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_amax_acc -- fp8_amax with the result max-accumulated into *amax_acc
 * instead of overwriting it: one kernel, no fill ahead of it.
 * [MPG] "Delayed scaling (the default recipe)": the step's amax goes into
 * the tensor's history slot, which fp8_amax_history_update_reset clears
 * after reading it, so the next step accumulates into zero.
 *   amax_acc  1 float (device), required: on return max(old value, max |x|)
 *             (as binary32 bit patterns of |value|: a NaN element makes it
 *             NaN).  Calls that accumulate into one slot may overlap.
 * Other arguments and errors as fp8_amax.
 * ---------------------------------------------------------------------- */
fp8_status fp8_amax_acc(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                        float* amax_acc, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_compute_scale -- current scaling: scale = fl32(fmax / amax) * 2^-margin,
 * scale_inv = fl32(1 / scale), elementwise over n tensors.
 * [MPG] "Per-tensor scaling" (the scale puts the amax at the top of the FP8
 * range; the matmul result is multiplied by the inverse scale) and the
 * DelayedScaling recipe's `margin` argument (formula not given; read as a
 * division of the scale by 2^margin).
 *   amax       [n] floats (device).
 *   fmt        fmax = 448 (E4M3) or 57344 (E5M2).
 *   margin     0..64.
 *   scale, scale_inv  [n] floats, overwritten.
 * amax == 0 or non-finite: scale = 1, scale_inv = 1 ([MPG] "torch.compile
 * and FP8": no scale update for an all-zero tensor).  A quotient that
 * overflows binary32 is clamped to FLT_MAX.  Divisions are correctly
 * rounded.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE (n < 0), FP8_ERR_ARG (fmt, margin).
 * ---------------------------------------------------------------------- */
fp8_status fp8_compute_scale(const float* amax, int64_t n, fp8_format fmt, int margin,
                             float* scale, float* scale_inv, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_compute_scale_pow2 -- current scaling with power-of-two scales.
 * [P3] abstract and reviews: the scale is an exponent bias chosen from the
 * tensor's maximum (FP8-AMAX), matching its range to the format's; the
 * page does not print the formula.  Reading: scale = 2^e with e the largest
 * integer such that amax * 2^e <= fmax (the amax lands in (fmax/2, fmax],
 * nothing saturates), then e -= margin, e clamped to [-126, 126];
 * scale_inv = 2^-e.  Both are exact, so dequantisation is exact.
 * Arguments, fallback rule and errors as fp8_compute_scale.
 * ---------------------------------------------------------------------- */
fp8_status fp8_compute_scale_pow2(const float* amax, int64_t n, fp8_format fmt, int margin,
                                  float* scale, float* scale_inv, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_amax_history_update -- delayed scaling from an amax history.
 * [MPG] "Delayed scaling (the default recipe)" and "History-based scaling":
 * the scale used at step t+1 comes from the maxima of the last `len` steps.
 * For each tensor i < n:
 *   history[i][len-1..1] = history[i][len-2..0]; history[i][0] = amax_new[i];
 *   eff = max_j history[i][j] (FP8_AMAX_MAX; NaN propagates) or
 *         history[i][0] (FP8_AMAX_MOST_RECENT);
 *   if eff > 0 and finite: scale[i] = fl32(fmax/eff)*2^-margin,
 *                          scale_inv[i] = fl32(1/scale[i]);
 *   otherwise scale[i], scale_inv[i] keep their previous values.
 *   history    [n][len] floats, newest first, updated in place (initialise
 *              to 0 with scale = scale_inv = 1 before the first step).
 *   amax_new   [n] floats (e.g. the fused amax of the step's casts).
 * Stream order makes the update happen after the step's casts and GEMMs
 * that read the old scale when all are enqueued on one stream.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE (n < 0, len < 1 or > 1024),
 * FP8_ERR_ARG (fmt, margin, algo).
 * ---------------------------------------------------------------------- */
fp8_status fp8_amax_history_update(float* history, int64_t n, int64_t len,
                                   const float* amax_new, fp8_format fmt, int margin,
                                   fp8_amax_algo algo, float* scale, float* scale_inv,
                                   hipStream_t stream);

/* fp8_amax_history_update_pow2 -- the same update with the power-of-two
 * scale of fp8_compute_scale_pow2 ([P3] exponent bias) from the effective
 * amax; arguments and errors as fp8_amax_history_update. */
fp8_status fp8_amax_history_update_pow2(float* history, int64_t n, int64_t len,
                                        const float* amax_new, fp8_format fmt, int margin,
                                        fp8_amax_algo algo, float* scale, float* scale_inv,
                                        hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_amax_history_update_reset -- fp8_amax_history_update, after which
 * every consumed amax_new[i] is set to 0.
 * [MPG] "Delayed scaling (the default recipe)": the amax observed at step t
 * enters the history that sets the scale of step t+1.  With the slots
 * cleared here, the casts of the next step accumulate into them with
 * fp8_cast_amax_acc and no separate zeroing is needed between steps: one
 * step is then casts -> GEMMs -> this update, with amax_new starting at 0.
 *   amax_new   [n] floats (device), read, then overwritten with 0.
 *   Other arguments, order and errors as fp8_amax_history_update.
 * ---------------------------------------------------------------------- */
fp8_status fp8_amax_history_update_reset(float* history, int64_t n, int64_t len, float* amax_new,
                                         fp8_format fmt, int margin, fp8_amax_algo algo,
                                         float* scale, float* scale_inv, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_amax_ewma_update -- delayed scaling from an exponentially weighted
 * amax.  [MPG] "Delayed scaling (the default recipe)": the scale used at
 * step t is the one right for step t-1, or an exponentially weighted
 * average of recent steps (read as an average of the amax, from which the
 * scale follows).  For each tensor i < n, with a = amax_new[i]:
 *   a == 0 or non-finite: nothing changes;
 *   ewma[i] == 0 (no step seen yet): ewma[i] = a;
 *   else ewma[i] = fl32(fl32(beta * ewma[i]) + fl32(fl32(1 - beta) * a));
 *   then scale[i] = fl32(fmax / ewma[i]) * 2^-margin, scale_inv[i] =
 *   fl32(1 / scale[i]) (overflow clamped to FLT_MAX).
 *   ewma       [n] floats, in place (initialise to 0, scale = scale_inv = 1).
 *   beta       weight of the past, 0 <= beta <= 1 (0: the newest amax).
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE (n < 0), FP8_ERR_ALIGN, FP8_ERR_ARG
 * (fmt, margin outside 0..64, beta outside [0, 1] or NaN).
 * ---------------------------------------------------------------------- */
fp8_status fp8_amax_ewma_update(float* ewma, int64_t n, const float* amax_new, float beta,
                                fp8_format fmt, int margin, float* scale, float* scale_inv,
                                hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_e4m3 / fp8_cast_e5m2 -- per-tensor saturating RNE cast,
 * q = encode(fl32(x * scale)), with optional fused transpose and amax.
 * [MPG] "Per-tensor scaling" (multiply by the scale before quantising);
 * [TALK] outline 05:00-15:00 (E4M3 for activations and weights, E5M2 for
 * gradients).
 *   x_bf16    [rows][cols] bf16, 16-byte aligned.
 *   scale     1 float (device): the quantisation scale (not the inverse).
 *   y         [rows][cols] FP8 codes, or NULL.
 *   y_t       [cols][rows] FP8 codes (y_t[c][r] = y[r][c]), or NULL.
 *   amax_out  1 float, overwritten with max |x| (as fp8_amax), or NULL.
 *   y and y_t must not both be NULL (unless the tensor is empty); y, y_t
 *   16-byte aligned.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN.
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_e4m3(const void* x_bf16, int64_t rows, int64_t cols, const float* scale,
                         uint8_t* y, uint8_t* y_t, float* amax_out, hipStream_t stream);
fp8_status fp8_cast_e5m2(const void* x_bf16, int64_t rows, int64_t cols, const float* scale,
                         uint8_t* y, uint8_t* y_t, float* amax_out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_amax_acc -- the per-tensor cast of fp8_cast_e4m3 / e5m2 with the
 * fused amax max-accumulated into *amax_acc instead of overwriting it.
 * [MPG] "Per-tensor scaling" (the cast), "Delayed scaling (the default
 * recipe)" (the amax of the step feeds the next step's scale): with the
 * slot cleared by fp8_amax_history_update_reset, a delayed-scaling step
 * needs no zeroing kernel before its casts.
 *   fmt        FP8_E4M3 or FP8_E5M2.
 *   amax_acc   1 float (device), required: on return
 *              max(previous value, max |x|), compared as binary32 bit
 *              patterns, so the previous value must be +0 or positive
 *              (NaN in x propagates as in fp8_amax).
 *   Other arguments, layouts and errors as fp8_cast_e4m3, plus FP8_ERR_ARG
 *   (fmt) and FP8_ERR_NULL (amax_acc).  Calls that accumulate into one slot
 *   may run concurrently on several streams.
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_amax_acc(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                             const float* scale, uint8_t* y, uint8_t* y_t, float* amax_acc,
                             hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_sr -- per-tensor cast with stochastic rounding.
 * [MPG] "Stochastic rounding": round up or down at random according to the
 * remainder, which keeps the rounded value unbiased (used for gradients);
 * [TALK] outline: "rounding techniques".
 * With v = fl32(x * scale) and lo <= |v| < hi the two neighbouring FP8
 * magnitudes, the code is hi when r < (|v| - lo) / (hi - lo) * 2^32, else
 * lo (sign kept), where r is the element's random word; |v| >= fmax and
 * +-Inf saturate to +-fmax, NaN gives 0x7F | sign.  The word of element i
 * (row-major index) is word i % 4 of Philox4x32-10 (Salmon et al., SC 2011)
 * with counter (i / 4 low, i / 4 high, offset low, offset high) and key
 * (seed low, seed high); y_t holds the same codes transposed.  Calls with the
 * same (seed, offset) repeat the same draw; a call with another offset draws
 * fresh words (the offset is its own pair of counter words).  The values are
 * baked into a captured graph: see fp8_cast_sr_state.
 *   fmt        FP8_E4M3 or FP8_E5M2.
 *   Other arguments, layouts and errors as fp8_cast_e4m3, plus FP8_ERR_ARG
 *   (fmt).
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_sr(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                       const float* scale, uint64_t seed, uint64_t offset, uint8_t* y,
                       uint8_t* y_t, float* amax_out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_sr_state -- fp8_cast_sr with the generator state in device
 * memory, for steps captured once and replayed.  [MPG] "Stochastic
 * rounding": the rounding is unbiased only if every step draws fresh random
 * words, which by-value (seed, offset) cannot give a replayed graph.
 *   rng_state  2 x uint64 (device, 8-byte aligned, caller-owned): seed and
 *              offset, read by the cast when it runs on the stream; the codes
 *              equal fp8_cast_sr with those values.  Afterwards, in stream
 *              order, rng_state[1] += advance (modulo 2^64).
 *   advance    any nonzero value gives the next call fresh words: the offset
 *              is its own pair of Philox counter words, distinct from the
 *              element index; 0 repeats the draw.
 *   Other arguments, layouts and errors as fp8_cast_sr, plus FP8_ERR_NULL
 *   (rng_state) and FP8_ERR_ALIGN (rng_state not 8-byte aligned).  Calls on
 *   one rng_state must be stream-ordered (concurrent calls race on it).
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_sr_state(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                             const float* scale, uint64_t* rng_state, uint64_t advance,
                             uint8_t* y, uint8_t* y_t, float* amax_out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_block -- block-wise cast with per-tile scales computed on the fly.
 * [MPG] "DeepSeek FP8 training recipe in detail > Block-wise scaling at 128
 * granularity": one scale per 128x128 weight block, one per 128-element
 * activation segment, stored next to the data and applied in the matmul.
 * Per tile: amax over the elements present, scale = fl32(fmax/amax)
 * (1 for an all-zero or non-finite tile), scale_inv = fl32(1/scale), then
 * the cast of fp8_cast_e4m3 with that scale.
 *   x_bf16   [rows][cols] bf16, 16-byte aligned.
 *   tile == FP8_SCALE_1x128:
 *     y         [rows][cols], tiles of 128 consecutive columns in one row;
 *     scale_inv [ceil(cols/128)][rows]  (kb-major);
 *     y_t       [cols][rows], tiles of 128 consecutive ROWS in one column
 *               (the token-axis tiles of the transposed operand), each
 *               quantised from bf16 with its own scale;
 *     scale_inv_t [ceil(rows/128)][cols].
 *   tile == FP8_SCALE_128x128:
 *     one scale per 128x128 block; y_t is the byte transpose of y;
 *     scale_inv   [ceil(cols/128)][ceil(rows/128)];
 *     scale_inv_t [ceil(rows/128)][ceil(cols/128)] (same values, transposed).
 *   Each of (y, scale_inv) and (y_t, scale_inv_t) is either both given or
 *   both NULL, and at least one pair is given (an empty tensor needs no
 *   pointers and enqueues nothing).  y, y_t 16-byte aligned.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN, FP8_ERR_ARG.
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_block(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                          fp8_scaling tile, uint8_t* y, float* scale_inv, uint8_t* y_t,
                          float* scale_inv_t, hipStream_t stream);

/* fp8_cast_block_pow2 -- fp8_cast_block with power-of-two tile scales (the
 * rule of fp8_compute_scale_pow2 on each tile's amax, margin 0; [P3]
 * exponent bias applied per DeepSeek-style block).  The scales it writes
 * are valid FP8_SCALE_1x128_POW2 / FP8_SCALE_128x128_POW2 GEMM operands.
 * Arguments (tile is FP8_SCALE_1x128 or FP8_SCALE_128x128) and errors as
 * fp8_cast_block. */
fp8_status fp8_cast_block_pow2(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                               fp8_scaling tile, uint8_t* y, float* scale_inv, uint8_t* y_t,
                               float* scale_inv_t, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_cast_rowwise -- row-wise (per-channel) cast with scales computed on
 * the fly.  [MPG] "Per-row vs per-tensor scaling": one scale per row of the
 * matrix rather than one per tensor, so an outlier row or column only
 * coarsens its own scale (torchao's row-wise recipe).
 *   x_bf16       [rows][cols] bf16, 16-byte aligned.
 *   y            [rows][cols]: row r quantised with s_r = fl32(fmax / amax_r),
 *                amax_r = max_c |x[r][c]| (s_r = 1 for an all-zero or
 *                non-finite row), codes as fp8_cast_e4m3 / e5m2;
 *   scale_inv    [rows]: fl32(1 / s_r)  (an FP8_SCALE_ROW GEMM operand);
 *   y_t          [cols][rows]: y_t[c][r] quantised with the scale of column
 *                c, s_c = fl32(fmax / max_r |x[r][c]|) (same fallback) -- the
 *                K-contiguous operand of the GEMMs that reduce over rows;
 *   scale_inv_t  [cols]: fl32(1 / s_c).
 *   Each of (y, scale_inv) and (y_t, scale_inv_t) is either both given or
 *   both NULL, and at least one pair is given (an empty tensor needs no
 *   pointers and enqueues nothing).  y, y_t 16-byte aligned.  The memory
 *   of y_t and scale_inv_t also serves as workspace while the call runs
 *   (column maxima); both hold their final values once the call's work
 *   has completed in stream order.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN, FP8_ERR_ARG (fmt).
 * ---------------------------------------------------------------------- */
fp8_status fp8_cast_rowwise(const void* x_bf16, int64_t rows, int64_t cols, fp8_format fmt,
                            uint8_t* y, float* scale_inv, uint8_t* y_t, float* scale_inv_t,
                            hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_scaled_gemm -- D[m][n] = sum_k A[m][k] * B[n][k] with FP8 operands,
 * FP32 accumulation and dequantisation.
 * [MPG] "Per-tensor scaling" (multiply the matmul result by the inverse
 * scales), "Skipping the BAcc accumulator promotion" and "Mixed-precision
 * accumulation" (partial products accumulate in FP32; the result is cast to
 * BF16), "Block-wise scaling at 128 granularity" (block scales applied
 * during the matmul).
 * Both operands are K-contiguous ("TN"): A [M][lda], B [N][ldb] FP8 codes.
 * The layer's three GEMMs are operand choices (weights stored [in][out]):
 *   forward  Y  = X W      : A = X_q   [T][in],  B = W^T_q  [out][in]
 *   dgrad    dX = dY W^T   : A = dY_q  [T][out], B = W_q    [in][out]
 *   wgrad    dW = X^T dY   : A = X^T_q [in][T],  B = dY^T_q [out][T]
 * Inverse-scale layouts (as produced by the casts):
 *   FP8_SCALE_TENSOR  : 1 float;
 *   FP8_SCALE_1x128   : [ceil(K/128)][rows]       (rows = M for A, N for B);
 *   FP8_SCALE_128x128 : [ceil(K/128)][ceil(rows/128)];
 *   FP8_SCALE_1x128_POW2, FP8_SCALE_128x128_POW2: the same layouts, every
 *   value an exact power of two 2^e with |e| <= 126 (fp8_cast_block_pow2);
 *   other values give unspecified (memory-safe) results.  When every
 *   block-scaled operand is a *_POW2 one, the block scales are applied
 *   inside the matrix instruction (exact power-of-two scaling of each
 *   128-wide K block) and a per-tensor operand's scale in the epilogue;
 *   mixed with a plain block operand, all block scales are promoted in
 *   FP32 as for FP8_SCALE_1x128 / FP8_SCALE_128x128;
 *   FP8_SCALE_ROW     : [rows] (one per row of the operand; combines with
 *   FP8_SCALE_TENSOR or FP8_SCALE_ROW only, else FP8_ERR_UNSUPPORTED).
 * Result: tensor or row x tensor or row: D = ((sum_k a b) * sa(m)) * sb(n),
 * one FP32 sum over all of K scaled in the epilogue; any block scaling:
 * D = sum_kb (sum_{k in kb} a b) * sa(m,kb) * sb(n,kb), each 128-wide K
 * block promoted into the FP32 accumulator.  D is [M][ldd], BF16 (round
 * to nearest even) or FP32.  accumulate = 1 (FP32 output only) adds the
 * result to the existing D.  d_amax (nullable, 1 float) is overwritten with
 * max |D| of the stored output values (a one-word fill runs ahead of the
 * GEMM on the stream), or, with amax_accumulate = 1, max-accumulated into
 * the value already there (no fill: the caller owns the slot, e.g. one
 * cleared by fp8_amax_history_update_reset; calls that accumulate into one
 * slot may overlap).
 * FP8 output (d_dtype FP8_OUT_E4M3 / FP8_OUT_E5M2; [TALK] outline
 * "quantisation fusions"; [MPG] "Transformer Engine internals": the cast
 * that the next layer would do, fused into this GEMM's epilogue): with v the
 * FP32 result above (before any BF16 rounding), D[m][n] = encode(fl32(v *
 * d_scale[0])) as in fp8_cast_e4m3 / e5m2; D_t (nullable) [N][ldt] receives
 * the same codes transposed (the next layer's wgrad operand); d_amax is
 * max |v| (the amax of the quantised tensor, for its delayed scaling).
 * accumulate must be 0; requires ldt >= M when D_t is given.
 * amax_accumulate: 0 or 1 (FP8_ERR_ARG otherwise), see d_amax.
 * Shape rules: M, N, K >= 0; K % 16 == 0 (tensor and row modes) or
 * K % 128 == 0 (block modes); lda, ldb >= K and multiples of 16; ldd >= N; A, B 16-byte
 * aligned; D 4-byte aligned.  K == 0 gives D = 0 (or D unchanged when
 * accumulating).
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN, FP8_ERR_ARG (also
 * D_t with a non-FP8 output), FP8_ERR_UNSUPPORTED (accumulate with a BF16
 * or FP8 output; FP8 output with lda or ldb beyond the large-tile kernel's
 * 32-bit panel offsets, i.e. 256 * ld >= 2^31; FP8_SCALE_ROW with a block
 * operand).
 * ---------------------------------------------------------------------- */
typedef struct {
  int64_t M, N, K;
  int64_t lda, ldb, ldd;
  const uint8_t* A; fp8_format a_fmt; fp8_scaling a_scaling; const float* a_scale_inv;
  const uint8_t* B; fp8_format b_fmt; fp8_scaling b_scaling; const float* b_scale_inv;
  void* D; fp8_out_dtype d_dtype;
  float* d_amax;
  int accumulate;
  const float* d_scale;   /* FP8 output: quantisation scale (1 float); else ignored */
  uint8_t* D_t;           /* FP8 output: transposed codes [N][ldt], or NULL */
  int64_t ldt;
  int amax_accumulate;    /* 1: max-accumulate into *d_amax instead of overwriting */
} fp8_gemm_args;

fp8_status fp8_scaled_gemm(const fp8_gemm_args* args, hipStream_t stream);

/* ========================================================================
 * The operators around the linears of a transformer block: norms with the
 * block's gate and residual scale, the GEMM with the linear's bias,
 * activation and residual, and rotary positions, each with its gradient.
 * They were added to version 10 without changing any structure or call above:
 * the version alone does not tell a caller that they are there.  One that may
 * meet an older library looks for the symbols (dlsym), one that is compiled
 * against a header of unknown age for FP8LIN_BLOCK_OPERATORS.  Beyond the
 * conventions at the top:
 *   - rows may be strided (ld >= columns, in elements); pointers need the
 *     alignment of their element only, unless stated otherwise;
 *   - an optional output or input is NULL when absent;
 *   - parameters (weights, biases, a per-channel gate) and their gradients
 *     have one type per call, param_dtype;
 *   - a workspace is caller-owned device memory, 16-byte aligned, that the
 *     call may overwrite; its contents mean nothing afterwards.  Calls that
 *     may overlap need one each.
 * Every sum, norm statistic and column sum is held in binary32 and taken in
 * a fixed order: equal inputs on equal hardware give equal bits.
 * ===================================================================== */
#define FP8LIN_BLOCK_OPERATORS 1
#define FP8LIN_GATED_OPERATORS 1   /* fp8_gated_linear, fp8_checkpoint_*: later still, the same way */
typedef enum { FP8_DT_BF16 = 0, FP8_DT_F32 = 1 } fp8_dtype;
typedef enum { FP8_NORM_RMS = 0, FP8_NORM_LAYER = 1 } fp8_norm_kind;
/* Gate of a block's output: none, one value per channel [cols]
 * (param_dtype), per token [rows] (FP32), or per element [rows][ldg] (BF16);
 * used as it is, or through a sigmoid or a hyperbolic tangent. */
typedef enum {
  FP8_GATE_NONE = 0, FP8_GATE_CHANNEL = 1, FP8_GATE_TOKEN = 2, FP8_GATE_FULL = 3
} fp8_gate_kind;
typedef enum { FP8_GATE_LINEAR = 0, FP8_GATE_SIGMOID = 1, FP8_GATE_TANH = 2 } fp8_gate_act;

/* ------------------------------------------------------------------------
 * fp8_block_norm -- per row of `cols` values, with N the norm of `kind`:
 *   h = res_scale * x + branch_scale * G(gate) * (N(z) * w_post + b_post)
 *   y = N(h) * w_pre + b_pre,   N(v) = (v - mean) * rstd,
 *   rstd = 1 / sqrt(mean((v - mean)^2) + eps), mean taken as 0 for the RMS
 *   norm.
 *   x       [rows][ldx], stream_dtype: the residual stream.
 *   z       [rows][ldz] BF16: the block's output.  NULL: no block ends here,
 *           h is x itself (res_scale unused) and `h` must be NULL.
 *   h       [rows][ldh], stream_dtype: the new stream; may be x in place.
 *   w_post, b_post, w_pre, b_pre  [cols]; NULL weight: 1, NULL bias: 0.  Biases
 *           belong to the layer norm only.
 *   stats_z, stats_h  [rows][2] FP32 (mean, rstd), for the gradient.
 *   y       [rows][ldy] BF16, and / or
 *   y8      [rows][ldy8] FP8 codes of y (of its binary32 value; row by row, no
 *           transposed copy), y8_format, with y8_scaling
 *             FP8_SCALE_TENSOR: y8_scale (1 float) as in fp8_cast_e4m3 /
 *               e5m2; y8_amax (1 float, optional) is max-accumulated with
 *               max |y| as in fp8_amax_acc;
 *             FP8_SCALE_ROW: the row's own scale, y8_scale_inv [rows], as
 *               fp8_cast_rowwise;
 *             FP8_SCALE_1x128: y8_scale_inv [ceil(cols/128)][rows], as
 *               fp8_cast_block.
 *   With neither y nor y8 only h is made (then z is required).
 *   rows == 0 or cols == 0: nothing is written.
 * y is taken from h in binary32, before h is rounded to stream_dtype.  No
 * other output may overlap an input.
 * Errors: FP8_ERR_NULL (args, x, h with z, a scale), FP8_ERR_SHAPE (negative
 * size, ld < cols), FP8_ERR_ARG (an enum, eps negative or NaN, h without z, a
 * gate without z or unlike gate_kind, a bias with the RMS norm, nothing to
 * make), FP8_ERR_UNSUPPORTED (cols > 32768; y8_scaling), FP8_ERR_ALIGN.
 * ---------------------------------------------------------------------- */
typedef struct {
  int64_t rows, cols;
  fp8_norm_kind kind;
  fp8_dtype stream_dtype, param_dtype;
  float eps, res_scale, branch_scale;
  const void* x; int64_t ldx;
  const void* z; int64_t ldz;
  const void* w_post; const void* b_post; const void* w_pre; const void* b_pre;
  const void* gate; int64_t ldg; fp8_gate_kind gate_kind; fp8_gate_act gate_act;
  void* h; int64_t ldh;
  float* stats_z; float* stats_h;
  void* y; int64_t ldy;
  uint8_t* y8; int64_t ldy8; fp8_format y8_format; fp8_scaling y8_scaling;
  const float* y8_scale; float* y8_scale_inv; float* y8_amax;
} fp8_norm_args;

fp8_status fp8_block_norm(const fp8_norm_args* args, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_block_norm_bwd -- gradients of fp8_block_norm.
 *   dy       [rows][lddy] BF16: gradient of y (of the values that y8 stands
 *            for); NULL: y was not made.
 *   dh       [rows][lddh] stream_dtype: gradient that reaches h from above;
 *            NULL: 0.
 *   h, stats_h  as written by the forward pass (h: x where there was no z);
 *            needed with dy.   z, stats_z, w_post, gate: as given to it;
 *            needed where there was a z.  b_post only for dgate.
 *   dx       [rows][lddx] stream_dtype, may be dh in place;  dz [rows][lddz]
 *            BF16, may be dy in place;  dgate: gate's shape and type ([rows][lddg]
 *            for FP8_GATE_FULL);  dw_pre, db_pre, dw_post, db_post [cols],
 *            param_dtype: overwritten.
 *   Each output is optional.  rows == 0 sets the column sums to 0, cols == 0
 *   a per-token dgate.
 *   workspace  fp8_block_norm_bwd_workspace(rows, cols) bytes (0 for sizes
 *            that the call refuses).
 * Errors: as fp8_block_norm; FP8_ERR_NULL also for the workspace,
 * FP8_ERR_SHAPE for one that is too small, FP8_ERR_ARG for an output whose
 * input is missing.
 * ---------------------------------------------------------------------- */
typedef struct {
  int64_t rows, cols;
  fp8_norm_kind kind;
  fp8_dtype stream_dtype, param_dtype;
  float res_scale, branch_scale;
  const void* dy; int64_t lddy;
  const void* dh; int64_t lddh;
  const void* h; int64_t ldh; const float* stats_h;
  const void* z; int64_t ldz; const float* stats_z;
  const void* w_post; const void* b_post; const void* w_pre;
  const void* gate; int64_t ldg; fp8_gate_kind gate_kind; fp8_gate_act gate_act;
  void* dx; int64_t lddx;
  void* dz; int64_t lddz;
  void* dgate; int64_t lddg;
  void* dw_pre; void* db_pre; void* dw_post; void* db_post;
  void* workspace; int64_t workspace_bytes;
} fp8_norm_bwd_args;

int64_t fp8_block_norm_bwd_workspace(int64_t rows, int64_t cols);
fp8_status fp8_block_norm_bwd(const fp8_norm_bwd_args* args, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_scaled_gemm_ep -- fp8_scaled_gemm with the linear's epilogue.  With v
 * the dequantised product in binary32 (every operand format and scaling of
 * fp8_scaled_gemm):
 *   forward  (backward = 0):  u = v + bias[n];  aux[m][n] = bf16(u);
 *                             d = act(u) + res_scale * residual[m][n]
 *   backward (backward = 1):  d = v * act'(aux[m][n]);
 *                             dbias[n] = sum_m d
 * and D = d in gemm->d_dtype: BF16, FP32, or FP8 codes of d * d_scale with the
 * transposed copy D_t; d_amax as in fp8_scaled_gemm (max |d|).  The forward
 * call is a linear with its bias and activation (the next linear's cast in the
 * same pass, if FP8); the backward call is the dgrad product of the linear
 * after the activation, and gives the gradient before it: the operand of the
 * wgrad and dgrad of the linear before.
 *   bias      [N] param_dtype, optional.   dbias [N] param_dtype, optional.
 *   act       FP8_ACT_GELU_TANH is the tanh form of GELU.
 *   aux       [M][ldaux] BF16.  Forward: optional output, the pre-activation.
 *             Backward: input, required unless act is FP8_ACT_NONE.
 *   residual  [M][ldres] residual_dtype, optional; may be D in place if the
 *             types agree.
 *   workspace fp8_scaled_gemm_ep_workspace(M, N, K, a_scaling, b_scaling)
 *             bytes.
 * Shape rules, scalings and errors as fp8_scaled_gemm, and: FP8_ERR_ARG (act,
 * dtypes, bias or residual in a backward call, dbias in a forward one),
 * FP8_ERR_NULL (aux of a backward call, workspace), FP8_ERR_SHAPE (ldaux,
 * ldres < N, a workspace that is too small), FP8_ERR_UNSUPPORTED (gemm's
 * accumulate; 256 * lda or 256 * ldb >= 2^31; K > 65536; more than 2^23 tiles
 * of 128 x 128 outputs; N > 2^28 - 64 with up to 16 rows or with dbias; an FP32
 * residual beside an FP8 output).
 * ---------------------------------------------------------------------- */
typedef enum {
  FP8_ACT_NONE = 0, FP8_ACT_RELU = 1, FP8_ACT_GELU = 2, FP8_ACT_GELU_TANH = 3, FP8_ACT_SILU = 4
} fp8_activation;

typedef struct {
  int backward;
  fp8_activation act;
  fp8_dtype param_dtype;
  const void* bias;
  const void* residual; int64_t ldres; fp8_dtype residual_dtype; float res_scale;
  void* aux; int64_t ldaux;
  void* dbias;
  void* workspace; int64_t workspace_bytes;
} fp8_epilogue_args;

int64_t fp8_scaled_gemm_ep_workspace(int64_t M, int64_t N, int64_t K, fp8_scaling a_scaling,
                                     fp8_scaling b_scaling);
fp8_status fp8_scaled_gemm_ep(const fp8_gemm_args* gemm, const fp8_epilogue_args* ep,
                              hipStream_t stream);

/* fp8_scaled_gemm_ep_plan -- which kernel fp8_scaled_gemm_ep takes with these
 * arguments on the current device (nothing is enqueued, no pointer is read; the
 * workspace is not looked at): for tests and profiles, since the choice goes by
 * measured times and may change.  Errors: as the call's; FP8_ERR_NULL (plan). */
typedef enum {
  FP8_EP_FEW_ROWS = 0,   /* up to 16 rows, weights streamed from memory */
  FP8_EP_TILES = 1,      /* tiles of tile_rows x 128, K in k_parts parts */
  FP8_EP_LARGE = 2       /* tiles of tile_rows x 256 (256, of the gated pair also 160) */
} fp8_ep_kernel;
typedef struct {
  fp8_ep_kernel kernel;
  int tile_rows, k_parts;
} fp8_ep_plan;

fp8_status fp8_scaled_gemm_ep_plan(const fp8_gemm_args* gemm, const fp8_epilogue_args* ep, fp8_ep_plan* plan);

/* ------------------------------------------------------------------------
 * fp8_gated_linear -- the gated pair of a feed-forward block as one product.
 * With F outputs per token (gemm->N = F) and every sum in binary32:
 *   forward (backward = 0):  B holds 2 F rows, those of the gate's weights and
 *     then those of the up projection's;  g[f] = A . B[f] + bias[f],
 *     u[f] = A . B[F + f] + bias[F + f], dequantised as in fp8_scaled_gemm;
 *     h = act(g) u, from the unrounded g and u;  D [M][F] = h.
 *   backward (backward = 1):  B holds F rows (the next linear's weights, its
 *     input dimension outermost);  v[f] = A . B[f], the gradient of h;
 *     D [M][2 F] = (dg | du),  dg = v u act'(g),  du = v act(g);
 *     dbias[2 F] = column sums of D before its rounding.
 * D is BF16, FP32 or FP8 codes of d_scale times it (backward: one scale for
 * both halves) with the transposed copy D_t ([F][ldt]; backward [2 F][ldt]);
 * d_amax as in fp8_scaled_gemm; of a forward call with FP8 output it is D's largest
 * output summed again in binary32, without the matrix unit's cut (it may differ by some
 * 1e-5 from what D's codes were made of).  With codes in both orders, D and D_t of a
 * backward call are the operands of the products that follow, each one product
 * over 2 F: the input's gradient (K = 2 F) and the weights' (2 F rows).
 *   a_fmt     FP8_E4M3; backward also FP8_E5M2.   b_fmt  FP8_E4M3.
 *   a_scaling, b_scaling  every combination of fp8_scaled_gemm; B's scales are
 *             those of its rows, all 2 F of them forward.
 *   act       as in fp8_scaled_gemm_ep (SiLU: SwiGLU, GELU: GEGLU, ReLU: ReGLU;
 *             none: the product of the two).
 *   bias [2 F], dbias [2 F]  param_dtype, optional.
 *   What the backward call needs of the forward one, g beside u, in either form;
 *   forward each is an optional output, backward one of them is the input:
 *   aux       [M][ldaux] BF16, 2 F columns.
 *   ck        [M][ldck] E4M3 codes, 2 F columns, and ck_exp [M][ldexp], 2 ceil(F /
 *             32) bytes: g's and u's as fp8_checkpoint_save writes each.
 *   workspace fp8_gated_linear_workspace(M, F, K, a_scaling, b_scaling, backward)
 *             bytes; calls that may run at the same time need one each.
 * Products of many rows are fastest (1.3 to 2 times) where F is a multiple of 32 (forward
 * with block scales: of 128) and every row of D, D_t, aux and ck starts on a multiple of 4
 * bytes, D_t's too: ldt a multiple of 4 where M is none.  (A product over the M tokens
 * takes D_t with its rows padded by zeros to a multiple of 16; what lies behind the M-th
 * code of a row is left as it was.)
 * No output may overlap an input.  K == 0 is a sum of nothing; M == 0 sets dbias
 * to 0.  Every pointer is memory of the current device, and the stream is one of its.
 * Errors: as fp8_scaled_gemm, and FP8_ERR_ARG (backward, act, param_dtype; a
 * bias in a backward call, dbias in a forward one; aux and ck both in a backward
 * one), FP8_ERR_NULL (one of ck and ck_exp alone; neither aux nor ck in a backward call;
 * workspace), FP8_ERR_SHAPE (ldd of a backward call, ldaux, ldck < 2 F, ldexp < 2
 * ceil(F / 32), a workspace that is too small), FP8_ERR_ALIGN,
 * FP8_ERR_UNSUPPORTED (other formats; gemm's accumulate; 256 * lda or 256 * ldb >=
 * 2^31; K > 65536; F > 2^26; more than 2^23 tiles of 128 x 128 of M x 2 F).
 * ---------------------------------------------------------------------- */
typedef struct {
  int backward;
  fp8_activation act;
  fp8_dtype param_dtype;
  const void* bias;
  void* aux; int64_t ldaux;
  uint8_t* ck; int64_t ldck;
  uint8_t* ck_exp; int64_t ldexp;
  void* dbias;
  void* workspace; int64_t workspace_bytes;
} fp8_gated_args;

int64_t fp8_gated_linear_workspace(int64_t M, int64_t F, int64_t K, fp8_scaling a_scaling, fp8_scaling b_scaling,
                                   int backward);
fp8_status fp8_gated_linear(const fp8_gemm_args* gemm, const fp8_gated_args* gated, hipStream_t stream);
/* Which kernel the call takes (see fp8_scaled_gemm_ep_plan). */
fp8_status fp8_gated_linear_plan(const fp8_gemm_args* gemm, const fp8_gated_args* gated, fp8_ep_plan* plan);

/* ------------------------------------------------------------------------
 * fp8_checkpoint_save, fp8_checkpoint_load -- a tensor that the backward pass
 * needs, kept in 8 bits: E4M3 codes and one power of two for every 32 columns of
 * a row (the last block of a row may be shorter), 8.25 bits a value.
 * save:  with a = max |x| of the block and e the largest integer with a 2^e <= 448,
 *   |e| <= 126 (0 for a block of zeros or one that holds an infinity or a NaN),
 *   ck = encode(x 2^e) as in fp8_cast_e4m3, ck_exp = 127 - e.
 * load:  y = value(ck) 2^(ck_exp - 127), rounded to nearest (exact in FP32 and, down
 *   to its smallest normal value, in BF16); ck_exp is an E8M0 number (255: NaN).
 *   x, y      [rows][ld] dtype.
 *   ck        [rows][ldck] codes.   ck_exp [rows][ldexp], ceil(cols / 32) bytes.
 * A value of a block without infinities or NaN is kept to 2^-4 of itself, to 2^-17 of
 * its block's largest or to 2^-136, whichever is most (the last only where the largest is
 * below 2^-119: e ends at 126; all of a block below 2^-136 is lost).  From 1.9375 2^127
 * on, a step from binary32's end, a value's code stands for 2^128, which load gives as an
 * infinity.  save's outputs may not overlap x, load's not ck or ck_exp.  Every pointer is
 * memory of the current device, and the stream is one of its.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE (negative size, ld < cols, ldexp < ceil(cols /
 * 32)), FP8_ERR_ARG (dtype), FP8_ERR_ALIGN (x, y: their element), FP8_ERR_UNSUPPORTED
 * (cols > 2^28).
 * ---------------------------------------------------------------------- */
fp8_status fp8_checkpoint_save(const void* x, fp8_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* ck,
                               int64_t ldck, uint8_t* ck_exp, int64_t ldexp, hipStream_t stream);
fp8_status fp8_checkpoint_load(const uint8_t* ck, int64_t ldck, const uint8_t* ck_exp, int64_t ldexp, int64_t rows,
                               int64_t cols, void* y, fp8_dtype dtype, int64_t ldy, hipStream_t stream);

/* ------------------------------------------------------------------------
 * fp8_rope -- rotary positions of the query and key heads of a QKV product.
 * Pair i < pairs of a head is (i, i + pairs) (FP8_ROPE_HALF) or (2i, 2i + 1)
 * (FP8_ROPE_INTERLEAVED); with theta = (position + offset) * freqs[i], reduced
 * in binary64,
 *   (x0, x1) -> scale * (x0 cos - x1 sin, x1 cos + x0 sin),
 * and elements 2 * pairs .. dim - 1 are copied.  inverse = 1 turns by -theta:
 * the gradient of the call with inverse = 0.
 *   q, k          [tokens][heads][dim] in dtype: unit stride inside a head,
 *                 strides of tokens and heads in elements (views of one QKV
 *                 tensor, for instance); k NULL: no key heads.
 *   q_out, k_out  the same shapes, strides of their own; may be q, k in place
 *                 (same pointer and strides), else no overlap.
 *   positions     [tokens] int32 or int64 (positions_i64); NULL: 0, 1, ...
 *   offset        added to every position.
 *   freqs         [pairs] binary64, as fp8_rope_freqs makes them.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE (negative sizes, 2 * pairs > dim),
 * FP8_ERR_ARG (enums), FP8_ERR_ALIGN, FP8_ERR_UNSUPPORTED (pairs > 1024, dim,
 * q_heads + k_heads > 65535, tokens > 2^23).
 * ---------------------------------------------------------------------- */
typedef enum { FP8_ROPE_HALF = 0, FP8_ROPE_INTERLEAVED = 1 } fp8_rope_layout;

typedef struct {
  int64_t tokens, q_heads, k_heads, dim, pairs;
  fp8_dtype dtype; fp8_rope_layout layout;
  int inverse;
  float scale;
  const double* freqs;
  const void* positions; int positions_i64; int64_t offset;
  const void* q; int64_t q_token_stride, q_head_stride;
  const void* k; int64_t k_token_stride, k_head_stride;
  void* q_out; int64_t q_out_token_stride, q_out_head_stride;
  void* k_out; int64_t k_out_token_stride, k_out_head_stride;
} fp8_rope_args;

fp8_status fp8_rope(const fp8_rope_args* args, hipStream_t stream);

/* fp8_rope_freqs -- the frequencies, once per model: freqs[i] = base^(-i /
 * pairs), i < pairs, scaled for contexts beyond the trained length:
 *   FP8_ROPE_PLAIN   as they are;
 *   FP8_ROPE_LINEAR  divided by factor (positions interpolated);
 *   FP8_ROPE_BASE    base replaced by base * factor^(pairs / (pairs - 1)): the
 *                    fastest pair is left, the slowest divided by factor;
 *   FP8_ROPE_PARTS   f keep + f / factor (1 - keep), keep = clamp((trained f /
 *                    (2 pi) - low) / (high - low), 0, 1): pairs that turn
 *                    more than `high` times over the trained length are left,
 *                    those that turn less than `low` times interpolated.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE (pairs < 0), FP8_ERR_ALIGN, FP8_ERR_ARG
 * (enum; base, factor or trained not positive and finite; high <= low). */
typedef enum {
  FP8_ROPE_PLAIN = 0, FP8_ROPE_LINEAR = 1, FP8_ROPE_BASE = 2, FP8_ROPE_PARTS = 3
} fp8_rope_scaling;

fp8_status fp8_rope_freqs(double* freqs, int64_t pairs, double base, fp8_rope_scaling scaling,
                          double factor, double trained, double low, double high,
                          hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8LIN_H */
