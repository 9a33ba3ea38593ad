// gemm_ep_tile.h -- the FP8 product with the linear's epilogue on tiles of
// BM x BN, for outputs that the 256 x 256 tiles of the large kernels would not
// spread over the card; instantiated by gemm_ep_tile.hip (which also
// holds the dispatch), gemm_ep_tile_fp8out.hip and, for promoted block scales,
// gemm_ep_tile_blk.hip and gemm_ep_tile_blk_fp8out.hip.
//
// A workgroup of four wavefronts takes one tile and, where tiles alone would
// leave compute units idle, one of `splits` parts of K; the parts' binary32
// sums go to the workspace and k_ep_join adds them in order and applies the
// epilogue.  Operands come through LDS in steps of 128 bytes of K, STAGES
// stages deep, by buffer loads straight into LDS (layout, swizzle and
// fragments as in gemm_big_kernel.h); rows past an operand's end fail the
// buffer's range check and read zeros, and so do chunks past K.
// Scales (MODE): per-tensor and per-row ones are applied to the whole sum.  Block
// scales arrive in LDS with the operands, one per row of the step: powers of two go
// into the matrix instruction (EP_MX); others promote each step's product into the
// binary32 accumulator, by the row's scale times the tile's one scale of B (EP_BLK:
// B's columns lie in one 128 x 128 block) or each column's (EP_BLKCOL).
//
// Bound: the latency of a step between its barriers (0.44 us at 64 rows and one
// workgroup per compute unit, of which the products are 0.12).  Measured on an MI355X:
// 300 x 14336 x 4096 with SiLU and pre-activation 32.9 us, 1.07 PFLOP/s; 256 x 8192 x
// 8192 per-tensor 35 us, power-of-two scales 41, promoted 40; backward 1037 x 1999 x
// 2304 24 us, of which the bias gradient's join is 4.
#pragma once

#include "gemm_big_kernel.h"
#include "gemm_ep.h"

namespace fp8lin {

namespace {

constexpr int EP_THREADS = 256;
enum : int { EP_SUM = 0, EP_BLK = 1, EP_BLKCOL = 2, EP_MX = 3 };

// One step's scale of an operand's row: the inverse scales' base and the row's
// offset in it.
__device__ __forceinline__ int64_t scale_base(int scaling, int64_t rows, int64_t kb) {
  return scaling == 0 ? 0 : (scaling == 1 ? kb * rows : kb * ((rows + 127) / 128));
}
__device__ __forceinline__ int64_t scale_row(int scaling, int64_t row) {
  return scaling == 0 ? 0 : (scaling == 1 ? row : row / 128);
}

// WM x WN wavefronts of (16 TI) x (16 TJ).
template <int AF, int BF, int MODE, bool OUT8, int WM, int WN, int TI, int TJ, int STAGES>
__global__ void __launch_bounds__(EP_THREADS) __attribute__((amdgpu_waves_per_eu(STAGES < 4 ? 2 : 1))) k_ep_tile(GemmParams p, EpParams e, int tiles_m, int tiles_n) {
  constexpr int BM_ = 16 * TI * WM, BN_ = 16 * TJ * WN;
  constexpr bool BLOCK = MODE != EP_SUM;
  static_assert(WM * WN == 4 && BM_ % 32 == 0 && BN_ % 32 == 0, "four wavefronts");
  constexpr int ABYTES = BM_ * BK, BBYTES = BN_ * BK;
  constexpr int SCALES = BLOCK ? 4 * ((BM_ + 63) / 64 * 64 + (BN_ + 63) / 64 * 64) : 0;
  constexpr int SA0 = ABYTES + BBYTES, SB0 = SA0 + (BM_ + 63) / 64 * 64 * 4;
  constexpr int STAGE_ = ABYTES + BBYTES + SCALES;
  constexpr int WREG = EpWave<16 * TJ, OUT8, EP_ANY, false>::bytes(TI) > EpWave<16 * TJ, false, EP_ANY, false>::bytes(TI)
                           ? EpWave<16 * TJ, OUT8, EP_ANY, false>::bytes(TI) : EpWave<16 * TJ, false, EP_ANY, false>::bytes(TI);
  constexpr int LDS_ = STAGES * STAGE_ > 4 * WREG ? STAGES * STAGE_ : 4 * WREG;
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS_];
  __shared__ float rs_tab[BLOCK ? 1 : BM_ + BN_];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t M = p.M, N = p.N, K = p.K;

  // tile id as in the large kernels: contiguous runs per XCD, 8 tile-rows at a time
  const int nblk = tiles_m * tiles_n;
  int bid = blockIdx.x;
  if ((nblk & 7) == 0) bid = (bid & 7) * (nblk >> 3) + (bid >> 3);
  const int group = bid / (GROUP_M * tiles_n), first_m = group * GROUP_M;
  const int gm = min(tiles_m - first_m, GROUP_M), in_group = bid - group * GROUP_M * tiles_n;
  const int tm = first_m + in_group % gm, tn = in_group / gm;
  const int64_t m0 = (int64_t)tm * BM_, n0 = (int64_t)tn * BN_;
  const int64_t rows_a = min((int64_t)BM_, M - m0), rows_b = min((int64_t)BN_, N - n0);
  const i32x4 ra = make_rsrc(p.A + m0 * p.lda, (uint32_t)(rows_a * p.lda));
  const i32x4 rb = make_rsrc(p.B + n0 * p.ldb, (uint32_t)(rows_b * p.ldb));
  const int lda = (int)p.lda, ldb = (int)p.ldb;

  // this workgroup's part of the K steps
  const int nk_all = (int)((K + BK - 1) / BK);
  const int z = blockIdx.y;
  const int kb0 = (int)((int64_t)nk_all * z / e.splits), kb1 = (int)((int64_t)nk_all * (z + 1) / e.splits);

  // Block scales of a stage: chunks of 64 rows' scales, A's then B's, PER of them
  // per wavefront (the last may be fetched twice).  Only the base moves from step to
  // step: worked out there, the addresses held every step up by 0.45 us.
  constexpr int CA = (BM_ + 63) / 64, CB = (BN_ + 63) / 64, PER = BLOCK ? (CA + CB + 3) / 4 : 1;
  const uint8_t* sc_base[PER];
  int64_t sc_step[PER];
  uint32_t sc_bytes[PER], sc_off[PER], sc_lds[PER];
  if constexpr (BLOCK) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int ch = min(wave * PER + u, CA + CB - 1);
      const bool a = ch < CA;
      const int sc = a ? p.a_scaling : p.b_scaling, r = 64 * (a ? ch : ch - CA) + lane;
      const int64_t rows = a ? M : N, r0 = a ? m0 : n0, first = scale_row(sc, r0), last = scale_row(sc, rows - 1);
      sc_base[u] = reinterpret_cast<const uint8_t*>((a ? p.a_sinv : p.b_sinv) + first);
      sc_step[u] = scale_base(sc, rows, 1) * 4;
      sc_bytes[u] = (uint32_t)min(4 * (last - first + 1), (int64_t)2048);   // (at most 128 + 64 rows' are read)
      sc_off[u] = (uint32_t)(4 * (min(scale_row(sc, r0 + r), last) - first));
      sc_lds[u] = (uint32_t)((a ? SA0 : SB0) + 256 * (a ? ch : ch - CA));
    }
  }

  // a wavefront's share of a stage: 8 rows per instruction
  constexpr int QA = BM_ / 32, QB = BN_ / 32;
  auto load = [&](int kb, int stage) {
    const uint32_t base = lds_addr(lds) + stage * STAGE_;
#pragma unroll
    for (int it = 0; it < QA + QB; ++it) {
      const bool a = it < QA;
      const int row = (a ? (BM_ / 4) * wave + 8 * it : (BN_ / 4) * wave + 8 * (it - QA)) + (lane >> 3);
      const int kc = kb * BK + 16 * ((lane & 7) ^ swz(row));
      const uint32_t dst =
          base + (a ? 0 : ABYTES) + ((a ? (BM_ / 4) * wave + 8 * it : (BN_ / 4) * wave + 8 * (it - QA))) * BK;
      dma16(dst, kc < (int)K ? (uint32_t)(row * (a ? lda : ldb)) + (uint32_t)kc : kOOB, a ? ra : rb);
    }
    if constexpr (BLOCK) {
#pragma unroll
      for (int u = 0; u < PER; ++u)
        dma4(base + sc_lds[u], sc_off[u], make_rsrc(sc_base[u] + kb * sc_step[u], sc_bytes[u]));
    }
  };

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  if constexpr (!BLOCK) {
    for (int r = tid; r < BM_ + BN_; r += EP_THREADS) {
      const bool a = r < BM_;
      const int64_t row = min((a ? m0 + r : n0 + r - BM_), (a ? M : N) - 1);
      const bool per_row = (a ? p.a_scaling : p.b_scaling) == 5;
      rs_tab[r] = K > 0 ? (a ? p.a_sinv : p.b_sinv)[per_row ? row : 0] : 0.0f;
    }
  }

  // STAGES - 1 stages ahead; a step waits for its own stage only (the stages after
  // it were issued later, PL instructions each, and may still be on their way).
  constexpr int PL = QA + QB + (BLOCK ? PER : 0);
  static_assert((STAGES - 2) * PL < 64, "counter of outstanding loads");
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (kb0 + s < kb1) load(kb0 + s, s);
  // What the epilogue reads beside the product is on its way from here on: fetched
  // strip by strip after the sums, it held a 64 x 128 tile up by 4 us.
  const int64_t r0 = m0 + wm * 16 * TI, c0 = n0 + wn * 16 * TJ;
  using W = EpWave<16 * TJ, OUT8, EP_ANY, false>;
  W w(p, e, c0, lane);
  constexpr int AHEAD = TI <= 2 ? TI : 1;
  typename W::Words src[AHEAD][W::RPL];
  if (e.splits == 1) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) w.fetch(r0 + 16 * i, src[i]);
  }
  // EP_MX: a per-tensor operand's exponent is 127 (its scale is applied to the sum).  By
  // masks: as a choice, each scale's read was a branch of its own that waited for LDS,
  // 0.24 us per step.
  const int keep_a = p.a_scaling == 0 ? 0 : 255, one_a = p.a_scaling == 0 ? 127 : 0;
  const int keep_b = p.b_scaling == 0 ? 0 : 255, one_b = p.b_scaling == 0 ? 127 : 0;
  int st = 0;
  for (int kb = kb0; kb < kb1; ++kb, st = st + 1 == STAGES ? 0 : st + 1) {
    // Every wavefront's share of this step's stage has to be in LDS, and every
    // wavefront done with the stage that the next load fills.
    if (kb + STAGES - 2 < kb1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((STAGES - 2) * PL) : "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    if (kb + STAGES - 1 < kb1) load(kb + STAGES - 1, st == 0 ? STAGES - 1 : st - 1);
    const uint8_t* S = lds + st * STAGE_;
    v8i b[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) b[j] = frag(S + ABYTES, wn * 16 * TJ + 16 * j + l16, g);
    float4 sb[MODE == EP_BLKCOL ? TJ : 1];
    int eb[MODE == EP_MX ? TJ : 1];
    float sb0 = 1.0f;
    if constexpr (MODE == EP_BLK) sb0 = *reinterpret_cast<const float*>(S + SB0);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const uint8_t* at = S + SB0 + 4 * (wn * 16 * TJ + 16 * j);
      if constexpr (MODE == EP_BLKCOL) sb[j] = *reinterpret_cast<const float4*>(at + 16 * g);
      if constexpr (MODE == EP_MX) eb[j] = (e8m0_of(*reinterpret_cast<const float*>(at + 4 * l16)) & keep_b) | one_b;
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int row = wm * 16 * TI + 16 * i + l16;
      const v8i a = frag(S, row, g);
      float sa = 1.0f;
      if constexpr (BLOCK) sa = *reinterpret_cast<const float*>(S + SA0 + 4 * row);
      if constexpr (MODE == EP_BLK) sa *= sb0;
      const int ea = MODE == EP_MX ? (e8m0_of(sa) & keep_a) | one_a : 127;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if constexpr (MODE == EP_SUM) {
          acc[i][j] = mfma<BF, AF>(b[j], a, acc[i][j]);
        } else if constexpr (MODE == EP_MX) {
          acc[i][j] = mfma_mx<BF, AF>(b[j], a, acc[i][j], eb[j], ea);
        } else {
          const v4f part = mfma<BF, AF>(b[j], a, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (MODE == EP_BLK) acc[i][j][q] = __builtin_fmaf(part[q], sa, acc[i][j][q]);
            else {
              const float c = q == 0 ? sb[j].x : (q == 1 ? sb[j].y : (q == 2 ? sb[j].z : sb[j].w));
              acc[i][j][q] = __builtin_fmaf(part[q] * sa, c, acc[i][j][q]);
            }
          }
        }
      }
    }
  }
  __syncthreads();   // the stages are free for the epilogue, rs_tab is written

  float ta = 1.0f, tb = 1.0f;   // EP_MX: a per-tensor operand's scale (without K there may be none)
  if constexpr (MODE == EP_MX) {
    if (p.a_scaling == 0 && K > 0) ta = p.a_sinv[0];
    if (p.b_scaling == 0 && K > 0) tb = p.b_sinv[0];
  }
  auto deq = [&](int i, int j, int q, float x) -> float {
    if constexpr (MODE == EP_BLK || MODE == EP_BLKCOL) return x;
    else if constexpr (MODE == EP_MX) return (x * ta) * tb;
    else
      return (x * rs_tab[wm * 16 * TI + 16 * i + l16]) * rs_tab[BM_ + wn * 16 * TJ + 16 * j + 4 * g + q];
  };
  uint8_t* wl = lds + wave * WREG;
  if (e.splits > 1) {   // this part's sums, [split][M][ldw]
    EpParams es = {};
    es.splits = 1;
    GemmParams ps = p;
    ps.D = e.sums + (int64_t)z * M * e.ldw;
    ps.ldd = e.ldw;
    ps.d_f32 = 1;
    ps.d_amax = nullptr;
    EpWave<16 * TJ, false, EP_FWD, false> ws(ps, es, c0, lane);
    ws.template tile<TI, TJ>(acc, deq, r0, c0, wl);
    return;
  }
  w.template tile<TI, TJ>(acc, deq, r0, c0, wl, src);
  w.put_dbias((int64_t)tm * WM + wm);   // (rows of the sum: WM per tile-row)
  if (p.d_amax) ep_amax<4>(p.d_amax, w.amax_bits(), lane, wave);
}

template <int AF, int BF, int MODE, bool OUT8>
hipError_t launch_tile(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  const int tiles_m = (int)((p.M + plan.bm - 1) / plan.bm), tiles_n = (int)((p.N + plan.bn - 1) / plan.bn);
  const dim3 grid((unsigned)(tiles_m * tiles_n), (unsigned)plan.splits), block(EP_THREADS);
#define FP8LIN_TILE(...) \
  hipLaunchKernelGGL((k_ep_tile<AF, BF, MODE, OUT8, __VA_ARGS__>), grid, block, 0, s, p, e, tiles_m, tiles_n)
  if (plan.bm == 32) FP8LIN_TILE(1, 4, 2, 2, 6);
  else if (plan.bm == 64) FP8LIN_TILE(2, 2, 2, 4, 3);
  else FP8LIN_TILE(2, 2, 4, 4, 2);
#undef FP8LIN_TILE
  return hipGetLastError();
}

template <int MODE, bool OUT8>
hipError_t launch_tile_fmt(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  if (p.a_fmt == 0 && p.b_fmt == 0) return launch_tile<0, 0, MODE, OUT8>(p, e, plan, s);
  if (p.a_fmt == 1 && p.b_fmt == 0) return launch_tile<1, 0, MODE, OUT8>(p, e, plan, s);
  if (p.a_fmt == 0 && p.b_fmt == 1) return launch_tile<0, 1, MODE, OUT8>(p, e, plan, s);
  return launch_tile<1, 1, MODE, OUT8>(p, e, plan, s);
}

// Per-tensor, per-row and power-of-two block scales: no promotion.
template <bool OUT8>
hipError_t launch_tile_sum(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  const bool per_a = p.a_scaling == 0 || p.a_scaling == 5, per_b = p.b_scaling == 0 || p.b_scaling == 5;
  return per_a && per_b ? launch_tile_fmt<EP_SUM, OUT8>(p, e, plan, s) : launch_tile_fmt<EP_MX, OUT8>(p, e, plan, s);
}
// Other block scales.
template <bool OUT8>
hipError_t launch_tile_blk(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  return p.b_scaling == 1 ? launch_tile_fmt<EP_BLKCOL, OUT8>(p, e, plan, s) : launch_tile_fmt<EP_BLK, OUT8>(p, e, plan, s);
}

}  // namespace

}  // namespace fp8lin
