// gemm_ep_skinny.h -- the FP8 product with the linear's epilogue for few rows of
// A (up to 16), where the weights' bytes are the work; instantiated by
// gemm_ep_skinny.hip and gemm_ep_skinny_fp8out.hip.
//
// A workgroup owns 32 columns; its eight wavefronts take every eighth 128-byte
// step of K each.  Weights go from memory straight into the registers that feed
// the matrix instruction: lane (g, l16) reads 16 bytes at 16 g and 16 at
// 64 + 16 g of row l16, so the four lanes of a row read 64 bytes in a piece, and A's
// fragments (from L2: A is small and shared) take the same bytes of K.  U steps are in flight per wavefront, each
// reloaded as soon as its products are issued, so a compute unit keeps
// 8 U 4 KB = 128 KB of weights under way; there is no barrier until the end, where
// the wavefronts' sums are added in order through LDS and one wavefront applies the
// epilogue.  No part of K goes to another workgroup: even 32
// workgroups (1024 columns) can draw more than memory gives, and the join of
// parts through memory would be a second launch.
//
// Bound: HBM.  Measured on an MI355X, per-row scales, bias and residual: one token,
// 8192 x 8192, 18.4 us, 3.6 TB/s; 28672 x 8192 53 us, 4.4 TB/s; 16 tokens, 8192 x
// 8192, 19.9 us.
#pragma once

#include "gemm_big_kernel.h"
#include "gemm_ep.h"

namespace fp8lin {

namespace {

constexpr int SK_WAVES = 8, SK_COLS = 32;

// Address of a row's inverse scale of K block kb; step: what it moves per block.
__device__ __forceinline__ const float* scale_ptr(int scaling, const float* s, int64_t rows, int64_t row, int64_t& step) {
  step = scaling == 0 ? 0 : (scaling == 1 ? rows : (rows + 127) / 128);
  return s + (scaling == 0 ? 0 : (scaling == 1 ? row : row / 128));
}

// BLOCK: block scales, promoted into binary32 per step;
// SBCOL: B's differ by column (1x128 segments), else one per step.  OP: whose
// epilogue; a PAIRED one's 32 columns are 16 rows of B's one factor and 16 of the
// other, so a workgroup makes 16 outputs (one scale per step: of each factor).
template <int AF, int BF, bool BLOCK, bool SBCOL, bool OUT8, typename OP = LinearOp>
__global__ void __launch_bounds__(SK_WAVES * 64) k_ep_skinny(GemmParams p, typename OP::Params e) {
  constexpr int NT = SK_COLS / 16, U = 4;
  constexpr bool PAIRED = OP::PAIRED;
  using W = typename OP::template Wave<SK_COLS, OUT8>;
  constexpr int TS = 32, EPB = W::bytes(1), SUMS = 16 * SK_COLS * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[SK_WAVES * SUMS + EPB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t M = p.M, N = p.N, n0 = (int64_t)blockIdx.x * (PAIRED ? SK_COLS / 2 : SK_COLS);
  auto b_row = [&](int c) -> int64_t {   // B's row of column c
    if constexpr (PAIRED) return half_of(c) * N + min(n0 + pair_of(c), N - 1);
    else return min(n0 + c, N - 1);
  };
  const int nk = (int)((p.K + BK - 1) / BK), K = (int)p.K;

  const uint8_t* arow = p.A + min((int64_t)l16, M - 1) * p.lda + 16 * g;
  const uint8_t* brow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) brow[j] = p.B + b_row(16 * j + l16) * p.ldb + 16 * g;
  // block scales: A's of this lane's row, B's of its 4 columns or of the block
  const float* asc = nullptr;
  const float* bsc[NT][SBCOL ? 4 : 1];
  int64_t astep = 0, bstep = 0;
  if constexpr (BLOCK) {
    asc = scale_ptr(p.a_scaling, p.a_sinv, M, min((int64_t)l16, M - 1), astep);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < (SBCOL ? 4 : 1); ++q)
        bsc[j][q] = scale_ptr(p.b_scaling, p.b_sinv, PAIRED ? 2 * N : N,
                              SBCOL ? b_row(16 * j + 4 * g + q) : (PAIRED ? j * N + n0 : n0), bstep);
  }

  struct Step {
    v8i a, b[NT];
    float sa, sb[BLOCK ? NT : 1][SBCOL ? 4 : 1];
  };
  auto line = [&](const uint8_t* row, int k) -> v8i {   // zeros past K (a multiple of 16)
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (k + 16 * g < K) lo = *reinterpret_cast<const uint4*>(row + k);
    if (k + 16 * g + 64 < K) hi = *reinterpret_cast<const uint4*>(row + k + 64);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  auto whole = [&](const uint8_t* row, int k) -> v8i {
    const uint4 lo = *reinterpret_cast<const uint4*>(row + k), hi = *reinterpret_cast<const uint4*>(row + k + 64);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  auto load = [&](int kb, Step& s) {
    const int k = kb * BK;
    if (k + BK <= K) {
#pragma unroll
      for (int j = 0; j < NT; ++j) s.b[j] = whole(brow[j], k);
      s.a = whole(arow, k);
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) s.b[j] = line(brow[j], k);
      s.a = line(arow, k);
    }
    if constexpr (BLOCK) {
      s.sa = asc[kb * astep];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < (SBCOL ? 4 : 1); ++q) s.sb[j][q] = bsc[j][q][kb * bstep];
    }
  };
  v4f acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Step& s) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (BLOCK) {
        const v4f part = mfma<BF, AF>(s.b[j], s.a, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = __builtin_fmaf(part[q] * s.sa, s.sb[j][SBCOL ? q : 0], acc[j][q]);
      } else {
        acc[j] = mfma<BF, AF>(s.b[j], s.a, acc[j]);
      }
    }
  };
  Step ring[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (wave + u * SK_WAVES < nk) load(wave + u * SK_WAVES, ring[u]);
  for (int kb = wave; kb < nk; kb += U * SK_WAVES) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int now = kb + u * SK_WAVES, next = now + U * SK_WAVES;
      if (now < nk) {
        use(ring[u]);
        if (next < nk) load(next, ring[u]);
      }
    }
  }

  // the wavefronts' sums, each [16][32], then the rows' epilogue by the first, whose
  // scales, bias and residual are on their way before the wavefronts meet
  float* mine = reinterpret_cast<float*>(lds + wave * SUMS);
  uint32_t top = 0;
  W w(p, e, (int64_t)blockIdx.x * SK_COLS, lane);
  static_assert(W::RPL == 1, "a lane has one row of 8 columns");
  const int r = lane / (SK_COLS / 8), c8 = lane % (SK_COLS / 8);   // the row and 8 columns it adds up
  typename W::Words o[1];
  float sa = 0.0f, sb[8] = {};
  if (wave == 0) {
    w.fetch(0, o);
    if (!BLOCK && K > 0) {
      sa = p.a_sinv[p.a_scaling == 5 ? min((int64_t)r, M - 1) : 0];
#pragma unroll
      for (int k = 0; k < 8; ++k) sb[k] = p.b_sinv[p.b_scaling == 5 ? b_row(8 * c8 + k) : 0];
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
    *reinterpret_cast<float4*>(mine + l16 * SK_COLS + 16 * j + 4 * g) =
        make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  if (wave == 0) {
    uint8_t* wl = lds + SK_WAVES * SUMS;
    float v[8] = {};
#pragma unroll
    for (int s = 0; s < SK_WAVES; ++s) {
      const float4* q = reinterpret_cast<const float4*>(lds + s * SUMS) + (r * SK_COLS + 8 * c8) / 4;
      const float4 a = q[0], b = q[1];
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    if constexpr (!BLOCK) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = (v[k] * sa) * sb[k];
    }
    *w.place(wl, r, 2 * c8) = make_float4(v[0], v[1], v[2], v[3]);
    *w.place(wl, r, 2 * c8 + 1) = make_float4(v[4], v[5], v[6], v[7]);
    w.stage(0, o, wl + W::src_at);
    w.template rows<TS>(0, wl, wl + W::src_at, wl + W::codes_at, 0);
    if constexpr (OUT8) {
      if (p.D_t) w.template flush_t<TS, 16>(wl + W::codes_at, 0, (int64_t)blockIdx.x * SK_COLS);
    }
    w.put_dbias(0);
    top = w.amax_bits();
  }
  if (p.d_amax) ep_amax<SK_WAVES>(p.d_amax, top, lane, wave);
}

template <int AF, int BF, bool OUT8, typename OP = LinearOp>
hipError_t launch_skinny_f(const GemmParams& p, const typename OP::Params& e, hipStream_t s) {
  const int64_t columns = OP::PAIRED ? paired_columns(p.N) : p.N;
  const dim3 grid((unsigned)((columns + SK_COLS - 1) / SK_COLS)), block(SK_WAVES * 64);
  const bool blk = !((p.a_scaling == 0 || p.a_scaling == 5) && (p.b_scaling == 0 || p.b_scaling == 5));
  // (16 columns of the second factor lie in one 128 x 128 block if it starts at a multiple of 16)
  const bool by_column = p.b_scaling == 1 || (OP::PAIRED && p.b_scaling == 2 && p.N % 16 != 0);
  if (!blk) hipLaunchKernelGGL((k_ep_skinny<AF, BF, false, false, OUT8, OP>), grid, block, 0, s, p, e);
  else if (by_column) hipLaunchKernelGGL((k_ep_skinny<AF, BF, true, true, OUT8, OP>), grid, block, 0, s, p, e);
  else hipLaunchKernelGGL((k_ep_skinny<AF, BF, true, false, OUT8, OP>), grid, block, 0, s, p, e);
  return hipGetLastError();
}
template <bool OUT8>
hipError_t launch_skinny_out(const GemmParams& p, const EpParams& e, hipStream_t s) {
  if (p.a_fmt == 0 && p.b_fmt == 0) return launch_skinny_f<0, 0, OUT8>(p, e, s);
  if (p.a_fmt == 1 && p.b_fmt == 0) return launch_skinny_f<1, 0, OUT8>(p, e, s);
  if (p.a_fmt == 0 && p.b_fmt == 1) return launch_skinny_f<0, 1, OUT8>(p, e, s);
  return launch_skinny_f<1, 1, OUT8>(p, e, s);
}

}  // namespace

}  // namespace fp8lin
