// gemm_ep_tile.hip -- the FP8 product with the linear's epilogue: its tile
// kernels, the join of K parts, the bias gradient's join and the dispatch.
#include "gemm_ep_tile.h"

namespace fp8lin {

namespace {

// The parts' sums added in order, then the epilogue: a wavefront takes 16 rows of
// 32 columns (one row of 8 columns per lane), a workgroup 16 rows of 128.
template <bool OUT8>
__global__ void __launch_bounds__(256) k_ep_join(GemmParams p, EpParams e) {
  constexpr int TS = 32;
  using W = EpWave<32, OUT8, EP_ANY, false>;
  constexpr int BYTES = W::bytes(1);
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * BYTES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * 128 + 32 * wave, m0 = (int64_t)blockIdx.y * 16;
  uint8_t* wl = lds + wave * BYTES;
  W w(p, e, n0, lane);
  typename W::Words o[1];
  w.fetch(m0, o);
  const int64_t m = m0 + w.rg;
  float v[8] = {};
  if (w.nv > 0 && m < p.M) {   // (rows of the sums are padded to whole vectors)
    const float* s = e.sums + m * e.ldw + w.c;
    const int64_t next = p.M * e.ldw;
#pragma unroll 8
    for (int z = 0; z < e.splits; ++z) {
      const float4 a = *reinterpret_cast<const float4*>(s + z * next), b = *reinterpret_cast<const float4*>(s + z * next + 4);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
  }
  *w.place(wl, w.rg, 2 * w.cq) = make_float4(v[0], v[1], v[2], v[3]);
  *w.place(wl, w.rg, 2 * w.cq + 1) = make_float4(v[4], v[5], v[6], v[7]);
  w.stage(m0, o, wl + W::src_at);
  w.template rows<TS>(m0, wl, wl + W::src_at, wl + W::codes_at, 0);
  if constexpr (OUT8) {
    if (p.D_t) w.template flush_t<TS, 16>(wl + W::codes_at, m0, n0);
  }
  w.put_dbias(blockIdx.y);
  if (p.d_amax) ep_amax<4>(p.d_amax, w.amax_bits(), lane, wave);
}

// dbias[n] = sum of the parts' column sums, 64 columns by 16 parts at a time,
// in a fixed order.
__global__ void __launch_bounds__(1024) k_ep_dbias(const float* part, int64_t parts, int64_t N, void* dbias, int f32) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (n < N)
    for (int64_t q = wave; q < parts; q += 16) s += part[q * N + n];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || n >= N) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += lds[w][lane];
  if (f32) reinterpret_cast<float*>(dbias)[n] = s;
  else reinterpret_cast<uint16_t*>(dbias)[n] = f32_to_bf16_rne(s);
}

}  // namespace

namespace {

// Times (us) of one 128-byte step of K, measured with every compute unit busy: a
// workgroup alone on its compute unit, and two of them (the 32-row tiles' stages
// fill its LDS).  Without and with block scales (measured with promoted ones, taken for
// powers of two as well); 256: the large kernels with their own formats.  (The tiles'
// steps with block scales have since become some 20% shorter; scaled by that, the
// choices were 0.7% slower on average over 135 products, 19% at worst, so these stay:
// they rank the cuts and no longer are what a step takes.)
struct TileCost {
  int bm;
  float alone, two;
};
constexpr TileCost kCost[2][4] = {{{32, 0.35f, 0.0f}, {64, 0.44f, 0.64f}, {128, 0.74f, 0.95f}, {256, 1.45f, 0.0f}},
                                  {{32, 0.50f, 0.0f}, {64, 0.66f, 0.92f}, {128, 1.15f, 1.50f}, {256, 1.75f, 0.0f}}};

// What a product takes on tiles of c.bm rows with K in `splits` parts: a launch
// and an epilogue, rounds of as many workgroups as run at once, and for parts a
// second launch and the sums' way through memory.
float tile_time(const TileCost& c, int64_t M, int64_t N, int64_t nk, int splits, int64_t cu) {
  const int64_t bn = c.bm == 256 ? 256 : 128;
  const int64_t wgs = (M + c.bm - 1) / c.bm * ((N + bn - 1) / bn) * splits;
  const int64_t at_once = c.two > 0.0f ? 2 * cu : cu, full = wgs / at_once, rest = wgs - full * at_once;
  const float round = c.two > 0.0f ? c.two : c.alone;
  const float steps = (float)((nk + splits - 1) / splits);
  float t = 5.0f + steps * ((float)full * round + (rest == 0 ? 0.0f : (rest <= cu ? c.alone : round)));
  if (splits > 1) t += 5.0f + (float)(splits * M * N) * 8.0f / 3.5e6f;
  return t;
}
int64_t tile_parts(int64_t M, int bm) { return (M + bm - 1) / bm * (bm == 32 ? 1 : 2); }

}  // namespace

// Up to 16 rows: the few-row kernel (16 x 8192 x 8192: 19.9 us against 26 on
// tiles).  Beyond: the cut that the measured steps above make shortest.  Over 72
// products (48 to 1500 rows, 1024 to 14336 columns, K 2304 to 8192, per-tensor and
// block scales) it took 2% more than the fastest of all cuts on average, 24% at
// worst (300 x 1024 x 4096, 16.1 us against 13.0).
EpPlan ep_plan(const GemmParams& p) {
  EpPlan plan = {};
  const bool per_a = p.a_scaling == 0 || p.a_scaling == 5, per_b = p.b_scaling == 0 || p.b_scaling == 5;
  const bool layer = per_a ? per_b : p.a_scaling == 1 ? p.b_scaling == 2 : p.a_scaling == 3 ? p.b_scaling == 4 : false;
  const int64_t cu = device_cu_count(), nk = (p.K + BK - 1) / BK;
  const bool parts = (p.M + 15) / 16 <= 65535;   // the join's grid: 16 rows per workgroup in y
  plan.skinny = p.M <= 16;
  plan.bm = 32;
  plan.bn = 128;
  plan.splits = 1;
  if (!plan.skinny) {
    const TileCost* cost = kCost[per_a && per_b ? 0 : 1];
    float best = 0.0f;
    for (int i = 0; i < 3; ++i)
      for (int splits = 1; splits <= 16 && (splits == 1 || (parts && nk / splits >= 2)); splits *= 2) {
        const float t = tile_time(cost[i], p.M, p.N, nk, splits, cu);
        if (best != 0.0f && t >= best) continue;
        best = t;
        plan.bm = cost[i].bm;
        plan.splits = splits;
      }
    plan.large = layer && p.K > 0 && tile_time(cost[3], p.M, p.N, nk, 1, cu) < best;
  }
  // Rows of column sums: the wavefronts' of the tiles, of the join or of the
  // few-row kernel; room for the tiles' too where a product of the large kernels'
  // size may run on them (large_takes).
  const int64_t tiled = plan.splits > 1 || plan.skinny ? (p.M + 15) / 16 : tile_parts(p.M, plan.bm);
  const int64_t large = plan.large ? (p.M + 255) / 256 * 2 : 0;
  plan.parts = tiled;
  plan.large_parts = large;
  plan.ldw = (p.N + 7) / 8 * 8;
  plan.part_bytes = ((tiled > large ? tiled : large) * p.N * 4 + 255) / 256 * 256;
  plan.sums_bytes = plan.splits > 1 ? plan.splits * p.M * plan.ldw * 4 : 0;
  return plan;
}

namespace {
// The large kernels' formats, and rows of whole vectors that start on a dword
// (see FAST in gemm_ep.h).
bool large_takes(const GemmParams& p, const EpParams& e) {
  auto dwords = [](const void* q, int64_t ld, int size) {
    return q == nullptr || (((reinterpret_cast<uintptr_t>(q) & 3u) == 0) && ((ld * size) & 3) == 0);
  };
  return p.b_fmt == 0 && p.a_fmt == e.backward && p.N % 8 == 0 &&
         dwords(p.D, p.ldd, p.d_fp8 ? 1 : (p.d_f32 ? 4 : 2)) && dwords(e.aux, e.ldaux, 2) &&
         dwords(e.residual, e.ldres, e.res_f32 ? 4 : 2);
}
}  // namespace

EpPlan ep_plan(const GemmParams& p, const EpParams& e) {
  EpPlan plan = ep_plan(p);
  plan.large = plan.large && large_takes(p, e);
  if (plan.large) {
    plan.splits = 1;
    plan.parts = plan.large_parts;
  }
  return plan;
}

hipError_t launch_gemm_ep_tile(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  return launch_tile_sum<false>(p, e, plan, s);
}

hipError_t launch_gemm_ep(const GemmParams& p0, EpParams e, uint8_t* ws, hipStream_t s) {
  GemmParams p = p0;
  if (p.d_amax && !p.amax_acc) {
    const hipError_t err = launch_fill_u32(reinterpret_cast<uint32_t*>(p.d_amax), 1, 0u, s);
    if (err != hipSuccess) return err;
  }
  if (p.N == 0) return hipSuccess;
  const EpPlan plan = ep_plan(p, e);
  e.part = reinterpret_cast<float*>(ws);
  e.sums = reinterpret_cast<float*>(ws + plan.part_bytes);
  e.ldw = plan.ldw;
  e.splits = plan.splits;
  // Power-of-two block scales on every block-scaled operand go into the matrix
  // instruction; beside others they are binary32 scales of the same layouts, as
  // they are for the few-row kernel (bound by memory, not by the promotion).
  const bool promoted = p.a_scaling == 1 || p.a_scaling == 2 || p.b_scaling == 1 || p.b_scaling == 2;
  if (!plan.large) {
    if (p.a_scaling == 3 || p.a_scaling == 4) p.a_scaling -= 2;
    if (p.b_scaling == 3 || p.b_scaling == 4) p.b_scaling -= 2;
  }
  if (p.M > 0) {
    hipError_t err;
    if (plan.large) err = p.d_fp8 ? launch_gemm_ep_large_fp8out(p, e, s) : launch_gemm_ep_large(p, e, s);
    else if (plan.skinny) err = p.d_fp8 ? launch_gemm_ep_skinny_fp8out(p, e, s) : launch_gemm_ep_skinny(p, e, s);
    else if (promoted) err = p.d_fp8 ? launch_gemm_ep_tile_blk_fp8out(p, e, plan, s) : launch_gemm_ep_tile_blk(p, e, plan, s);
    else err = p.d_fp8 ? launch_gemm_ep_tile_fp8out(p, e, plan, s) : launch_gemm_ep_tile(p, e, plan, s);
    if (err != hipSuccess) return err;
    if (e.splits > 1) {
      const dim3 grid((unsigned)((p.N + 127) / 128), (unsigned)((p.M + 15) / 16));
      if (p.d_fp8) hipLaunchKernelGGL((k_ep_join<true>), grid, dim3(256), 0, s, p, e);
      else hipLaunchKernelGGL((k_ep_join<false>), grid, dim3(256), 0, s, p, e);
      err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
  }
  if (e.dbias) {
    hipLaunchKernelGGL(k_ep_dbias, dim3((unsigned)((p.N + 63) / 64)), dim3(1024), 0, s, e.part, plan.parts, p.N,
                       e.dbias, e.bias_f32);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace fp8lin
