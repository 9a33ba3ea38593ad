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
  uint32_t o[1][W::SW];
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

template <int AF, int BF, bool BLOCK, bool OUT8>
hipError_t launch_tile(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  const int tiles_m = (int)((p.M + plan.bm - 1) / plan.bm), tiles_n = (int)((p.N + plan.bn - 1) / plan.bn);
  const dim3 grid((unsigned)(tiles_m * tiles_n), (unsigned)plan.splits), block(EP_THREADS);
  if (plan.bm == 32)
    hipLaunchKernelGGL((k_ep_tile<AF, BF, BLOCK, OUT8, 1, 4, 2, 2, 6>), grid, block, 0, s, p, e, tiles_m, tiles_n);
  else if (plan.bm == 64)
    hipLaunchKernelGGL((k_ep_tile<AF, BF, BLOCK, OUT8, 2, 2, 2, 4, 5>), grid, block, 0, s, p, e, tiles_m, tiles_n);
  else
    hipLaunchKernelGGL((k_ep_tile<AF, BF, BLOCK, OUT8, 2, 2, 4, 4, 4>), grid, block, 0, s, p, e, tiles_m, tiles_n);
  return hipGetLastError();
}

template <bool BLOCK, bool OUT8>
hipError_t launch_fmt(const GemmParams& p, const EpParams& e, const EpPlan& plan, hipStream_t s) {
  if (p.a_fmt == 0 && p.b_fmt == 0) return launch_tile<0, 0, BLOCK, OUT8>(p, e, plan, s);
  if (p.a_fmt == 1 && p.b_fmt == 0) return launch_tile<1, 0, BLOCK, OUT8>(p, e, plan, s);
  if (p.a_fmt == 0 && p.b_fmt == 1) return launch_tile<0, 1, BLOCK, OUT8>(p, e, plan, s);
  return launch_tile<1, 1, BLOCK, OUT8>(p, e, plan, s);
}

}  // namespace

namespace {
int64_t tile_parts(int64_t M, int bm) { return (M + bm - 1) / bm * (bm == 32 ? 1 : 2); }
}  // namespace

EpPlan ep_plan(const GemmParams& p) {
  EpPlan plan = {};
  const int64_t big_tiles = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  const bool layer = (p.a_scaling == 0 || p.a_scaling == 5) ? (p.b_scaling == 0 || p.b_scaling == 5)
                     : p.a_scaling == 1 ? p.b_scaling == 2 : p.a_scaling == 3 ? p.b_scaling == 4 : false;
  plan.large = p.M > 64 && layer && p.K > 0 && 2 * big_tiles >= device_cu_count();
  plan.skinny = p.M <= 16;
  plan.bm = p.M <= 32 ? 32 : (p.M <= 64 ? 64 : 128);
  plan.bn = 128;
  plan.splits = 1;
  const int64_t tiles = ((p.M + plan.bm - 1) / plan.bm) * ((p.N + 127) / 128), cu = device_cu_count();
  const int64_t nk = (p.K + BK - 1) / BK;
  // Split K while the tiles leave compute units without work and every part
  // keeps at least four steps.
  int64_t splits = 1;
  while (!plan.large && !plan.skinny && splits < 16 && tiles * splits * 2 <= cu && nk / (splits * 2) >= 4) splits *= 2;
  plan.splits = (int)splits;
  // rows of column sums: the wavefronts' rows of tiles, or of the join
  plan.parts = splits > 1 || plan.skinny ? (p.M + 15) / 16
               : plan.large ? (p.M + 255) / 256 * 2 : tile_parts(p.M, plan.bm);
  plan.ldw = (p.N + 7) / 8 * 8;
  // (a product of the large kernels' size may still run on the tiles: large_takes)
  const int64_t parts = plan.large && tile_parts(p.M, plan.bm) > plan.parts ? tile_parts(p.M, plan.bm) : plan.parts;
  plan.part_bytes = (parts * p.N * 4 + 255) / 256 * 256;
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

hipError_t launch_gemm_ep(const GemmParams& p0, EpParams e, uint8_t* ws, hipStream_t s) {
  GemmParams p = p0;
  if (p.d_amax && !p.amax_acc) {
    const hipError_t err = launch_fill_u32(reinterpret_cast<uint32_t*>(p.d_amax), 1, 0u, s);
    if (err != hipSuccess) return err;
  }
  if (p.N == 0) return hipSuccess;
  const EpPlan plan = ep_plan(p);
  e.part = reinterpret_cast<float*>(ws);
  e.sums = reinterpret_cast<float*>(ws + plan.part_bytes);
  e.ldw = plan.ldw;
  e.splits = plan.splits;
  const bool large = plan.large && large_takes(p, e);
  int64_t parts = plan.parts;
  if (!large) {
    // power-of-two block scales are binary32 scales of the same layouts here
    if (p.a_scaling == 3 || p.a_scaling == 4) p.a_scaling -= 2;
    if (p.b_scaling == 3 || p.b_scaling == 4) p.b_scaling -= 2;
    if (plan.large) parts = tile_parts(p.M, plan.bm);
  }
  const bool block = !((p.a_scaling == 0 || p.a_scaling == 5) && (p.b_scaling == 0 || p.b_scaling == 5));
  if (p.M > 0) {
    hipError_t err;
    if (large) err = p.d_fp8 ? launch_gemm_ep_large_fp8out(p, e, s) : launch_gemm_ep_large(p, e, s);
    else if (plan.skinny) err = p.d_fp8 ? launch_gemm_ep_skinny_fp8out(p, e, s) : launch_gemm_ep_skinny(p, e, s);
    else if (block) err = p.d_fp8 ? launch_fmt<true, true>(p, e, plan, s) : launch_fmt<true, false>(p, e, plan, s);
    else err = p.d_fp8 ? launch_fmt<false, true>(p, e, plan, s) : launch_fmt<false, false>(p, e, plan, s);
    if (err != hipSuccess) return err;
    if (plan.splits > 1) {
      const dim3 grid((unsigned)((p.N + 127) / 128), (unsigned)((p.M + 15) / 16));
      if (p.d_fp8) hipLaunchKernelGGL((k_ep_join<true>), grid, dim3(256), 0, s, p, e);
      else hipLaunchKernelGGL((k_ep_join<false>), grid, dim3(256), 0, s, p, e);
      err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
  }
  if (e.dbias) {
    hipLaunchKernelGGL(k_ep_dbias, dim3((unsigned)((p.N + 63) / 64)), dim3(1024), 0, s, e.part, parts, p.N,
                       e.dbias, e.bias_f32);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace fp8lin
