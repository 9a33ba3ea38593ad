// gemm_gated.hip -- the gated pair of a feed-forward block: the join of K parts, and
// which kernel a call takes.
#include "gemm_gated.h"

namespace fp8lin {

namespace {

// The parts' sums added in order, then the epilogue: a wavefront takes 16 rows of 32
// outputs (a lane one row of eight), a workgroup 16 rows of 128.
template <typename W>
__device__ __forceinline__ void add_parts(const GatedParams& e, const float* s, int64_t next, float (&v)[8]) {
#pragma unroll 8
  for (int z = 0; z < e.splits; ++z) {
    const float4 a = *reinterpret_cast<const float4*>(s + z * next), b = *reinterpret_cast<const float4*>(s + z * next + 4);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
}
template <bool BACK, bool OUT8>
__global__ void __launch_bounds__(256) k_gated_join(GemmParams p, GatedParams e) {
  constexpr int TS = 32, COLS = BACK ? 32 : 64;   // columns of the sums
  using W = typename std::conditional<BACK, GatedGradWave<COLS, OUT8, false, 2>, GatedWave<COLS, OUT8, false>>::type;
  constexpr int BYTES = W::bytes(1);
  static_assert(W::RPL == 1, "a lane has one row of 8 outputs");
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * BYTES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * COLS, m0 = (int64_t)blockIdx.y * 16;
  uint8_t* wl = lds + wave * BYTES;
  W w(p, e, n0, lane);
  typename W::Words o[1];
  w.fetch(m0, o);
  const int64_t m = m0 + w.rg;
  // eight outputs' columns: their own, or 16 of each factor in turn
  const int at = BACK ? 8 * w.cq : 32 * (w.cq >> 1) + 8 * (w.cq & 1);
#pragma unroll
  for (int h = 0; h < (BACK ? 1 : 2); ++h) {
    float v[8] = {};
    if (w.nv > 0 && m < p.M) add_parts<W>(e, e.sums + m * e.ldw + n0 + at + 16 * h, p.M * e.ldw, v);
    *w.place(wl, w.rg, at / 4 + 4 * h) = make_float4(v[0], v[1], v[2], v[3]);
    *w.place(wl, w.rg, at / 4 + 4 * h + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
  w.stage(m0, o, wl + W::src_at);
  w.template rows<TS>(m0, wl, wl + W::src_at, wl + W::codes_at, 0);
  if constexpr (OUT8) {
    if (p.D_t) w.template flush_t<TS, 16>(wl + W::codes_at, m0, n0);
  }
  w.put_dbias(blockIdx.y);
  if (p.d_amax) ep_amax<4>(p.d_amax, w.amax_bits(), lane, wave);
}

template <bool OUT8>
hipError_t launch_join(const GemmParams& p, const GatedParams& e, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 127) / 128), (unsigned)((p.M + 15) / 16));
  if (e.backward) hipLaunchKernelGGL((k_gated_join<true, OUT8>), grid, dim3(256), 0, s, p, e);
  else hipLaunchKernelGGL((k_gated_join<false, OUT8>), grid, dim3(256), 0, s, p, e);
  return hipGetLastError();
}

// The cut of the linear's products (ep_plan), over the columns that B's rows make: the
// sums do not differ.  `tiles`: never the few-row kernel.
EpPlan plan_of(const GemmParams& p, int backward, bool tiles) {
  GemmParams v = p;
  if (!backward) v.N = paired_columns(p.N);
  if (tiles && v.M > 0 && v.M <= 16) v.M = 17;
  EpPlan plan = ep_plan(v);
  const int64_t parts = plan.parts > plan.large_parts ? plan.parts : plan.large_parts;   // (either may be taken)
  plan.part_bytes = backward ? (parts * 2 * p.N * 4 + 255) / 256 * 256 : 0;
  plan.sums_bytes = plan.splits > 1 ? plan.splits * p.M * plan.ldw * 4 : 0;
  return plan;
}

}  // namespace

// The workspace has to do for a call that keeps a checkpoint, which few rows take to
// the tiles (the few-row kernel's 16 outputs are half a block), and for one that does not.
EpPlan gated_plan(const GemmParams& p, int backward) { return plan_of(p, backward, !backward); }

namespace {
bool blocks(const GemmParams& p) { return p.a_scaling != 0 && p.a_scaling != 5; }
// What the large kernels take: see gemm_gated_large.h.
bool large_takes(const GemmParams& p, const GatedParams& e) {
  auto dwords = [](const void* q, int64_t ld, int size) {
    return q == nullptr || (((reinterpret_cast<uintptr_t>(q) & 3u) == 0) && ((ld * size) & 3) == 0);
  };
  // (a wavefront's 128 rows, and 128 of D_t's, stay inside a buffer's 31 bits)
  auto near = [](const void* q, int64_t ld, int size) { return q == nullptr || ld <= ((int64_t)1 << 23) / size; };
  const int es = p.d_fp8 ? 1 : (p.d_f32 ? 4 : 2);
  return p.N % (blocks(p) && !e.backward ? 128 : 32) == 0 && dwords(p.D, p.ldd, es) && dwords(p.D_t, p.ldt, 1) &&
         dwords(e.aux, e.ldaux, 2) && dwords(e.ck, e.ldck, 1) && near(p.D, p.ldd, es) && near(p.D_t, p.ldt, 1) &&
         near(e.aux, e.ldaux, 2) && near(e.ck, e.ldck, 1) && near(e.ck_exp, e.ldexp, 1);
}
}  // namespace

EpPlan gated_plan(const GemmParams& p, const GatedParams& e) {
  EpPlan plan = plan_of(p, e.backward, !e.backward && e.ck != nullptr);
  const bool takes = large_takes(p, e);
  plan.mid = plan.mid && takes && !e.backward && !blocks(p);
  plan.large = plan.large && takes && !plan.mid;
  if (plan.large || plan.mid) plan.splits = 1;
  return plan;
}

hipError_t launch_gated(const GemmParams& p0, GatedParams e, uint8_t* ws, hipStream_t s) {
  GemmParams p = p0;
  if (p.d_amax && !p.amax_acc) {
    const hipError_t err = launch_fill_u32(reinterpret_cast<uint32_t*>(p.d_amax), 1, 0u, s);
    if (err != hipSuccess) return err;
  }
  if (p.N == 0) return hipSuccess;
  const EpPlan plan = gated_plan(p, e);
  // (the only row of column sums is the bias gradient: up to 32 rows, 3 us less)
  const bool joined = e.dbias != nullptr && (plan.large || plan.parts != 1);
  e.part = e.dbias && !joined ? static_cast<float*>(e.dbias) : reinterpret_cast<float*>(ws);
  e.part_f32 = joined || e.bias_f32;
  e.sums = reinterpret_cast<float*>(ws + plan.part_bytes);
  e.ldw = plan.ldw;
  e.splits = plan.splits;
  // (powers of two on every block-scaled operand go into the matrix instruction; beside
  // others, and for few rows, they are binary32 scales of the same layouts)
  if (plan.mid) return launch_gated_mid(p, e, s);
  if (plan.large) {
    const hipError_t err = !e.backward ? launch_gated_large(p, e, s)
                           : p.a_fmt == 0 ? launch_gated_grad_large(p, e, s) : launch_gated_grad_large_e5m2(p, e, s);
    if (err != hipSuccess) return err;
    return joined ? launch_ep_dbias(e.part, plan.large_parts, 2 * p.N, e.dbias, e.bias_f32, s) : hipSuccess;
  }
  const bool promoted = p.a_scaling == 1 || p.a_scaling == 2 || p.b_scaling == 1 || p.b_scaling == 2;
  if (p.a_scaling == 3 || p.a_scaling == 4) p.a_scaling -= 2;
  if (p.b_scaling == 3 || p.b_scaling == 4) p.b_scaling -= 2;
  if (p.M > 0) {
    hipError_t err;
    if (plan.skinny) err = launch_gated_skinny(p, e, s);
    else if (e.backward) err = promoted ? launch_gated_grad_tile_blk(p, e, plan, s) : launch_gated_grad_tile(p, e, plan, s);
    else err = promoted ? launch_gated_tile_blk(p, e, plan, s) : launch_gated_tile(p, e, plan, s);
    if (err != hipSuccess) return err;
    if (e.splits > 1) {
      err = p.d_fp8 ? launch_join<true>(p, e, s) : launch_join<false>(p, e, s);
      if (err != hipSuccess) return err;
    }
  }
  return joined ? launch_ep_dbias(e.part, plan.parts, 2 * p.N, e.dbias, e.bias_f32, s) : hipSuccess;
}

}  // namespace fp8lin
