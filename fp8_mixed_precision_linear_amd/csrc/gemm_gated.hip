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

// The amax of a forward product with FP8 output: the largest |d| taken again in binary32.
// The matrix unit cuts the bits of each eight products below 2^-13 of the largest, 1.2e-5 of
// a row's norm, and d multiplies two such sums, which in a row of large activations put the
// amax up to 4e-5 off.  (A backward d holds one such sum, 1.7e-5 off at most, and its amax
// is that of the matrix unit's values, as the linear's.)  So every wavefront leaves a key
// (its largest |d| and the up to 16 outputs among which a lane met it) in place of an atomic
// maximum, and this workgroup takes the largest key's outputs again in binary32, 32 lanes to
// a sum.  Equal keys: the first.  The value is right to binary32's roundings for the outputs
// taken again; another wavefront's, within the cut of the largest, may be the larger one.
// Infinities, NaN and zeros stay as they are.
// Bound by latency, a chain of six loads: the kernel takes 5.7 us at K = 256, 7.7 at 4096 (8.4
// with block scales), 15.8 at 8192 x 28672 x 8192 (28 672 keys).  A call among others takes 33.3
// us with an amax and 25.2 without at 1 x 14336 x 4096, 53.1 and 43.8 at 300 rows, 2759 and 2754
// at 8192 x 28672 x 8192.
constexpr int AMAX_THREADS = 1024;
__device__ __forceinline__ float scale_at(const float* s, int scaling, int64_t rows, int64_t kb, int64_t row) {
  if (scaling == 1 || scaling == 3) return s[kb * rows + row];
  return scaling == 2 || scaling == 4 ? s[kb * ((rows + 127) / 128) + row / 128] : 1.0f;
}
__global__ void __launch_bounds__(AMAX_THREADS) k_gated_amax(GemmParams p, GatedParams e, uint32_t keys, float* amax) {
  __shared__ uint32_t wbits[AMAX_THREADS / 64], wat[AMAX_THREADS / 64];
  __shared__ float sums[32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t best = 0, at = 0;
  auto take = [&](uint32_t b, uint32_t i) {
    if (b > best || (b == best && i < at)) { best = b; at = i; }
  };
  constexpr int AT_ONCE = 8, CHUNKS = 4;   // loads on their way together
  for (uint32_t i0 = tid; i0 < keys; i0 += AT_ONCE * AMAX_THREADS) {
    uint32_t b[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) b[k] = e.keys[min(i0 + k * AMAX_THREADS, keys - 1)];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) take(b[k], min(i0 + k * AMAX_THREADS, keys - 1));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) take(__shfl_xor(best, off, 64), __shfl_xor(at, off, 64));
  if (lane == 0) { wbits[wave] = best; wat[wave] = at; }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < AMAX_THREADS / 64; ++w) take(wbits[w], wat[w]);
  if (best != 0 && best < 0x7F800000u) {
    const uint2 key = e.key_at[at];
    const int64_t F = p.N, K = p.K, m = key.x, d = tid >> 5, f = (int64_t)(key.y & ~7u) + (d & 15);
    const bool on = (d & 15) < ((key.y & 1) ? 16 : 8) && f < F;
    const int64_t n = d < 16 ? f : F + f;   // B's row
    float v = 0.0f, sa = 1.0f, sb = 1.0f, bias = 0.0f;
    if (on) {
      if (K > 0 && (p.a_scaling == 0 || p.a_scaling == 5)) sa = p.a_sinv[p.a_scaling == 5 ? m : 0];
      if (K > 0 && (p.b_scaling == 0 || p.b_scaling == 5)) sb = p.b_sinv[p.b_scaling == 5 ? n : 0];
      if (e.bias) bias = e.bias_f32 ? static_cast<const float*>(e.bias)[n] : bf16_lo(static_cast<const uint16_t*>(e.bias)[n]);
      const int64_t last = K / 16 - 1;
      for (int64_t c0 = tid & 31; c0 <= last; c0 += 32 * CHUNKS) {
        uint4 as[CHUNKS], bs[CHUNKS];
        float w[CHUNKS];
#pragma unroll
        for (int u = 0; u < CHUNKS; ++u) {   // (past the end: the last one again, without weight)
          const int64_t c = min(c0 + 32 * u, last);
          as[u] = *reinterpret_cast<const uint4*>(p.A + m * p.lda + 16 * c);
          bs[u] = *reinterpret_cast<const uint4*>(p.B + n * p.ldb + 16 * c);
          w[u] = scale_at(p.a_sinv, p.a_scaling, p.M, c >> 3, m) * scale_at(p.b_sinv, p.b_scaling, 2 * F, c >> 3, n);
        }
#pragma unroll
        for (int u = 0; u < CHUNKS; ++u) {
          const uint4 a = as[u], b = bs[u];
          const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
          float s = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const auto x0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[q], false), x1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[q], true);
            const auto y0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)y[q], false), y1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)y[q], true);
            s = __builtin_fmaf(x0[0], y0[0], s);
            s = __builtin_fmaf(x0[1], y0[1], s);
            s = __builtin_fmaf(x1[0], y1[0], s);
            s = __builtin_fmaf(x1[1], y1[1], s);
          }
          v = c0 + 32 * u <= last ? __builtin_fmaf(s, w[u], v) : v;
        }
      }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((tid & 31) == 0) sums[d] = on ? (v * sa) * sb + bias : 0.0f;
    __syncthreads();
    best = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float g[8], a[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = sums[8 * h + k];
      act_of(e.act, g, a);
#pragma unroll
      for (int k = 0; k < 8; ++k) best = max_u32(best, abs_bits(a[k] * sums[16 + 8 * h + k]));
    }
  }
  if (tid == 0) {
    if (p.amax_acc) atomic_max_bits(amax, best);   // (calls on other streams may add to it)
    else *reinterpret_cast<uint32_t*>(amax) = best;
  }
}

// How many wavefronts leave keys: of a call's kernel, and of any that a call may take.
int64_t tiles_of(int64_t M, int64_t N, int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); }
int64_t keys_of(const GemmParams& p, const EpPlan& plan, int waves_of_large) {
  const int64_t columns = paired_columns(p.N);
  if (plan.large) return tiles_of(p.M, columns, 256, 256) * waves_of_large;
  if (plan.mid) return tiles_of(p.M, columns, 160, 256) * 4;
  if (plan.skinny) return (columns + 31) / 32;
  return 4 * (plan.splits > 1 ? tiles_of(p.M, p.N, 16, 128) : tiles_of(p.M, columns, plan.bm, plan.bn));
}
int64_t most_keys(const GemmParams& p, EpPlan plan) {
  int64_t most = 0;
  for (int kind = 0; kind < 4; ++kind) {
    plan.large = kind == 0;
    plan.mid = kind == 1;
    plan.skinny = kind == 2;
    const int64_t n = keys_of(p, plan, 8);
    most = n > most ? n : most;
  }
  return most;
}

// The cut of the linear's products (ep_plan), over the columns that B's rows make: the
// sums do not differ.  `tiles`: never the few-row kernel.
EpPlan plan_of(const GemmParams& p, int backward, bool tiles) {
  GemmParams v = p;
  if (!backward) v.N = paired_columns(p.N);
  if (tiles && v.M > 0 && v.M <= 16) v.M = 17;
  EpPlan plan = ep_plan(v);
  const int64_t parts = plan.parts > plan.large_parts ? plan.parts : plan.large_parts;   // (either may be taken)
  const int64_t keys = backward ? 0 : most_keys(p, plan);
  plan.part_bytes = backward ? (parts * 2 * p.N * 4 + 255) / 256 * 256 : (4 * keys + 255) / 256 * 256 + (8 * keys + 255) / 256 * 256;
  plan.sums_bytes = plan.splits > 1 ? plan.splits * p.M * plan.ldw * 4 : 0;
  return plan;
}

}  // namespace

// The workspace has to do for a call that keeps a checkpoint, which few rows take to
// the tiles (the few-row kernel's 16 outputs are half a block), and for one that does not.
EpPlan gated_plan(const GemmParams& p, int backward) { return plan_of(p, backward, !backward); }

namespace {
bool blocks(const GemmParams& p) { return p.a_scaling != 0 && p.a_scaling != 5; }
// What the large kernels take (gemm_gated_large.h): their stores are dwords and more.  So a
// contiguous D_t with a number of rows that is no multiple of 4 is written on tiles: 8191 x
// 28672 x 8192 in 3822 us forward and 2326 backward, with D_t's rows padded to a dword 2770
// and 1698.
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
  float* amax = !e.backward && p.d_fp8 && p.M > 0 && p.N > 0 ? p.d_amax : nullptr;   // k_gated_amax writes it
  if (amax) p.d_amax = nullptr;
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
  const int waves = p.a_scaling == 1 ? 8 : 4;
  const GemmParams given = p;
  const int64_t keys = amax ? keys_of(p, plan, waves) : 0;
  e.keys = amax ? reinterpret_cast<uint32_t*>(ws) : nullptr;
  e.key_at = reinterpret_cast<uint2*>(ws + (4 * keys + 255) / 256 * 256);
  e.key_waves = plan.large ? waves : plan.skinny ? 1 : 4;
  auto join_amax = [&](hipError_t err) {
    if (err != hipSuccess || amax == nullptr) return err;
    hipLaunchKernelGGL(k_gated_amax, dim3(1), dim3(AMAX_THREADS), 0, s, given, e, (uint32_t)keys, amax);
    return hipGetLastError();
  };
  if (plan.mid) return join_amax(launch_gated_mid(p, e, s));
  if (plan.large) {
    const hipError_t err = !e.backward ? launch_gated_large(p, e, s)
                           : p.a_fmt == 0 ? launch_gated_grad_large(p, e, s) : launch_gated_grad_large_e5m2(p, e, s);
    if (err != hipSuccess) return err;
    return joined ? launch_ep_dbias(e.part, plan.large_parts, 2 * p.N, e.dbias, e.bias_f32, s) : join_amax(hipSuccess);
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
  return joined ? launch_ep_dbias(e.part, plan.parts, 2 * p.N, e.dbias, e.bias_f32, s) : join_amax(hipSuccess);
}

}  // namespace fp8lin
