// norm_kernels.hip -- the norms before and after a block, fused with the
// block's gate and residual scale, and their gradients.
//
// Forward, per row of D columns (N the RMS or layer norm, its statistics and
// every sum in binary32):
//   n = (z - mz) rz w_post + b_post       rz = 1 / sqrt(mean (z - mz)^2 + eps)
//   h = res_scale x + branch_scale G(gate) n            (h = x without z)
//   y = (h - mh) rh w_pre + b_pre
// with mz = mh = 0 for the RMS norm.  y is taken from h in binary32, before h
// is rounded to the stream's type (the rounding would add its own half step
// to y), and leaves as BF16 and / or as FP8 codes with the per-tensor scale of
// the steps before, or the scale of the row or of each 128 columns of it:
// the cast of the next linear's operand without a pass over y of its own.  (Codes
// row by row: the transposed ones that a weight gradient multiplies are a cast of
// their own.)
//
// Backward, from dy and dh (the gradient that reaches h from above):
//   a = dy w_pre, xh = (h - mh) rh
//   dH = dh + rh (a - mean a [layer] - xh mean(a xh))
//   dn = branch_scale G dH,  c = dn w_post, zh = (z - mz) rz
//   dz = rz (c - mean c [layer] - zh mean(c zh)),   dx = res_scale dH
//   dw_pre = sum_t dy xh, db_pre = sum_t dy,
//   dw_post = sum_t dn zh, db_post = sum_t dn,
//   dgate = branch_scale G' dH n, summed to the gate's shape.
// A channel gate is constant down a column, so the sums S1 = sum_t dH zh and
// S0 = sum_t dH give all of dw_post = bs G S1, db_post = bs G S0 and
// dgate = bs G' (w S1 + b S0).
//
// Bound: HBM.  Up to 8192 columns, one vector of eight per thread, a row stays in
// registers between its loads and its stores (but for up to 60 bytes per lane in some
// kernels), so each element is read and written once; the column sums are kept in
// registers or LDS over the rows that a workgroup takes and joined by a second, small
// kernel in a fixed order (no atomics: equal inputs give equal bits).  Wider rows, with
// two vectors per thread up to 16384 columns and four beyond, do not fit the 128
// registers of a 1024-thread workgroup's threads: 64 .. 256 and 464 .. 880 bytes per lane
// of the forward pass, 184 .. 648 and 1104 .. 1772 of the gradient wait in scratch
// memory, and these are bound by that.
//
// Measured (MI355X, inputs that change from call to call; a copy of 2 x 2 GiB moves
// 4.94 TB/s): 8192 x 8192 with channel gate and FP8 out 107 us, 4.4 TB/s; its gradient
// 160 us, 5.0 TB/s, of which the join is 6; 1 x 8192 6.4 us of kernel; layer norm of
// 1531 x 2053 in binary32 17.4 us, 2.5 TB/s; gradient of 777 x 4095 33 us, 1.7 TB/s,
// bound by its partial column sums.  Wide rows: 4096 x 12288 138 us, gradient 232 (at 5
// TB/s 81 and 121); 4096 x 16384 170 and 276 (107 and 161); 2048 x 28672 215 and 939 (94
// and 141).  Rows of an XCD kept contiguous: 5-8% slower.
#include <atomic>

#include "op_device.h"
#include "launch.h"

namespace fp8lin {

namespace {

// The wavefronts of a row share sums and maxima: each by lane permutations,
// then (more than one) through one LDS word group per wavefront, of which lane l
// reads group l % 16.  Two buffers in turn, so one barrier per exchange is
// enough: whoever writes a buffer again has passed the barrier in between, which
// every reader of its old values reached after reading.
constexpr int kMaxWaves = 16;
template <bool ONE>   // ONE: a wavefront has a row to itself, no barrier
struct Row {
  float4* lds;   // 2 * kMaxWaves
  int nw, first, turn = 0;   // the row's wavefronts, the first of them
  __device__ __forceinline__ Row(float4* l, int nw_, int first_) : lds(l), nw(nw_), first(first_) {}

  // this wavefront's group out, this lane's group in (0 past the last)
  __device__ __forceinline__ float4 swap(float4 w) {
    float4* b = lds + turn * kMaxWaves;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = w;
    __syncthreads();
    const int l = threadIdx.x & 15;
    return l < nw ? b[first + l] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  template <int NV>
  __device__ __forceinline__ void sum(float (&v)[NV]) {
    static_assert(NV <= 3, "one group");
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = wave_sum(v[k]);
    if constexpr (!ONE) {
      float4 w = make_float4(v[0], 0.0f, 0.0f, 0.0f);
      if constexpr (NV > 1) w.y = v[1];
      if constexpr (NV > 2) w.z = v[2];
      w = swap(w);
      v[0] = row16_sum(w.x);
      if constexpr (NV > 1) v[1] = row16_sum(w.y);
      if constexpr (NV > 2) v[2] = row16_sum(w.z);
    }
  }
  __device__ __forceinline__ uint32_t max(uint32_t m) {
    m = wave_max(m);
    if constexpr (!ONE)
      m = row16_max(__float_as_uint(swap(make_float4(__uint_as_float(m), 0.0f, 0.0f, 0.0f)).x));
    return m;
  }
  // Mean (0 for the RMS norm) and the sum of squares about it.  Layer norm:
  // each wavefront sums about its own mean first, the wavefronts' sums are
  // joined as M2 = sum (M2_w + n_w (m_w - m)^2): no cancellation and one
  // exchange.  count: this wavefront's columns.
  template <bool LN, int VPT>
  __device__ __forceinline__ void stats(const float (&v)[VPT][8], const RowVec (&x)[VPT], float count, float inv_d,
                                        float& mean, float& m2) {
    float s = 0.0f, q = 0.0f, mw = 0.0f;
    if constexpr (LN) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) s += k >= x[i].skip ? v[i][k] : 0.0f;
      s = wave_sum(s);
      mw = count > 0.0f ? s / count : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float c = k >= x[i].skip ? v[i][k] - mw : 0.0f;
        q = __builtin_fmaf(c, c, q);
      }
    q = wave_sum(q);
    if constexpr (ONE) {
      mean = mw;
      m2 = q;
    } else if constexpr (!LN) {
      mean = 0.0f;
      m2 = row16_sum(swap(make_float4(q, 0.0f, 0.0f, 0.0f)).x);
    } else {
      const float4 w = swap(make_float4(s, q, count, 0.0f));
      mean = row16_sum(w.x) * inv_d;
      const float off = w.z > 0.0f ? w.x / w.z - mean : 0.0f;
      m2 = row16_sum(__builtin_fmaf(w.z * off, off, w.y));
    }
  }
};

// A row takes G threads, the multiple of 64 that covers its vectors of 8 columns
// with VPT of them per thread, vector t + i G for thread t.
template <int VPT>
struct Cols {
  RowVec x[VPT];
  __device__ __forceinline__ Cols(int64_t cols, int t, int G) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = RowVec((int)cols, t + i * G);
  }
};

// The rows of a workgroup: every gridDim.x-th group of `rpw`.  (A contiguous run
// of rows per XCD, so that neighbouring rows share their boundary lines in one
// L2, was 5-8% slower at 8192 and 4096 columns and no faster at 4104.)
struct Rows {
  int64_t first, end, step;
  __device__ __forceinline__ Rows(int64_t rows, int rpw) {
    first = (int64_t)blockIdx.x * rpw;
    end = rows;
    step = (int64_t)gridDim.x * rpw;
  }
};

// Whether the next row's loads fit in registers beside this row: not for
// several vectors per thread of up to 1024 threads (128 registers each).
constexpr bool ahead(bool one, int VPT) { return VPT == 1 || one; }

// Keeps the compiler from working on a thread's vectors side by side, which
// would need the registers of all of them.
template <int VPT>
__device__ __forceinline__ void one_at_a_time() {
  if constexpr (VPT > 1) __builtin_amdgcn_sched_barrier(0);
}

// Row `row` of a matrix of bf16 (f32 = 0) or binary32 values.
__device__ __forceinline__ const void* row_of(const void* base, int64_t row, int64_t ld, int f32) {
  return reinterpret_cast<const char*>(base) + row * ld * (f32 ? 4 : 2);
}
__device__ __forceinline__ void* row_of(void* base, int64_t row, int64_t ld, int f32) {
  return reinterpret_cast<char*>(base) + row * ld * (f32 ? 4 : 2);
}

// A vector of a row at once, of either type.
template <bool TINY>
__device__ __forceinline__ void load_vec(const void* row, int f32, const RowVec& x, float (&v)[8]) {
  if (f32) unpack(load_raw<true, TINY>(row, x), row, x, v);
  else unpack(load_raw<false, TINY>(row, x), row, x, v);
}

// A parameter vector's values for this thread (optionally times a channel gate
// and a factor): kept in registers for one vector per thread, read again (from
// L2) beyond, where they would not fit.
template <int VPT, bool TINY, bool KEEP = true>
struct Param {
  static constexpr bool KEPT = VPT <= 1 && KEEP;
  float v[KEPT ? VPT : 1][8];
  const void *p, *gate;
  int f32, act;
  float other, factor;
  __device__ __forceinline__ Param(const Cols<VPT>& c, const void* p_, int f32_, float other_,
                                   const void* gate_ = nullptr, int act_ = 0, float factor_ = 1.0f)
      : p(p_), gate(gate_), f32(f32_), act(act_), other(other_), factor(factor_) {
    if constexpr (KEPT) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) read(c.x[i], v[i]);
    }
  }
  __device__ __forceinline__ void read(const RowVec& x, float (&o)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = other;
    if (p) load_vec<TINY>(p, f32, x, o);
    if (gate) {
      float g[8];
      load_vec<TINY>(gate, f32, x, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= gate_value(act, g[k]);
    }
    if (factor != 1.0f) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= factor;
    }
  }
  __device__ __forceinline__ void get(int i, const RowVec& x, float (&o)[8]) const {
    if constexpr (KEPT) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = v[i][k];
    } else {
      read(x, o);
    }
  }
};

// VPT vectors of 8 columns per thread.  ONE: a wavefront per row (four rows per
// workgroup); else the workgroup's threads share a row.  FULL: a gate per
// element.  Where registers allow (ahead), the next row's loads are in flight
// while this row is worked on.
template <int VPT, bool ONE, bool LN, bool XF32, bool FULL, bool TINY>
__global__ void __launch_bounds__(ONE ? 256 : 1024)
    __attribute__((amdgpu_waves_per_eu(VPT == 1 ? (LN ? 5 : 6) : 1))) k_norm_fwd(NormParams p) {
  constexpr bool AHEAD = ahead(ONE, VPT);
  __shared__ float4 red[ONE ? 1 : 2 * kMaxWaves];
  __shared__ uint32_t amax_part[kMaxWaves];
  const int G = ONE ? 64 : (int)blockDim.x, RPW = ONE ? 4 : 1;
  const int t = ONE ? threadIdx.x & 63 : threadIdx.x, sub = ONE ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  Row<ONE> rs(red, G >> 6, 0);
  const float inv_d = 1.0f / (float)p.cols;
  const bool post = p.z != nullptr, pre = p.y != nullptr || p.y8 != nullptr;
  const Cols<VPT> c(p.cols, t, G);
  float count = 0.0f;
  if constexpr (LN) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) count += (float)(8 - c.x[i].skip);
    count = wave_sum(count);
  }
  const void* cgate = p.gate_kind == 1 ? p.gate : nullptr;
  // branch_scale G(gate) w_post and (layer norm) branch_scale G(gate) b_post
  const Param<VPT, TINY> w_post(c, p.w_post, p.p_f32, 1.0f, cgate, p.gate_act, p.branch_scale);
  const Param<LN ? VPT : 2, TINY> b_post(Cols<LN ? VPT : 2>(p.cols, t, G), p.b_post, p.p_f32, 0.0f, cgate, p.gate_act,
                                   p.branch_scale);
  const Param<VPT, TINY> w_pre(c, p.w_pre, p.p_f32, 1.0f);
  const float s_tensor = p.y8_scale ? p.y8_scale[0] : 1.0f;
  uint32_t amax = 0;

  struct Held {
    Raw8<XF32> x[VPT];
    Raw8<false> z[VPT], g[FULL ? VPT : 1];
  };
  auto fetch = [&](int64_t row, Held& f) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (post) {
        f.z[i] = load_raw<false, TINY>(row_of(p.z, row, p.ldz, false), c.x[i]);
        if constexpr (FULL) f.g[i] = load_raw<false, TINY>(row_of(p.gate, row, p.ldg, false), c.x[i]);
      }
      f.x[i] = load_raw<XF32, TINY>(row_of(p.x, row, p.ldx, XF32), c.x[i]);
    }
  };
  const Rows mine(p.rows, RPW);
  int64_t row = mine.first + sub;
  Held next;
  if (AHEAD && row < mine.end) fetch(row, next);
  for (; row < mine.end; row += mine.step) {
    if constexpr (!AHEAD) fetch(row, next);
    const Held f = next;
    if (AHEAD && row + mine.step < mine.end) fetch(row + mine.step, next);
    float h[VPT][8];
    if (post) {
      float m, q, z[VPT][8];
#pragma unroll
      for (int i = 0; i < VPT; ++i) unpack(f.z[i], row_of(p.z, row, p.ldz, false), c.x[i], z[i]);
      rs.template stats<LN>(z, c.x, count, inv_d, m, q);
      const float r = rsqrtf(q * inv_d + p.eps);
      if (p.stats_z && t == 0) {
        p.stats_z[2 * row] = m;
        p.stats_z[2 * row + 1] = r;
      }
      float gt = 1.0f;
      if (!FULL && p.gate_kind == 2) gt = gate_value(p.gate_act, reinterpret_cast<const float*>(p.gate)[row]);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float w[8], b[8];
        w_post.get(i, c.x[i], w);
        unpack(f.z[i], row_of(p.z, row, p.ldz, false), c.x[i], z[i]);
        unpack(f.x[i], row_of(p.x, row, p.ldx, XF32), c.x[i], h[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) z[i][k] = ((z[i][k] - m) * r) * w[k];
        if constexpr (LN) {
          if (p.b_post) {
            b_post.get(i, c.x[i], b);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[i][k] += b[k];
          }
        }
        if constexpr (FULL) {
          float g[8];
          unpack(f.g[i], row_of(p.gate, row, p.ldg, false), c.x[i], g);
#pragma unroll
          for (int k = 0; k < 8; ++k) z[i][k] *= gate_value(p.gate_act, g[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[i][k] = __builtin_fmaf(p.res_scale, h[i][k], gt * z[i][k]);
        }
        store_vec<TINY>(row_of(p.h, row, p.ldh, XF32), XF32, c.x[i], true, h[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) unpack(f.x[i], row_of(p.x, row, p.ldx, XF32), c.x[i], h[i]);
    }
    if (!pre) continue;
    float m, q;
    rs.template stats<LN>(h, c.x, count, inv_d, m, q);
    const float r = rsqrtf(q * inv_d + p.eps);
    if (p.stats_h && t == 0) {
      p.stats_h[2 * row] = m;
      p.stats_h[2 * row + 1] = r;
    }
    uint32_t row_max = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8];
      w_pre.get(i, c.x[i], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = ((h[i][k] - m) * r) * w[k];
      if constexpr (LN) {
        if (p.b_pre) {
          float b[8];
          load_vec<TINY>(p.b_pre, p.p_f32, c.x[i], b);
#pragma unroll
          for (int k = 0; k < 8; ++k) h[i][k] += b[k];
        }
      }
      if (p.y) store_vec<TINY>(row_of(p.y, row, p.ldy, 0), 0, c.x[i], true, h[i]);
      if (p.y8) {
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = max_u32(mx, k >= c.x[i].skip ? abs_bits(h[i][k]) : 0u);
        if (p.y8_scaling == 1) {   // one scale per 128 columns: 16 neighbouring lanes
          mx = row16_max(mx);
          float s = 1.0f, si = 1.0f;
          scale_from_amax(__uint_as_float(mx), p.y8_fmt == 0 ? kMaxE4M3 : kMaxE5M2, 0, s, si);
          if (c.x[i].skip < 8 && (t & 15) == 0) p.y8_sinv[(int64_t)((t + i * G) >> 4) * p.rows + row] = si;
          uint32_t lo, hi;
          codes8(p.y8_fmt, h[i], s, lo, hi);
          store_vec_codes<TINY>(p.y8 + row * p.ldy8, c.x[i], lo, hi);
        } else {
          row_max = max_u32(row_max, mx);
        }
      }
    }
    if (p.y8 && p.y8_scaling != 1) {
      float s = s_tensor, si = 1.0f;
      if (p.y8_scaling == 5) {
        row_max = rs.max(row_max);
        s = 1.0f;
        scale_from_amax(__uint_as_float(row_max), p.y8_fmt == 0 ? kMaxE4M3 : kMaxE5M2, 0, s, si);
        if (t == 0) p.y8_sinv[row] = si;
      } else {
        amax = max_u32(amax, row_max);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        uint32_t lo, hi;
        codes8(p.y8_fmt, h[i], s, lo, hi);
        store_vec_codes<TINY>(p.y8 + row * p.ldy8, c.x[i], lo, hi);
      }
    }
  }
  if (p.y8_amax) {   // one filtered atomic maximum per workgroup (order-free)
    amax = wave_max(amax);
    if ((threadIdx.x & 63) == 0) amax_part[threadIdx.x >> 6] = amax;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < (int)blockDim.x / 64; ++w) amax = max_u32(amax, amax_part[w]);
      if (amax != 0u) atomic_max_bits(p.y8_amax, amax);
    }
  }
}

// Column sums of the backward pass, in this order in the workspace: dw_pre,
// db_pre, S1 (dw_post), S0 (db_post); without LN only the first and third.
// EACH: a gate per token or element, whose gradient leaves row by row; without
// it the gate is absent or per channel and goes into one vector with w_post.
// The row waits packed, as loaded, and is unpacked where it is used: with the
// next row's loads in flight and the column sums beside it, the unpacked
// values would not fit the 128 registers of a 1024-thread workgroup.
// A workgroup takes `rpw` rows at a time (ONE: a wavefront each, without a
// barrier), and every group of threads goes through the same number of them, so
// that the barriers match: past the last row it works on zeros.
template <int VPT, bool ONE, bool LN, bool XF32, bool EACH, bool TINY>
__global__ void __launch_bounds__(ONE ? 512 : 1024) k_norm_bwd(NormGradParams p, int G, int rpw) {
  constexpr int NA = LN ? 4 : 2;
  // The widest rows (binary32, four sums, a gate's values) have no registers left for
  // the next row's loads: 8192 x 4096 155 us with them, 150 without; in bf16 112
  // against 123.
  constexpr bool AHEAD = ahead(ONE, VPT) && !(EACH && LN && XF32);
  __shared__ float4 red[ONE ? 1 : 2 * kMaxWaves];
  // The column sums, NA VPT vectors of 8 per thread, live in registers, or, where
  // they would spill (the layer norm's four, several vectors per thread, or a gate's
  // values beside them: 8192 x 4096 in binary32 with a gate per token 140 us so, 133
  // as here), the first four of them in LDS: each thread its own words, up to 128 KB.
  constexpr int SLOTS = ONE ? 0 : NA * VPT >= 4 ? 4 : EACH ? NA * VPT : 0;
  __shared__ __attribute__((aligned(16))) float sums[(SLOTS ? SLOTS : 1) * 8 * 1024];
  const int sub = __builtin_amdgcn_readfirstlane((int)threadIdx.x / G), t = (int)threadIdx.x - sub * G;
  Row<ONE> rs(red, G >> 6, (sub * G) >> 6);
  const float inv_d = 1.0f / (float)p.cols;
  const bool post = p.z != nullptr, pre = p.dy != nullptr;
  const Cols<VPT> c(p.cols, t, G);
  const Param<VPT, TINY> w_pre(c, pre ? p.w_pre : nullptr, p.p_f32, 1.0f);
  // without EACH, branch_scale G(gate) w_post
  const Param<VPT, TINY, !EACH> w_post(c, post ? p.w_post : nullptr, p.p_f32, 1.0f, post && p.gate_kind == 1 ? p.gate : nullptr,
                          p.gate_act, EACH ? 1.0f : p.branch_scale);
  float acc[NA * VPT][8];
  auto slot = [&](int at, int half) {
    return reinterpret_cast<float4*>(sums) + (at * 2 + half) * 1024 + threadIdx.x;
  };
#pragma unroll
  for (int at = 0; at < NA * VPT; ++at) {
    if (at < SLOTS) *slot(at, 0) = *slot(at, 1) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[at][k] = 0.0f;
  }
  auto add = [&](int a, int i, const float (&v)[8]) {
    const int at = a * VPT + i;
    if (at < SLOTS) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float4* s = slot(at, half);
        float4 o = *s;
        o.x += v[4 * half];
        o.y += v[4 * half + 1];
        o.z += v[4 * half + 2];
        o.w += v[4 * half + 3];
        *s = o;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[at][k] += v[k];
    }
  };

  struct Held {
    Raw8<XF32> dh[VPT], h[VPT];
    Raw8<false> dy[VPT], z[VPT];
    float mh, rh, mz, rz;
  };
  const Rows mine(p.rows, rpw);
  auto fetch = [&](int64_t row, Held& f) {
    const bool live = row < mine.end;
    f.mh = f.rh = f.mz = f.rz = 0.0f;
    if (pre && live) {
      if constexpr (LN) f.mh = p.stats_h[2 * row];
      f.rh = p.stats_h[2 * row + 1];
    }
    if (post && live) {
      if constexpr (LN) f.mz = p.stats_z[2 * row];
      f.rz = p.stats_z[2 * row + 1];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      RowVec x = c.x[i];
      if (!live) x.skip = 8;
      if (pre) {
        f.dy[i] = load_raw<false, TINY>(row_of(p.dy, row, p.lddy, false), x);
        f.h[i] = load_raw<XF32, TINY>(row_of(p.h, row, p.ldh, XF32), x);
      }
      if (p.dh) f.dh[i] = load_raw<XF32, TINY>(row_of(p.dh, row, p.lddh, XF32), x);
      if (post) f.z[i] = load_raw<false, TINY>(row_of(p.z, row, p.ldz, false), x);
    }
  };
  int64_t row0 = mine.first;
  Held next;
  if (AHEAD && row0 < mine.end) fetch(row0 + sub, next);
  for (; row0 < mine.end; row0 += mine.step) {
    const int64_t row = row0 + sub;
    const bool live = row < mine.end;
    if constexpr (!AHEAD) fetch(row, next);
    const Held f = next;
    if (AHEAD && row0 + mine.step < mine.end) fetch(row + mine.step, next);
    float d[VPT][8];   // dH
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) d[i][k] = 0.0f;
    if (p.dh) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) unpack(f.dh[i], row_of(p.dh, row, p.lddh, XF32), c.x[i], d[i]);
    }
    if (pre) {
      float s[LN ? 2 : 1] = {};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float w[8], a[8], xh[8];
        unpack(f.dy[i], row_of(p.dy, row, p.lddy, false), c.x[i], a);
        unpack(f.h[i], row_of(p.h, row, p.ldh, XF32), c.x[i], xh);
        w_pre.get(i, c.x[i], w);
        #pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] = k >= c.x[i].skip ? a[k] : 0.0f;
          xh[k] = a[k] * ((xh[k] - f.mh) * f.rh);
          s[0] = __builtin_fmaf(w[k], xh[k], s[0]);
          if constexpr (LN) s[LN ? 1 : 0] = __builtin_fmaf(w[k], a[k], s[LN ? 1 : 0]);
        }
        if constexpr (LN) add(1, i, a);
        add(0, i, xh);
        one_at_a_time<VPT>();
      }
      rs.sum(s);
      const float s0 = s[0] * inv_d, s1 = LN ? s[LN ? 1 : 0] * inv_d : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float w[8], a[8], xh[8];
        unpack(f.dy[i], row_of(p.dy, row, p.lddy, false), c.x[i], a);
        unpack(f.h[i], row_of(p.h, row, p.ldh, XF32), c.x[i], xh);
        w_pre.get(i, c.x[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          xh[k] = (xh[k] - f.mh) * f.rh;
          const float v = __builtin_fmaf(-xh[k], s0, __builtin_fmaf(a[k], w[k], -s1));
          d[i][k] = __builtin_fmaf(f.rh, v, d[i][k]);
        }
        one_at_a_time<VPT>();
      }
    }
    if (p.dx) {
      const float rscale = post ? p.res_scale : 1.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = rscale * d[i][k];
        store_vec<TINY>(row_of(p.dx, row, p.lddx, XF32), XF32, c.x[i], live, o);
      }
    }
    if (!post) continue;
    float gt = 1.0f, gt_slope = 1.0f;
    if constexpr (EACH) {
      if (p.gate_kind == 2 && live) {
        const float g = reinterpret_cast<const float*>(p.gate)[row];
        gt = gate_value(p.gate_act, g);
        gt_slope = gate_slope(p.gate_act, g);
      }
    }
    // d becomes c = dn w_post; sums of c zh, c, and (EACH) dH n
    float q[EACH ? 3 : (LN ? 2 : 1)] = {};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8], zh[8];
      unpack(f.z[i], row_of(p.z, row, p.ldz, false), c.x[i], zh);
      w_post.get(i, c.x[i], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        zh[k] = (zh[k] - f.mz) * f.rz;
        d[i][k] = k >= c.x[i].skip ? d[i][k] : 0.0f;
      }
      if constexpr (EACH) {
        // (bias and gate one after the other: both in flight, this spilled twice the
        // registers, and layer norm of 8192 x 4096 in binary32 took 177 us, now 155)
        float g[8], dg[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) dg[k] = 0.0f;
        if (LN && p.b_post) load_vec<TINY>(p.b_post, p.p_f32, c.x[i], dg);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dg[k] = d[i][k] * __builtin_fmaf(zh[k], w[k], dg[k]);
          q[EACH ? 2 : 0] += dg[k];
          g[k] = gt;
        }
        __builtin_amdgcn_sched_barrier(0);
        if (p.gate_kind == 3) {
          if (live) load_vec<TINY>(row_of(p.gate, row, p.ldg, 0), 0, c.x[i], g);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            dg[k] = p.branch_scale * dg[k] * gate_slope(p.gate_act, g[k]);
            g[k] = gate_value(p.gate_act, g[k]);
          }
          if (p.dgate) store_vec<TINY>(row_of(p.dgate, row, p.lddg, 0), 0, c.x[i], live, dg);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) d[i][k] *= g[k];
      }
      if constexpr (LN) add(3, i, d[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        zh[k] *= d[i][k];
        w[k] = EACH ? p.branch_scale * w[k] : w[k];
        d[i][k] *= w[k];
        q[0] = __builtin_fmaf(w[k], zh[k], q[0]);
        if constexpr (LN) q[LN ? 1 : 0] += d[i][k];
      }
      add(LN ? 2 : 1, i, zh);
      one_at_a_time<VPT>();
    }
    rs.sum(q);
    const float s0 = q[0] * inv_d, s1 = LN ? q[LN ? 1 : 0] * inv_d : 0.0f;
    if constexpr (EACH) {
      if (p.dgate && p.gate_kind == 2 && t == 0 && live)
        reinterpret_cast<float*>(p.dgate)[row] = p.branch_scale * gt_slope * q[EACH ? 2 : 0];
    }
    if (p.dz) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float zh[8];
        unpack(f.z[i], row_of(p.z, row, p.ldz, false), c.x[i], zh);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          zh[k] = (zh[k] - f.mz) * f.rz;
          zh[k] = f.rz * (__builtin_fmaf(-zh[k], s0, d[i][k]) - s1);
        }
        store_vec<TINY>(row_of(p.dz, row, p.lddz, 0), 0, c.x[i], live, zh);
      }
    }
  }
  // this workgroup's column sums, its rows joined in order: part[a][blockIdx.x][cols]
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    if (a < NA / 2 ? !pre : !post) continue;
    float* out = p.part + ((int64_t)a * gridDim.x + blockIdx.x) * p.cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int slot_at = a * VPT + i;
      const int at = slot_at < SLOTS ? slot_at * 2048 : 0;   // in float4; the registers' through slot 0
      if (slot_at >= SLOTS) {
        __syncthreads();
        float4* s = reinterpret_cast<float4*>(sums) + threadIdx.x;
        const float (&v)[8] = acc[slot_at];
        s[0] = make_float4(v[0], v[1], v[2], v[3]);
        s[1024] = make_float4(v[4], v[5], v[6], v[7]);
      }
      __syncthreads();
      if (sub == 0) {
        float v[8] = {};
        for (int w = 0; w < rpw; ++w)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float4 o = reinterpret_cast<const float4*>(sums)[at + half * 1024 + w * G + t];
            v[4 * half] += o.x;
            v[4 * half + 1] += o.y;
            v[4 * half + 2] += o.z;
            v[4 * half + 3] += o.w;
          }
        store_vec<TINY>(out, 1, c.x[i], true, v);
      }
    }
  }
}

// The column sums over the workgroups: 32 columns per workgroup, 32 groups of
// threads that take every 32nd part, then the groups in order; and from them the
// parameters' gradients.
__global__ void __launch_bounds__(1024) k_norm_join(NormGradParams p, int nparts, int ln) {
  __shared__ float lds[4][32][33];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int na = ln ? 4 : 2;
  const bool post = p.z != nullptr, pre = p.dy != nullptr;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < p.cols) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a >= na || !(a < na / 2 ? pre : post)) continue;
      const float* part = p.part + (int64_t)a * nparts * p.cols + col;
#pragma unroll 8
      for (int q = group; q < nparts; q += 32) s[a] += part[q * p.cols];
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) lds[a][group][lane] = s[a];
  __syncthreads();
  // wavefront a: sum a of the 32 columns, lane's half of the groups
  if (threadIdx.x < 256) {
    const int a = threadIdx.x >> 6, half = (threadIdx.x >> 5) & 1;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += lds[a][half * 16 + w][lane];
    v += __shfl_xor(v, 32, 64);
    __builtin_amdgcn_wave_barrier();
    lds[a][0][lane] = v;   // read by this wavefront only, above, before
  }
  __syncthreads();
  if (threadIdx.x >= 32 || col >= p.cols) return;
#pragma unroll
  for (int a = 0; a < 4; ++a) s[a] = lds[a][0][lane];
  auto put = [&](void* dst, float v) {
    if (dst == nullptr) return;
    if (p.p_f32) reinterpret_cast<float*>(dst)[col] = v;
    else reinterpret_cast<uint16_t*>(dst)[col] = f32_to_bf16_rne(v);
  };
  auto get = [&](const void* src, float other) {
    if (src == nullptr) return other;
    return p.p_f32 ? reinterpret_cast<const float*>(src)[col]
                   : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(src)[col] << 16);
  };
  // (without rows, dy and z may be absent: the sums are then 0)
  put(p.dw_pre, s[0]);
  if (ln) put(p.db_pre, s[1]);
  const float s1 = ln ? s[2] : s[1], s0 = ln ? s[3] : 0.0f;
  const float raw = p.gate_kind == 1 ? get(p.gate, 1.0f) : 1.0f;
  const float g = p.gate_kind == 1 ? gate_value(p.gate_act, raw) : 1.0f;
  put(p.dw_post, p.branch_scale * g * s1);
  if (ln) put(p.db_post, p.branch_scale * g * s0);
  if (p.gate_kind == 1)
    put(p.dgate, p.branch_scale * gate_slope(p.gate_act, raw) *
                     (get(p.w_post, 1.0f) * s1 + (ln ? get(p.b_post, 0.0f) * s0 : 0.0f)));
}

// Vectors per thread, threads per row and rows per workgroup.  A wavefront has
// a row to itself up to 1024 columns, where a barrier would cost more than the
// second vector.
struct Shape {
  int vpt, G, rpw;
  bool one;
};
Shape shape_of(int64_t cols, bool backward) {
  const int v = (int)((cols + 7) / 8);
  if (v <= 128) return {v <= 64 ? 1 : 2, 64, backward ? 8 : 4, true};
  const int vpt = v <= 1024 ? 1 : (v <= 2048 ? 2 : 4);
  const int G = ((v + vpt - 1) / vpt + 63) / 64 * 64;
  return {vpt, G, backward ? 1024 / G : 1, false};
}

// Workgroups of `rpw` rows at a time, at most `most`.
int64_t row_groups(int64_t rows, int rpw, int64_t most) {
  const int64_t n = (rows + rpw - 1) / rpw;
  return n < 1 ? 1 : (n < most ? n : most);
}

// Workgroups of a kernel that run at once on a compute unit, asked once per
// kernel and workgroup size: a grid of more would run its rest after the others
// (4096 rows of 4104 columns: 768 workgroups of which 512 run at once, 47 us).
template <void (*KERNEL)(NormParams)>
int64_t resident(int threads) {
  static std::atomic<int> known[17];
  std::atomic<int>& k = known[threads / 64];
  int n = k.load(std::memory_order_relaxed);
  if (n <= 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, threads, 0) != hipSuccess || n < 1) n = 1;
    k.store(n, std::memory_order_relaxed);
  }
  return n;
}

// f(vectors per thread, ONE) as compile-time constants.
template <typename F>
hipError_t with_shape(const Shape& s, F&& f) {
  using std::integral_constant;
  const integral_constant<bool, true> yes{};
  const integral_constant<bool, false> no{};
  if (s.one) return s.vpt == 1 ? f(integral_constant<int, 1>{}, yes) : f(integral_constant<int, 2>{}, yes);
  if (s.vpt == 1) return f(integral_constant<int, 1>{}, no);
  if (s.vpt == 2) return f(integral_constant<int, 2>{}, no);
  return f(integral_constant<int, 4>{}, no);
}

template <void (*KERNEL)(NormParams)>
hipError_t launch_rows(const NormParams& p, const Shape& sh, hipStream_t s) {
  const int threads = sh.G * sh.rpw;
  const dim3 grid((unsigned)row_groups(p.rows, sh.rpw, device_cu_count() * resident<KERNEL>(threads)));
  hipLaunchKernelGGL(KERNEL, grid, dim3((unsigned)threads), 0, s, p);
  return hipGetLastError();
}
template <int VPT, bool ONE, bool LN, bool XF32>
hipError_t launch_fwd(const NormParams& p, const Shape& sh, hipStream_t s) {
  if constexpr (ONE && VPT == 1) {
    if (p.cols < 8) return p.gate_kind == 3 ? launch_rows<k_norm_fwd<VPT, ONE, LN, XF32, true, true>>(p, sh, s)
                                            : launch_rows<k_norm_fwd<VPT, ONE, LN, XF32, false, true>>(p, sh, s);
  }
  return p.gate_kind == 3 ? launch_rows<k_norm_fwd<VPT, ONE, LN, XF32, true, false>>(p, sh, s)
                          : launch_rows<k_norm_fwd<VPT, ONE, LN, XF32, false, false>>(p, sh, s);
}
template <int VPT, bool ONE, bool LN, bool XF32, bool TINY>
hipError_t launch_bwd_k(const NormGradParams& p, const Shape& sh, dim3 grid, dim3 block, hipStream_t s) {
  if (p.gate_kind >= 2)
    hipLaunchKernelGGL((k_norm_bwd<VPT, ONE, LN, XF32, true, TINY>), grid, block, 0, s, p, sh.G, sh.rpw);
  else
    hipLaunchKernelGGL((k_norm_bwd<VPT, ONE, LN, XF32, false, TINY>), grid, block, 0, s, p, sh.G, sh.rpw);
  return hipGetLastError();
}
template <int VPT, bool ONE, bool LN, bool XF32>
hipError_t launch_bwd(const NormGradParams& p, const Shape& sh, dim3 grid, dim3 block, hipStream_t s) {
  if constexpr (ONE && VPT == 1) {
    if (p.cols < 8) return launch_bwd_k<VPT, ONE, LN, XF32, true>(p, sh, grid, block, s);
  }
  return launch_bwd_k<VPT, ONE, LN, XF32, false>(p, sh, grid, block, s);
}

}  // namespace

int64_t norm_max_cols() { return 1024 * 4 * 8; }

// Workgroups of the backward pass: as many as run at once (each ends in a row of
// column sums, so no more than that).
int64_t norm_parts(int64_t rows, int64_t cols) {
  const Shape sh = shape_of(cols, true);
  return row_groups(rows, sh.rpw, device_cu_count());
}

hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const Shape sh = shape_of(p.cols, false);
  return with_shape(sh, [&](auto vpt, auto one) {
    constexpr int VPT = decltype(vpt)::value;
    constexpr bool ONE = decltype(one)::value;
    if (p.layer) return p.x_f32 ? launch_fwd<VPT, ONE, true, true>(p, sh, s)
                                : launch_fwd<VPT, ONE, true, false>(p, sh, s);
    return p.x_f32 ? launch_fwd<VPT, ONE, false, true>(p, sh, s)
                   : launch_fwd<VPT, ONE, false, false>(p, sh, s);
  });
}

hipError_t launch_norm_bwd(const NormGradParams& p, hipStream_t s) {
  const int64_t parts = norm_parts(p.rows, p.cols);
  const Shape sh = shape_of(p.cols, true);
  const dim3 grid((unsigned)parts), block((unsigned)(sh.G * sh.rpw));
  const hipError_t e = with_shape(sh, [&](auto vpt, auto one) {
    constexpr int VPT = decltype(vpt)::value;
    constexpr bool ONE = decltype(one)::value;
    if (p.layer) return p.x_f32 ? launch_bwd<VPT, ONE, true, true>(p, sh, grid, block, s)
                                : launch_bwd<VPT, ONE, true, false>(p, sh, grid, block, s);
    return p.x_f32 ? launch_bwd<VPT, ONE, false, true>(p, sh, grid, block, s)
                   : launch_bwd<VPT, ONE, false, false>(p, sh, grid, block, s);
  });
  if (e != hipSuccess) return e;
  if (!p.dw_pre && !p.db_pre && !p.dw_post && !p.db_post && !(p.dgate && p.gate_kind == 1)) return hipSuccess;
  hipLaunchKernelGGL(k_norm_join, dim3((unsigned)((p.cols + 31) / 32)), dim3(1024), 0, s, p, (int)parts, p.layer);
  return hipGetLastError();
}

}  // namespace fp8lin
