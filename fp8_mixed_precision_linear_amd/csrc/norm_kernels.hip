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
// the cast of the next linear's operand without a pass over y of its own.
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
// Bound: HBM.  A row stays in registers between its loads and its stores, so
// each element is read and written once; the column sums are kept in
// registers over the rows that a workgroup takes and joined by a second, small
// kernel in a fixed order (no atomics: equal inputs give equal bits).
#include "op_device.h"
#include "launch.h"

namespace fp8lin {

namespace {

// Sums of NV values per thread over the G threads of a row (G = 64: one
// wavefront, no barrier).  Two LDS buffers in turn, so one barrier per sum is
// enough: whoever writes a buffer again has passed the barrier in between,
// which every reader of its old values reached after reading.
template <int G>
struct RowSum {
  float* lds;   // 2 * (G / 64) * 2 floats
  int turn = 0;
  __device__ explicit RowSum(float* l) : lds(l) {}
  template <int NV>
  __device__ __forceinline__ void sum(float (&v)[NV]) {
    static_assert(NV <= 4, "two buffers of four values per wavefront");
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = wave_sum(v[k]);
    if constexpr (G > 64) {
      constexpr int NW = G / 64;
      float* b = lds + turn * NW * 4;
      turn ^= 1;
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k) b[wave * 4 + k] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += b[w * 4 + k];
        v[k] = s;
      }
    }
  }
  __device__ __forceinline__ uint32_t max(uint32_t m) {
    m = wave_max(m);
    if constexpr (G > 64) {
      constexpr int NW = G / 64;
      uint32_t* b = reinterpret_cast<uint32_t*>(lds + turn * NW * 4);
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) b[(threadIdx.x >> 6) * 4] = m;
      __syncthreads();
      m = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) m = max_u32(m, b[w * 4]);
    }
    return m;
  }
};

constexpr int threads_of(int G) { return G < 256 ? 256 : G; }

// G threads per row (G = 64: four rows per 256-thread workgroup), VPT vectors
// of 8 columns per thread.
template <int G, int VPT, bool LN>
__global__ void __launch_bounds__(threads_of(G)) k_norm_fwd(NormParams p) {
  constexpr int NT = threads_of(G), RPW = NT / G;
  __shared__ float red[2 * 4 * (NT / 64)];
  __shared__ uint32_t amax_part[NT / 64];
  const int t = threadIdx.x % G, sub = threadIdx.x / G;
  RowSum<G> rs(red);
  const float inv_d = 1.0f / (float)p.cols;
  const bool post = p.z != nullptr, pre = p.y != nullptr || p.y8 != nullptr;
  uint32_t amax = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < p.rows; row += (int64_t)gridDim.x * RPW) {
    float h[VPT][8];
    int n[VPT];
    int64_t c[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      c[i] = 8 * (int64_t)(t + i * G);
      const int64_t left = p.cols - c[i];
      n[i] = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
      load8(p.x, p.x_f32, row * p.ldx + c[i], n[i], h[i]);
    }
    if (post) {
      float z[VPT][8];
#pragma unroll
      for (int i = 0; i < VPT; ++i) load8(p.z, 0, row * p.ldz + c[i], n[i], z[i]);
      float m = 0.0f;
      if constexpr (LN) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) s[0] += z[i][k];
        rs.sum(s);
        m = s[0] * inv_d;
      }
      float q[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          z[i][k] = LN && k >= n[i] ? 0.0f : z[i][k] - m;
          q[0] = __builtin_fmaf(z[i][k], z[i][k], q[0]);
        }
      rs.sum(q);
      const float r = rsqrtf(q[0] * inv_d + p.eps);
      if (p.stats_z && t == 0) {
        p.stats_z[2 * row] = m;
        p.stats_z[2 * row + 1] = r;
      }
      const float gt = p.gate_kind == 2 ? gate_value(p.gate_act, reinterpret_cast<const float*>(p.gate)[row]) : 1.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float w[8], g[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) { w[k] = 1.0f; b[k] = 0.0f; g[k] = gt; }
        if (p.w_post) load8(p.w_post, p.p_f32, c[i], n[i], w);
        if (LN && p.b_post) load8(p.b_post, p.p_f32, c[i], n[i], b);
        if (p.gate_kind == 1 || p.gate_kind == 3) {
          if (p.gate_kind == 1) load8(p.gate, p.p_f32, c[i], n[i], g);
          else load8(p.gate, 0, row * p.ldg + c[i], n[i], g);
          if (p.gate_act != 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = gate_value(p.gate_act, g[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float nv = __builtin_fmaf(z[i][k] * r, w[k], b[k]);
          h[i][k] = __builtin_fmaf(p.res_scale, h[i][k], p.branch_scale * (g[k] * nv));
        }
        store8(p.h, p.x_f32, row * p.ldh + c[i], n[i], h[i]);
      }
    }
    if (!pre) continue;
    float m = 0.0f;
    if constexpr (LN) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] += k < n[i] ? h[i][k] : 0.0f;
      rs.sum(s);
      m = s[0] * inv_d;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][k] = k < n[i] ? h[i][k] - m : 0.0f;
        q[0] = __builtin_fmaf(h[i][k], h[i][k], q[0]);
      }
    rs.sum(q);
    const float r = rsqrtf(q[0] * inv_d + p.eps);
    if (p.stats_h && t == 0) {
      p.stats_h[2 * row] = m;
      p.stats_h[2 * row + 1] = r;
    }
    uint32_t row_max = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8], b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) { w[k] = 1.0f; b[k] = 0.0f; }
      if (p.w_pre) load8(p.w_pre, p.p_f32, c[i], n[i], w);
      if (LN && p.b_pre) load8(p.b_pre, p.p_f32, c[i], n[i], b);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __builtin_fmaf(h[i][k] * r, w[k], b[k]);
      if (p.y) store8(p.y, 0, row * p.ldy + c[i], n[i], h[i]);
      if (p.y8) {
        if (p.y8_scaling == 1) {   // one scale per 128 columns: 16 neighbouring lanes
          uint32_t mx = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = max_u32(mx, k < n[i] ? abs_bits(h[i][k]) : 0u);
          mx = row16_max(mx);
          float s = 1.0f, si = 1.0f;
          scale_from_amax(__uint_as_float(mx), p.y8_fmt == 0 ? kMaxE4M3 : kMaxE5M2, 0, s, si);
          if (n[i] > 0) {
            if ((t & 15) == 0) p.y8_sinv[(c[i] >> 7) * p.rows + row] = si;
            uint32_t lo, hi;
            codes8(p.y8_fmt, h[i], s, lo, hi);
            store8_codes(p.y8, row * p.ldy8 + c[i], n[i], lo, hi);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) row_max = max_u32(row_max, k < n[i] ? abs_bits(h[i][k]) : 0u);
        }
      }
    }
    if (p.y8 && p.y8_scaling != 1) {
      float s = 1.0f, si = 1.0f;
      if (p.y8_scaling == 5) {
        row_max = rs.max(row_max);
        scale_from_amax(__uint_as_float(row_max), p.y8_fmt == 0 ? kMaxE4M3 : kMaxE5M2, 0, s, si);
        if (t == 0) p.y8_sinv[row] = si;
      } else {
        s = p.y8_scale[0];
        amax = max_u32(amax, row_max);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        uint32_t lo, hi;
        codes8(p.y8_fmt, h[i], s, lo, hi);
        if (n[i] > 0) store8_codes(p.y8, row * p.ldy8 + c[i], n[i], lo, hi);
      }
    }
  }
  if (p.y8_amax) {   // one filtered atomic maximum per workgroup (order-free)
    amax = wave_max(amax);
    if ((threadIdx.x & 63) == 0) amax_part[threadIdx.x >> 6] = amax;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < NT / 64; ++w) amax = max_u32(amax, amax_part[w]);
      if (amax != 0u) atomic_max_bits(p.y8_amax, amax);
    }
  }
}

// Column sums of the backward pass, in this order in the workspace: dw_pre,
// db_pre, S1 (dw_post), S0 (db_post); without LN only the first and third.
template <int G, int VPT, bool LN>
__global__ void __launch_bounds__(threads_of(G)) k_norm_bwd(NormGradParams p) {
  constexpr int NT = threads_of(G), RPW = NT / G, NA = LN ? 4 : 2;
  __shared__ float red[2 * 4 * (NT / 64)];
  __shared__ float join[RPW > 1 ? RPW * G * 8 : 1];
  const int t = threadIdx.x % G, sub = threadIdx.x / G;
  RowSum<G> rs(red);
  const float inv_d = 1.0f / (float)p.cols;
  const bool post = p.z != nullptr, pre = p.dy != nullptr;
  float acc[NA][VPT][8];
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[a][i][k] = 0.0f;
  int n[VPT];
  int64_t c[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    c[i] = 8 * (int64_t)(t + i * G);
    const int64_t left = p.cols - c[i];
    n[i] = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  }
  for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < p.rows; row += (int64_t)gridDim.x * RPW) {
    float d[VPT][8];   // dH
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) d[i][k] = 0.0f;
      if (p.dh) load8(p.dh, p.x_f32, row * p.lddh + c[i], n[i], d[i]);
    }
    if (pre) {
      float a[VPT][8], xh[VPT][8];
      const float m = LN ? p.stats_h[2 * row] : 0.0f, r = p.stats_h[2 * row + 1];
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float w[8];
        load8(p.dy, 0, row * p.lddy + c[i], n[i], a[i]);
        load8(p.h, p.x_f32, row * p.ldh + c[i], n[i], xh[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 1.0f;
        if (p.w_pre) load8(p.w_pre, p.p_f32, c[i], n[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          xh[i][k] = (xh[i][k] - m) * r;
          acc[0][i][k] = __builtin_fmaf(a[i][k], xh[i][k], acc[0][i][k]);
          if constexpr (LN) acc[1][i][k] += a[i][k];
          a[i][k] *= w[k];   // dy is 0 past the row's end
          s[0] = __builtin_fmaf(a[i][k], xh[i][k], s[0]);
          if constexpr (LN) s[1] += a[i][k];
        }
      }
      rs.sum(s);
      const float s0 = s[0] * inv_d, s1 = LN ? s[1] * inv_d : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          d[i][k] = __builtin_fmaf(r, a[i][k] - s1 - xh[i][k] * s0, d[i][k]);
    }
    const float rscale = post ? p.res_scale : 1.0f;
    if (p.dx) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = rscale * d[i][k];
        store8(p.dx, p.x_f32, row * p.lddx + c[i], n[i], o);
      }
    }
    if (post) {
      float zh[VPT][8];
      const float m = LN ? p.stats_z[2 * row] : 0.0f, r = p.stats_z[2 * row + 1];
      const float gt = p.gate_kind == 2 ? gate_value(p.gate_act, reinterpret_cast<const float*>(p.gate)[row]) : 1.0f;
      float s[3] = {0.0f, 0.0f, 0.0f};   // c zh, c, dH n
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float w[8], g[8], b[8];
        load8(p.z, 0, row * p.ldz + c[i], n[i], zh[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) { w[k] = 1.0f; b[k] = 0.0f; g[k] = gt; }
        if (p.w_post) load8(p.w_post, p.p_f32, c[i], n[i], w);
        if (LN && p.b_post && p.dgate) load8(p.b_post, p.p_f32, c[i], n[i], b);
        if (p.gate_kind == 1 || p.gate_kind == 3) {
          if (p.gate_kind == 1) load8(p.gate, p.p_f32, c[i], n[i], g);
          else load8(p.gate, 0, row * p.ldg + c[i], n[i], g);
          if (p.gate_act != 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = gate_value(p.gate_act, g[k]);
          }
        }
        float dg[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          zh[i][k] = (zh[i][k] - m) * r;
          const float dk = k < n[i] ? d[i][k] : 0.0f;
          // a channel gate leaves its factor to the join
          const float u = p.gate_kind == 1 ? dk : g[k] * dk;
          constexpr int A1 = LN ? 2 : 1;
          acc[A1][i][k] = __builtin_fmaf(u, zh[i][k], acc[A1][i][k]);
          if constexpr (LN) acc[LN ? 3 : 0][i][k] += u;
          const float nv = __builtin_fmaf(zh[i][k], w[k], b[k]);
          s[2] = __builtin_fmaf(dk, nv, s[2]);
          dg[k] = p.branch_scale * dk * nv * gate_slope(p.gate_act, g[k]);
          const float cc = p.branch_scale * g[k] * dk * w[k];
          s[0] = __builtin_fmaf(cc, zh[i][k], s[0]);
          s[1] += cc;
          d[i][k] = cc;
        }
        if (p.dgate && p.gate_kind == 3) store8(p.dgate, 0, row * p.lddg + c[i], n[i], dg);
      }
      rs.sum(s);
      const float s0 = s[0] * inv_d, s1 = LN ? s[1] * inv_d : 0.0f;
      if (p.dgate && p.gate_kind == 2 && t == 0)
        reinterpret_cast<float*>(p.dgate)[row] = p.branch_scale * gate_slope(p.gate_act, gt) * s[2];
      if (p.dz) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = r * (d[i][k] - s1 - zh[i][k] * s0);
          store8(p.dz, 0, row * p.lddz + c[i], n[i], o);
        }
      }
    }
  }
  // this workgroup's column sums: part[a][blockIdx.x][cols]
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    const bool of_pre = a < NA / 2;
    if (of_pre ? !pre : !post) continue;
    float* out = p.part + ((int64_t)a * gridDim.x + blockIdx.x) * p.cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if constexpr (RPW > 1) {   // the rows' wavefronts are joined first
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) join[(sub * G + t) * 8 + k] = acc[a][i][k];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < RPW; ++w) s += join[(w * G + t) * 8 + k];
            acc[a][i][k] = s;
          }
        }
      }
      if (sub == 0) store8(out, 1, c[i], n[i], acc[a][i]);
    }
  }
}

// The column sums over the workgroups, 64 columns by 16 parts at a time, and
// from them the parameters' gradients.
__global__ void __launch_bounds__(1024) k_norm_join(NormGradParams p, int nparts, int ln) {
  __shared__ float lds[4][16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  const int na = ln ? 4 : 2;
  const bool post = p.z != nullptr, pre = p.dy != nullptr;
  for (int a = 0; a < na; ++a) {
    float s = 0.0f;
    if (col < p.cols && (a < na / 2 ? pre : post))
      for (int q = wave; q < nparts; q += 16) s += p.part[((int64_t)a * nparts + q) * p.cols + col];
    lds[a][wave][lane] = s;
  }
  __syncthreads();
  if (wave != 0 || col >= p.cols) return;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int a = 0; a < na; ++a)
    for (int w = 0; w < 16; ++w) s[a] += lds[a][w][lane];
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
  const float g = p.gate_kind == 1 ? gate_value(p.gate_act, get(p.gate, 1.0f)) : 1.0f;
  put(p.dw_post, p.branch_scale * g * s1);
  if (ln) put(p.db_post, p.branch_scale * g * s0);
  if (p.gate_kind == 1)
    put(p.dgate, p.branch_scale * gate_slope(p.gate_act, g) *
                     (get(p.w_post, 1.0f) * s1 + (ln ? get(p.b_post, 0.0f) * s0 : 0.0f)));
}

// Threads per row and vectors per thread for a number of columns.
template <typename F>
hipError_t for_cols(int64_t cols, F&& f) {
  const int64_t v = (cols + 7) / 8;
#define FP8LIN_ROW(G, VPT) \
  if (v <= (int64_t)(G) * (VPT)) return f(std::integral_constant<int, G>{}, std::integral_constant<int, VPT>{})
  FP8LIN_ROW(64, 1);
  FP8LIN_ROW(64, 2);
  FP8LIN_ROW(256, 1);
  FP8LIN_ROW(256, 2);
  FP8LIN_ROW(512, 2);
  FP8LIN_ROW(1024, 2);
  FP8LIN_ROW(1024, 4);
#undef FP8LIN_ROW
  return hipErrorInvalidValue;
}

}  // namespace

int64_t norm_max_cols() { return 1024 * 4 * 8; }

int64_t norm_parts(int64_t rows) {
  const int64_t cu = device_cu_count();
  return rows < cu ? (rows > 0 ? rows : 1) : cu;
}

hipError_t launch_norm_fwd(const NormParams& p, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  return for_cols(p.cols, [&](auto g, auto vpt) {
    constexpr int G = decltype(g)::value, VPT = decltype(vpt)::value, NT = threads_of(G), RPW = NT / G;
    const int64_t want = (p.rows + RPW - 1) / RPW, most = device_cu_count() * (2048 / NT);
    const dim3 grid((unsigned)(want < most ? want : most)), block(NT);
    if (p.layer) hipLaunchKernelGGL((k_norm_fwd<G, VPT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((k_norm_fwd<G, VPT, false>), grid, block, 0, s, p);
    return hipGetLastError();
  });
}

hipError_t launch_norm_bwd(const NormGradParams& p, hipStream_t s) {
  const int64_t parts = norm_parts(p.rows);
  const hipError_t e = for_cols(p.cols, [&](auto g, auto vpt) {
    constexpr int G = decltype(g)::value, VPT = decltype(vpt)::value;
    const dim3 grid((unsigned)parts), block(threads_of(G));
    if (p.layer) hipLaunchKernelGGL((k_norm_bwd<G, VPT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((k_norm_bwd<G, VPT, false>), grid, block, 0, s, p);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_norm_join, dim3((unsigned)((p.cols + 63) / 64)), dim3(1024), 0, s, p, (int)parts, p.layer);
  return hipGetLastError();
}

}  // namespace fp8lin
