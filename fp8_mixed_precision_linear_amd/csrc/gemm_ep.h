// gemm_ep.h -- what the linear's epilogue does to a row of eight outputs, and
// how a wavefront's accumulators become such rows.
//
// With v the dequantised product in binary32:
//   forward   u = v + bias[n],  aux = bf16(u),  d = act(u) + res_scale residual
//   backward  d = v act'(aux),  dbias[n] = sum_m d
// and D = d as BF16 or FP32, or as FP8 codes encode(d * d_scale) with their
// transposed copy; amax = max |d| (of the rounded values for BF16).
//
// The matrix instruction leaves a lane with 4 columns of 16 different rows;
// rows of D, aux and residual want 16 bytes per lane and whole lines.  So the
// accumulators pass through LDS in strips of 16 rows, in binary32 (the
// activation and the residual act on the unrounded product), each wavefront in
// its own region, without a barrier.  A lane then holds RPL neighbouring rows
// of the same 8 columns throughout: bias is read once, the bias gradient is
// summed in registers, and the transposed codes of RPL rows leave as one word.
#pragma once

#include "op_device.h"
#include "launch.h"

namespace fp8lin {

namespace {

typedef float v4f_ep __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(1))) Pk16a1 { uint32_t v[4]; };

template <int ACT>
__device__ __forceinline__ void act8(float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = act_value<ACT>(v[k]);
}
template <int ACT>
__device__ __forceinline__ void slope8(float (&v)[8], const float (&u)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= act_slope<ACT>(u[k]);
}
// A uniform run-time choice per eight values: one scalar branch.
__device__ __forceinline__ void apply_act(int act, float (&v)[8]) {
  switch (act) {
    case 1: act8<1>(v); break;
    case 2: act8<2>(v); break;
    case 3: act8<3>(v); break;
    case 4: act8<4>(v); break;
    default: break;
  }
}
__device__ __forceinline__ void apply_slope(int act, float (&v)[8], const float (&u)[8]) {
  switch (act) {
    case 1: slope8<1>(v, u); break;
    case 2: slope8<2>(v, u); break;
    case 3: slope8<3>(v, u); break;
    case 4: slope8<4>(v, u); break;
    default: break;
  }
}

// One wavefront's columns n0 .. n0 + WTN - 1, lane's columns c .. c + 7.
template <int WTN, bool OUT8>
struct EpWave {
  static constexpr int LPR = WTN / 8;        // lanes per row
  static constexpr int RPL = WTN / 32;       // rows per lane and strip of 16
  const GemmParams& p;
  const EpParams& e;
  int lane, cq, rg, nv;
  int64_t c;
  float bias[8], db[8];
  uint32_t amax = 0;
  float so;

  __device__ __forceinline__ EpWave(const GemmParams& p_, const EpParams& e_, int64_t n0, int lane_)
      : p(p_), e(e_), lane(lane_), cq(lane_ % LPR), rg(lane_ / LPR), c(n0 + 8 * (lane_ % LPR)) {
    const int64_t left = p.N - c;
    nv = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) { bias[k] = 0.0f; db[k] = 0.0f; }
    if (e.bias) load8(e.bias, e.bias_f32, c, nv, bias);
    so = OUT8 ? p.d_scale[0] : 1.0f;
  }

  // What the strip of rows m0 .. m0 + 15 reads beside the product: the
  // pre-activation (backward) or the residual.
  __device__ __forceinline__ void fetch(int64_t m0, float (&o)[RPL][8]) {
    const void* src = e.backward ? (e.act ? e.aux : nullptr) : e.residual;
    if (src == nullptr) return;
    const int f32 = e.backward ? 0 : e.res_f32;
    const int64_t ld = e.backward ? e.ldaux : e.ldres;
#pragma unroll
    for (int t = 0; t < RPL; ++t) {
      const int64_t m = m0 + rg * RPL + t;
      load8(src, f32, m * ld + c, m < p.M ? nv : 0, o[t]);
    }
  }

  // The strip: v[t] is row m0 + rg RPL + t.  tl: column-major codes of the
  // wavefront (TS bytes per column, this strip's rows at byte tr), if D_t.
  template <int TS>
  __device__ __forceinline__ void strip(int64_t m0, float (&v)[RPL][8], const float (&o)[RPL][8], uint8_t* tl,
                                        int tr) {
    uint32_t lo[RPL], hi[RPL];
#pragma unroll
    for (int t = 0; t < RPL; ++t) {
      const int64_t m = m0 + rg * RPL + t;
      const int n = m < p.M ? nv : 0;
      if (!e.backward) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[t][k] += bias[k];
        if (e.aux) store8(const_cast<void*>(e.aux), 0, m * e.ldaux + c, n, v[t]);
        apply_act(e.act, v[t]);
        if (e.residual) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[t][k] = __builtin_fmaf(e.res_scale, o[t][k], v[t][k]);
        }
      } else {
        apply_slope(e.act, v[t], o[t]);
#pragma unroll
        for (int k = 0; k < 8; ++k) db[k] += k < n ? v[t][k] : 0.0f;
      }
      if (p.d_amax) {
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max_u32(amax, k < n ? abs_bits(v[t][k]) : 0u);
      }
      if constexpr (OUT8) {
        codes8(p.d_fp8 - 1, v[t], so, lo[t], hi[t]);
        store8_codes(reinterpret_cast<uint8_t*>(p.D), m * p.ldd + c, n, lo[t], hi[t]);
      } else {
        store8(p.D, p.d_f32, m * p.ldd + c, n, v[t]);
      }
    }
    if constexpr (OUT8) {
      if (p.D_t) {
        uint8_t* dst = tl + (8 * cq) * TS + tr + rg * RPL;
        if constexpr (RPL == 4) {
          uint32_t w[8];
          transpose4x4(lo[0], lo[1], lo[2], lo[3], w[0], w[1], w[2], w[3]);
          transpose4x4(hi[0], hi[1], hi[2], hi[3], w[4], w[5], w[6], w[7]);
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint32_t*>(dst + k * TS) = w[k];
        } else {
          static_assert(RPL == 2, "two or four rows per lane");
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t a = (k < 4 ? lo[0] : hi[0]) >> (8 * (k & 3)), b = (k < 4 ? lo[1] : hi[1]) >> (8 * (k & 3));
            *reinterpret_cast<uint16_t*>(dst + k * TS) = (uint16_t)((a & 0xFFu) | ((b & 0xFFu) << 8));
          }
        }
      }
    }
  }

  // Accumulators to strips.  acc[i][j] of lane (g, l16): row r0 + 16 i + l16,
  // columns n0 + 16 j + 4 g .. + 3.  wl: 64 WTN bytes for the strip, then
  // (D_t) WTN columns of 16 TI + 16 bytes, wavefront-private.
  template <int TI, int TJ, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl) {
    static_assert(16 * TJ == WTN, "the wavefront's columns");
    constexpr int TS = 16 * TI + 16, CH = WTN / 4;
    const int g = lane >> 4, l16 = lane & 15;
    uint8_t* tl = wl + 64 * WTN;
    float o[2][RPL][8];
    fetch(r0, o[0]);
    ep_for<0, TI>([&](auto itag) {
      constexpr int i = decltype(itag)::value;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        float4 w;
        w.x = deq(i, j, 0, acc[i][j][0]);
        w.y = deq(i, j, 1, acc[i][j][1]);
        w.z = deq(i, j, 2, acc[i][j][2]);
        w.w = deq(i, j, 3, acc[i][j][3]);
        *reinterpret_cast<float4*>(wl + l16 * (WTN * 4) + (((4 * j + g) ^ (l16 & (CH - 1))) << 4)) = w;
      }
      if constexpr (i + 1 < TI) fetch(r0 + 16 * (i + 1), o[(i + 1) & 1]);
      float v[RPL][8];
#pragma unroll
      for (int t = 0; t < RPL; ++t) {
        const int r = rg * RPL + t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 w =
              *reinterpret_cast<const float4*>(wl + r * (WTN * 4) + (((2 * cq + h) ^ (r & (CH - 1))) << 4));
          v[t][4 * h] = w.x;
          v[t][4 * h + 1] = w.y;
          v[t][4 * h + 2] = w.z;
          v[t][4 * h + 3] = w.w;
        }
      }
      strip<TS>(r0 + 16 * i, v, o[i & 1], tl, 16 * i);
    });
    if constexpr (OUT8) {
      asm volatile("" ::: "memory");   // the codes were written as other types than they are read
      if (p.D_t) flush_t<TS, 16 * TI>(tl, r0, n0);
    }
  }

  // The column-major codes of ROWS rows to D_t, 16 bytes per lane.
  template <int TS, int ROWS>
  __device__ __forceinline__ void flush_t(const uint8_t* tl, int64_t r0, int64_t n0) {
    constexpr int LPC = ROWS / 16;
    const int q = lane % LPC;
    const int64_t m = r0 + 16 * q, left = p.M - m;
#pragma unroll 4
    for (int k = lane / LPC; k < WTN; k += 64 / LPC) {
      const int64_t n = n0 + k;
      if (n >= p.N || left <= 0) continue;
      const uint4 w = *reinterpret_cast<const uint4*>(tl + k * TS + 16 * q);
      uint8_t* dst = p.D_t + n * p.ldt + m;
      if (left >= 16) {
        Pk16a1 a;
        a.v[0] = w.x; a.v[1] = w.y; a.v[2] = w.z; a.v[3] = w.w;
        *reinterpret_cast<Pk16a1*>(dst) = a;
      } else {
        for (int b = 0; b < (int)left; ++b) dst[b] = tl[k * TS + 16 * q + b];
      }
    }
  }

  // Column sums of the wavefront's rows to part[row][N] (row: which rows of
  // the sum these are), joined in a fixed order by k_ep_dbias.
  __device__ __forceinline__ void put_dbias(int64_t row) {
    if (e.dbias == nullptr) return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int off = LPR; off < 64; off <<= 1) db[k] += __shfl_xor(db[k], off, 64);
    if (rg == 0 && nv > 0) store8(e.part, 1, row * p.N + c, nv, db);
  }

  // max |d| of the wavefront as stored.
  __device__ __forceinline__ uint32_t amax_bits() {
    uint32_t a = wave_max(amax);
    if (!OUT8 && !p.d_f32) a = (uint32_t)f32_to_bf16_rne(__uint_as_float(a)) << 16;
    return a;
  }

  // compile-time loop: an array indexed by it stays in registers
  template <int B, int E, typename F>
  static __device__ __forceinline__ void ep_for(F&& f) {
    if constexpr (B < E) {
      f(std::integral_constant<int, B>{});
      ep_for<B + 1, E>(f);
    }
  }
};

template <int NW>
__device__ __forceinline__ void ep_amax(float* d_amax, uint32_t bits, int lane, int wave) {
  __shared__ uint32_t wmax[NW];
  if (lane == 0) wmax[wave] = bits;
  __syncthreads();
  if (wave == 0 && lane == 0) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = max_u32(m, wmax[w]);
    if (m != 0u) atomic_max_bits(d_amax, m);
  }
}

}  // namespace

}  // namespace fp8lin
