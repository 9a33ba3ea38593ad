// gemm_gated.h -- the gated pair of a feed-forward block as the epilogue of an FP8
// product: what happens to a row of eight outputs, forward and backward, and how a
// wavefront's sums become such rows.
//
// Forward, with g and u the two halves of a token's product (gate and up projection, in
// binary32, biases added):  h = act(g) u;  D = h as BF16 or FP32, or as FP8 codes
// encode(h * d_scale) with their transposed copy.  g and u may be kept, in BF16 or as a
// checkpoint (checkpoint.h).
// Backward, with v the product with the next linear's weights and g, u as kept:
//   dg = v u act'(g),  du = v act(g);  D = (dg | du), dbias = their column sums.
//
// Forward the two factors of an output have to meet in one lane.  So B's rows are taken
// 16 of the gate, the same 16 of the up projection, and so on (half_of, pair_of in
// fp8_device.h): the matrix instruction's column tiles alternate, and a strip of 16 rows in
// LDS (see gemm_ep.h) holds both factors of the outputs.  A lane reads eight of each.
// The checkpoint's blocks are 32 outputs of a row, four neighbouring lanes: no exchange
// beyond a quad, and none between wavefronts.
#pragma once

#include "gemm_ep.h"
#include "checkpoint.h"

namespace fp8lin {

namespace {

// act(u), and act(u) beside act'(u), which share their exponential and reciprocal.  A
// uniform run-time choice per eight values.  SiLU, with s = 1 / (1 + e^-u), has the
// slope s + u s (1 - s).
__device__ __forceinline__ void act_of(int act, const float (&u)[8], float (&a)[8]) {
  if (act == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = u[k] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * u[k]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = u[k];
    activate<false>(act, a, u);
  }
}
template <int E>
__device__ __forceinline__ void act_and_slope(int act, const float (&u)[E], float (&a)[E], float (&s)[E]) {
  if (act == 4) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float g = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * u[k]));
      a[k] = u[k] * g;
      s[k] = __builtin_fmaf(a[k], 1.0f - g, g);
    }
  } else if (act == 3) {
    const SigmoidForm f(act);
#pragma unroll
    for (int k = 0; k < E; ++k) f.both(u[k], a[k], s[k]);
  } else if (act == 2) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      a[k] = gelu_erf<false>(u[k]);
      s[k] = gelu_erf<true>(u[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      a[k] = act == 1 && u[k] <= 0.0f ? 0.0f : u[k];
      s[k] = act == 1 && !(u[k] > 0.0f) ? 0.0f : 1.0f;
    }
  }
}

// Eight values x as FP8 codes.  `tame`: none of them is a NaN or beyond the format's
// largest, so they need neither saturation nor a patch (a third of the instructions).
template <int FMT>
__device__ __forceinline__ void encode_tame(const float (&x)[8], uint32_t& lo, uint32_t& hi) {
  int a, b;
  if constexpr (FMT == 0) {
    a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], b, true);
  } else {
    a = __builtin_amdgcn_cvt_pk_bf8_f32(x[0], x[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_bf8_f32(x[2], x[3], a, true);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(x[4], x[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(x[6], x[7], b, true);
  }
  lo = (uint32_t)a;
  hi = (uint32_t)b;
}
__device__ __forceinline__ void codes_of(int fp8, bool tame, const float (&x)[8], uint32_t& lo, uint32_t& hi) {
  if (fp8 == 1) {
    if (__builtin_expect(tame, 1)) encode_tame<0>(x, lo, hi);
    else encode8<0>(x, lo, hi);
  } else {
    if (__builtin_expect(tame, 1)) encode_tame<1>(x, lo, hi);
    else encode8<1>(x, lo, hi);
  }
}
// The first `bytes` of NW dwords to byte address p, each lane by itself: what lies in
// whole dwords of memory as those, the ends as bytes and pairs of them.  A tile's few rows
// wait for instructions, not for memory: with the lanes' exchange of store_row, and
// partial vectors value by value, 4096 x 4095 x 4096 took 123 us backward instead of 111,
// 177 forward instead of 174, 1037 x 1999 x 2304 backward 29.8 instead of 27.7 (on rows
// that start on a dword 26.1 instead of 26.7).
template <int NW>
__device__ __forceinline__ void put_words(uint8_t* p, int bytes, const uint32_t (&w)[NW]) {
  struct __attribute__((packed, aligned(4))) Words { uint32_t v[NW]; };
  struct __attribute__((packed, aligned(4))) Rest { uint32_t v[NW - 1]; };
  const uint32_t lead = (0u - (uint32_t)reinterpret_cast<uintptr_t>(p)) & 3u;   // bytes before the first whole dword
  const bool whole = bytes <= 0 || (bytes == 4 * NW && lead == 0);
  if (__builtin_amdgcn_ballot_w64(!whole) == 0) {
    if (bytes > 0) {
      Words a;
#pragma unroll
      for (int k = 0; k < NW; ++k) a.v[k] = w[k];
      *reinterpret_cast<Words*>(p) = a;
    }
    return;
  }
  if (bytes <= 0) return;
  auto ends = [](uint8_t* q, uint32_t n, uint32_t v, bool odd_first) {   // up to three bytes
    uint32_t at = 0;
    if (odd_first && (n & 1)) { *q = (uint8_t)v; at = 1; }
    if (n & 2) { *reinterpret_cast<uint16_t*>(q + at) = (uint16_t)(v >> (8 * at)); at += 2; }
    if (!odd_first && (n & 1)) q[at] = (uint8_t)(v >> (8 * at));
  };
  const int first = (int)lead < bytes ? (int)lead : bytes, rest = bytes - first;
  uint8_t* q = p + first;
  uint32_t a[NW];
#pragma unroll
  for (int k = 0; k < NW; ++k) a[k] = __builtin_amdgcn_alignbyte(k + 1 < NW ? w[k + 1] : 0u, w[k], lead);
  ends(p, (uint32_t)first, w[0], lead == (uint32_t)first);
  if (bytes == 4 * NW) {   // (not aligned, so one dword is left of its own)
    Rest b;
#pragma unroll
    for (int k = 0; k < NW - 1; ++k) b.v[k] = a[k];
    *reinterpret_cast<Rest*>(q) = b;
    if (lead == 0) reinterpret_cast<uint32_t*>(q)[NW - 1] = a[NW - 1];
    else ends(q + 4 * (NW - 1), 4 - lead, a[NW - 1], false);
  } else {
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      if (4 * k + 4 <= rest) reinterpret_cast<uint32_t*>(q)[k] = a[k];
      else if (4 * k < rest) ends(q + 4 * k, (uint32_t)(rest - 4 * k), a[k], false);
    }
  }
}
// Eight bf16 or binary32 values, or eight codes, to p; n: how many are written.
template <bool FAST>
__device__ __forceinline__ void put_values(void* p, int f32, int n, const float (&v)[8]) {
  if (FAST || f32) {
    put8<16, FAST>(p, f32, n, v);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
    put_words<4>(reinterpret_cast<uint8_t*>(p), 2 * n, w);
  }
}
template <bool FAST>
__device__ __forceinline__ void put_codes(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
  if constexpr (FAST) {
    put8_codes<16, true>(p, n, lo, hi);
  } else {
    const uint32_t w[2] = {lo, hi};
    put_words<2>(p, n, w);
  }
}
// Code k to the top of column k's word, the rows before down a byte.
__device__ __forceinline__ void turn(uint32_t (&turned)[8], uint32_t lo, uint32_t hi) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    turned[k] = __builtin_amdgcn_perm(k < 4 ? lo : hi, turned[k], 0x00030201u | ((uint32_t)(4 + (k & 3)) << 24));
}
template <int RPL, int TS>
__device__ __forceinline__ void put_turned(uint8_t* dst, const uint32_t (&turned)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if constexpr (RPL == 4) *reinterpret_cast<uint32_t*>(dst + k * TS) = turned[k];
    else if constexpr (RPL == 2) *reinterpret_cast<uint16_t*>(dst + k * TS) = (uint16_t)(turned[k] >> 16);
    else dst[k * TS] = (uint8_t)(turned[k] >> 24);
  }
}
// Column-major codes of ROWS rows (TS bytes per column in LDS) to `cols` rows of D_t from
// row n on, 16 bytes per lane; m: the first row, left: how many there are from it on.
template <int TS, int ROWS>
__device__ __forceinline__ void put_columns(uint8_t* d_t, int64_t ldt, const uint8_t* tl, int lane, int64_t n, int cols,
                                            int64_t m, int64_t left) {
  constexpr int LPC = ROWS / 16;
  const int q = lane % LPC;
  left -= 16 * q;
  if (left <= 0 || lane >= 64 / LPC * LPC) return;
  uint8_t* dst = d_t + n * ldt + m + 16 * q;
#pragma unroll 2
  for (int k = lane / LPC; k < cols; k += 64 / LPC) {
    const uint4 w = *reinterpret_cast<const uint4*>(tl + k * TS + 16 * q);
    if (left >= 16) {
      Pk16a1 a;
      a.v[0] = w.x; a.v[1] = w.y; a.v[2] = w.z; a.v[3] = w.w;
      *reinterpret_cast<Pk16a1*>(dst + k * ldt) = a;
    } else {
      for (int b = 0; b < (int)left; ++b) dst[k * ldt + b] = tl[k * TS + 16 * q + b];
    }
  }
}

// A wavefront's largest |d|, and the row and first of n columns where a lane met it (see
// k_gated_amax).
__device__ __forceinline__ void put_key(const GatedParams& e, float top, int row, int col, int n) {
  const uint32_t b = __float_as_uint(top), m = wave_max(b);
  const int at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(b == m));
  const uint32_t r = lane_u32((uint32_t)row, at), c = lane_u32((uint32_t)col, at);
  const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if ((threadIdx.x & 63) == 0) {   // (c is a multiple of 8)
    e.keys[wg * e.key_waves + (threadIdx.x >> 6)] = m;
    e.key_at[wg * e.key_waves + (threadIdx.x >> 6)] = make_uint2(r, c | (n == 16 ? 1u : 0u));
  }
}

// What both directions share: WTN columns in LDS, OC of them outputs of the wavefront,
// lane's outputs c .. c + 7, RPL rows of a strip per lane (lanes past the strip's 16
// rows are idle: on).  FAST as in gemm_ep.h.
template <int WTN, int OC, bool OUT8, bool FAST>
struct GatedBase {
  static constexpr int LPR = OC / 8;
  static constexpr int RPL = LPR >= 4 ? LPR / 4 : 1;
  static constexpr int CH = WTN / 4;
  static_assert(LPR == 2 || LPR == 4 || LPR == 8 || LPR == 16, "16, 32, 64 or 128 outputs");
  const GemmParams& p;
  const GatedParams& e;
  int lane, cq, rg, nv;
  bool on;
  int64_t c;
  float top = 0.0f;      // max |d|
  float so;

  __device__ __forceinline__ GatedBase(const GemmParams& p_, const GatedParams& e_, int64_t first, int lane_)
      : p(p_), e(e_), lane(lane_), cq(lane_ % LPR), rg(lane_ / LPR), on(lane_ / LPR * RPL < 16),
        c(first + 8 * (lane_ % LPR)) {
    const int64_t left = p.N - c;
    nv = !on ? 0 : left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    if (!on) rg = 0;
    so = OUT8 ? p.d_scale[0] : 1.0f;
  }

  // Where the strip's row r keeps columns 4 q .. 4 q + 3.
  static __device__ __forceinline__ float4* place(uint8_t* wl, int r, int q) {
    return reinterpret_cast<float4*>(wl + r * (WTN * 4) + ((q ^ (r & (CH - 1))) << 4));
  }
  static __device__ __forceinline__ void read8(uint8_t* wl, int r, int q, float (&v)[8]) {
    const float4 a = *place(wl, r, q), b = *place(wl, r, q + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  // Accumulators of strip i into LDS: lane (g, l16) has row l16, columns 16 j + 4 g .. + 3.
  template <int TI, int TJ, int I, typename Deq>
  __device__ __forceinline__ void spill(const v4f (&acc)[TI][TJ], Deq&& deq, uint8_t* wl) {
    static_assert(16 * TJ == WTN, "the wavefront's columns");
    const int g = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      *place(wl, l16, 4 * j + g) = make_float4(deq(I, j, 0, acc[I][j][0]), deq(I, j, 1, acc[I][j][1]),
                                               deq(I, j, 2, acc[I][j][2]), deq(I, j, 3, acc[I][j][3]));
  }
  // Takes eight values into the maximum (n: how many of them count) and, as codes of
  // v * so, into lo and hi.
  __device__ __forceinline__ void see(const float (&v)[8], int n, uint32_t& lo, uint32_t& hi) {
    float m;
    if constexpr (FAST) {
      m = n > 0 ? max8(v) : 0.0f;
    } else {
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = k < n ? v[k] : 0.0f;
      m = max8(w);
    }
    top = __builtin_elementwise_maximum(top, m);
    if constexpr (OUT8) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = v[k] * so;
      const float most = p.d_fp8 == 1 ? Fmt<0>::max : Fmt<1>::max;
      const bool tame = __builtin_amdgcn_ballot_w64(!(max8(v) * __builtin_fabsf(so) <= most)) == 0;
      codes_of(p.d_fp8, tame, x, lo, hi);
    }
  }
  // max |d| of the wavefront as stored.
  __device__ __forceinline__ uint32_t amax_bits() {
    uint32_t a = wave_max(__float_as_uint(top));
    if (!OUT8 && !p.d_f32) a = (uint32_t)f32_to_bf16_rne(__uint_as_float(a)) << 16;
    return a;
  }
  template <int B, int E, typename F>
  static __device__ __forceinline__ void each(F&& f) {
    if constexpr (B < E) {
      f(std::integral_constant<int, B>{});
      each<B + 1, E>(f);
    }
  }
};

// Forward: WTN columns of B's rows are WTN / 2 outputs.
template <int WTN, bool OUT8, bool FAST>
struct GatedWave : GatedBase<WTN, WTN / 2, OUT8, FAST> {
  using Base = GatedBase<WTN, WTN / 2, OUT8, FAST>;
  using Base::LPR; using Base::RPL; using Base::p; using Base::e; using Base::lane; using Base::cq; using Base::rg;
  using Base::nv; using Base::on; using Base::c; using Base::so; using Base::read8;
  using Words = uint32_t;            // nothing is read beside the product
  static constexpr int OC = WTN / 2;
  static constexpr bool KEEPS = OC % 32 == 0;   // whole blocks of a checkpoint
  static constexpr int src_at = 64 * WTN, codes_at = src_at;
  static constexpr int bytes(int TI) { return codes_at + (OUT8 ? OC * (16 * TI + 16) : 0); }
  float bias[2][8];
  int where = 0;         // the row of the lane's largest |d|

  __device__ __forceinline__ GatedWave(const GemmParams& p_, const GatedParams& e_, int64_t n0, int lane_)
      : Base(p_, e_, n0 / 2, lane_) {
#pragma unroll
    for (int k = 0; k < 8; ++k) bias[0][k] = bias[1][k] = 0.0f;
    if (e.bias) {
      load8(e.bias, e.bias_f32, c, nv, bias[0]);
      load8(e.bias, e.bias_f32, p.N + c, nv, bias[1]);
    }
  }
  __device__ __forceinline__ void fetch(int64_t, Words (&)[RPL]) {}
  __device__ __forceinline__ void stage(int64_t, const Words (&)[RPL], uint8_t*) {}

  // The strip in wl, one row after the other (a loop that stays one: see EpWave).
  template <int TS>
  __device__ __forceinline__ void rows(int64_t m0, uint8_t* wl, const uint8_t*, uint8_t* tl, int tr) {
    uint32_t turned[8] = {};
    const int64_t first = m0 + rg * RPL;
    const int esz = OUT8 ? 1 : (p.d_f32 ? 4 : 2);
    char* d = reinterpret_cast<char*>(p.D) + (first * p.ldd + c) * esz;
    const int64_t F = p.N, nb = ck_blocks(F);
#pragma unroll 1
    for (int t = 0; t < RPL; ++t) {
      const int64_t m = first + t;
      const int n = m < p.M ? nv : 0;
      const int q = 8 * (cq >> 1) + 2 * (cq & 1);
      float g[8], u[8], v[8];
      read8(wl, rg * RPL + t, q, g);
      read8(wl, rg * RPL + t, q + 4, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] += bias[0][k];
        u[k] += bias[1][k];
      }
      if (e.aux) {
        uint16_t* a = reinterpret_cast<uint16_t*>(e.aux) + m * e.ldaux + c;
        put_values<FAST>(a, 0, n, g);
        put_values<FAST>(a + F, 0, n, u);
      }
      if constexpr (KEEPS) {
        if (e.ck) {
          uint8_t* a = e.ck + m * e.ldck + c;
          uint8_t* x = e.ck_exp + m * e.ldexp + (c >> 5);
          keep(g, n, a, x);
          keep(u, n, a + F, x + nb);
        }
      }
      act_of(e.act, g, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= u[k];
      uint32_t lo, hi;
      const float before = this->top;
      this->see(v, n, lo, hi);
      if constexpr (OUT8) {
        where = __float_as_uint(this->top) != __float_as_uint(before) ? (int)m : where;
        put_codes<FAST>(reinterpret_cast<uint8_t*>(d), n, lo, hi);
        if (p.D_t) turn(turned, lo, hi);
      } else {
        put_values<FAST>(d, p.d_f32, n, v);
      }
      d += p.ldd * esz;
    }
    if constexpr (OUT8) {
      if (p.D_t && on) put_turned<RPL, TS>(tl + (8 * cq) * TS + tr + rg * RPL, turned);
    }
    asm volatile("" ::: "memory");   // LDS is written and read as different types
  }

  // Eight values of a block's 32 to the checkpoint.  Columns past the last output
  // are zeros (B's rows past its end are read as zeros, their bias is 0), or NaN
  // where the whole row is, so the block's maximum needs no mask.
  __device__ __forceinline__ void keep(const float (&v)[8], int n, uint8_t* ck, uint8_t* exp) {
    uint32_t lo, hi, a = __float_as_uint(max8(v));
    const bool tame = __builtin_amdgcn_ballot_w64(a >= 0x7F800000u) == 0;
    a = max_u32(a, dpp<kXor1>(a));
    a = max_u32(a, dpp<kXor2>(a));
    const uint32_t byte = ck_exponent(a);
    if (__builtin_expect(tame, 1)) {
      ck_codes(v, byte, lo, hi);
    } else {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = v[k] * ck_scale(byte);
      encode8<0>(x, lo, hi);
    }
    put_codes<FAST>(ck, n, lo, hi);
    if ((cq & 3) == 0 && n > 0) *exp = (uint8_t)byte;
  }

  template <int TI, int TJ, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl) {
    constexpr int TS = 16 * TI + 16;
    this->template each<0, TI>([&](auto itag) {
      constexpr int i = decltype(itag)::value;
      this->template spill<TI, TJ, i>(acc, deq, wl);
      rows<TS>(r0 + 16 * i, wl, nullptr, wl + codes_at, 16 * i);
    });
    if constexpr (OUT8) {
      if (p.D_t) flush_t<TS, 16 * TI>(wl + codes_at, r0, n0);
    }
  }
  template <int TI, int TJ, int STRIPS, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl,
                                       Words (&)[STRIPS][RPL]) {
    tile(acc, deq, r0, n0, wl);
  }
  template <int TS, int ROWS>
  __device__ __forceinline__ void flush_t(const uint8_t* tl, int64_t r0, int64_t n0) {
    const int64_t first = n0 / 2, cols = p.N - first;
    put_columns<TS, ROWS>(p.D_t, p.ldt, tl, lane, first, cols < OC ? (int)cols : OC, r0, p.M - r0);
  }
  // (what a backward wavefront has to leave at its end, a forward one has not: the key of
  // its largest |d|)
  __device__ __forceinline__ void put_dbias(int64_t) {
    if constexpr (OUT8) {
      if (e.keys) put_key(e, this->top, where, (int)c, 8);
    }
  }
};

// Backward: WTN columns are as many outputs of each half.  KEPT: g and u come from BF16
// (0), from a checkpoint (1), or from either (2).
template <int WTN, bool OUT8, bool FAST, int KEPT>
struct GatedGradWave : GatedBase<WTN, WTN, OUT8, FAST> {
  using Base = GatedBase<WTN, WTN, OUT8, FAST>;
  using Base::LPR; using Base::RPL; using Base::p; using Base::e; using Base::lane; using Base::cq; using Base::rg;
  using Base::nv; using Base::c; using Base::so; using Base::read8;
  static_assert(LPR >= 4, "whole strips");
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  using Eight = typename std::conditional<FAST, v4u, v8u>::type;   // (vectors: arrays in arrays go to scratch memory)
  struct Words { Eight g, u; uint32_t xg, xu; };
  // LDS: the strip, each lane's own words of g and u (32 bytes a row), and (OUT8) the
  // column-major codes of dg and du of two strips, which leave 32 bytes a column.
  static constexpr int FLUSH = 2, TS_ = 16 * FLUSH + 16;
  static constexpr int src_at = 64 * WTN, codes_at = src_at + RPL * 64 * 32;
  static constexpr int bytes(int) { return codes_at + (OUT8 ? 2 * WTN * TS_ : 0); }
  float db[2][8];

  __device__ __forceinline__ GatedGradWave(const GemmParams& p_, const GatedParams& e_, int64_t n0, int lane_)
      : Base(p_, e_, n0, lane_) {
#pragma unroll
    for (int k = 0; k < 8; ++k) db[0][k] = db[1][k] = 0.0f;
  }
  __device__ __forceinline__ bool coded() const { return KEPT == 2 ? e.ck != nullptr : KEPT == 1; }

  // The strip of rows m0 .. m0 + 15 of g and u, in flight until stage().
  __device__ __forceinline__ void fetch(int64_t m0, Words (&o)[RPL]) {
#pragma unroll
    for (int t = 0; t < RPL; ++t) {
      const int64_t m = m0 + rg * RPL + t;
      const int n = m < p.M ? nv : 0;
      if (n <= 0) {   // zeros, so that no sum or maximum needs a mask
#pragma unroll
        for (int k = 0; k < (FAST ? 4 : 5); ++k) o[t].g[k] = o[t].u[k] = 0u;
        o[t].xg = o[t].xu = 127u;
      }
      if (coded()) {
        const uint8_t* a = e.ck + m * e.ldck + c;
        const uint8_t* x = e.ck_exp + m * e.ldexp + (c >> 5);
        load_codes(a, n, o[t].g);
        load_codes(a + p.N, n, o[t].u);
        if (n > 0) {
          o[t].xg = x[0];
          o[t].xu = x[ck_blocks(p.N)];
        }
      } else {
        const uint16_t* a = reinterpret_cast<const uint16_t*>(e.aux) + m * e.ldaux + c;
        load_packed<FAST, false>(a, 0, n, o[t].g);
        load_packed<FAST, false>(a + p.N, 0, n, o[t].u);
      }
    }
  }
  static __device__ __forceinline__ void load_codes(const uint8_t* a, int n, Eight& w) {
    if (n <= 0) return;
    if constexpr (FAST) {
      struct __attribute__((packed, aligned(4))) Two { uint32_t a, b; };
      const Two q = *reinterpret_cast<const Two*>(a);
      w[0] = q.a;
      w[1] = q.b;
    } else {   // the dwords of memory that hold one of them (see codes())
      const int o = (int)(reinterpret_cast<uintptr_t>(a) & 3u);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a - o);
      struct __attribute__((packed, aligned(4))) Two { uint32_t a, b; };
      w[1] = w[2] = 0u;
      if (o + n > 4) {
        const Two t = *reinterpret_cast<const Two*>(q);
        w[0] = t.a;
        w[1] = t.b;
      } else {
        w[0] = q[0];
      }
      if (o + n > 8) w[2] = q[2];
    }
  }
  // The n codes at a out of the dwords that load_codes took.
  static __device__ __forceinline__ uint2 codes(const Eight& w, const uint8_t* a, int n) {
    if constexpr (FAST) return make_uint2(w[0], w[1]);
    const uint32_t o = (uint32_t)reinterpret_cast<uintptr_t>(a);   // (alignbyte takes its two lowest bits)
    uint32_t lo = __builtin_amdgcn_alignbyte(w[1], w[0], o), hi = __builtin_amdgcn_alignbyte(w[2], w[1], o);
    if (n < 8) {
      lo = n >= 4 ? lo : (n <= 0 ? 0u : lo & (0xFFFFFFFFu >> (32 - 8 * n)));
      hi = n <= 4 ? 0u : hi & (0xFFFFFFFFu >> (64 - 8 * n));
    }
    return make_uint2(lo, hi);
  }
  // Each lane's own words: 16 bytes of g's eight values and 16 of u's a row, or 16 of
  // both's codes and exponents.
  __device__ __forceinline__ void stage(int64_t m0, const Words (&o)[RPL], uint8_t* ol) {
    uint4* q = reinterpret_cast<uint4*>(ol) + lane;
#pragma unroll
    for (int t = 0; t < RPL; ++t) {
      if (coded()) {
        const int64_t m = m0 + rg * RPL + t;
        const uint8_t* a = e.ck + m * e.ldck + c;
        const int n = m < p.M ? nv : 0;
        const uint2 g = codes(o[t].g, a, n), u = codes(o[t].u, a + p.N, n);
        q[t * 64] = make_uint4(g.x, g.y, u.x, u.y);
        reinterpret_cast<uint32_t*>(ol + RPL * 64 * 16)[t * 64 + lane] = o[t].xg | (o[t].xu << 8);
      } else {
        const uint16_t* a = reinterpret_cast<const uint16_t*>(e.aux) + (m0 + rg * RPL + t) * e.ldaux + c;
        q[t * 64] = words(o[t].g, FAST ? 0u : odd_of(a));
        q[(RPL + t) * 64] = words(o[t].u, FAST ? 0u : odd_of(a + p.N));
      }
    }
  }
  static __device__ __forceinline__ uint4 words(const Eight& w, uint32_t s) {
    if constexpr (FAST) return make_uint4(w[0], w[1], w[2], w[3]);
    else
      return make_uint4(__builtin_amdgcn_alignbyte(w[1], w[0], s), __builtin_amdgcn_alignbyte(w[2], w[1], s),
                        __builtin_amdgcn_alignbyte(w[3], w[2], s), __builtin_amdgcn_alignbyte(w[4], w[3], s));
  }
  static __device__ __forceinline__ void widen(const uint4& a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_lo(w[k]);
      v[2 * k + 1] = bf16_hi(w[k]);
    }
  }

  template <int TS>
  __device__ __forceinline__ void rows(int64_t m0, uint8_t* wl, const uint8_t* ol, uint8_t* tl, int tr) {
    uint32_t tg[8] = {}, tu[8] = {};
    const int64_t first = m0 + rg * RPL;
    const int esz = OUT8 ? 1 : (p.d_f32 ? 4 : 2);
    char* d = reinterpret_cast<char*>(p.D) + (first * p.ldd + c) * esz;
    const int64_t half = p.N * esz;
    const uint4* q = reinterpret_cast<const uint4*>(ol) + lane;
#pragma unroll 1
    for (int t = 0; t < RPL; ++t) {
      const int n = first + t < p.M ? nv : 0;
      float v[8], g[8], u[8], a[8], s[8];
      read8(wl, rg * RPL + t, 2 * cq, v);
      // (past the last row stand zeros; times an infinite scale they are NaN)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = n > 0 ? v[k] : 0.0f;
      const uint4 x = q[t * 64];
      if (coded()) {
        const uint32_t b = reinterpret_cast<const uint32_t*>(ol + RPL * 64 * 16)[t * 64 + lane];
        ck_values(x.x, x.y, b & 0xFFu, g);
        ck_values(x.z, x.w, b >> 8, u);
      } else {
        widen(x, g);
        widen(q[(RPL + t) * 64], u);
      }
      act_and_slope(e.act, g, a, s);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] = v[k] * u[k] * s[k];
        u[k] = v[k] * a[k];
      }
      // (rows past the last have v = g = u = 0, columns past the last are not stored)
      if (e.dbias) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          db[0][k] += g[k];
          db[1][k] += u[k];
        }
      }
      uint32_t lo, hi;
      this->see(g, n, lo, hi);
      if constexpr (OUT8) {
        put_codes<FAST>(reinterpret_cast<uint8_t*>(d), n, lo, hi);
        if (p.D_t) turn(tg, lo, hi);
      } else {
        put_values<FAST>(d, p.d_f32, n, g);
      }
      this->see(u, n, lo, hi);
      if constexpr (OUT8) {
        put_codes<FAST>(reinterpret_cast<uint8_t*>(d) + half, n, lo, hi);
        if (p.D_t) turn(tu, lo, hi);
      } else {
        put_values<FAST>(d + half, p.d_f32, n, u);
      }
      d += p.ldd * esz;
    }
    if constexpr (OUT8) {
      if (p.D_t) {
        uint8_t* dst = tl + (8 * cq) * TS + tr + rg * RPL;
        put_turned<RPL, TS>(dst, tg);
        put_turned<RPL, TS>(dst + WTN * TS, tu);
      }
    }
    asm volatile("" ::: "memory");   // LDS is written and read as different types
  }

  template <int TI, int TJ, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl) {
    Words o[1][RPL];
    fetch(r0, o[0]);
    tile(acc, deq, r0, n0, wl, o);
  }
  template <int TI, int TJ, int STRIPS, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl,
                                       Words (&o)[STRIPS][RPL]) {
    static_assert(STRIPS == 1 || STRIPS == TI, "one strip ahead, or all");
    static_assert(TI == 1 || TI % FLUSH == 0, "whole flushes");
    constexpr int EACH = TI < FLUSH ? TI : FLUSH;
    this->template each<0, TI>([&](auto itag) {
      constexpr int i = decltype(itag)::value;
      this->template spill<TI, TJ, i>(acc, deq, wl);
      stage(r0 + 16 * i, o[STRIPS == 1 ? 0 : i], wl + src_at);
      if constexpr (STRIPS == 1 && i + 1 < TI) fetch(r0 + 16 * (i + 1), o[0]);
      rows<TS_>(r0 + 16 * i, wl, wl + src_at, wl + codes_at, 16 * (i % EACH));
      if constexpr (OUT8 && i % EACH == EACH - 1) {
        if (p.D_t) flush_t<TS_, 16 * EACH>(wl + codes_at, r0 + 16 * (i - EACH + 1), n0);
      }
    });
  }
  template <int TS, int ROWS>
  __device__ __forceinline__ void flush_t(const uint8_t* tl, int64_t r0, int64_t n0) {
    const int cols = p.N - n0 < WTN ? (int)(p.N - n0) : WTN;
    put_columns<TS, ROWS>(p.D_t, p.ldt, tl, lane, n0, cols, r0, p.M - r0);
    put_columns<TS, ROWS>(p.D_t, p.ldt, tl + WTN * TS, lane, p.N + n0, cols, r0, p.M - r0);
    asm volatile("" ::: "memory");
  }

  // Column sums of the wavefront's rows to part[row][2 N] (see EpWave).
  __device__ __forceinline__ void put_dbias(int64_t row) {
    if (e.dbias == nullptr) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int off = LPR; off < 64; off <<= 1) db[h][k] += __shfl_xor(db[h][k], off, 64);
      if (rg == 0 && nv > 0) store8(e.part, e.part_f32, (2 * row + h) * p.N + c, nv, db[h]);
    }
  }
};

// What the tile and few-row kernels are built around (LinearOp in gemm_ep.h).
struct GatedOp {
  using Params = GatedParams;
  static constexpr bool PAIRED = true;
  template <int WTN, bool OUT8>
  using Wave = GatedWave<WTN, OUT8, false>;
};
struct GatedGradOp {
  using Params = GatedParams;
  static constexpr bool PAIRED = false;
  template <int WTN, bool OUT8>
  using Wave = GatedGradWave<WTN, OUT8, false, 2>;
};

// The epilogue as k_gemm_big takes it (see LinearEp): two wavefronts on a SIMD hide what a
// strip's way through LDS takes (8192 x 14336 x 4096 with 1x128 scales, backward, checkpoint: 570 us;
// from the accumulators, as in gemm_gated_direct.h, 630).
template <typename W, int TI, int TJ, int NW, typename Deq>
__device__ __forceinline__ void gated_finish(const GemmParams& p, const GatedParams& e, const v4f (&acc)[TI][TJ], Deq&& deq,
                                             int64_t r0, int64_t c0, int64_t part, int lane, int wave, uint8_t* wl) {
  static_assert(W::bytes(TI) <= 128 * 1024 / NW, "the wavefront's part of the stages");
  W w(p, e, c0, lane);
  w.template tile<TI, TJ>(acc, deq, r0, c0, wl);
  w.put_dbias(part);
  if (p.d_amax) ep_amax<NW>(p.d_amax, w.amax_bits(), lane, wave);
}
struct GatedStripEp {
  static constexpr bool PAIRED = true, DIRECT = false;
  GatedParams e;
  template <bool OUT8, int TI, int TJ, int NW, typename Deq>
  __device__ __forceinline__ void finish(const GemmParams& p, const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t c0,
                                         int64_t part, int lane, int wave, uint8_t* wl) const {
    gated_finish<GatedWave<16 * TJ, OUT8, true>, TI, TJ, NW>(p, e, acc, deq, r0, c0, part, lane, wave, wl);
  }
};
template <int KEPT>
struct GatedGradStripEp {
  static constexpr bool PAIRED = false, DIRECT = false;
  GatedParams e;
  template <bool OUT8, int TI, int TJ, int NW, typename Deq>
  __device__ __forceinline__ void finish(const GemmParams& p, const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t c0,
                                         int64_t part, int lane, int wave, uint8_t* wl) const {
    gated_finish<GatedGradWave<16 * TJ, OUT8, true, KEPT>, TI, TJ, NW>(p, e, acc, deq, r0, c0, part, lane, wave, wl);
  }
};

}  // namespace

}  // namespace fp8lin
