// op_device.h -- device helpers shared by the operators around the linears
// (norm_kernels.hip, rope_kernels.hip, gemm_ep*): 8-element loads and stores
// at any element alignment, wavefront and workgroup reductions in a fixed
// order, activations and gates with their derivatives.
#pragma once

#include "fp8_device.h"

namespace fp8lin {

namespace {

// 16-, 8- and 4-byte accesses at the alignment of the element: gfx950 serves
// global accesses at any byte address, so a row of odd length costs nothing
// but the lines it straddles.
struct __attribute__((packed, aligned(2))) Pk16a2 { uint32_t v[4]; };
struct __attribute__((packed, aligned(4))) Pk16a4 { uint32_t v[4]; };

typedef float f32x2_op __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_op __attribute__((ext_vector_type(2)));

// Two binary32 -> two bf16, round to nearest even (one instruction; binary32
// subnormals, below 2^-126, may be off by one bf16 step of 2^-133).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_op v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_op));
}

// ---- rows cut into vectors of eight, one per lane, for loads that are issued
// long before they are used.  Vector v of a row of `cols` elements starts at 8 v;
// the last one, if cols is no multiple of 8, starts at cols - 8, so that it is one
// 16-byte load like the others and needs no wait for what is in flight, and its
// first `skip` elements belong to the vector before: they are left out of sums
// and stores.  (Read element by element, the last vector waited for every load
// before it, and with it the whole workgroup: BF16 norm of 4096 x 4104, 45 us.)
// skip = 8: no such vector.  TINY: a row of fewer than 8 elements, whose only
// vector starts at c < 0 (kernels of their own: the accesses of single elements
// cost the others some 20 registers).
struct RowVec {
  int c, skip;
  __device__ __forceinline__ RowVec() {}
  __device__ __forceinline__ RowVec(int cols, int v) {
    const int left = cols - 8 * v;
    c = left >= 8 ? 8 * v : cols - 8;
    skip = left >= 8 ? 0 : (left > 0 ? 8 - left : 8);
  }
};
// Element i of an array.  With a 32-bit index and a base that is the same in all
// lanes the address is that base plus a 32-bit offset: one register for all the
// arrays of a row, where 64-bit addresses take two for each.
template <typename T, typename I>
__device__ __forceinline__ const T* elem(const void* base, I i) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + (I)(i * (I)sizeof(T)));
}
template <typename T, typename I>
__device__ __forceinline__ T* elem(void* base, I i) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + (I)(i * (I)sizeof(T)));
}

// Eight bf16 as whole dwords of memory: the four from the dword that holds the
// first, and, where that one starts in the middle of it, the last element by
// itself.  (A 16-byte load that does not start on a dword costs several times
// one that does: BF16 norm of 4096 x 4095, 62 us so, 44 us as here.)
__device__ __forceinline__ uint32_t odd_of(const void* p) { return (uint32_t)reinterpret_cast<uintptr_t>(p) & 2u; }
__device__ __forceinline__ void load_dwords(const uint16_t* p, uint32_t (&w)[5]) {
  const uint32_t o = odd_of(p);
  const Pk16a4 a = *reinterpret_cast<const Pk16a4*>(reinterpret_cast<const char*>(p) - o);
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = a.v[k];
  w[4] = 0u;
  if (o) w[4] = p[7];
}

// v[0..7] = elements i .. i+7 of a bf16 (F32 = 0) or binary32 (F32 = 1) array;
// n < 8: only the first n are there, the others become 0.
template <typename I>
__device__ __forceinline__ void load8(const void* base, int f32, I i, int n, float (&v)[8]) {
  if (f32) {
    const float* p = elem<float>(base, i);
    if (n >= 8) {
      const Pk16a4 a = *reinterpret_cast<const Pk16a4*>(p);
      const Pk16a4 b = *reinterpret_cast<const Pk16a4*>(p + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = __uint_as_float(a.v[k]);
        v[k + 4] = __uint_as_float(b.v[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : 0.0f;
    }
  } else {
    const uint16_t* p = elem<uint16_t>(base, i);
    if (n >= 8) {
      uint32_t w[5];
      load_dwords(p, w);
      const uint32_t o = odd_of(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t d = __builtin_amdgcn_alignbyte(w[k + 1], w[k], o);
        v[2 * k] = bf16_lo(d);
        v[2 * k + 1] = bf16_hi(d);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? __uint_as_float((uint32_t)p[k] << 16) : 0.0f;
    }
  }
}

template <typename I>
__device__ __forceinline__ void store8(void* base, int f32, I i, int n, const float (&v)[8]) {
  if (f32) {
    float* p = elem<float>(base, i);
    if (n >= 8) {
      Pk16a4 a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a.v[k] = __float_as_uint(v[k]);
        b.v[k] = __float_as_uint(v[k + 4]);
      }
      *reinterpret_cast<Pk16a4*>(p) = a;
      *reinterpret_cast<Pk16a4*>(p + 4) = b;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = v[k];
    }
  } else {
    uint16_t* p = elem<uint16_t>(base, i);
    Pk16a2 a;
#pragma unroll
    for (int k = 0; k < 4; ++k) a.v[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
    if (n >= 8) {
      *reinterpret_cast<Pk16a2*>(p) = a;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = (uint16_t)(a.v[k >> 1] >> (16 * (k & 1)));
    }
  }
}

// As the elements lie in memory: a bf16 vector waits in five registers, not in
// eight.
template <bool F32>
struct Raw8 {
  uint32_t v[F32 ? 8 : 5];
};
template <bool F32, bool TINY>
__device__ __forceinline__ Raw8<F32> load_raw(const void* row, const RowVec& x) {
  Raw8<F32> r;
#pragma unroll
  for (int k = 0; k < (F32 ? 8 : 5); ++k) r.v[k] = 0u;
  if (x.skip >= 8) return r;
  if constexpr (!TINY) {
    if constexpr (F32) {
      const float* p = elem<float>(row, (uint32_t)x.c);
      const Pk16a4 a = *reinterpret_cast<const Pk16a4*>(p);
      const Pk16a4 b = *reinterpret_cast<const Pk16a4*>(p + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        r.v[k] = a.v[k];
        r.v[k + 4] = b.v[k];
      }
    } else {
      load_dwords(elem<uint16_t>(row, (uint32_t)x.c), r.v);
    }
  } else if constexpr (F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= x.skip) r.v[k] = __float_as_uint(reinterpret_cast<const float*>(row)[x.c + k]);
  } else {
    uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= x.skip) d[k >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[x.c + k] << (16 * (k & 1));
    const bool o = ((odd_of(row) ^ (2u * (uint32_t)x.c)) & 2u) != 0u;
    r.v[0] = o ? d[0] << 16 : d[0];
#pragma unroll
    for (int k = 1; k < 4; ++k) r.v[k] = o ? __builtin_amdgcn_alignbyte(d[k], d[k - 1], 2) : d[k];
    r.v[4] = d[3] >> 16;
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack(const Raw8<F32>& r, const void* row, const RowVec& x, float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.v[k]);
  } else {
    const uint32_t o = (odd_of(row) ^ (2u * (uint32_t)x.c)) & 2u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t d = __builtin_amdgcn_alignbyte(r.v[k + 1], r.v[k], o);
      v[2 * k] = bf16_lo(d);
      v[2 * k + 1] = bf16_hi(d);
    }
  }
}

// fmt 0: E4M3, 1: E5M2 (a uniform run-time choice).
__device__ __forceinline__ void codes8(int fmt, const float (&v)[8], float s, uint32_t& lo, uint32_t& hi) {
  if (fmt == 0) {
    lo = cvt4<0>(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
    hi = cvt4<0>(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
  } else {
    lo = cvt4<1>(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
    hi = cvt4<1>(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
  }
}

// Lane permutations inside a row of 16 lanes: xor 1, xor 2, then mirrors of 8
// and of 16 (after the xor steps every lane of a quad / half row holds the
// same value, so a mirror pairs the halves).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ float row16_sum(float v) {
  v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kMirror>(__float_as_uint(v)));
  return v;
}
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max_u32(v, dpp<kXor1>(v));
  v = max_u32(v, dpp<kXor2>(v));
  v = max_u32(v, dpp<kHalfMirror>(v));
  return max_u32(v, dpp<kMirror>(v));
}
__device__ __forceinline__ uint32_t lane_u32(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
// The value of the lane before / after in a row of 16 lanes (0 at its ends).
__device__ __forceinline__ uint32_t lane_before(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);   // row_shr:1
}
__device__ __forceinline__ uint32_t lane_after(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x101, 0xF, 0xF, true);   // row_shl:1
}

// NW dwords per lane to byte address p, where SEG neighbouring lanes (SEG
// divides 16, and the group starts at a multiple of it) write one after the
// other into one row; every lane of the wavefront calls it, `full` for those
// that have a whole vector.  A vector that does not start on a dword costs
// several times an aligned one, so such a row is written as the dwords of memory: each lane takes the
// bytes that its first dword shares with the lane before, and only the ends of a
// group write single bytes.
template <int NW, int SEG>
__device__ __forceinline__ void store_row(uint8_t* p, const uint32_t (&w)[NW], bool full) {
  struct __attribute__((packed, aligned(4))) Words { uint32_t v[NW]; };
  struct __attribute__((packed, aligned(4))) Rest { uint32_t v[NW - 1]; };
  const uint32_t o = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3u);
  if (__builtin_expect(__any(o != 0 && full), 0)) {
    const int at = (int)(threadIdx.x & (SEG - 1));
    // (every lane takes part in each exchange: none inside a short-circuit)
    const uint32_t f = full ? 1u : 0u, carry = lane_before(w[NW - 1]), fb = lane_before(f), fa = lane_after(f);
    const bool before = (at != 0) & (fb != 0u), after = (at != SEG - 1) & (fa != 0u);
    if (!full) return;
    Words a;
    a.v[0] = o == 0 ? w[0] : __builtin_amdgcn_alignbyte(w[0], carry, 4 - o);
#pragma unroll
    for (int k = 1; k < NW; ++k) a.v[k] = o == 0 ? w[k] : __builtin_amdgcn_alignbyte(w[k], w[k - 1], 4 - o);
    if (o == 0 || before) {
      *reinterpret_cast<Words*>(p - o) = a;
    } else {
      Rest r;
#pragma unroll
      for (int k = 1; k < NW; ++k) r.v[k - 1] = a.v[k];
      *reinterpret_cast<Rest*>(p - o + 4) = r;
      for (uint32_t b = 0; b < 4 - o; ++b) p[b] = (uint8_t)(w[0] >> (8 * b));
    }
    if (o != 0 && !after)
      for (uint32_t b = 4 - o; b < 4; ++b) p[4 * (NW - 1) + b] = (uint8_t)(w[NW - 1] >> (8 * b));
    return;
  }
  if (full) {
    Words a;
#pragma unroll
    for (int k = 0; k < NW; ++k) a.v[k] = w[k];
    *reinterpret_cast<Words*>(p) = a;
  }
}

template <bool TINY, typename T>
__device__ __forceinline__ T* place(void* row, const RowVec& x, int k) {
  if constexpr (TINY) return reinterpret_cast<T*>(row) + (x.c + k);
  else return elem<T>(row, (uint32_t)x.c) + k;
}
// Eight bf16 or binary32 values, or eight codes, of a row's vector (see store_row
// and RowVec; every lane of the wavefront calls it).  live: whether to write.
template <bool TINY>
__device__ __forceinline__ void store_vec(void* row, int f32, const RowVec& x, bool live, const float (&v)[8]) {
  if (f32) {
    if (!live) return;
    if (x.skip == 0) {
      store8(row, 1, (uint32_t)x.c, 8, v);
    } else {
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k >= x.skip) *place<TINY, float>(row, x, k) = v[k];
    }
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
  store_row<4, 16>(reinterpret_cast<uint8_t*>(elem<uint16_t>(row, (uint32_t)x.c)), w, live && x.skip == 0);
  if (live && x.skip > 0 && x.skip < 8) {
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (k >= x.skip) *place<TINY, uint16_t>(row, x, k) = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
  }
}
template <bool TINY>
__device__ __forceinline__ void store_vec_codes(uint8_t* row, const RowVec& x, uint32_t lo, uint32_t hi) {
  const uint32_t w[2] = {lo, hi};
  store_row<2, 16>(elem<uint8_t>(row, (uint32_t)x.c), w, x.skip == 0);
  if (x.skip > 0 && x.skip < 8) {
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (k >= x.skip) *place<TINY, uint8_t>(row, x, k) = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
  }
}

// Over the 64 lanes, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  const uint32_t b = __float_as_uint(row16_sum(v));
  return (__uint_as_float(lane_u32(b, 0)) + __uint_as_float(lane_u32(b, 16))) +
         (__uint_as_float(lane_u32(b, 32)) + __uint_as_float(lane_u32(b, 48)));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = row16_max(v);
  return max_u32(max_u32(lane_u32(v, 0), lane_u32(v, 16)), max_u32(lane_u32(v, 32), lane_u32(v, 48)));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

constexpr float kLog2E = 1.44269504088896f;

// Gate G(g): 0 g itself, 1 sigmoid, 2 tanh.  With e = exp(-2 |g|), tanh |g| =
// (1 - e) / (1 + e), which loses bits where 1 - e cancels: below 1/4 the series to
// g^9 (the next term is below 2^-26 of it).
__device__ __forceinline__ float gate_value(int act, float g) {
  if (act == 1) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * g));
  if (act == 2) {
    const float a = __builtin_fabsf(g), e = __builtin_amdgcn_exp2f(-2.0f * kLog2E * a), q = g * g;
    const float series = g * __builtin_fmaf(
        q, __builtin_fmaf(q, __builtin_fmaf(q, __builtin_fmaf(q, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f),
                          -1.0f / 3.0f), 1.0f);
    const float far = __builtin_copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), g);
    return a < 0.25f ? series : far;
  }
  return g;
}
// Its derivative: e / (1 + e)^2 with e = exp(-|g|) for the sigmoid, 4 e / (1 + e)^2 with
// e = exp(-2 |g|) for tanh.  G (1 - G) and 1 - G^2 would lose every digit for a gate
// that is all but open or shut.
__device__ __forceinline__ float gate_slope(int act, float g) {
  if (act == 0) return 1.0f;
  const float e = __builtin_amdgcn_exp2f((act == 2 ? -2.0f * kLog2E : -kLog2E) * __builtin_fabsf(g));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return (act == 2 ? 4.0f : 1.0f) * e * r * r;
}

// Activations of the linear's epilogue: 0 none, 1 ReLU, 2 GELU (erf),
// 3 GELU (tanh form), 4 SiLU; u -> act(u), or act'(u).
// The sigmoid forms cost one exponential and one reciprocal: with s(x) = 1 /
// (1 + e^-x), SiLU is u s(u) and the tanh form of GELU u s(2 t), t = sqrt(2/pi)
// (u + 0.044715 u^3), because 0.5 (1 + tanh t) = s(2 t); both slopes are
// s + u s (1 - s) x'(u).  GELU's lower tail, erfc(x) / 2 with x = |u| / sqrt 2, is
// e^(-x^2) t P(t), t = 1 / (1 + 0.43 x): P of degree 7 has the least largest relative
// error over x = 0 .. 9.6 (beyond, e^(-x^2) is below 2^-132), 7e-8, so a value keeps its
// digits however small it is (as 1 + erf(u / sqrt 2) it would lose them all by u = -5);
// what is left is the rounding of the exponential's argument, 1.5 u^2 2^-24 of the
// value.  One reciprocal, and e^(-u^2/2), which the slope needs too.
constexpr float kRootTwoOverPi = 0.797884560802865f;
template <bool SLOPE>
__device__ __forceinline__ float gelu_erf(float u) {
  const float x = __builtin_fabsf(u) * 0.707106781186548f;
  const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2E * u * u);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.43f, x, 1.0f));
  float q = __builtin_fmaf(t, 0.0365416668f, -0.153960645f);
  q = __builtin_fmaf(t, q, 0.189873412f);
  q = __builtin_fmaf(t, q, -0.0411675461f);
  q = __builtin_fmaf(t, q, 0.122594289f);
  q = __builtin_fmaf(t, q, 0.102705248f);
  q = __builtin_fmaf(t, q, 0.122154258f);
  q = __builtin_fmaf(t, q, 0.12125928f);
  const float tail = q * t * e;                      // 0.5 (1 - erf x)
  const float cdf = u < 0.0f ? tail : 1.0f - tail;   // 0.5 (1 + erf(u / sqrt 2))
  return SLOPE ? __builtin_fmaf(u * 0.398942280401433f, e, cdf) : u * cdf;
}
// u s(x(u)), x(u) = u (a + b u^2).
struct SigmoidForm {
  float a, b;
  __device__ __forceinline__ explicit SigmoidForm(int act)
      : a(act == 3 ? 2.0f * kRootTwoOverPi : 1.0f), b(act == 3 ? 2.0f * kRootTwoOverPi * 0.044715f : 0.0f) {}
  __device__ __forceinline__ float sigmoid(float u, float q) const {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f((-kLog2E * u) * __builtin_fmaf(b, q, a)));
  }
  __device__ __forceinline__ float value(float u) const {
    // (u^2 stays finite: b u^2 is far past where s is 1 or 0, and 0 * inf is NaN)
    const float q = __builtin_fminf(u * u, 1e30f);
    return u * sigmoid(u, q);
  }
  // s + u s (1 - s) x'(u); beyond +-100 s is 1 or 0 in both forms and u no
  // longer matters, where u^2 might overflow into inf * 0.
  __device__ __forceinline__ float slope(float u) const {
    u = u == u ? __builtin_amdgcn_fmed3f(u, -100.0f, 100.0f) : u;
    const float q = u * u, s = sigmoid(u, q);
    return __builtin_fmaf(u * (s - s * s), __builtin_fmaf(3.0f * b, q, a), s);
  }
};

}  // namespace

}  // namespace fp8lin
