// checkpoint.h -- tensors kept for the backward pass in 8 bits: E4M3 codes, and for each
// block of 32 neighbouring columns of a row one power of two.
//
// With a = max |x| of the block (an exact maximum) and e the largest integer with
// a 2^e <= 448, |e| <= 126, a code is encode(x 2^e), x 2^e being exact, and the block's
// byte is 127 - e: 2^(byte - 127) takes a code back to a value.  Nothing saturates; a
// value is off by at most 2^-4 of itself, or 2^-10 2^-e: below 2^-17 of its block's
// largest, or, where e ends at 126, 2^-136 (a block that is below 2^-136 is lost).  What
// rounds to 2^128 (from 1.9375 2^127 on) reads back as an infinity.  A block of zeros, or
// one that holds an infinity or a NaN, has e = 0, as in the block casts.
// 448 = 1.75 2^8, so with a = 1.m 2^(E - 127):  e = 8 - (E - 127) - (1.m > 1.75), and the
// byte is E - 8 + (1.m > 1.75), at least 1 (a below 2^-118: e stays 126).
#pragma once

#include "op_device.h"

namespace fp8lin {

namespace {

constexpr int CK_BLOCK = 32;
__host__ __device__ constexpr int64_t ck_blocks(int64_t cols) { return (cols + CK_BLOCK - 1) / CK_BLOCK; }

// The block's byte from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t ck_exponent(uint32_t amax) {
  const int b = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0u || amax >= 0x7F800000u ? 127u : (uint32_t)(b < 1 ? 1 : b);
}
// 2^e.
__device__ __forceinline__ float ck_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight values of a block without infinities or NaN as codes: the conversion divides by
// 2^(byte - 127), given as a binary32 of which it takes the exponent.
typedef short ck_s2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void ck_codes(const float (&v)[8], uint32_t byte, uint32_t& lo, uint32_t& hi) {
  const float s = __uint_as_float(byte << 23);
  ck_s2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[0], v[1], s, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[2], v[3], s, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[4], v[5], s, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[6], v[7], s, true);
  lo = __builtin_bit_cast(uint32_t, a);
  hi = __builtin_bit_cast(uint32_t, b);
}
// Four and eight values from their codes and the block's byte.
__device__ __forceinline__ void ck_values(uint32_t w, uint32_t byte, float (&v)[4]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const float s = __uint_as_float(byte << 23);
  const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void ck_values(uint32_t lo, uint32_t hi, uint32_t byte, float (&v)[8]) {
  float a[4], b[4];
  ck_values(lo, byte, a);
  ck_values(hi, byte, b);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = a[k];
    v[k + 4] = b[k];
  }
}

// max |v| of eight; a NaN among them is the maximum.
__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = __builtin_elementwise_maximum(__builtin_fabsf(v[0]), __builtin_fabsf(v[1]));
#pragma unroll
  for (int k = 2; k < 8; k += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(v[k])), __builtin_fabsf(v[k + 1]));
  return m;
}

}  // namespace

}  // namespace fp8lin
