// checkpoint.h -- tensors kept for the backward pass in 8 bits: E4M3 codes, and for each
// block of 32 neighbouring columns of a row one power of two.
//
// With a = max |x| of the block (an exact maximum) and e the largest integer with
// a 2^e <= 448, |e| <= 126, a code is encode(x 2^e), x 2^e being exact, and the block's
// byte is 127 - e: 2^(byte - 127) takes a code back to a value.  Nothing saturates; a
// value is off by at most 2^-4 of itself, or 2^-10 2^-e, below 2^-17 of its block's largest.  A block of zeros, or one
// that holds an infinity or a NaN, has e = 0, as in the block casts.
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
// 2^e, and back: 2^-e.  (Bytes are 1 .. 247 as made here; read, 0 is 2^-127, a binary32
// subnormal, and 255 a NaN, as E8M0 has them.)
__device__ __forceinline__ float ck_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float ck_unscale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

// Eight values from their codes and the block's byte.
__device__ __forceinline__ void ck_values(uint32_t lo, uint32_t hi, uint32_t byte, float (&v)[8]) {
  const float s = ck_unscale(byte);
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, true);
  const f2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, true);
  v[0] = a.x * s; v[1] = a.y * s; v[2] = b.x * s; v[3] = b.y * s;
  v[4] = c.x * s; v[5] = c.y * s; v[6] = d.x * s; v[7] = d.y * s;
}

}  // namespace

}  // namespace fp8lin
