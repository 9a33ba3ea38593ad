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
struct __attribute__((packed, aligned(1))) Pk8a1 { uint32_t v[2]; };

typedef float f32x2_op __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_op __attribute__((ext_vector_type(2)));

// Two binary32 -> two bf16, round to nearest even (one instruction; binary32
// subnormals, below 2^-126, may be off by one bf16 step of 2^-133).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_op v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_op));
}

// v[0..7] = elements i .. i+7 of a bf16 (F32 = 0) or binary32 (F32 = 1) array;
// n < 8: only the first n are there, the others become 0.
__device__ __forceinline__ void load8(const void* base, int f32, int64_t i, int n, float (&v)[8]) {
  if (f32) {
    const float* p = reinterpret_cast<const float*>(base) + i;
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
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + i;
    if (n >= 8) {
      const Pk16a2 a = *reinterpret_cast<const Pk16a2*>(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo(a.v[k]);
        v[2 * k + 1] = bf16_hi(a.v[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? __uint_as_float((uint32_t)p[k] << 16) : 0.0f;
    }
  }
}

__device__ __forceinline__ void store8(void* base, int f32, int64_t i, int n, const float (&v)[8]) {
  if (f32) {
    float* p = reinterpret_cast<float*>(base) + i;
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
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + i;
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

// Eight FP8 codes (two dwords) to element i of a byte array.
__device__ __forceinline__ void store8_codes(uint8_t* base, int64_t i, int n, uint32_t lo, uint32_t hi) {
  uint8_t* p = base + i;
  if (n >= 8) {
    Pk8a1 a;
    a.v[0] = lo;
    a.v[1] = hi;
    *reinterpret_cast<Pk8a1*>(p) = a;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint8_t)((k < 4 ? lo : hi) >> (8 * (k & 3)));
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

// Gate G(g) and its derivative: 0 g itself, 1 sigmoid, 2 tanh.
__device__ __forceinline__ float gate_value(int act, float g) {
  if (act == 1) return 1.0f / (1.0f + expf(-g));
  if (act == 2) return tanhf(g);
  return g;
}
__device__ __forceinline__ float gate_slope(int act, float value) {
  if (act == 1) return value * (1.0f - value);
  if (act == 2) return 1.0f - value * value;
  return 1.0f;
}

// Activations of the linear's epilogue: 0 none, 1 ReLU, 2 GELU (erf),
// 3 GELU (tanh form), 4 SiLU.  The sigmoid forms cost one exponential and one
// reciprocal: the tanh form of GELU is u * sigmoid(2 t), t = sqrt(2/pi) (u +
// 0.044715 u^3), because 0.5 (1 + tanh t) = sigmoid(2 t).
constexpr float kLog2E = 1.44269504088896f;
constexpr float kRootTwoOverPi = 0.797884560802865f;
__device__ __forceinline__ float sigmoid_of_log2(float t) {   // 1 / (1 + 2^-t)
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-t));
}
template <int ACT>
__device__ __forceinline__ float act_value(float u) {
  if constexpr (ACT == 1) return u > 0.0f ? u : (u != u ? u : 0.0f);
  if constexpr (ACT == 2) return 0.5f * u * (1.0f + erff(u * 0.707106781186548f));
  if constexpr (ACT == 3) {
    constexpr float c = 2.0f * kRootTwoOverPi * kLog2E;
    return u * sigmoid_of_log2(u * (c + c * 0.044715f * u * u));
  }
  if constexpr (ACT == 4) return u * sigmoid_of_log2(u * kLog2E);
  return u;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float u) {
  if constexpr (ACT == 1) return u > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == 2)
    return 0.5f * (1.0f + erff(u * 0.707106781186548f)) +
           u * (0.398942280401433f * __builtin_amdgcn_exp2f(-0.5f * kLog2E * u * u));
  if constexpr (ACT == 3) {
    // d/du [u s(2t)] = s + u s (1 - s) 2 t'; beyond +-30 s is 1 or 0 and the
    // second term 0, where u * u could overflow and give inf * 0
    constexpr float c = 2.0f * kRootTwoOverPi;
    u = u == u ? __builtin_amdgcn_fmed3f(u, -30.0f, 30.0f) : u;
    const float s = sigmoid_of_log2(u * (c * kLog2E + c * kLog2E * 0.044715f * u * u));
    return s + u * s * (1.0f - s) * (c + 3.0f * c * 0.044715f * u * u);
  }
  if constexpr (ACT == 4) {
    const float s = sigmoid_of_log2(u * kLog2E);
    return s * (1.0f + u * (1.0f - s));
  }
  return 1.0f;
}

}  // namespace

}  // namespace fp8lin
