// checkpoint_kernels.hip -- 8-bit checkpoints (checkpoint.h) of whole tensors, written
// and read back.
//
// A lane takes eight neighbouring columns of a row, four lanes a block of 32, whose
// largest magnitude they exchange inside their quad; nothing is kept but the eight
// values.  Bound: HBM (8192 x 8192 BF16 saved in 40.5 us, 5.0 TB/s, a copy's rate; 8192 x 14336
// loaded in 63), small ones by a launch and a load's latency (1531 x 2053 FP32 7.4 us, of
// which the call's host part is 5.5).  A row per workgroup and step, 2048 columns of it: no
// lane has a division, but lanes past a row's end have no work.  Widths that fill the
// workgroups are at a copy's rate, others are not: 16.8 M values BF16 saved as 8192 x 2048 in 9.8
// us, as 8192 x 2053 in 20.5, as 65536 x 256 in 41.5, as 262144 x 64 in 98 (loaded in 9.5, 14.1,
// 30.8 and 35.8).
#include "checkpoint.h"
#include "launch.h"

namespace fp8lin {

namespace {

constexpr int CK_THREADS = 256;

__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
  const uint32_t w[2] = {lo, hi};
  store_row<2, 4>(p, w, n >= 8);
  if (n > 0 && n < 8) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) p[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
  }
}

template <bool F32>
__global__ void __launch_bounds__(CK_THREADS) k_checkpoint_save(const void* x, int64_t rows, int64_t cols, int64_t ldx,
                                                                uint8_t* ck, int64_t ldck, uint8_t* ck_exp,
                                                                int64_t ldexp) {
  const int64_t c = ((int64_t)blockIdx.x * CK_THREADS + threadIdx.x) * 8;
  const int n = cols - c >= 8 ? 8 : (cols > c ? (int)(cols - c) : 0);
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    float v[8] = {};
    if (n > 0) load8(x, F32, r * ldx + c, n, v);
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) a = max_u32(a, abs_bits(v[k]));
    const bool tame = __builtin_amdgcn_ballot_w64(a >= 0x7F800000u) == 0;
    a = max_u32(a, dpp<kXor1>(a));
    a = max_u32(a, dpp<kXor2>(a));
    const uint32_t byte = ck_exponent(a);
    uint32_t lo, hi;
    if (__builtin_expect(tame, 1)) {
      ck_codes(v, byte, lo, hi);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= ck_scale(byte);
      codes8(0, v, 1.0f, lo, hi);
    }
    store_codes(ck + r * ldck + c, n, lo, hi);
    if ((threadIdx.x & 3) == 0 && n > 0) ck_exp[r * ldexp + (c >> 5)] = (uint8_t)byte;
  }
}

template <bool F32>
__global__ void __launch_bounds__(CK_THREADS) k_checkpoint_load(const uint8_t* ck, int64_t ldck, const uint8_t* ck_exp,
                                                                int64_t ldexp, int64_t rows, int64_t cols, void* y,
                                                                int64_t ldy) {
  const int64_t c = ((int64_t)blockIdx.x * CK_THREADS + threadIdx.x) * 8;
  const int n = cols - c >= 8 ? 8 : (cols > c ? (int)(cols - c) : 0);
  if (n == 0) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const uint8_t* p = ck + r * ldck + c;
    uint32_t d[2] = {0u, 0u};
    if (n >= 8) {
      struct __attribute__((packed, aligned(1))) Two { uint32_t a, b; };
      const Two q = *reinterpret_cast<const Two*>(p);
      d[0] = q.a;
      d[1] = q.b;
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < n) d[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
    }
    float v[8];
    ck_values(d[0], d[1], ck_exp[r * ldexp + (c >> 5)], v);
    store8(y, F32, r * ldy + c, n, v);
  }
}

dim3 grid_of(int64_t rows, int64_t cols) {
  const int64_t x = (cols + 8 * CK_THREADS - 1) / (8 * CK_THREADS);
  return dim3((unsigned)x, (unsigned)(rows < 65535 ? rows : 65535));
}

}  // namespace

hipError_t launch_checkpoint_save(const void* x, int f32, int64_t rows, int64_t cols, int64_t ldx, uint8_t* ck,
                                  int64_t ldck, uint8_t* ck_exp, int64_t ldexp, hipStream_t s) {
  const dim3 grid = grid_of(rows, cols);
  if (f32)
    hipLaunchKernelGGL((k_checkpoint_save<true>), grid, dim3(CK_THREADS), 0, s, x, rows, cols, ldx, ck, ldck, ck_exp, ldexp);
  else
    hipLaunchKernelGGL((k_checkpoint_save<false>), grid, dim3(CK_THREADS), 0, s, x, rows, cols, ldx, ck, ldck, ck_exp, ldexp);
  return hipGetLastError();
}

hipError_t launch_checkpoint_load(const uint8_t* ck, int64_t ldck, const uint8_t* ck_exp, int64_t ldexp, int64_t rows,
                                  int64_t cols, void* y, int f32, int64_t ldy, hipStream_t s) {
  const dim3 grid = grid_of(rows, cols);
  if (f32)
    hipLaunchKernelGGL((k_checkpoint_load<true>), grid, dim3(CK_THREADS), 0, s, ck, ldck, ck_exp, ldexp, rows, cols, y, ldy);
  else
    hipLaunchKernelGGL((k_checkpoint_load<false>), grid, dim3(CK_THREADS), 0, s, ck, ldck, ck_exp, ldexp, rows, cols, y, ldy);
  return hipGetLastError();
}

}  // namespace fp8lin
