// gemm_ep.h -- what the linear's epilogue does to a row of eight outputs, and
// how a wavefront's accumulators become such rows.
//
// With v the dequantised product, summed in binary32 as fp8_scaled_gemm does (of each
// eight products that the matrix unit adds at a time it drops the bits below 2^-13 of
// the largest: 1.1e-5 to 1.5e-5 of v's norm for random operands, K 2304 to 8192, against
// 5e-8 to 1.6e-6 where the products are summed in binary32):
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

// A uniform run-time choice per eight values: one scalar branch.  The tanh form of
// GELU and SiLU are the same code with other factors.
template <bool SLOPE>
__device__ __forceinline__ void activate(int act, float (&v)[8], const float (&u)[8]) {
  if (act == 0) return;
  if (act >= 3) {
    const SigmoidForm f(act);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = SLOPE ? v[k] * f.slope(u[k]) : f.value(u[k]);
  } else if (act == 2) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = SLOPE ? v[k] * gelu_erf<true>(u[k]) : gelu_erf<false>(u[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = SLOPE ? (u[k] > 0.0f ? v[k] : 0.0f * v[k]) : (u[k] <= 0.0f ? 0.0f : u[k]);
  }
}

// Eight values of a row of bf16 or binary32 (WIDE: may be), as they lie in memory
// (see Raw8 in op_device.h); n: how many there are.  Words: a vector where several
// strips' are kept (arrays of arrays went to scratch memory), an array otherwise.  The
// first 16 bytes are loaded ahead of the choice of type: loads of the same words in two
// branches wait where the branches meet, 15% of a whole product's time.
typedef uint32_t v8u __attribute__((ext_vector_type(8)));

template <bool FAST, bool WIDE, typename Words>
__device__ __forceinline__ void load_packed(const void* p, int f32, int n, Words& w) {
  if (n <= 0) return;
  const bool wide = WIDE && f32;
  if (FAST || n >= 8) {
    const uint32_t odd = FAST ? 0u : odd_of(p);
    const Pk16a4 a = *reinterpret_cast<const Pk16a4*>(reinterpret_cast<const char*>(p) - odd);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = a.v[k];
    if constexpr (WIDE) {
      if (wide) {
        const Pk16a4 b = *(reinterpret_cast<const Pk16a4*>(p) + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k + 4] = b.v[k];
        return;
      }
    }
    if constexpr (!FAST) {
      w[4] = 0u;
      if (odd) w[4] = reinterpret_cast<const uint16_t*>(p)[7];
    }
    return;
  }
  if constexpr (!FAST) {
    if (wide) {
      const float* q = reinterpret_cast<const float*>(p);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = k < n ? __float_as_uint(q[k]) : 0u;
      return;
    }
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    uint32_t d[5] = {0u, 0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) d[k >> 1] |= (uint32_t)q[k] << (16 * (k & 1));
    if (odd_of(p)) {
#pragma unroll
      for (int k = 4; k >= 1; --k) d[k] = __builtin_amdgcn_alignbyte(d[k], d[k - 1], 2);
      d[0] <<= 16;
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = d[k];
  }
}

// Eight bf16 or binary32 values, or eight codes, to p, by SEG neighbouring lanes
// per row (see store_row); n: how many are written.
template <int SEG, bool FAST>
__device__ __forceinline__ void put8(void* p, int f32, int n, const float (&v)[8]) {
  if (f32) {
    if (!FAST) store8(p, 1, 0, n, v);
    else if (n > 0) store8(p, 1, 0, 8, v);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
  if constexpr (FAST) {
    if (n > 0) {
      Pk16a4 a;
#pragma unroll
      for (int k = 0; k < 4; ++k) a.v[k] = w[k];
      *reinterpret_cast<Pk16a4*>(p) = a;
    }
    return;
  }
  store_row<4, SEG>(reinterpret_cast<uint8_t*>(p), w, n >= 8);
  if (n > 0 && n < 8) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) reinterpret_cast<uint16_t*>(p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
  }
}
template <int SEG, bool FAST>
__device__ __forceinline__ void put8_codes(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
  if constexpr (FAST) {
    struct __attribute__((packed, aligned(4))) Two { uint32_t a, b; };
    if (n > 0) *reinterpret_cast<Two*>(p) = Two{lo, hi};
    return;
  }
  const uint32_t w[2] = {lo, hi};
  store_row<2, SEG>(p, w, n >= 8);
  if (n > 0 && n < 8) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) p[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
  }
}

// Eight codes; a NaN (rare) is patched in place, without a call, which would
// spill the caller's accumulators.
template <int FMT>
__device__ __forceinline__ void encode8(const float (&x)[8], uint32_t& lo, uint32_t& hi) {
  int a, b;
  if constexpr (FMT == 0) {
    a = __builtin_amdgcn_cvt_pk_fp8_f32(sat<0>(x[0]), sat<0>(x[1]), 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(sat<0>(x[2]), sat<0>(x[3]), a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(sat<0>(x[4]), sat<0>(x[5]), 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(sat<0>(x[6]), sat<0>(x[7]), b, true);
  } else {
    a = __builtin_amdgcn_cvt_pk_bf8_f32(sat<1>(x[0]), sat<1>(x[1]), 0, false);
    a = __builtin_amdgcn_cvt_pk_bf8_f32(sat<1>(x[2]), sat<1>(x[3]), a, true);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(sat<1>(x[4]), sat<1>(x[5]), 0, false);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(sat<1>(x[6]), sat<1>(x[7]), b, true);
  }
  lo = (uint32_t)a;
  hi = (uint32_t)b;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 8; k += 2) nan |= __builtin_isunordered(x[k], x[k + 1]);
  if (__builtin_expect(nan, 0)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t code = 0x7Fu | ((__float_as_uint(x[k]) >> 24) & 0x80u), w = k < 4 ? lo : hi;
      const int s = 8 * (k & 3);
      const uint32_t q = x[k] == x[k] ? w : ((w & ~(0xFFu << s)) | (code << s));
      if (k < 4) lo = q;
      else hi = q;
    }
  }
}

// FAST: whole vectors only (N a multiple of 8) that start on a dword in every row;
// the others' accesses of single elements are a third of the code, and in the
// large kernels, whose epilogue is unrolled over 8 strips, more than the
// instruction cache holds.
// Directions of an epilogue: fixed at compile time in the large kernels (half the
// code), by EpParams::backward in the others.
enum : int { EP_FWD = 0, EP_BWD = 1, EP_ANY = 2 };

// One wavefront's columns n0 .. n0 + WTN - 1, lane's columns c .. c + 7.
template <int WTN, bool OUT8, int DIR, bool FAST>
struct EpWave {
  static constexpr int LPR = WTN / 8;        // lanes per row
  static constexpr int RPL = WTN / 32;       // rows per lane and strip of 16
  static_assert(RPL == 1 || RPL == 2 || RPL == 4, "32, 64 or 128 columns");
  static constexpr bool WIDE = !OUT8 && DIR != EP_BWD;   // src may be binary32
  using Words = typename std::conditional<FAST, uint32_t[WIDE ? 8 : 4], v8u>::type;
  static constexpr int CH = WTN / 4;         // 16-byte chunks of a strip's row
  const GemmParams& p;
  const EpParams& e;
  int lane, cq, rg, nv;
  int64_t c;
  float bias[8], db[8];
  uint32_t amax = 0;
  float so;
  const char* src;      // what is read beside the product: pre-activation (backward) or residual
  int64_t src_ld;       // bytes per row
  int src_f32;

  __device__ __forceinline__ bool backward() const { return DIR == EP_ANY ? e.backward != 0 : DIR == EP_BWD; }

  __device__ __forceinline__ EpWave(const GemmParams& p_, const EpParams& e_, int64_t n0, int lane_)
      : p(p_), e(e_), lane(lane_), cq(lane_ % LPR), rg(lane_ / LPR), c(n0 + 8 * (lane_ % LPR)) {
    const int64_t left = p.N - c;
    nv = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) { bias[k] = 0.0f; db[k] = 0.0f; }
    if (!backward() && e.bias) load8(e.bias, e.bias_f32, c, nv, bias);
    so = OUT8 ? p.d_scale[0] : 1.0f;
    src_f32 = backward() || OUT8 ? 0 : e.res_f32;
    const int es = src_f32 ? 4 : 2;
    src = reinterpret_cast<const char*>(backward() ? (e.act ? e.aux : nullptr) : e.residual);
    src_ld = (backward() ? e.ldaux : e.ldres) * es;
    if (src) src += c * es;
  }

  // The strip of rows m0 .. m0 + 15 of src, in flight until stage() puts it into
  // LDS, where the loop over the rows can index it.
  __device__ __forceinline__ void fetch(int64_t m0, Words (&o)[RPL]) {
    if (src == nullptr) return;
#pragma unroll
    for (int t = 0; t < RPL; ++t) {
      const int64_t m = m0 + rg * RPL + t;
      load_packed<FAST, WIDE>(src + m * src_ld, src_f32, m < p.M ? nv : 0, o[t]);
    }
  }
  // Each lane's own words: 16 bytes per lane and row for bf16, twice that for
  // binary32.
  static constexpr int SRC_BYTES = RPL * 64 * 16;
  __device__ __forceinline__ void stage(int64_t m0, const Words (&o)[RPL], uint8_t* ol) {
    if (src == nullptr) return;
    uint4* q = reinterpret_cast<uint4*>(ol) + lane;
#pragma unroll
    for (int t = 0; t < RPL; ++t) {
      if (FAST || src_f32) q[t * 64] = make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
      if constexpr (WIDE) {
        if (src_f32) q[(RPL + t) * 64] = make_uint4(o[t][4], o[t][5], o[t][6], o[t][7]);
      }
      if constexpr (!FAST) {
        if (src_f32) continue;
        const uint32_t s = odd_of(src + (m0 + rg * RPL + t) * src_ld);
        q[t * 64] = make_uint4(__builtin_amdgcn_alignbyte(o[t][1], o[t][0], s), __builtin_amdgcn_alignbyte(o[t][2], o[t][1], s),
                               __builtin_amdgcn_alignbyte(o[t][3], o[t][2], s), __builtin_amdgcn_alignbyte(o[t][4], o[t][3], s));
      }
    }
  }

  // Where the strip's row r keeps columns 4 q .. 4 q + 3.
  static __device__ __forceinline__ float4* place(uint8_t* wl, int r, int q) {
    return reinterpret_cast<float4*>(wl + r * (WTN * 4) + ((q ^ (r & (CH - 1))) << 4));
  }

  // The strip in wl, rows m0 + rg RPL + t for t = 0 .. RPL - 1, one after the
  // other in a loop that stays one: unrolled over its 4 rows and a wavefront's 8
  // strips the epilogue was 44000 instructions, several times the instruction
  // cache.  ol: src's rows (stage); tl: column-major codes of the wavefront (TS
  // bytes per column, this strip's rows at byte tr), if D_t.
  template <int TS>
  __device__ __forceinline__ void rows(int64_t m0, uint8_t* wl, const uint8_t* ol, uint8_t* tl, int tr) {
    uint32_t turned[8] = {};
    const int64_t first = m0 + rg * RPL;
    const int esz = OUT8 ? 1 : (p.d_f32 ? 4 : 2);
    char* d = reinterpret_cast<char*>(p.D) + (first * p.ldd + c) * esz;
    char* aux = (!backward() && e.aux)
                    ? reinterpret_cast<char*>(const_cast<void*>(e.aux)) + (first * e.ldaux + c) * 2 : nullptr;
    const uint4* q = reinterpret_cast<const uint4*>(ol) + lane;
    const bool wide = WIDE && src != nullptr && src_f32;
#pragma unroll 1
    for (int t = 0; t < RPL; ++t) {
      const float4 w0 = *place(wl, rg * RPL + t, 2 * cq), w1 = *place(wl, rg * RPL + t, 2 * cq + 1);
      float v[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      const int n = first + t < p.M ? nv : 0;
      float u[8];
      if (src) {
        const uint4 a = q[t * 64];
        if (wide) {
          const uint4 b = q[(RPL + t) * 64];
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = __uint_as_float(w[k]);
        } else {
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            u[2 * k] = bf16_lo(w[k]);
            u[2 * k + 1] = bf16_hi(w[k]);
          }
        }
      }
      if (!backward()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += bias[k];
        if (aux) put8<LPR, FAST>(aux, 0, n, v);
        activate<false>(e.act, v, v);
        if (src) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __builtin_fmaf(e.res_scale, u[k], v[k]);
        }
      } else {
        if (src) activate<true>(e.act, v, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) db[k] += (FAST ? n > 0 : k < n) ? v[k] : 0.0f;
      }
      if (p.d_amax) {
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max_u32(amax, (FAST ? n > 0 : k < n) ? abs_bits(v[k]) : 0u);
      }
      if constexpr (OUT8) {
        uint32_t lo, hi;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= so;
        if (p.d_fp8 == 1) encode8<0>(v, lo, hi);
        else encode8<1>(v, lo, hi);
        put8_codes<LPR, FAST>(reinterpret_cast<uint8_t*>(d), n, lo, hi);
        if (p.D_t) {   // code k to the top of column k's word, the rows before down a byte
#pragma unroll
          for (int k = 0; k < 8; ++k)
            turned[k] = __builtin_amdgcn_perm(k < 4 ? lo : hi, turned[k], 0x00030201u | ((uint32_t)(4 + (k & 3)) << 24));
        }
      } else {
        put8<LPR, FAST>(d, p.d_f32, n, v);
      }
      d += p.ldd * esz;
      if (aux) aux += e.ldaux * 2;
    }
    if constexpr (OUT8) {
      if (p.D_t) {
        uint8_t* dst = tl + (8 * cq) * TS + tr + rg * RPL;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (RPL == 4) *reinterpret_cast<uint32_t*>(dst + k * TS) = turned[k];
          else if constexpr (RPL == 2) *reinterpret_cast<uint16_t*>(dst + k * TS) = (uint16_t)(turned[k] >> 16);
          else dst[k * TS] = (uint8_t)(turned[k] >> 24);
        }
      }
    }
    asm volatile("" ::: "memory");   // LDS is written and read as different types
  }

  // LDS of a wavefront of TI strips: the strip (64 WTN bytes), src's rows, then
  // (OUT8) the column-major codes.  (An FP8
  // output takes a bf16 residual only, so its src words are half as many.)
  static constexpr int strip_at = 0, src_at = 64 * WTN;
  static constexpr int codes_at = src_at + (OUT8 ? 1 : 2) * SRC_BYTES;
  static constexpr int bytes(int TI) { return codes_at + (OUT8 ? WTN * (16 * TI + 16) : 0); }

  // Accumulators to strips.  acc[i][j] of lane (g, l16): row r0 + 16 i + l16,
  // columns n0 + 16 j + 4 g .. + 3.  wl: bytes(TI) of LDS, wavefront-private.  Here src
  // is fetched strip by strip; below (o) every strip's words are there already.
  template <int TI, int TJ, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl) {
    Words o[1][RPL];
    fetch(r0, o[0]);
    tile(acc, deq, r0, n0, wl, o);
  }
  template <int TI, int TJ, int STRIPS, typename Deq>
  __device__ __forceinline__ void tile(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0, int64_t n0, uint8_t* wl,
                                       Words (&o)[STRIPS][RPL]) {
    static_assert(16 * TJ == WTN, "the wavefront's columns");
    static_assert(STRIPS == 1 || STRIPS == TI, "one strip ahead, or all");
    constexpr int TS = 16 * TI + 16;
    const int g = lane >> 4, l16 = lane & 15;
    ep_for<0, TI>([&](auto itag) {
      constexpr int i = decltype(itag)::value;
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        *place(wl, l16, 4 * j + g) = make_float4(deq(i, j, 0, acc[i][j][0]), deq(i, j, 1, acc[i][j][1]),
                                                 deq(i, j, 2, acc[i][j][2]), deq(i, j, 3, acc[i][j][3]));
      stage(r0 + 16 * i, o[STRIPS == 1 ? 0 : i], wl + src_at);
      if constexpr (STRIPS == 1 && i + 1 < TI) fetch(r0 + 16 * (i + 1), o[0]);
      rows<TS>(r0 + 16 * i, wl, wl + src_at, wl + codes_at, 16 * i);
    });
    if constexpr (OUT8) {
      if (p.D_t) flush_t<TS, 16 * TI>(wl + codes_at, r0, n0);
    }
  }

  // The column-major codes of ROWS rows to D_t, 16 bytes per lane.
  template <int TS, int ROWS>
  __device__ __forceinline__ void flush_t(const uint8_t* tl, int64_t r0, int64_t n0) {
    constexpr int LPC = ROWS / 16;
    const int q = lane % LPC;
    const int64_t m = r0 + 16 * q, left = p.M - m;
#pragma unroll 2
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
    if (!backward() || e.dbias == nullptr) return;
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
__device__ __forceinline__ void ep_amax(float* d_amax, uint32_t bits, int lane, int wave);

// What the kernels on tiles and on few rows are built around: the epilogue's
// arguments, and who takes a wavefront's sums of WTN columns of B's rows.  PAIRED: B's
// rows come in pairs of a product with two factors (see half_of in fp8_device.h).
struct LinearOp {
  using Params = EpParams;
  static constexpr bool PAIRED = false;
  template <int WTN, bool OUT8>
  using Wave = EpWave<WTN, OUT8, EP_ANY, false>;
};

// The epilogue as the large kernels take it (FAST): accumulators of a wavefront whose
// rows start at r0 and columns at c0; part: its row of column sums.
template <int DIR>
struct LinearEp {
  static constexpr bool PAIRED = false, DIRECT = false;
  EpParams e;
  template <bool OUT8, int TI, int TJ, int NW, typename Deq>
  __device__ __forceinline__ void finish(const GemmParams& p, const v4f (&acc)[TI][TJ], Deq&& deq, int64_t r0,
                                         int64_t c0, int64_t part, int lane, int wave, uint8_t* wl) const {
    using W = EpWave<16 * TJ, OUT8, DIR, true>;
    static_assert(W::bytes(TI) <= 128 * 1024 / NW, "the wavefront's part of the stages");
    W w(p, e, c0, lane);
    w.template tile<TI, TJ>(acc, deq, r0, c0, wl);
    w.put_dbias(part);
    if (p.d_amax) ep_amax<NW>(p.d_amax, w.amax_bits(), lane, wave);
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
