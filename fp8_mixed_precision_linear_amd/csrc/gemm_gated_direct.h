// gemm_gated_direct.h -- the gated pair's epilogue (gemm_gated.h has the formulas) as the
// four-wavefront kernel (k_gemm_w4) takes it: from the accumulators, without LDS.
//
// The matrix instruction leaves lane (g, l16) with four neighbouring rows of its B operand
// and one row of its A operand of each 16 x 16 tile.  Which rows of A and B those stand for
// is the DMA's choice (TilePlace in gemm_w4_kernel.h), and it is made so that a lane ends up
// with neighbouring rows and columns: of its wavefront's 128 rows, rows 64 h + 4 l16 + t
// (h = 0, 1; t = 0 .. 3); of its columns, runs of 16, the four lanes of a row side by side
// (forward one run of outputs, both factors; backward two runs).  So a row's codes leave as
// 16 bytes a lane and 64 together, four rows' transposed codes as one word a column, a
// checkpoint's block of 32 is two lanes, and a bias gradient is summed in registers.
//
// With one wavefront on a SIMD nothing hides what an instruction takes: by way of LDS
// (gemm_gated.h), 8192 x 28672 x 8192 took 1990 us backward (checkpoint, E5M2 codes, both
// orders, bias gradient) and 2990 forward (checkpoint, E4M3 codes, both orders), here 1690
// and 2760 (with the amax; 2745 the kernel); fp8_scaled_gemm alone is 1400 and 2640.  Runs of 16 columns per lane that were
// not side by side cost 80 us more backward, and 16-byte halves of a row's 64 with BF16 400.
// What is read beside the sums is on its way four rows ahead, the first rows before the last
// step of K; every access is a buffer access whose range check drops rows and columns past
// the end, so that none is branched around.
#pragma once

#include "gemm_big_kernel.h"
#include "gemm_gated.h"

namespace fp8lin {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Rows r0 .. of an array, ld bytes each, as a buffer: rows past the end are out of range.
// `off` is the lane's place in it, `more` what is the same for all of them (the range check
// may take it off the buffer's size, so it is less than ld, and there is a row).
struct RowsOf {
  __amdgpu_buffer_rsrc_t r;
  int ld;
  __device__ __forceinline__ RowsOf(const void* base, int64_t r0, int64_t ld_, int64_t rows) : ld((int)ld_) {
    const char* b = reinterpret_cast<const char*>(base) + (base ? r0 * ld_ : 0);
    const int64_t n = base && rows > 0 ? rows * ld_ : 0;
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(b), 0, (int)n, kRsrcWord3);
  }
  __device__ __forceinline__ void put16(uint32_t off, uint32_t more, const uint32_t* w) const {
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, r, off, more, 0);
  }
  __device__ __forceinline__ u32x4 get16(uint32_t off, uint32_t more) const {
    return __builtin_amdgcn_raw_buffer_load_b128(r, off, more, 0);
  }
  __device__ __forceinline__ uint32_t get1(uint32_t off, uint32_t more) const {
    return __builtin_amdgcn_raw_buffer_load_b8(r, off, more, 0);
  }
};

// max |v| of N values; a NaN among them is the maximum.
template <int N>
__device__ __forceinline__ float max_of(const float (&v)[N]) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int k = 1; k + 1 < N; k += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(v[k])), __builtin_fabsf(v[k + 1]));
  return __builtin_elementwise_maximum(m, __builtin_fabsf(v[N - 1]));
}
template <int N>
__device__ __forceinline__ const float (&eight(const float (&v)[N], int i))[8] {
  return *reinterpret_cast<const float(*)[8]>(&v[8 * i]);
}
template <int N>
__device__ __forceinline__ float (&eight(float (&v)[N], int i))[8] {
  return *reinterpret_cast<float(*)[8]>(&v[8 * i]);
}

// N values times s as codes; tame: see encode_tame.
template <int N>
__device__ __forceinline__ void codes_to(int fp8, bool tame, const float (&v)[N], float s, uint32_t (&w)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = v[8 * i + k] * s;
    codes_of(fp8, tame, x, w[2 * i], w[2 * i + 1]);
  }
}
__device__ __forceinline__ void codes_to(int fp8, bool tame, const float (&v)[4], float s, uint32_t (&w)[1]) {
  const float x[4] = {v[0] * s, v[1] * s, v[2] * s, v[3] * s};
  if (__builtin_expect(tame, 1)) {
    int a;
    if (fp8 == 1) {
      a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
      a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], a, true);
    } else {
      a = __builtin_amdgcn_cvt_pk_bf8_f32(x[0], x[1], 0, false);
      a = __builtin_amdgcn_cvt_pk_bf8_f32(x[2], x[3], a, true);
    }
    w[0] = (uint32_t)a;
  } else {
    w[0] = fp8 == 1 ? cvt4<0, true>(x[0], x[1], x[2], x[3]) : cvt4<1, true>(x[0], x[1], x[2], x[3]);
  }
}
// N values to a row: binary32, or bf16 too.
template <int N>
__device__ __forceinline__ void put_f32(const RowsOf& d, uint32_t off, uint32_t more, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t w[4] = {__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                           __float_as_uint(v[4 * i + 3])};
    d.put16(off, more + 16 * i, w);
  }
}
template <int N>
__device__ __forceinline__ void put_wide(const RowsOf& d, int f32, uint32_t off, uint32_t more, const float (&v)[N]) {
  if (f32) {
    put_f32(d, off, more, v);
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = pack_bf16(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
      d.put16(off, more + 16 * i, w);
    }
  }
}

// Four rows' codes of N columns to N rows of D_t, a word each.
struct TurnedOf {
  __amdgpu_buffer_rsrc_t r;
  int ld;
  uint32_t at;      // the lane's first column, first row of the wavefront's first half
  int left;         // rows from there on
  __device__ __forceinline__ TurnedOf(const GemmParams& p, int64_t r0, int64_t n0, int64_t cols, int lane_col, int l16, bool on)
      : ld((int)p.ldt), at(on ? (uint32_t)(lane_col * (int)p.ldt + 4 * l16) : kOOB), left((int)min(p.M - r0, (int64_t)128) - 4 * l16) {
    uint8_t* b = p.D_t + (p.D_t ? n0 * p.ldt + r0 : 0);
    // (rows past the last are told by `left`: they would be the next column's first)
    const int64_t n = p.D_t && cols > 0 && p.M > r0 ? (cols - 1) * p.ldt + min(p.M - r0, (int64_t)128) : 0;
    r = __builtin_amdgcn_make_buffer_rsrc(b, 0, (int)n, kRsrcWord3);
  }
  template <int N>
  __device__ __forceinline__ void put(int h, int col, const uint32_t (&w)[4][N / 4]) const {
    uint32_t o = at + (uint32_t)(col * ld + 64 * h);
    const int n = left - 64 * h;
    if (at == kOOB || n < 4) o = kOOB;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      uint32_t t[4];
      transpose4x4(w[0][i], w[1][i], w[2][i], w[3][i], t[0], t[1], t[2], t[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        __builtin_amdgcn_raw_buffer_store_b32(t[k], r, o == kOOB ? kOOB : o + (uint32_t)((4 * i + k) * ld), 0, 0);
      if (at != kOOB && n > 0 && n < 4) {   // the last rows of D, fewer than four
#pragma unroll
        for (int k = 0; k < 4; ++k)
          for (int b = 0; b < n; ++b)
            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(t[k] >> (8 * b)), r,
                                                 at + (uint32_t)((col + 4 * i + k) * ld + 64 * h + b), 0, 0);
      }
    }
  }
};

// The rows' values: rows 64 h + 4 l16 + t are accumulator rows 4 h + t.  h and the run of
// columns are known at run time (the loops over them are not unrolled, so that the
// epilogue stays in the instruction cache); the branches are told apart, since merged they
// would index the accumulators, which would then live in scratch memory.
template <int BEGIN, int END, typename F>
__device__ __forceinline__ void one_of(int i, F&& f) {
  if constexpr (BEGIN < END) {
    if (i == BEGIN) {
      asm volatile("; rows %0" ::"n"(BEGIN) : "memory");
      f(std::integral_constant<int, BEGIN>{});
      asm volatile("; rows %0 taken" ::"n"(BEGIN) : "memory");
    }
    one_of<BEGIN + 1, END>(i, f);
  }
}

// max |d| of the wavefront as stored, from its lanes'.
template <bool OUT8>
__device__ __forceinline__ uint32_t amax_bits(const GemmParams& p, float top) {
  const uint32_t a = wave_max(__float_as_uint(top));
  return !OUT8 && !p.d_f32 ? (uint32_t)f32_to_bf16_rne(__uint_as_float(a)) << 16 : a;
}

// Four sums, read where this stands: their scaling, which does not change from turn to
// turn of the loops, would be taken out of them for all sums at once, and spill.
__device__ __forceinline__ v4f here(const v4f& x) {
  float a = x[0], b = x[1], c = x[2], d = x[3];
  asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
  return v4f{a, b, c, d};
}
__device__ __forceinline__ float pick(bool c, float a, float b) { return c ? a : b; }   // (by value)
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

template <bool OUT8, int TI, int TJ, int NW>
struct GatedRun {
  static constexpr int N = 16;           // outputs of a lane
  static_assert(TI == 8 && TJ == 8, "128 rows, 64 outputs");
  const GemmParams& p;
  const GatedParams& e;
  int g, l16, rows;
  int64_t r0, c0;
  bool on;
  uint32_t col;      // the lane's first output, from c0 on
  __device__ __forceinline__ GatedRun(const GemmParams& p_, const GatedParams& e_, int64_t r0_, int64_t cb, int lane)
      : p(p_), e(e_), g(lane >> 4), l16(lane & 15), rows((int)min(p_.M - r0_, (int64_t)128)), r0(r0_), c0(cb / 2),
        on(cb / 2 + N * (lane >> 4) < p_.N), col((uint32_t)(N * (lane >> 4))) {}
  __device__ __forceinline__ void ahead() {}

  // N of a block's 32 values to the checkpoint.
  __device__ __forceinline__ void keep(const float (&v)[N], const RowsOf& ck, uint32_t off, uint32_t more, const RowsOf& exp, uint32_t xoff,
                                       uint32_t xmore) const {
    uint32_t a = __float_as_uint(max_of(v));
    const bool tame = __builtin_amdgcn_ballot_w64(a >= 0x7F800000u) == 0;
    auto s = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    a = max_u32(s[0], s[1]);
    const uint32_t byte = ck_exponent(a);
    uint32_t w[N / 4];
    if (__builtin_expect(tame, 1)) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) ck_codes(eight(v, i), byte, w[2 * i], w[2 * i + 1]);
    } else {
      codes_to(1, false, v, ck_scale(byte), w);
    }
    ck.put16(off, more, w);
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)byte, exp.r, (g & 1) == 0 ? xoff : kOOB, xmore, 0);
  }

  template <typename Deq>
  __device__ __forceinline__ void finish(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t, int lane, int wave) const {
    int where = 0;
    const float top = rows > 0 ? body(acc, deq, where) : 0.0f;
    if constexpr (OUT8) {
      if (e.keys) put_key(e, top, (int)r0 + where, (int)c0 + (int)col, N);
    }
    if (p.d_amax) ep_amax<NW>(p.d_amax, amax_bits<OUT8>(p, top), lane, wave);
  }
  template <typename Deq>
  __device__ __forceinline__ float body(const v4f (&acc)[TI][TJ], Deq&& deq, int& where) const {
    const int64_t F = p.N;
    const int esz = OUT8 ? 1 : (p.d_f32 ? 4 : 2);
    const RowsOf D(p.D, r0, p.ldd * esz, rows), aux(e.aux, r0, e.ldaux * 2, rows), ck(e.ck, r0, e.ldck, rows),
        exp(e.ck_exp, r0, e.ldexp, rows);
    const TurnedOf D_t(p, r0, c0, min(F - c0, (int64_t)(4 * N)), (int)col, l16, on);
    const uint32_t c = (uint32_t)c0 + col, nb = (uint32_t)ck_blocks(F);
    float bg[N], bu[N];
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const int n = on && e.bias ? 8 : 0;
      load8(e.bias, e.bias_f32, (int64_t)c + 8 * i, n, eight(bg, i));
      load8(e.bias, e.bias_f32, F + c + 8 * i, n, eight(bu, i));
    }
    const float so = OUT8 ? p.d_scale[0] : 1.0f, most = p.d_fp8 == 1 ? Fmt<0>::max : Fmt<1>::max;
    float top = 0.0f;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t turned[4][N / 4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float G[N], U[N], v[N];
        __builtin_amdgcn_sched_barrier(0);
        one_of<0, 2>(h, [&](auto hh) {
          constexpr int i = 4 * decltype(hh)::value;
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            const v4f x = here(acc[i + t][j]);
#pragma unroll
            for (int q = 0; q < 4; ++q) (j & 1 ? U : G)[4 * (j >> 1) + q] = deq(i + t, j, q, x[q]);
          }
        });
#pragma unroll
        for (int k = 0; k < N; ++k) {
          G[k] += bg[k];
          U[k] += bu[k];
        }
        const int row = 64 * h + 4 * l16 + t;
        if (e.aux) {
          const uint32_t off = on ? (uint32_t)(row * aux.ld) + 2 * c : kOOB;
          put_wide(aux, 0, off, 0, G);
          put_wide(aux, 0, off, 2 * (uint32_t)F, U);
        }
        if (e.ck) {
          const uint32_t off = on ? (uint32_t)(row * ck.ld) + c : kOOB, x = on ? (uint32_t)(row * exp.ld) + (c >> 5) : kOOB;
          keep(G, ck, off, 0, exp, x, 0);
          keep(U, ck, off, (uint32_t)F, exp, x, nb);
        }
#pragma unroll
        for (int i = 0; i < N / 8; ++i) act_of(e.act, eight(G, i), eight(v, i));
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] *= U[k];
        const float m = row < rows && on ? max_of(v) : 0.0f;
        if constexpr (OUT8) where = __float_as_uint(__builtin_elementwise_maximum(top, m)) != __float_as_uint(top) ? row : where;
        top = __builtin_elementwise_maximum(top, m);
        const uint32_t off = on ? (uint32_t)(row * D.ld) + c * (uint32_t)esz : kOOB;
        if constexpr (OUT8) {
          const bool tame = __builtin_amdgcn_ballot_w64(!(m * __builtin_fabsf(so) <= most)) == 0;
          codes_to(p.d_fp8, tame, v, so, turned[t]);
          D.put16(off, 0, turned[t]);
        } else {
          put_wide(D, p.d_f32, off, 0, v);
        }
      }
      if constexpr (OUT8) {
        if (p.D_t) D_t.put<N>(h, 0, turned);
      }
    }
    return top;
  }
};

// KEPT: g and u come from BF16 (0) or from a checkpoint (1).
template <bool OUT8, int KEPT, int TI, int TJ, int NW>
struct GatedGradRun {
  // a unit: 4 rows of one of the two runs of 16 columns; the runs of four rows follow each
  // other, so that a line of memory is touched twice in a row
  static constexpr int N = 16, UNITS = 4;
  static_assert(TI == 8 && TJ == 8, "128 rows and columns");
  const GemmParams& p;
  const GatedParams& e;
  int g, l16, rows;
  int64_t r0, c0;
  RowsOf in, exp;
  static constexpr int GV = KEPT ? 1 : 2;
  struct In {
    u32x4 g[GV], u[GV];
    uint32_t xg, xu;
  } in4[4];   // the next four rows, on their way

  __device__ __forceinline__ GatedGradRun(const GemmParams& p_, const GatedParams& e_, int64_t r0_, int64_t cb, int lane)
      : p(p_), e(e_), g(lane >> 4), l16(lane & 15), rows((int)min(p_.M - r0_, (int64_t)128)), r0(r0_), c0(cb),
        in(KEPT ? e_.ck : e_.aux, r0_, KEPT ? e_.ldck : 2 * e_.ldaux, rows), exp(KEPT ? e_.ck_exp : nullptr, r0_, e_.ldexp, rows) {}
  // A unit's first column, from c0 on, and whether it is there.
  __device__ __forceinline__ uint32_t col(int unit) const { return (uint32_t)(4 * N * (unit & 1) + N * g); }
  __device__ __forceinline__ bool on(int unit) const { return c0 + col(unit) < p.N; }
  __device__ __forceinline__ void load(int unit, int t) {
    const int row = 64 * (unit >> 1) + 4 * l16 + t;
    const uint32_t c = (uint32_t)c0 + col(unit), F = (uint32_t)p.N;
    const bool there = unit < UNITS && on(unit);   // (past the last unit: nothing is read)
    In& x = in4[t];
    const uint32_t off = there ? (uint32_t)(row * in.ld) + (KEPT ? c : 2 * c) : kOOB;
    if constexpr (KEPT) {
      const uint32_t b = there ? (uint32_t)(row * exp.ld) + (c >> 5) : kOOB;
      x.g[0] = in.get16(off, 0);
      x.u[0] = in.get16(off, F);
      x.xg = exp.get1(b, 0);
      x.xu = exp.get1(b, (uint32_t)ck_blocks(p.N));
    } else {
#pragma unroll
      for (int i = 0; i < GV; ++i) {
        x.g[i] = in.get16(off, 16 * i);
        x.u[i] = in.get16(off, 2 * F + 16 * i);
      }
    }
  }
  // Before the last step: as many rows as its registers leave room for; the others when
  // it is done.
  static constexpr int AHEAD = KEPT ? 4 : 2;
  __device__ __forceinline__ void ahead() {
    if (rows <= 0) return;
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) load(0, t);
  }
  // E columns at a time: as few as the registers want.
  static constexpr int E = N / 2;
  // g and u of columns E i .. of the run.
  static __device__ __forceinline__ void kept(const In& x, int i, float (&g)[E], float (&u)[E]) {
#pragma unroll
    for (int k = 0; k < E; k += 4) {
      float a[4], b[4];
      const int w = KEPT ? (E * i + k) / 4 : (E * i + k) / 2;   // the word that these start in
      if constexpr (KEPT) {
        ck_values(x.g[0][w], x.xg, a);
        ck_values(x.u[0][w], x.xu, b);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t p = x.g[(w + j) / 4][(w + j) % 4], q = x.u[(w + j) / 4][(w + j) % 4];
          a[2 * j] = bf16_lo(p);
          a[2 * j + 1] = bf16_hi(p);
          b[2 * j] = bf16_lo(q);
          b[2 * j + 1] = bf16_hi(q);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[k + j] = a[j];
        u[k + j] = b[j];
      }
    }
  }

  template <typename Deq>
  __device__ __forceinline__ void finish(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t part, int lane, int wave) {
    const float top = body(acc, deq, part);
    if (p.d_amax) ep_amax<NW>(p.d_amax, amax_bits<OUT8>(p, top), lane, wave);
  }
  // Column sums of no rows are zeros to part[part][2 F].
  __device__ __forceinline__ void no_rows(int64_t part) const {
    if (e.dbias == nullptr) return;
    for (int unit = 0; unit < 2; ++unit)
      if (on(unit))
        for (int half = 0; half < 2; ++half) e.part[(2 * part + half) * p.N + c0 + col(unit) + l16] = 0.0f;
  }
  template <typename Deq>
  __device__ __forceinline__ float body(const v4f (&acc)[TI][TJ], Deq&& deq, int64_t part) {
    if (rows <= 0) {
      no_rows(part);
      return 0.0f;
    }
    const int64_t F = p.N;
    const int esz = OUT8 ? 1 : (p.d_f32 ? 4 : 2);
    const RowsOf D(p.D, r0, p.ldd * esz, rows);
    const float so = OUT8 ? p.d_scale[0] : 1.0f, most = p.d_fp8 == 1 ? Fmt<0>::max : Fmt<1>::max;
    float top = 0.0f, sum[2][2] = {};   // (lane l16's columns' of the first half's rows, by run)
#pragma unroll
    for (int t = AHEAD; t < 4; ++t) load(0, t);
#pragma unroll 1
    for (int unit = 0; unit < UNITS; ++unit) {
      const int h = unit >> 1;
      const uint32_t c = (uint32_t)c0 + col(unit);
      const bool there = on(unit);
      uint32_t tg[4][N / 4], tu[4][N / 4];
      float db[2][N];   // (of four rows: kept from one turn to the next, they spilled)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 64 * h + 4 * l16 + t;
        const uint32_t off = there ? (uint32_t)(row * D.ld) + c * (uint32_t)esz : kOOB;
        uint32_t wide[2][OUT8 ? 1 : N / 2];   // (bf16 pairs)
        // (rows and parts of a row are kept apart: interleaved they spill)
#pragma unroll
        for (int i = 0; i < N / E; ++i) {
          float v[E], G[E], U[E], a[E], s[E];
          __builtin_amdgcn_sched_barrier(0);
          one_of<0, UNITS>(unit, [&](auto uu) {
            constexpr int i0 = 4 * (decltype(uu)::value >> 1), j0 = N / 4 * (decltype(uu)::value & 1);
#pragma unroll
            for (int j = 0; j < E / 4; ++j) {
              const v4f x = here(acc[i0 + t][j0 + E / 4 * i + j]);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[4 * j + q] = deq(i0 + t, j0 + E / 4 * i + j, q, x[q]);
            }
          });
          // (past the last row and column stand zeros, and an infinity times a zero is a NaN)
#pragma unroll
          for (int k = 0; k < E; ++k) v[k] = there && row < rows ? v[k] : 0.0f;
          kept(in4[t], i, G, U);
          __builtin_amdgcn_sched_barrier(0);
          if (i == N / E - 1) load(unit + 1, t);
          __builtin_amdgcn_sched_barrier(0);
          // (rows and columns past the last have v = g = u = 0: no sum or maximum needs a mask)
          act_and_slope(e.act, G, a, s);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            G[k] = v[k] * U[k] * s[k];
            U[k] = v[k] * a[k];
          }
#pragma unroll
          for (int k = 0; k < E; ++k) {
            db[0][E * i + k] = t == 0 ? G[k] : db[0][E * i + k] + G[k];
            db[1][E * i + k] = t == 0 ? U[k] : db[1][E * i + k] + U[k];
          }
          const float m = __builtin_elementwise_maximum(max_of(G), max_of(U));
          top = __builtin_elementwise_maximum(top, m);
          if constexpr (OUT8) {
            const bool tame = __builtin_amdgcn_ballot_w64(!(m * __builtin_fabsf(so) <= most)) == 0;
            uint32_t w[2][E / 4];
            codes_to(p.d_fp8, tame, G, so, w[0]);
            codes_to(p.d_fp8, tame, U, so, w[1]);
#pragma unroll
            for (int k = 0; k < E / 4; ++k) {
              tg[t][E / 4 * i + k] = w[0][k];
              tu[t][E / 4 * i + k] = w[1][k];
            }
          } else if (p.d_f32) {
            put_f32(D, off, (uint32_t)(4 * E * i), G);
            put_f32(D, off, (uint32_t)(4 * (F + E * i)), U);
          } else {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
              wide[0][E / 2 * i + k] = pack_bf16(G[2 * k], G[2 * k + 1]);
              wide[1][E / 2 * i + k] = pack_bf16(U[2 * k], U[2 * k + 1]);
            }
          }
        }
        if constexpr (!OUT8) {
          if (!p.d_f32) {
#pragma unroll
            for (int k = 0; k < N / 8; ++k) {
              D.put16(off, (uint32_t)(16 * k), &wide[0][4 * k]);
              D.put16(off, (uint32_t)(2 * F + 16 * k), &wide[1][4 * k]);
            }
          }
        }
        if constexpr (OUT8) {
          D.put16(off, 0, tg[t]);
          D.put16(off, (uint32_t)F, tu[t]);
        }
      }
      if constexpr (OUT8) {
        if (p.D_t) {
          const int64_t cols = min(F - c0, (int64_t)(16 * TJ));
          TurnedOf(p, r0, c0, cols, (int)col(unit), l16, there).put<N>(h, 0, tg);
          TurnedOf(p, r0, F + c0, cols, (int)col(unit), l16, there).put<N>(h, 0, tu);
        }
      }
      // column sums of the 128 rows to part[part][2 F]: lane l16 takes column l16
      if (e.dbias) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float w = 0.0f;
          const int mine = here(l16);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float x = row16_sum(db[half][k]);
            w = mine == k ? x : w;
          }
          const bool second = (unit & 1) != 0;
          if (h == 1 && there) e.part[(2 * part + half) * F + c + l16] = pick(second, sum[1][half], sum[0][half]) + w;
          sum[0][half] = pick(second, sum[0][half], w);
          sum[1][half] = pick(second, w, sum[1][half]);
        }
      }
    }
    return top;
  }
};

// The epilogue as the large kernels name it.
struct GatedEp {
  static constexpr bool PAIRED = true, DIRECT = true;
  GatedParams e;
  template <bool OUT8, int TI, int TJ, int NW>
  using Run = GatedRun<OUT8, TI, TJ, NW>;
};
template <int KEPT>
struct GatedGradEp {
  static constexpr bool PAIRED = false, DIRECT = true;
  GatedParams e;
  template <bool OUT8, int TI, int TJ, int NW>
  using Run = GatedGradRun<OUT8, KEPT, TI, TJ, NW>;
};

}  // namespace

}  // namespace fp8lin
