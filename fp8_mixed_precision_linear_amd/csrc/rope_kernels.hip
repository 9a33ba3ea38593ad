// rope_kernels.hip -- rotary positions of the heads of a QKV product.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) is turned by
// theta = position * f_i and scaled:
//   (x0, x1) -> scale (x0 cos theta - x1 sin theta, x1 cos theta + x0 sin theta)
// and the inverse (the gradient: the transpose of the turn) takes -theta.
// Elements past rot are copied.
//
// theta / (2 pi) is formed and reduced to a fraction of a turn in binary64 (a
// position of 2^20 times a frequency near 1 leaves 2^-33 of a turn; in
// binary32 it would leave 2^-4 radians); the cosine and sine of the fraction
// are binary32.  They are computed once per token and pair by the workgroup,
// into LDS, and read from there by all its heads.
//
// Bound: HBM, one read and one write of each head element; angles cost
// rot / 2 per token however many heads turn by them.  Measured on an MI355X: 8192
// tokens, 64 + 8 heads of 128, half of each turned, 69 us, 4.4 TB/s (a copy: 4.94);
// 16 tokens 4.6 us of kernel.
#include "op_device.h"
#include "launch.h"

namespace fp8lin {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 1024;   // (token, pair) angles of one workgroup
constexpr double kInvTwoPi = 0.15915494309189533577;

template <bool F32>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeParams p) {
  __shared__ float2 cs[kRopeAngles];
  const int np = (int)p.pairs;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_wg;
  const int nt = (int)(p.tokens - t0 < p.tokens_wg ? p.tokens - t0 : p.tokens_wg);
  // Units of a head: two vectors of 8 elements each.  Half layout: elements i0 ..
  // and np + i0 ..; interleaved, and the elements past rot (other buffer than the
  // input): vectors w and w + half the number of them, so that neighbouring lanes
  // read neighbouring vectors.
  const bool halves = !p.interleaved;
  const int rest = p.copy_rest ? (int)p.dim - 2 * np : 0;
  const int pu = halves ? (np + 7) / 8 : (2 * np + 15) / 16, ru = (rest + 15) / 16, units = pu + ru;
  const int64_t heads = p.q_heads + p.k_heads, h0 = (int64_t)blockIdx.y * p.heads_wg;
  const int nh = (int)(heads - h0 < p.heads_wg ? heads - h0 : p.heads_wg);
  const int all = nt * nh * units;
  // u / d for u, d < 2^16 (see launch_rope): exact, as u (d - 2^32 mod d) < 2^32
  const uint32_t per_unit = 0xFFFFFFFFu / (uint32_t)units + 1u, per_head = 0xFFFFFFFFu / (uint32_t)nh + 1u;
  constexpr int ES = F32 ? 4 : 2;
  float x[2][8], y[2][8];
  char* dst[2];
  int w[2], tk[2], n[2], n2[2], second[2];   // unit of the head, token, elements of each vector, from first to second
  auto fetch = [&](int u0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int u = u0 + q * kRopeThreads, uc = u < all ? u : 0;
      const int th = units == 1 ? uc : (int)__umulhi((uint32_t)uc, per_unit);
      w[q] = uc - th * units;
      tk[q] = nh == 1 ? th : (int)__umulhi((uint32_t)th, per_head);
      int64_t h = h0 + (th - tk[q] * nh);
      const int64_t tok = t0 + tk[q];
      const bool is_k = h >= p.q_heads;
      if (is_k) h -= p.q_heads;
      const char* src = reinterpret_cast<const char*>(is_k ? p.k : p.q) +
                        (tok * (is_k ? p.k_st : p.q_st) + h * (is_k ? p.k_sh : p.q_sh)) * ES;
      dst[q] = reinterpret_cast<char*>(is_k ? p.k_out : p.q_out) +
               (tok * (is_k ? p.ko_st : p.qo_st) + h * (is_k ? p.ko_sh : p.qo_sh)) * ES;
      const bool turned = w[q] < pu;
      const int first = turned ? 8 * w[q] : 2 * np + 8 * (w[q] - pu);
      const int end = !turned ? (int)p.dim : (halves ? np : 2 * np);
      second[q] = !turned ? 8 * ru : (halves ? np : 8 * pu);
      n[q] = u < all ? end - first : 0;
      n2[q] = turned && halves ? n[q] : n[q] - second[q];
      dst[q] += first * ES;
      load8(src, F32, first, n[q], x[q]);
      load8(src, F32, first + second[q], n2[q], y[q]);
    }
  };
  // the first units' elements are on their way while the angles are computed
  fetch(threadIdx.x);
  for (int a = threadIdx.x; a < nt * np; a += kRopeThreads) {
    const int t = a / np, i = a - t * np;
    const int64_t tok = t0 + t;
    const int64_t pos = p.pos == nullptr ? p.offset + tok
                        : p.pos_i64      ? reinterpret_cast<const int64_t*>(p.pos)[tok] + p.offset
                                         : (int64_t) reinterpret_cast<const int32_t*>(p.pos)[tok] + p.offset;
    const double turns = (double)pos * (p.freqs[i] * kInvTwoPi);
    // (the fraction's part beyond binary32 turns the result a little further: without it
    // a cosine next to 0 would be off by up to 2^-23 and keep no digit)
    const double part = turns - rint(turns);
    const float f = (float)part, beyond = (float)((part - (double)f) * (1.0 / kInvTwoPi));
    float s0, c0;
    sincospif(2.0f * f, &s0, &c0);
    float s = __builtin_fmaf(c0, beyond, s0);
    const float c = __builtin_fmaf(-s0, beyond, c0);
    if (p.inverse) s = -s;
    cs[a] = make_float2(c * p.scale, s * p.scale);
  }
  __syncthreads();
  for (int u0 = threadIdx.x; u0 < all; u0 += 2 * kRopeThreads) {
    if (u0 != (int)threadIdx.x) fetch(u0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (w[q] < pu) {
        const float2* a = cs + tk[q] * np;
        if (halves) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 r = a[min(8 * w[q] + j, np - 1)];
            const float v0 = x[q][j], v1 = y[q][j];
            x[q][j] = v0 * r.x - v1 * r.y;
            y[q][j] = v1 * r.x + v0 * r.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 r = a[min(4 * w[q] + j, np - 1)], r2 = a[min(4 * (w[q] + pu) + j, np - 1)];
            const float v0 = x[q][2 * j], v1 = x[q][2 * j + 1], v2 = y[q][2 * j], v3 = y[q][2 * j + 1];
            x[q][2 * j] = v0 * r.x - v1 * r.y;
            x[q][2 * j + 1] = v1 * r.x + v0 * r.y;
            y[q][2 * j] = v2 * r2.x - v3 * r2.y;
            y[q][2 * j + 1] = v3 * r2.x + v2 * r2.y;
          }
        }
      }
      store8(dst[q], F32, 0, n[q], x[q]);
      store8(dst[q], F32, second[q], n2[q], y[q]);
    }
  }
}

// f_i = base^(-i / pairs), in binary64, scaled for contexts longer than the
// trained ones: 1, all positions divided by `factor`; 2, a larger base, which
// leaves the fastest pair and divides the slowest by `factor`; 3, by parts: a
// pair that turns more than `high` times over the trained length is left, one
// that turns less than `low` times is divided by `factor`, a linear ramp
// between the two.
__global__ void k_rope_freqs(double* f, int64_t pairs, double base, int scaling, double factor, double trained,
                             double low, double high) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= pairs) return;
  if (scaling == 2 && pairs > 1) base *= pow(factor, (double)pairs / (double)(pairs - 1));
  double v = pow(base, -(double)i / (double)pairs);
  if (scaling == 1) v /= factor;
  if (scaling == 3) {
    double keep = (trained * v * kInvTwoPi - low) / (high - low);
    keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
    v = v * keep + v / factor * (1.0 - keep);
  }
  f[i] = v;
}

}  // namespace

int64_t rope_max_pairs() { return kRopeAngles; }

hipError_t launch_rope(RopeParams p, hipStream_t s) {
  const int64_t heads = p.q_heads + p.k_heads;
  if (p.tokens == 0 || heads == 0 || p.dim == 0) return hipSuccess;
  // Tokens of a workgroup: enough angles for its threads (fewer tokens would
  // leave threads idle while the angles are computed), and, when that leaves
  // compute units without work, fewer heads each.
  int64_t tw = p.pairs > 0 ? kRopeThreads / p.pairs : 1;
  tw = tw < 1 ? 1 : (tw > 8 ? 8 : tw);
  const int64_t cu = device_cu_count();
  while (tw > 1 && (p.tokens + tw - 1) / tw < 2 * cu) tw >>= 1;
  const int64_t units = (p.interleaved ? (2 * p.pairs + 15) / 16 : (p.pairs + 7) / 8) +
                        (p.copy_rest ? (p.dim - 2 * p.pairs + 15) / 16 : 0);
  if (units == 0) return hipSuccess;   // no pair and nothing to copy
  int64_t hw = heads < 256 ? heads : 256;
  while (hw > 1 && tw * hw * units > 65535) hw = (hw + 1) / 2;   // units are divided in 16 bits
  while (tw > 1 && tw * hw * units > 65535) tw >>= 1;
  const int64_t tb = (p.tokens + tw - 1) / tw;
  while (hw > 8 && tb * ((heads + hw - 1) / hw) < 2 * cu) hw = (hw + 1) / 2;
  p.tokens_wg = (int)tw;
  p.heads_wg = (int)hw;
  const dim3 grid((unsigned)tb, (unsigned)((heads + hw - 1) / hw));
  if (p.f32) hipLaunchKernelGGL((k_rope<true>), grid, dim3(kRopeThreads), 0, s, p);
  else hipLaunchKernelGGL((k_rope<false>), grid, dim3(kRopeThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_rope_freqs(double* f, int64_t pairs, double base, int scaling, double factor, double trained,
                             double low, double high, hipStream_t s) {
  if (pairs == 0) return hipSuccess;
  hipLaunchKernelGGL(k_rope_freqs, dim3((unsigned)((pairs + 63) / 64)), dim3(64), 0, s, f, pairs, base, scaling,
                     factor, trained, low, high);
  return hipGetLastError();
}

}  // namespace fp8lin
