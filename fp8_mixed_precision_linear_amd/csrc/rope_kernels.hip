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
// rot / 2 per token however many heads turn by them.
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
  for (int a = threadIdx.x; a < nt * np; a += kRopeThreads) {
    const int t = a / np, i = a - t * np;
    const int64_t tok = t0 + t;
    const int64_t pos = p.pos == nullptr ? p.offset + tok
                        : p.pos_i64      ? reinterpret_cast<const int64_t*>(p.pos)[tok] + p.offset
                                         : (int64_t) reinterpret_cast<const int32_t*>(p.pos)[tok] + p.offset;
    const double turns = (double)pos * (p.freqs[i] * kInvTwoPi);
    const float f = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    if (p.inverse) s = -s;
    cs[a] = make_float2(c * p.scale, s * p.scale);
  }
  __syncthreads();
  // units of a head: 8 pairs each, then (other buffer than the input) the
  // elements past rot, 16 each
  const int pu = (np + 7) / 8, rest = (int)p.dim - 2 * np;
  const int cu = p.copy_rest ? (rest + 15) / 16 : 0;
  const int units = pu + cu;
  const int64_t heads = p.q_heads + p.k_heads;
  const int64_t h0 = (int64_t)blockIdx.y * p.heads_wg;
  const int nh = (int)(heads - h0 < p.heads_wg ? heads - h0 : p.heads_wg);
  const int all = nt * nh * units;
  for (int u = threadIdx.x; u < all; u += kRopeThreads) {
    const int th = u / units, w = u - th * units;
    const int t = th / nh;
    const int64_t tok = t0 + t;
    int64_t h = h0 + (th - t * nh);
    const bool is_k = h >= p.q_heads;
    if (is_k) h -= p.q_heads;
    const void* src = is_k ? p.k : p.q;
    void* dst = is_k ? p.k_out : p.q_out;
    const int64_t si = tok * (is_k ? p.k_st : p.q_st) + h * (is_k ? p.k_sh : p.q_sh);
    const int64_t di = tok * (is_k ? p.ko_st : p.qo_st) + h * (is_k ? p.ko_sh : p.qo_sh);
    if (w >= pu) {
      const int e = 2 * np + 16 * (w - pu), left = (int)p.dim - e;
      float v[8], v2[8];
      load8(src, F32, si + e, left, v);
      load8(src, F32, si + e + 8, left - 8, v2);
      store8(dst, F32, di + e, left, v);
      store8(dst, F32, di + e + 8, left - 8, v2);
      continue;
    }
    const int i0 = 8 * w, n = np - i0 < 8 ? np - i0 : 8;
    const float2* a = cs + t * np + i0;
    float x[8], y[8];
    if (p.interleaved) {
      load8(src, F32, si + 2 * i0, 2 * n, x);
      load8(src, F32, si + 2 * i0 + 8, 2 * n - 8, y);
      auto turn = [&](float (&v)[8], int j0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 r = j0 + j < n ? a[j0 + j] : make_float2(0.0f, 0.0f);
          const float v0 = v[2 * j], v1 = v[2 * j + 1];
          v[2 * j] = v0 * r.x - v1 * r.y;
          v[2 * j + 1] = v1 * r.x + v0 * r.y;
        }
      };
      turn(x, 0);
      turn(y, 4);
      store8(dst, F32, di + 2 * i0, 2 * n, x);
      store8(dst, F32, di + 2 * i0 + 8, 2 * n - 8, y);
    } else {
      load8(src, F32, si + i0, n, x);
      load8(src, F32, si + np + i0, n, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 r = j < n ? a[j] : make_float2(0.0f, 0.0f);
        const float v0 = x[j], v1 = y[j];
        x[j] = v0 * r.x - v1 * r.y;
        y[j] = v1 * r.x + v0 * r.y;
      }
      store8(dst, F32, di + i0, n, x);
      store8(dst, F32, di + np + i0, n, y);
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
  const int64_t tb = (p.tokens + tw - 1) / tw;
  int64_t hw = heads < 256 ? heads : 256;
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
