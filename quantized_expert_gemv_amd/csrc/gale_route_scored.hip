// Expert choice from softmax or sigmoid scores, with a selection bias, expert groups and renormalised weights.
//
// One wavefront per token.  Each of the n_groups groups gets L = 64 / (n_groups rounded up to a power of two) lanes, and
// lane i of a group holds its experts i, i + L, ...: a group's value is a reduction over L neighbouring lanes, and with one
// group the wavefront reads the logits in whole lines.  Scores, their sums with the bias and the group values are
// computed and compared in 64 bits: rounding them to 32 would let the order of close experts hang on the exponential's last
// bit.  Without a bias the order is that of the logits, compared exactly in 32 bits.
#include "gale_internal.h"
#include "gale_lanes.h"
#include "gale_mx.h"
#include "gale_route.h"

namespace gale {

struct ScoredParams {
  const void* logits;
  int64_t stride;
  int n_tok, E, k;
  const float* bias;     // NULL: none
  int score, G, keep, rule;
  int gsize;             // experts per group
  int log2L;             // lanes per group
  int renorm;
  float scale;
  int32_t* idx;
  float* w;
};

__device__ __forceinline__ double shfl_xor_f64(double v, int m) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)b, m, 64), hi = (uint32_t)__shfl_xor((int)(uint32_t)(b >> 32), m, 64);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double readlane_f64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Order-preserving 64-bit key of a finite or +infinite value; 0 stands for "none".
__device__ __forceinline__ uint64_t f64_key(double v) {
  uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);   // -0 becomes +0
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, m, 64), hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), m, 64);
    const uint64_t o = (uint64_t)hi << 32 | lo;
    v = o > v ? o : v;
  }
  return v;
}

// NJ: experts per lane, NJ * L >= gsize.
template <typename T, int NJ>
__global__ void __launch_bounds__(256) route_scored_kernel(const ScoredParams p) {
  const int lane = threadIdx.x & 63;
  const int t = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6);
  if (t >= p.n_tok) return;
  const typename T::bits* lg = (const typename T::bits*)p.logits + (int64_t)t * p.stride;
  const int L = 1 << p.log2L, g = lane >> p.log2L, li = lane & (L - 1);
  float l[NJ];       // logit; -infinity: no expert, or one that cannot be chosen
  float b[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int i = li + (j << p.log2L);
    const bool in = g < p.G && i < p.gsize;
    const int e = in ? g * p.gsize + i : 0;
    const float v = T::to_f32(lg[e]);
    b[j] = p.bias ? p.bias[e] : 0.f;
    l[j] = in && v == v && b[j] == b[j] && b[j] != -INFINITY ? fminf(v, 3.402823466e38f) : -INFINITY;
  }
  // scores in 64 bits
  double s[NJ], m = 0.0, Z = 0.0;
  if (p.score == GALE_SCORE_SOFTMAX) {
    float mf = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) mf = fmaxf(mf, l[j]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) mf = fmaxf(mf, __shfl_xor(mf, x, 64));
    m = mf;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = l[j] == -INFINITY ? 0.0 : exp((double)l[j] - m);
      Z += s[j];
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) Z += shfl_xor_f64(Z, x);
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = l[j] == -INFINITY ? 0.0 : s[j] / Z;
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = l[j] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[j]));
  }
  double c[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) c[j] = l[j] == -INFINITY ? -INFINITY : s[j] + (double)b[j];
  // group values: the largest c, or the sum of the two largest
  bool kept = g < p.G;
  if (p.keep < p.G) {
    double v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v2 = fmax(v2, fmin(v1, c[j]));
      v1 = fmax(v1, c[j]);
    }
    for (int x = 1; x < L; x <<= 1) {
      const double o1 = shfl_xor_f64(v1, x), o2 = shfl_xor_f64(v2, x);
      v2 = fmax(fmin(v1, o1), fmax(v2, o2));
      v1 = fmax(v1, o1);
    }
    const double v = p.rule == GALE_GROUP_TOP2 && v2 != -INFINITY ? v1 + v2 : v1;
    int rank = 0;
    for (int o = 0; o < p.G; ++o) {
      const double ov = readlane_f64(v, o << p.log2L);
      rank += ov > v || (ov == v && o < g) ? 1 : 0;
    }
    kept = kept && rank < p.keep;
  }
  // keys: 0 is no candidate
  uint64_t key[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    key[j] = kept && l[j] != -INFINITY ? (p.bias ? f64_key(c[j]) : f64_key((double)l[j])) : 0ull;
  double mine = 0.0, sum = 0.0;
  int my_e = -1;
  for (int r = 0; r < p.k; ++r) {
    uint64_t best = key[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) best = key[j] > best ? key[j] : best;
    best = wave_max_u64(best);
    if (best == 0ull) break;          // no candidate is left
    // the lowest expert among the equal ones
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int j = NJ - 1; j >= 0; --j)
      if (key[j] == best) e = (uint32_t)(g * p.gsize + li + (j << p.log2L));
    const uint32_t w = wave_min_u32(e);
    double sv = 0.0;
    bool have = false;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (e == w && key[j] == best && !have) {   // the lowest j of this lane is the one that e names
        sv = s[j];
        key[j] = 0ull;
        have = true;
      }
    const uint64_t who = __ballot(have);
    const double ws = readlane_f64(sv, __builtin_ctzll(who));
    sum += ws;
    if (lane == r) {
      mine = ws;
      my_e = (int)w;
    }
  }
  if (lane < p.k) {
    const double f = p.renorm ? (sum > 0.0 ? mine / sum : 0.0) : mine;
    p.idx[(int64_t)t * p.k + lane] = my_e;
    p.w[(int64_t)t * p.k + lane] = my_e < 0 ? 0.f : (float)(f * (double)p.scale);
  }
}

template <typename T>
static hipError_t launch_scored_t(const ScoredParams& p, hipStream_t s) {
  const int L = 1 << p.log2L, nj = (p.gsize + L - 1) / L;
  const dim3 grid((unsigned)((p.n_tok + 3) / 4));
  if (nj <= 2) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 2>), grid, dim3(256), 0, s, p);
  else if (nj <= 4) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 4>), grid, dim3(256), 0, s, p);
  else if (nj <= 8) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 8>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 16>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

// n_groups rounded up to a power of two has at most 64 groups of at least one lane, so a lane holds at most
// 2 * GALE_MAX_EXPERTS / 64 = 16 experts.
hipError_t launch_route_scored(const void* logits, int dtype, int64_t stride, int n_tok, int E, const float* bias,
                               int score, int G, int keep, int rule, int k, int renorm, float scale, int32_t* idx,
                               float* w, hipStream_t s) {
  int lg = 0;
  while ((1 << lg) < G) ++lg;
  ScoredParams p;
  p.logits = logits;
  p.stride = stride;
  p.n_tok = n_tok;
  p.E = E;
  p.k = k;
  p.bias = bias;
  p.score = score;
  p.G = G;
  p.keep = keep;
  p.rule = rule;
  p.gsize = E / G;
  p.log2L = 6 - lg;
  p.renorm = renorm;
  p.scale = scale;
  p.idx = idx;
  p.w = w;
  if (dtype == GALE_F16) return launch_scored_t<F16>(p, s);
  if (dtype == GALE_BF16) return launch_scored_t<BF16>(p, s);
  return launch_scored_t<F32>(p, s);
}

}  // namespace gale
