// Expert choice from softmax or sigmoid scores, with a selection bias, expert groups and renormalised weights.
//
// One wavefront chooses for one token.  Each of the n_groups groups gets L = 64 / (n_groups rounded up to a power of two) lanes, and
// lane i of a group holds its experts i, i + L, ...: a group's value is a reduction over L neighbouring lanes, and with one
// group the wavefront reads the logits in whole lines.  The choice is that of scores, sums and group values in 64 bits: in
// 32 the order of close experts would hang on the exponential's last bit.  64-bit exponentials of every expert and
// 64-bit keys cost most of the time, though, and nearly every token's choice is clear in 32 bits: so the choice is
// made in 32 bits with margins, and made again in 64 where a margin is not kept.
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

// LDS accesses of one wavefront complete in order: this keeps the compiler from reordering them.
__device__ __forceinline__ void wave_lds_done() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A key that the lanes' largest keys reach at least `need` times, by a bitwise search over their counts that ends early
// where only a few more do; at least 1, which leaves out the lanes without a candidate.
__device__ __forceinline__ uint32_t head_threshold(uint32_t head, int need) {
  uint32_t thr = 0;
  for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1) {
    const int n = __builtin_popcountll(__ballot(head >= (thr | bit)));
    if (n >= need) {
      thr |= bit;
      if (n <= need + 6) break;
    }
  }
  return max(thr, 1u);
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// What both ways of choosing leave: lane r < k holds slot r's expert (-1: none).  NJ: experts per lane, NJ * L >= gsize.
// l: the lane's logits (-infinity: no expert, or one that cannot be chosen), b its biases.

// Scores, sums with the bias and group values in 64 bits, compared exactly; equal values are ties.
template <int NJ>
__device__ __forceinline__ int choose_exact(const ScoredParams& p, const float l[NJ], const float b[NJ], int lane, int g,
                                            int li, uint64_t* s_cand, uint32_t* s_id) {
  double s[NJ];
  if (p.score == GALE_SCORE_SOFTMAX) {
    float mf = l[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) mf = fmaxf(mf, l[j]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) mf = fmaxf(mf, __shfl_xor(mf, x, 64));
    double Z = 0.0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = l[j] == -INFINITY ? 0.0 : exp((double)l[j] - (double)mf);
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
  bool kept = true;
  if (p.keep < p.G) {
    double v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v2 = fmax(v2, fmin(v1, c[j]));
      v1 = fmax(v1, c[j]);
    }
    for (int x = 1; x < (1 << p.log2L); x <<= 1) {
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
    kept = rank < p.keep;
  }
  uint64_t key[NJ];      // 0: no candidate
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    key[j] = kept && l[j] != -INFINITY ? (p.bias ? f64_key(c[j]) : f64_key((double)l[j])) : 0ull;
  // Candidates by the keys' upper halves, as below in 32 bits: equal halves come along, and their ranks compare whole keys.
  uint32_t head = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) head = max(head, (uint32_t)(key[j] >> 32));
  const uint32_t thr = head_threshold(head, p.k);
  int at = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool in = (uint32_t)(key[j] >> 32) >= thr;
    const uint64_t mask = __ballot(in);
    const int pos = at + lanes_below(mask);
    if (in && pos < 64) {
      s_cand[pos] = key[j];
      s_id[pos] = (uint32_t)(g * p.gsize + li + (j << p.log2L));
    }
    at += __builtin_popcountll(mask);
  }
  wave_lds_done();
  if (at <= 64) {
    const uint64_t mine = lane < at ? s_cand[lane] : 0ull;
    const uint32_t id = lane < at ? s_id[lane] : 0xFFFFFFFFu;
    int rank = 0;
    for (int i = 0; i < at; ++i) {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mine, i);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(mine >> 32), i);
      const uint64_t o = (uint64_t)hi << 32 | lo;
      rank += o > mine || (o == mine && (uint32_t)__builtin_amdgcn_readlane((int)id, i) < id) ? 1 : 0;
    }
    wave_lds_done();
    if (lane < at) s_id[rank] = id;          // ranks are all different
    wave_lds_done();
    return lane < p.k && lane < at ? (int)s_id[lane] : -1;
  }
  // more than 64 candidates (as many equal keys): slot by slot
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
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if ((uint32_t)(g * p.gsize + li + (j << p.log2L)) == w) key[j] = 0ull;
    my_e = lane == r ? (int)w : my_e;
  }
  return my_e;
}

// The same in 32 bits, with margins: returns false (and no choice) when two values that the choice compares lie closer
// than their errors could explain; the exact way then decides.
//   Without a bias the candidates compare by their logits: exact, ties included.
//   The scores' errors.  Sigmoid: x = l log2 e is off by 2^-24 |x|, which moves e^-|l| by |l| e^-|l| 2^-24 < 2^-25; the hardware
//   exponential and reciprocal are within 1 ulp, two additions within half of one: below 2^-21 together.  Softmax: the
//   same for each e^(l - max), and below 2^-20 after a sum of 512 terms (a tree of nine levels) and the reciprocal.
//   Adding the bias rounds by 2^-24 |c|, adding two sums for a group the same once more.
// So two experts' c are apart in truth when they differ here by more than 2^-18 + 2^-22 |c|, two groups' values by twice that
// with the largest |c| that any group adds.
template <int NJ>
__device__ __forceinline__ bool choose_fast(const ScoredParams& p, const float l[NJ], const float b[NJ], int lane, int g,
                                            int li, uint64_t* s_cand, int& my_e) {
  const bool by_score = p.bias != nullptr || p.keep < p.G;
  float c[NJ];
  if (by_score) {
    if (p.score == GALE_SCORE_SOFTMAX) {
      float m = l[0];
#pragma unroll
      for (int j = 1; j < NJ; ++j) m = fmaxf(m, l[j]);
      m = key_to_logit(wave_max_u32_v(logit_key(m)));
      float Z = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        c[j] = l[j] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((l[j] - m) * 1.44269504088896341f);
        Z += c[j];
      }
      Z += lane_xor<1>(Z);
      Z += lane_xor<2>(Z);
      Z += lane_xor<4>(Z);
      Z += lane_xor<8>(Z);
      Z += lane_xor<16>(Z);
      Z += lane_xor<32>(Z);
      const float inv = __builtin_amdgcn_rcpf(Z);
#pragma unroll
      for (int j = 0; j < NJ; ++j) c[j] *= inv;
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float z = __builtin_amdgcn_exp2f(-fabsf(l[j]) * 1.44269504088896341f);   // e^-|l| in [0, 1]
        c[j] = (l[j] < 0.f ? z : 1.f) * __builtin_amdgcn_rcpf(1.f + z);
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) c[j] = l[j] == -INFINITY ? -INFINITY : c[j] + b[j];
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) c[j] = l[j];
  }
  constexpr float kAbs = 0x1p-18f, kRel = 0x1p-22f;
  bool kept = true;
  if (p.keep < p.G) {
    float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v2 = fmaxf(v2, fminf(v1, c[j]));
      v1 = fmaxf(v1, c[j]);
    }
    auto merge = [&](float o1, float o2) {
      v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
      v1 = fmaxf(v1, o1);
    };
    if (p.log2L > 0) merge(lane_xor<1>(v1), lane_xor<1>(v2));
    if (p.log2L > 1) merge(lane_xor<2>(v1), lane_xor<2>(v2));
    if (p.log2L > 2) merge(lane_xor<4>(v1), lane_xor<4>(v2));
    if (p.log2L > 3) merge(lane_xor<8>(v1), lane_xor<8>(v2));
    if (p.log2L > 4) merge(lane_xor<16>(v1), lane_xor<16>(v2));
    const float v = p.rule == GALE_GROUP_TOP2 && v2 != -INFINITY ? v1 + v2 : v1;
    // the terms' size, not their sum's, sets the error: large biases may cancel
    float size = fmaxf(fabsf(v1), v2 == -INFINITY ? 0.f : fabsf(v2));
    size = g < p.G && v1 != -INFINITY ? size : 0.f;
    const float margin = 2.f * (kAbs + kRel * __uint_as_float(wave_max_u32_v(__float_as_uint(size))));
    int over = 0, near = 0;       // groups surely better, groups at least nearly as good (this one among them)
    for (int o = 0; o < p.G; ++o) {
      const float ov = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), o << p.log2L));
      over += ov > v + margin ? 1 : 0;
      near += ov >= v - margin ? 1 : 0;
    }
    kept = near <= p.keep;
    // infinite values have no margin: they go the exact way, except the empty groups behind enough others
    if (__ballot(g < p.G && !kept && over < p.keep) != 0ull) return false;
  }
  uint32_t key[NJ];      // 0: no candidate
#pragma unroll
  for (int j = 0; j < NJ; ++j) key[j] = kept && l[j] != -INFINITY ? logit_key(p.bias ? c[j] : l[j]) : 0u;
  // The slots' keys (one more with a bias, for the last margin) are found among few candidates: those that reach a
  // threshold which as many lanes' largest keys reach, at most 64 or the exact way decides.  Compacted one per lane, their
  // ranks are counted directly.
  my_e = -1;
  uint32_t head = key[0];
#pragma unroll
  for (int j = 1; j < NJ; ++j) head = max(head, key[j]);
  const uint32_t thr = head_threshold(head, p.bias ? p.k + 1 : p.k);
  int count = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) count += __builtin_popcountll(__ballot(key[j] >= thr));
  if (count > 64) return false;
  int at = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const uint64_t mask = __ballot(key[j] >= thr);
    if (key[j] >= thr)
      s_cand[at + lanes_below(mask)] =
          (uint64_t)key[j] << 32 | (uint32_t)~(g * p.gsize + li + (j << p.log2L));   // lower experts are larger
    at += __builtin_popcountll(mask);
  }
  wave_lds_done();
  const uint64_t mine = lane < count ? s_cand[lane] : 0ull;
  int rank = 0;
  for (int i = 0; i < count; ++i) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mine, i);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(mine >> 32), i);
    rank += ((uint64_t)hi << 32 | lo) > mine ? 1 : 0;
  }
  wave_lds_done();
  if (lane < count) s_cand[rank] = mine;        // ranks are all different: a permutation
  wave_lds_done();
  const uint64_t own = lane < count ? s_cand[lane] : 0ull;
  if (p.bias) {
    const uint64_t after = lane + 1 < count ? s_cand[lane + 1] : 0ull;
    const float c0 = key_to_logit((uint32_t)(own >> 32)), c1 = key_to_logit((uint32_t)(after >> 32));
    if (__ballot(lane < p.k && after != 0ull && !(c0 - c1 > kAbs + kRel * fabsf(c0))) != 0ull) return false;
  }
  if (lane < p.k && own != 0ull) my_e = (int)~(uint32_t)own;
  return true;
}

// Eight tokens per workgroup, one wavefront each; then one wavefront computes the weights of all eight, a lane per slot
// (64-bit exponentials and divisions of 8 tokens at the price of one).
constexpr int kScoredTokens = 8;

template <typename T, int NJ>
__global__ void __launch_bounds__(64 * kScoredTokens) route_scored_kernel(const ScoredParams p) {
  __shared__ float s_l[kScoredTokens][GALE_MAX_EXPERTS];
  __shared__ uint64_t s_cand[kScoredTokens][64];
  __shared__ uint32_t s_id[kScoredTokens][64];
  __shared__ int s_e[kScoredTokens][GALE_MAX_TOPK];
  __shared__ float s_m[kScoredTokens];       // a softmax: the token's largest logit
  __shared__ double s_Z[kScoredTokens];      // and the sum relative to it, where it is needed
  const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int t0 = (int)blockIdx.x * kScoredTokens, t = t0 + wave;
  if (t < p.n_tok) {
    const typename T::bits* lg = (const typename T::bits*)p.logits + (int64_t)t * p.stride;
    const int g = lane >> p.log2L, li = lane & ((1 << p.log2L) - 1);
    float l[NJ], b[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int i = li + (j << p.log2L);
      const bool in = g < p.G && i < p.gsize;
      const int e = in ? g * p.gsize + i : 0;
      const float v = T::to_f32(lg[e]);
      b[j] = p.bias ? p.bias[e] : 0.f;
      l[j] = in && v == v && b[j] == b[j] && b[j] != -INFINITY ? fminf(v, 3.402823466e38f) : -INFINITY;
      if (in) s_l[wave][e] = l[j];
    }
    int my_e = -1;
    if (!choose_fast<NJ>(p, l, b, lane, g, li, s_cand[wave], my_e)) my_e = choose_exact<NJ>(p, l, b, lane, g, li, s_cand[wave], s_id[wave]);
    if (lane < GALE_MAX_TOPK) s_e[wave][lane] = lane < p.k ? my_e : -1;
    if (p.score == GALE_SCORE_SOFTMAX) {
      float m = l[0];
#pragma unroll
      for (int j = 1; j < NJ; ++j) m = fmaxf(m, l[j]);
      m = key_to_logit(wave_max_u32_v(logit_key(m)));
      if (lane == 0) s_m[wave] = m;
      if (!p.renorm) {
        double Z = 0.0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) Z += l[j] == -INFINITY ? 0.0 : exp((double)l[j] - (double)m);
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) Z += shfl_xor_f64(Z, x);
        if (lane == 0) s_Z[wave] = Z;
      }
    }
  }
  __syncthreads();
  if (wave != 0) return;
  const int w = lane >> 3, slot = lane & 7;         // token of the eight, and its slot
  const bool there = t0 + w < p.n_tok;
  const int e = there ? s_e[w][slot] : -1;
  const float lv = e >= 0 ? s_l[w][e] : -INFINITY;
  double s, f = 1.0;
  if (p.score == GALE_SCORE_SOFTMAX) {
    if (!p.renorm) f = s_Z[w];       // renormalised, the sum of all cancels
    s = e >= 0 ? exp((double)lv - (double)s_m[w]) : 0.0;
  } else {
    s = e >= 0 ? 1.0 / (1.0 + exp(-(double)lv)) : 0.0;
  }
  if (p.renorm) {
    f = s;
    f += shfl_xor_f64(f, 1);
    f += shfl_xor_f64(f, 2);
    f += shfl_xor_f64(f, 4);
  }
  if (there && slot < p.k) {
    p.idx[(int64_t)(t0 + w) * p.k + slot] = e;
    p.w[(int64_t)(t0 + w) * p.k + slot] = e >= 0 && f > 0.0 ? (float)(s / f * (double)p.scale) : 0.f;
  }
}

template <typename T>
static hipError_t launch_scored_t(const ScoredParams& p, hipStream_t s) {
  const int L = 1 << p.log2L, nj = (p.gsize + L - 1) / L;
  const dim3 grid((unsigned)((p.n_tok + kScoredTokens - 1) / kScoredTokens)), block(64 * kScoredTokens);
  if (nj <= 1) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 1>), grid, block, 0, s, p);
  else if (nj <= 2) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 2>), grid, block, 0, s, p);
  else if (nj <= 4) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 4>), grid, block, 0, s, p);
  else if (nj <= 6) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 6>), grid, block, 0, s, p);
  else if (nj <= 8) hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 8>), grid, block, 0, s, p);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(route_scored_kernel<T, 16>), grid, block, 0, s, p);
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
  p.stride = stride;
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
  // a grid has fewer than 2^32 threads, 64 for a token: four million tokens per launch
  for (int64_t t = 0; t < n_tok; t += 1 << 22) {
    p.n_tok = (int)std::min<int64_t>(n_tok - t, 1 << 22);
    p.logits = (const char*)logits + t * stride * (dtype == GALE_F32 ? 4 : 2);
    p.idx = idx + t * k;
    p.w = w + t * k;
    const hipError_t e = dtype == GALE_F16    ? launch_scored_t<F16>(p, s)
                         : dtype == GALE_BF16 ? launch_scored_t<BF16>(p, s)
                                              : launch_scored_t<F32>(p, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gale
