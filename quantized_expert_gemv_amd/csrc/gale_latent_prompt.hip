// Latent attention of prompts, expanded form.
#include "gale_latent.h"

namespace gale {

constexpr int kNope = GALE_HEAD_NOPE, kValue = GALE_HEAD_VALUE;

// A workgroup per query (token and head): scores of 256 keys at a time, one thread each, then the 128 sums over those keys.
template <typename T>
__global__ void __launch_bounds__(256) prompt_simple_kernel(const PromptParams p) {
  __shared__ int part[4];
  __shared__ float fpart[4], x[(kNope + kRope)], w[256];
  const int tid = threadIdx.x, t = (int)(blockIdx.x / (unsigned)p.n_heads), h = (int)(blockIdx.x % (unsigned)p.n_heads);
  const int r = request_of(p.q_starts, p.n_req, p.n_tok, t, part);
  if (r == p.n_req) return;
  const int q0 = start_at(p.q_starts, r, p.n_tok), n = start_at(p.q_starts, r + 1, p.n_tok) - q0;
  const int k0 = start_at(p.kv_starts, r, p.n_kv), keys = max(0, start_at(p.kv_starts, r + 1, p.n_kv) - k0);
  const int seen = p.causal ? max(0, min(keys, keys - n + (t - q0) + 1)) : keys;
  for (int d = tid; d < (kNope + kRope); d += 256) x[d] = T::to_f32(p.q[t * p.q_stride + (int64_t)h * (kNope + kRope) + d]);
  float m = -INFINITY, l = 0.f, o[kValue / 128] = {};
  __syncthreads();
  for (int j0 = 0; j0 < seen; j0 += 256) {
    const int j = j0 + tid;
    float s = -INFINITY;
    if (j < seen) {
      const uint16_t* k = p.k + (k0 + j) * p.k_stride + h * p.k_head;
      const uint16_t* kr = p.kr + (k0 + j) * p.kr_stride;
      float sum = 0.f;
      for (int d = 0; d < kNope; ++d) sum += x[d] * T::to_f32(k[d]);
      for (int d = 0; d < kRope; ++d) sum += x[kNope + d] * T::to_f32(kr[d]);
      s = sum * p.scale;
    }
    float top = s;
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((tid & 63) == 0) fpart[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(m, fmaxf(fmaxf(fpart[0], fpart[1]), fmaxf(fpart[2], fpart[3])));
    const float ref = top == -INFINITY ? 0.f : top, back = m == -INFINITY ? 0.f : expf(m - ref);
    const float e = s == -INFINITY ? 0.f : expf(s - ref);
    w[tid] = e;
    float sum = e;
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    __syncthreads();
    if ((tid & 63) == 0) fpart[tid >> 6] = sum;
    __syncthreads();
    l = l * back + fpart[0] + fpart[1] + fpart[2] + fpart[3];
    m = top;
    for (int i = 0; i < kValue / 128; ++i) o[i] *= back;
    for (int i = 0; i < min(256, seen - j0); ++i) {
      const float e2 = w[i];
      if (e2 == 0.f) continue;
      if (tid < kValue) o[0] += e2 * T::to_f32(p.v[(k0 + j0 + i) * p.v_stride + h * p.v_head + tid]);
    }
    __syncthreads();
  }
  if (tid < kValue) p.out[t * p.out_stride + (int64_t)h * kValue + tid] = T::from_f32(l == 0.f ? 0.f : o[0] / l);
  if (tid == 0 && p.lse) p.lse[(int64_t)t * p.n_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

hipError_t launch_prompt_attention(const PromptParams& p, int dtype, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.n_tok * p.n_heads)), dim3(256), 0, s, p);
    return hipGetLastError();
  };
  return dtype == GALE_F16 ? go(prompt_simple_kernel<F16>) : go(prompt_simple_kernel<BF16>);
}

}  // namespace gale
