// Latent attention over a paged cache, absorbed form.
#include "gale_latent.h"

namespace gale {

// Number d of the latent vector in a slot, as a number of T.
template <typename T, bool MX>
__device__ __forceinline__ float cached(const LatentParams& p, int slot, int d) {
  if constexpr (!MX) {
    return T::to_f32(((const uint16_t*)(p.latent + (int64_t)slot * p.latent_bytes))[d]);
  } else {
    const uint32_t c = (p.latent[(int64_t)slot * (kLat / 2) + (d >> 1)] >> (4 * (d & 1))) & 15u;
    const uint32_t s = p.scales[(int64_t)slot * (kLat / 32) + (d >> 5)];
    const float scale = s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s ? s << 23 : 0x400000u);
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float a = e == 0 ? 0.5f * (float)m : __uint_as_float(((e + 126u) << 23) | (m << 22));
    return T::to_f32(T::from_f32((c & 8u ? -a : a) * scale));
  }
}

// A workgroup per query (token and head): scores of 256 keys at a time, one thread each, then the 512 sums over those keys.
template <typename T, bool MX>
__global__ void __launch_bounds__(256) latent_simple_kernel(const LatentParams p) {
  __shared__ int part[4];
  __shared__ float fpart[4], x[kQk], w[256];
  __shared__ int slot[256];
  const int tid = threadIdx.x, t = (int)(blockIdx.x / (unsigned)p.n_heads), h = (int)(blockIdx.x % (unsigned)p.n_heads);
  const int r = request_of(p.q_starts, p.n_req, p.n_tok, t, part);
  if (r == p.n_req) return;
  const int q0 = start_at(p.q_starts, r, p.n_tok), n = start_at(p.q_starts, r + 1, p.n_tok) - q0;
  const int keys = keys_of(p.kv_lens, r, p.max_blocks, p.block_shift);
  const int32_t* row = p.table + (int64_t)r * p.table_stride;
  const int seen = p.causal ? max(0, min(keys, keys - n + (t - q0) + 1)) : keys;
  for (int d = tid; d < kQk; d += 256) x[d] = T::to_f32(p.q[t * p.q_stride + (int64_t)h * kQk + d]);
  float m = -INFINITY, l = 0.f, o[kLat / 2 / 128] = {};
  __syncthreads();
  for (int j0 = 0; j0 < seen; j0 += 256) {
    const int j = j0 + tid;
    float s = -INFINITY;
    const int at = j < seen ? slot_of(row, j, p.block_shift, p.n_blocks) : -1;
    slot[tid] = at;
    if (at >= 0) {
      float sum = 0.f;
      for (int d = 0; d < kLat; ++d) sum += x[d] * cached<T, MX>(p, at, d);
      const uint16_t* kr = (const uint16_t*)(p.rope + (int64_t)at * p.rope_bytes);
      for (int d = 0; d < kRope; ++d) sum += x[kLat + d] * T::to_f32(kr[d]);
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
    for (int i = 0; i < kLat / 2 / 128; ++i) o[i] *= back;
    for (int i = 0; i < min(256, seen - j0); ++i) {
      const float e2 = w[i];
      if (e2 == 0.f) continue;
      for (int k = 0; k < 2; ++k) o[k] += e2 * cached<T, MX>(p, slot[i], tid + 256 * k);
    }
    __syncthreads();
  }
  for (int k = 0; k < 2; ++k)
    p.out[t * p.out_stride + (int64_t)h * kLat + tid + 256 * k] = T::from_f32(l == 0.f ? 0.f : o[k] / l);
  if (tid == 0 && p.lse) p.lse[(int64_t)t * p.n_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t latent_workspace_bytes(int n_tok, int n_req, int n_heads) { return 256; }

hipError_t launch_latent_attention(const LatentParams& p, int dtype, int fmt, void* ws, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.n_tok * p.n_heads)), dim3(256), 0, s, p);
    return hipGetLastError();
  };
  if (dtype == GALE_F16) return fmt ? go(latent_simple_kernel<F16, true>) : go(latent_simple_kernel<F16, false>);
  return fmt ? go(latent_simple_kernel<BF16, true>) : go(latent_simple_kernel<BF16, false>);
}

}  // namespace gale
