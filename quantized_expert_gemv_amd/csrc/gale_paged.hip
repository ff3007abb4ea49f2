// Block tables and slot maps of a batch, and the paged cache's writer.
#include "gale_mx.h"

namespace gale {

// Inclusive sum over the workgroup's 256 threads; total: the sum of all.  part: 4 words of LDS.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();                     // part of the sum before is read
  if (lane == 63) part[wave] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) v += part[w];
    total += part[w];
  }
  return v;
}

// One launch.  Request r's tokens and new blocks begin where the sums over the requests before it end, so a workgroup
// scans the requests (256 threads, four each per turn) and then places its own share of the batch's tokens, each found
// by a binary search over the turn's ends in LDS.  A new block begins with a token of the batch, and that token writes
// its table entry: every place and every entry has one writer, which reads nothing that another writes.  The turns stop with
// the workgroup's last token; the per-request outputs of turn c belong to workgroup c % gridDim.x, and taken to the last.
// Latency bound: a turn is one round of loads and two scans (5 us for one turn, 10 to 12 for 2047 requests of up to 256 tokens).
constexpr int kPlanPer = 4, kPlanTurn = 256 * kPlanPer;

__global__ void __launch_bounds__(256) paged_plan_kernel(
    const int32_t* __restrict__ past_lens, const int32_t* __restrict__ new_lens, int n_req, int shift,
    const int32_t* __restrict__ free_blocks, int free_cap, const int32_t* __restrict__ n_free, int32_t* __restrict__ table,
    int64_t table_stride, int max_blocks, int n_tok, int per, int64_t* __restrict__ slots, int32_t* __restrict__ q_starts,
    int32_t* __restrict__ kv_lens, int32_t* __restrict__ taken) {
  __shared__ int64_t part[4];
  __shared__ int32_t s_end[kPlanTurn], s_past[kPlanTurn], s_base[kPlanTurn];   // s_base: -1 for a refused request
  const int64_t free_n = max(0, min(*n_free, free_cap));
  const int t0 = (int)min((int64_t)n_tok, (int64_t)blockIdx.x * per), t1 = (int)min((int64_t)n_tok, (int64_t)t0 + per);
  const bool last_group = blockIdx.x == gridDim.x - 1;
  const int64_t mask = ((int64_t)1 << shift) - 1;
  int64_t tok0 = 0, need0 = 0, used = 0;       // sums over the turns before; used: blocks of this thread's granted requests
  int64_t total;
  for (int turn = 0;; ++turn) {
    const int r0 = turn * kPlanTurn;
    if (r0 >= n_req) break;
    const int64_t turn_first = tok0;
    int64_t past[kPlanPer], want[kPlanPer], end[kPlanPer], need[kPlanPer];
    int64_t sum = 0;
    const int first = r0 + (int)threadIdx.x * kPlanPer;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = first + i;
      past[i] = r < n_req ? max(0, past_lens[r]) : 0;
      const int64_t fresh = r < n_req ? max(0, new_lens[r]) : 0;
      want[i] = (past[i] + fresh + mask) >> shift;
      sum += fresh;
      end[i] = sum;
    }
    const int64_t before = tok0 + block_scan(sum, part, total) - sum;
    tok0 += total;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      end[i] += before;
      const bool fits = want[i] <= max_blocks && end[i] <= n_tok;
      need[i] = fits ? want[i] - ((past[i] + mask) >> shift) : -1;
      sum += max((int64_t)0, need[i]);
    }
    int64_t base = need0 + block_scan(sum, part, total) - sum;
    need0 += total;
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = first + i, c = (int)threadIdx.x * kPlanPer + i;
      const bool granted = need[i] == 0 || (need[i] > 0 && base + need[i] <= free_n);
      const int64_t prev = i == 0 ? before : end[i - 1];
      s_end[c] = (int)min(end[i], (int64_t)n_tok);
      s_past[c] = (int)past[i];
      s_base[c] = granted ? (int)min(base, free_n) : -1;      // past free_n only where nothing is taken
      if (granted) used += need[i];
      if (r < n_req && turn % (int)gridDim.x == (int)blockIdx.x) {
        q_starts[r] = (int)min(prev, (int64_t)n_tok);
        kv_lens[r] = (int)min((int64_t)INT32_MAX, granted ? past[i] + (end[i] - prev) : past[i]);
      }
      base += max((int64_t)0, need[i]);
    }
    __syncthreads();
    // the workgroup's own tokens among this turn's
    const int lo = (int)max((int64_t)t0, min(turn_first, (int64_t)n_tok)), hi = (int)min((int64_t)t1, tok0);
    for (int64_t t = lo + (int64_t)threadIdx.x; t < hi; t += 256) {
      int a = 0, b = kPlanTurn - 1;                           // the first request that ends behind t
      while (a < b) {
        const int m = (a + b) >> 1;
        if (s_end[m] > t) b = m;
        else a = m + 1;
      }
      const int begin = a ? s_end[a - 1] : (int)turn_first;
      int64_t slot = -1;
      if (s_base[a] >= 0) {
        const int64_t pos = s_past[a] + (t - begin);
        const int64_t blk = pos >> shift, have = ((int64_t)s_past[a] + mask) >> shift;
        int32_t* entry = table + (int64_t)(r0 + a) * table_stride + blk;
        int32_t id;
        if (blk >= have) {
          id = free_blocks[s_base[a] + (blk - have)];
          if ((pos & mask) == 0) *entry = id;
        } else {
          id = *entry;
        }
        if (id >= 0) slot = ((int64_t)id << shift) + (pos & mask);
      }
      slots[t] = slot;
    }
    __syncthreads();                    // the next turn writes s_end, s_past, s_base
    // nothing left for this workgroup: its tokens are placed and no later turn's outputs are its own
    const int grid = (int)gridDim.x, next = turn + 1 + ((int)blockIdx.x - (turn + 1) % grid + grid) % grid;
    if (tok0 >= t1 && !last_group && (int64_t)next * kPlanTurn >= n_req) return;
  }
  for (int64_t t = max((int64_t)t0, min(tok0, (int64_t)n_tok)) + threadIdx.x; t < t1; t += 256) slots[t] = -1;
  if (last_group) {
    (void)block_scan(used, part, total);
    if (threadIdx.x == 0) {
      q_starts[n_req] = (int)min(tok0, (int64_t)n_tok);
      taken[0] = (int)total;
    }
  }
}

hipError_t launch_paged_plan(const int32_t* past, const int32_t* news, int n_req, int shift, const int32_t* free_blocks,
                             int free_cap, const int32_t* n_free, int32_t* table, int64_t table_stride, int max_blocks,
                             int n_tok, int64_t* slots, int32_t* q_starts, int32_t* kv_lens, int32_t* taken, hipStream_t s) {
  const int grid = (int)std::min<int64_t>(256, std::max<int64_t>(1, ((int64_t)n_tok + 1023) / 1024));
  const int per = (int)(((int64_t)n_tok + grid - 1) / grid);
  hipLaunchKernelGGL(paged_plan_kernel, dim3(grid), dim3(256), 0, s, past, news, n_req, shift, free_blocks, free_cap, n_free,
                     table, table_stride, max_blocks, n_tok, per, slots, q_starts, kv_lens, taken);
  return hipGetLastError();
}

// A wavefront per token: 1 KB of latents is one 16-byte load of every lane, and eight lanes take the rope row.  In 4 bits
// a lane holds eight columns and a quad one MX block; 16-bit numbers times a power of two are exact in fp32, so the
// conversion's rounding is the only one.  Bound by HBM (16384 tokens to 4 bits: 7 us, 3.6 TB/s); a few tokens by latency (2.5 us).
template <typename T, bool MX>
__global__ void __launch_bounds__(256) latent_append_kernel(const uint16_t* __restrict__ latent, int64_t latent_stride,
                                                            const uint16_t* __restrict__ rope, int64_t rope_stride,
                                                            const int64_t* __restrict__ slots, int n_tok, int n_slots,
                                                            uint8_t* __restrict__ c, int64_t c_bytes,
                                                            uint8_t* __restrict__ scales, uint8_t* __restrict__ r,
                                                            int64_t r_bytes) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < n_tok; t += (int64_t)gridDim.x * 4) {
    const uint16_t* src = latent + t * latent_stride;
    const mx_u32x4 a = *reinterpret_cast<const mx_u32x4*>(src + 8 * lane);
    mx_u32x4 b = {0, 0, 0, 0};
    if (lane < 8) b = *reinterpret_cast<const mx_u32x4*>(rope + t * rope_stride + 8 * lane);
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= n_slots) continue;
    if constexpr (MX) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = T::to_f32((uint16_t)(a[i] & 0xFFFFu));
        v[2 * i + 1] = T::to_f32((uint16_t)(a[i] >> 16));
      }
      uint32_t words[2];
      const uint32_t s = mx_encode8<GALE_MX_E2M1>(v, words);
      mx_store8<GALE_MX_E2M1>(c + slot * (GALE_LATENT_DIM / 2), scales + slot * (GALE_LATENT_DIM / 32), lane, s, words);
    } else {
      *reinterpret_cast<mx_u32x4*>(c + slot * c_bytes + 16 * lane) = a;
    }
    if (lane < 8) *reinterpret_cast<mx_u32x4*>(r + slot * r_bytes + 16 * lane) = b;
  }
}

hipError_t launch_latent_append(const gale_latent_cache& c, const void* latent, int64_t latent_stride, const void* rope,
                                int64_t rope_stride, const int64_t* slots, int n_tok, hipStream_t s) {
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)n_tok + 3) / 4, 1 << 23);      // a grid has less than 2^32 threads
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, s, (const uint16_t*)latent, latent_stride,
                       (const uint16_t*)rope, rope_stride, slots, n_tok, c.n_blocks * c.block_size, (uint8_t*)c.latent,
                       2 * c.latent_stride, c.scales, (uint8_t*)c.rope, 2 * c.rope_stride);
    return hipGetLastError();
  };
  if (c.fmt == 0) return go(latent_append_kernel<F16, false>);      // 16-bit rows are copied: the type does not matter
  return c.dtype == GALE_F16 ? go(latent_append_kernel<F16, true>) : go(latent_append_kernel<BF16, true>);
}

}  // namespace gale
