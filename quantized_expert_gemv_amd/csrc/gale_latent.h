// Device pieces shared by the kernels of latent attention.
#pragma once
#include "gale_mx.h"

namespace gale {

constexpr int kLat = GALE_LATENT_DIM, kRope = GALE_LATENT_ROPE, kQk = kLat + kRope;

// Entry r of an ascending array of starts, within [0, n].
__device__ __forceinline__ int start_at(const int32_t* starts, int r, int n) { return min(max(starts[r], 0), n); }

// The request that token t belongs to, n_req if none: the number of requests that end at or before t.  For a workgroup
// of 256 threads; part: 4 words of LDS.
__device__ __forceinline__ int request_of(const int32_t* starts, int n_req, int n_tok, int t, int* part) {
  int n = 0;
  for (int r = threadIdx.x; r < n_req; r += 256) n += start_at(starts, r + 1, n_tok) <= t;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = n;
  __syncthreads();
  n = part[0] + part[1] + part[2] + part[3];
  return n < n_req && start_at(starts, n, n_tok) <= t ? n : n_req;
}

// Row of the cache that holds a request's key at position pos, -1 if its block does not exist.  row: the request's row
// of the block table; pos is below max_blocks * block_size.
__device__ __forceinline__ int slot_of(const int32_t* row, int pos, int shift, int n_blocks) {
  const int id = row[pos >> shift];
  return id >= 0 && id < n_blocks ? (id << shift) + (pos & ((1 << shift) - 1)) : -1;
}

// Keys of request r.
__device__ __forceinline__ int keys_of(const int32_t* kv_lens, int r, int max_blocks, int shift) {
  return (int)min((int64_t)max(kv_lens[r], 0), (int64_t)max_blocks << shift);
}

}  // namespace gale
