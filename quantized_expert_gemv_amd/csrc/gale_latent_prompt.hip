// Latent attention of prompts, expanded form.
#include <climits>
#include <type_traits>

#include "gale_latent.h"

namespace gale {

constexpr int kNope = GALE_HEAD_NOPE, kValue = GALE_HEAD_VALUE, kQuery = kNope + kRope;

// A workgroup takes 128 queries of one head, 32 to each wavefront, and walks the keys in tiles of 64 with a running maximum
// and sum.  The tiles (keys' own parts, rope rows, values: 40 KB) come by direct copies into two LDS buffers, the next one's
// during the products of this one, so two workgroups share a CU and one's softmax runs beside the other's products.  S^T = K Q^T and
// O^T = V^T P^T: a query is a lane's column in both.  Bound by the matrix cores, the softmax between them, and the card's power (16384
// tokens, 16 heads: 1390 us, 990 TFLOP/s, MFMA busy half of the time at the clock that it gets); prompts of many lengths
// also by tiles that only some wavefronts need and by the start of each workgroup (12 of 20 to 2000 tokens: 684 TFLOP/s).
constexpr int kBq = 128, kBk = 64, kHeads = 8;
constexpr int kTileK = kBk * 256, kTileR = kBk * 128, kTileV = kBk * 256, kTile = kTileK + kTileR + kTileV;

struct Found {
  int q0, n, k0, keys, block;
};
__device__ __forceinline__ int wave_sum(int v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  v += lane_xor<8>(v);
  v += lane_xor<16>(v);
  v += lane_xor<32>(v);
  return __builtin_amdgcn_readfirstlane(v);
}

// Up to 64 requests, a lane for each: blocks go by the number of keys that they look at, in steps of kBq, most first, so that the
// grid ends with short ones (12 prompts of 20 to 2000 tokens, 32 heads: 352 us; in the order of the batch 371).  Of a request whose
// last block has level ceil(keys / kBq), blocks of level `at` and more are as many as the last of them: N(at) over the
// requests falls with `at`, and a binary search finds the level that the rank lies in.
__device__ __forceinline__ bool find_by_length(const PromptParams& p, int rank, Found& f) {
  const int lane = threadIdx.x & 63, r = min(lane, p.n_req - 1);
  const int q0 = start_at(p.q_starts, r, p.n_tok), q1 = start_at(p.q_starts, r + 1, p.n_tok);
  const int k0 = start_at(p.kv_starts, r, p.n_kv), k1 = start_at(p.kv_starts, r + 1, p.n_kv);
  const int n = lane < p.n_req ? max(0, q1 - q0) : 0, keys = max(0, k1 - k0);
  const int blocks = n / kBq + (n % kBq != 0), top = keys / kBq + (keys % kBq != 0);
  const int back = p.causal ? (n - keys) >> 7 : INT_MIN / 2;      // floor: block j's level is more than j - back, where it has keys
  auto from = [&](int at) { return at <= 0 ? blocks : top < at ? 0 : blocks - min(max(at - 1 + back, 0), blocks); };
  if (rank >= wave_sum(blocks)) return false;
  int lo = 0, hi = n > 0 ? top : 0, behind = 0;      // N(lo) > rank >= N(hi) = behind
  hi = max(hi, lane_xor<1>(hi));
  hi = max(hi, lane_xor<2>(hi));
  hi = max(hi, lane_xor<4>(hi));
  hi = max(hi, lane_xor<8>(hi));
  hi = max(hi, lane_xor<16>(hi));
  hi = __builtin_amdgcn_readfirstlane(max(hi, lane_xor<32>(hi))) + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, count = wave_sum(from(mid));
    if (count > rank) lo = mid;
    else hi = mid, behind = count;
  }
  const int mine = from(lo) - from(hi);
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(sum, d);
    if (lane >= d) sum += u;
  }
  const int at = rank - behind, place = at - (sum - mine);
  const uint64_t here = __ballot(place >= 0 && place < mine);
  if (here == 0) return false;
  const int it = __builtin_ctzll(here);
  f.q0 = __builtin_amdgcn_readlane(q0, it);
  f.n = __builtin_amdgcn_readlane(n, it);
  f.k0 = __builtin_amdgcn_readlane(k0, it);
  f.keys = __builtin_amdgcn_readlane(keys, it);
  f.block = __builtin_amdgcn_readlane(blocks - from(lo) + place, it);
  return true;
}

// More requests: request r's blocks begin at number start_r / kBq + r, which is at most one number more than its blocks behind the
// request before it, so a block's request is found by a search in the starts alone: 64 places at a time, two rounds of loads
// for up to 4096 requests and three for the most.  Every wavefront does it by itself.
__device__ __forceinline__ bool find_block(const PromptParams& p, int idx, Found& f) {
  const int lane = threadIdx.x & 63;
  for (int lo = 0, hi = p.n_req;;) {
    const int step = (hi - lo + 63) >> 6, r = lo + lane * step, at = min(r, p.n_req - 1);
    const int q = start_at(p.q_starts, at, p.n_tok), q1 = start_at(p.q_starts, at + 1, p.n_tok);
    const int k = start_at(p.kv_starts, at, p.n_kv), k1 = start_at(p.kv_starts, at + 1, p.n_kv);
    const uint64_t ahead = __ballot(r < hi && q / kBq + r <= idx);
    if (ahead == 0) return false;
    const int last = 63 - __builtin_clzll(ahead);
    if (step > 1) {
      lo += last * step;
      hi = min(hi, lo + step);
      continue;
    }
    f.q0 = __builtin_amdgcn_readlane(q, last);
    f.n = __builtin_amdgcn_readlane(q1, last) - f.q0;
    f.k0 = __builtin_amdgcn_readlane(k, last);
    f.keys = max(0, __builtin_amdgcn_readlane(k1, last) - f.k0);
    f.block = idx - (f.q0 / kBq + lo + last);
    return (int64_t)f.block * kBq < f.n;
  }
}

template <typename T>
__global__ void __launch_bounds__(256, 2) prompt_kernel(const PromptParams p, int n_blocks) {
#if defined(__HIP_DEVICE_COMPILE__)   // buffer resources are a device type: the host pass needs the kernel's name only
  __shared__ __attribute__((aligned(1024))) uint8_t tiles[2 * kTile];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups go round robin over the 8 XCDs: of kHeads heads at a time an XCD takes one, so the blocks that read one head's keys
  // share an L2 (those prompts: 0.94 GB from memory; 32 heads at a time 1.5 GB and 359 us, 16 362 us).
  const int64_t place = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (place >= (int64_t)n_blocks * p.n_heads) return;
  const int group = (int)(place / ((int64_t)n_blocks * kHeads)), width = min(kHeads, p.n_heads - group * kHeads);
  const int inside = (int)(place - (int64_t)group * n_blocks * kHeads), idx = inside / width;
  const int head = group * kHeads + inside - idx * width;
  Found f;
  if (p.n_req <= 64 ? !find_by_length(p, idx, f) : !find_block(p, n_blocks - 1 - idx, f)) return;
  const int q0 = f.q0, n = f.n, k0 = f.k0, keys = f.keys, b0 = f.block * kBq;
  const int qi = b0 + 32 * wave + col;                        // this lane's query
  const int gap = keys - n;
  const int seen = qi >= n ? 0 : p.causal ? max(0, min(keys, gap + qi + 1)) : keys;
  // keys that the workgroup, and this wavefront, look at; keys that all of the wavefront's queries see
  const int last = min(n, b0 + kBq) - 1, wlast = min(n, b0 + 32 * wave + 32) - 1, wfirst = b0 + 32 * wave;
  const int wg_keys = __builtin_amdgcn_readfirstlane(p.causal ? max(0, min(keys, gap + last + 1)) : keys);
  const int w_keys = __builtin_amdgcn_readfirstlane(wfirst >= n ? 0 : p.causal ? max(0, min(keys, gap + wlast + 1)) : keys);
  const int w_all = __builtin_amdgcn_readfirstlane(wfirst >= n ? 0 : p.causal ? max(0, min(keys, gap + wfirst + 1)) : keys);

  // copies: 1 KB of consecutive LDS places, lane l the place 16 l; wavefront w takes the copies 4 j + w
  lds_u8* smem = (lds_u8*)tiles;
  const int kr = 4 * wave + (lane >> 4), rr = 8 * wave + (lane >> 3);      // first row of this lane: + 16 j, + 32 j
  const int kb = (int)(2 * p.k_stride), vb = (int)(2 * p.v_stride), rb = (int)(2 * p.kr_stride);   // the host keeps 64 rows in 32 bits
  const int vk = kr * kb + 16 * ((lane & 15) ^ swizzle(kr)), vv = kr * vb + 16 * ((lane & 15) ^ swizzle(kr));
  const int vr = rr * rb + 16 * ((lane & 7) ^ swizzle8(rr));
  auto copy = [&](int j0, lds_u8* to) {
    // rows behind the last key come as zeros, also where a copy's scalar offset alone is past the end: it counts in the range check
    // (measured for 1 to 64 rows, 256 bytes to 32 MB apart)
    const int rows = min(kBk, keys - j0);
    const auto rk = __builtin_amdgcn_make_buffer_rsrc((void*)(p.k + (int64_t)(k0 + j0) * p.k_stride + head * p.k_head), 0,
                                                      (rows - 1) * kb + 256, 0x00020000);
    const auto rv = __builtin_amdgcn_make_buffer_rsrc((void*)(p.v + (int64_t)(k0 + j0) * p.v_stride + head * p.v_head), 0,
                                                      (rows - 1) * vb + 256, 0x00020000);
    const auto rp = __builtin_amdgcn_make_buffer_rsrc((void*)(p.kr + (int64_t)(k0 + j0) * p.kr_stride), 0,
                                                      (rows - 1) * rb + 128, 0x00020000);
    typedef __attribute__((address_space(3))) void* lds_ptr;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_ptr)(to + 1024 * (4 * j + wave)), 16, vk, 16 * j * kb, 0, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (lds_ptr)(to + kTileK + 1024 * (4 * j + wave)), 16, vr, 32 * j * rb, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_ptr)(to + kTileK + kTileR + 1024 * (4 * j + wave)), 16, vv, 16 * j * vb, 0, 0);
  };

  // this lane's query: 12 operands of 16 columns
  s16x8 xq[12];
  {
    const int64_t t = q0 + min(qi, n - 1);
    const uint16_t* src = p.q + t * p.q_stride + (int64_t)head * kQuery + 8 * half;
#pragma unroll
    for (int s = 0; s < 12; ++s) xq[s] = signed_query<T>(*reinterpret_cast<const s16x8*>(src + 16 * s), p.scale);
  }
  const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * 1.44269504088896341f;
  if (wg_keys > 0) copy(0, smem);

  const float lift = Mma<T>::lift(keys);
  f32x16 o[4] = {};
  float m = -INFINITY, l = 0.f;

  // The next tile's copies and the use of this one stand in one function with pointers that do not meet: the compiler, which does not
  // see how the places alternate, would otherwise wait for all copies in front of every transposing read.
  auto step = [&](int j0, lds_u8* __restrict to, const lds_u8* __restrict at) __attribute__((always_inline)) {
    if (j0 + kBk < wg_keys) copy(j0 + kBk, to);
    if (j0 >= w_keys) return;
    // LDS places of operands: K, block k of 16 columns: chunk 2 k + half of row col (+ 32); V^T, column block b of 32: chunks 4 b .. of
    // rows vrow, vrow + 8 (+ 16 t).  Blocks change the same bits of a place as a row's swizzle: by exclusive or.
    const int lane = here(tid & 63), col = lane & 31, half = lane >> 5, vrow = 4 * half + ((lane & 15) >> 2);
    const int ak = col * 256 + ((half ^ swizzle(col)) << 4), ar = col * 128 + ((half ^ swizzle8(col)) << 4);
    const int chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int av0 = vrow * 256 + ((chunk ^ swizzle(vrow)) << 4) + 8 * (lane & 1);
    const int av1 = (vrow + 8) * 256 + ((chunk ^ swizzle(vrow + 8)) << 4) + 8 * (lane & 1);
    const lds_u8* const rows = at + kTileK;
    const lds_u8* const vals = rows + kTileR;
    f32x16 s[2] = {};
#pragma unroll
    for (int k = 0; k < 12; ++k)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const s16x8 a = k < 8 ? lds_operand(at + (ak ^ (k << 5)) + g * 32 * 256) : lds_operand(rows + (ar ^ ((k & 3) << 5)) + g * 32 * 128);
        s[g] = Mma<T>::mma(a, xq[k], s[g]);
      }
    const bool masked = j0 + kBk > w_all;
    if (masked) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j0 + 32 * g + 8 * (i >> 2) + 4 * half + (i & 3) >= seen) s[g][i] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[g][i]);
    top = fmaxf(top, other_half(top)) * c;
    if (__any(top > m + kSlack)) {
      const float up = fmaxf(m, top), back = m == up ? 1.f : __builtin_amdgcn_exp2f(m - up);
#pragma unroll
      for (int b = 0; b < 4; ++b) o[b] *= back;
      l *= back;
      m = up;
    }
    const float ref = (m == -INFINITY ? 0.f : m) - lift;
    s16x8 pt[4];
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = __builtin_amdgcn_exp2f(fmaf(s[t >> 1][8 * (t & 1) + i], c, -ref));
        sum += w[i];
      }
      pt[t] = Mma<T>::pack(w);
    }
    l += sum;
    auto values = [&](auto clean) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const s16x4 lo = lds_transposed(vals + (av0 ^ (b << 6)) + t * 16 * 256), hi = lds_transposed(vals + (av1 ^ (b << 6)) + t * 16 * 256);
          s16x8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          if constexpr (clean.value) a = finite_only<T>(a);
          o[b] = Mma<T>::mma(a, pt[t], o[b]);
          if constexpr (clean.value) __builtin_amdgcn_sched_barrier(0);      // the rare way takes no more registers
        }
      }
    };
    // A product takes the weight 0 of a key that a query does not see times its value, and NaN times 0 is NaN.  So where only some
    // of the queries see a key, values that are not finite stay out of the product and are added to those that do.
    uint32_t odd = 0;
    if (masked && w_all < w_keys) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const mx_u32x4 v = *(const __attribute__((address_space(3))) mx_u32x4*)(vals + 1024 * i + 16 * lane);
        odd |= not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w);
      }
    }
    if (__builtin_expect(__any(odd != 0), 0)) {
      values(std::true_type{});
      for (int j = 0; j < kBk; ++j) {
        if (j0 + j >= w_keys) break;
#pragma unroll
        for (int u = 0; u < 16; ++u) {          // columns 8 u + 4 half ..
          const s16x4 v = *(const __attribute__((address_space(3))) s16x4*)(vals + j * 256 + ((u ^ swizzle(j)) << 4) + 8 * half);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = T::to_f32((uint16_t)v[i]);
            if (!(fabsf(f) < INFINITY) && j0 + j < seen) o[u >> 2][4 * (u & 3) + i] += f;
          }
        }
      }
    } else {
      values(std::false_type{});
    }
  };

  int buf = 0;
  for (int j0 = 0; j0 < wg_keys; j0 += kBk, buf ^= 1) {
    tiles_ready();
    step(j0, smem + (buf ^ 1) * kTile, smem + buf * kTile);
  }

  l += other_half(l);
  if (l == 0.f && seen > 0) l = kNoScore;
  if (qi < n) {
    const int64_t t = q0 + qi;
    const float r = normaliser(l);
    uint16_t* out = p.out + t * p.out_stride + (int64_t)head * kValue + 4 * half;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mx_u32x2 v;
        v.x = (uint32_t)T::from_f32(o[b][4 * i] * r) | ((uint32_t)T::from_f32(o[b][4 * i + 1] * r) << 16);
        v.y = (uint32_t)T::from_f32(o[b][4 * i + 2] * r) | ((uint32_t)T::from_f32(o[b][4 * i + 3] * r) << 16);
        *reinterpret_cast<mx_u32x2*>(out + 32 * b + 8 * i) = v;
      }
    if (half == 0 && p.lse)
      p.lse[t * p.n_heads + head] = l == 0.f ? -INFINITY : (m - lift + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
  }
#endif
}

hipError_t launch_prompt_attention(const PromptParams& p, int dtype, hipStream_t s) {
  const int64_t blocks = (int64_t)p.n_tok / kBq + p.n_req, total = blocks * p.n_heads;
  // a dimension of a grid is less than 2^32 threads
  const unsigned x = (unsigned)std::min<int64_t>(total, 1 << 23);
  const dim3 grid(x, (unsigned)((total + x - 1) / x));
  if (dtype == GALE_F16) hipLaunchKernelGGL(prompt_kernel<F16>, grid, dim3(256), 0, s, p, (int)blocks);
  else hipLaunchKernelGGL(prompt_kernel<BF16>, grid, dim3(256), 0, s, p, (int)blocks);
  return hipGetLastError();
}

}  // namespace gale
