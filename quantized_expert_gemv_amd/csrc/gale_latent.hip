// Latent attention over a paged cache, absorbed form.
#include <climits>
#include <cmath>

#include "gale_latent.h"

namespace gale {

// The queries of a request are its tokens' heads, token by token; a run is 16 RG of them against all of the request's keys.
// A workgroup of W wavefronts has RG row groups of 16 queries and KG = W / RG key groups: wavefront (rg, kg) walks every KG-th
// tile of 32 keys with its own running maximum and sums, which are joined at the end of the run.  A wavefront keeps its
// queries (72 registers) and its sums (128) to itself, and a tile (32 KB of latents, 4 KB of rope rows) is read from LDS
// twice: as K by rows and, transposed by the read, as V.  That is a 1 KB operand for each MFMA of 16 cycles: many rows
// are bound by the LDS, few by HBM.
//
// S^T = K Q^T and O^T = V^T P^T with the 16x16x32 MFMA: first operand: lane l holds row l % 16, columns 8 (l / 16) .. + 7, second
// alike; result register i of lane l: row 4 (l / 16) + i, column l % 16.  So the weights of keys 4 g .. 4 g + 3 and 16 + 4 g .. of
// a tile's two halves are lane group g's operand of the second product as they are, and V^T takes the same keys.
//
// All runs' tiles form one line, cut into up to kGroups equal parts, one for each workgroup (one to a CU): a run that lies in several
// parts leaves unnormalised sums in the workspace, two places to a workgroup (a run that began before its part, and one that goes
// on behind it), and latent_join_kernel adds them in the order of the parts.
constexpr int kGroups = 256;
constexpr int kKeys = 32, kTileL = kKeys * 2 * kLat, kTileR = kKeys * 2 * kRope, kTile = kTileL + kTileR;
constexpr int kScaleArea = 1024;                           // MX: scales of a tile's rows, for each wavefront
constexpr int kLds = 4 * kTile + 8 * kScaleArea + 1024 + 64;      // and maxima and sums of the wavefronts, a word of each
constexpr int kRows = 16, kSumBytes = kRows * kLat * 4;    // a row group and its sums

// Wavefronts of a workgroup with RG row groups.  LDS holds four tiles: one for each of four key groups, two for each of two, or four.
template <int RG>
constexpr int waves_of() { return RG == 8 ? 8 : 4; }

struct Run {
  int32_t parts, first, req, block;      // 0 parts: nothing to join
};
struct Workspace {
  int32_t* count;                        // runs of the batch
  Run* runs;                             // by run if there are at most kGroups, else by the workgroup that a run begins in
  float* stats;                          // [2 kGroups][RG][2][16]: maxima (powers of two), sums of weights
  float* sums;                           // [2 kGroups][RG][32 blocks of 16 columns][64 lanes] of 4: as a wavefront holds them
};

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Units (KG tiles) of request r's runs: blocks of rows, and units of each.
template <int RG>
__device__ __forceinline__ void run_units(const LatentParams& p, int r, int64_t& blocks, int64_t& units) {
  const int64_t n = max(0, start_at(p.q_starts, r + 1, p.n_tok) - start_at(p.q_starts, r, p.n_tok));
  const int64_t keys = keys_of(p.kv_lens, r, p.max_blocks, p.block_shift);
  blocks = (n * p.n_heads + kRows * RG - 1) / (kRows * RG);
  constexpr int kUnit = kKeys * (waves_of<RG>() / RG);
  units = max((int64_t)1, (keys + kUnit - 1) / kUnit);
}

template <typename T, bool MX, int RG>
__global__ void __launch_bounds__(64 * waves_of<RG>(), waves_of<RG>() / 4) latent_kernel(const LatentParams p, const Workspace ws, bool by_run) {
#if defined(__HIP_DEVICE_COMPILE__)   // buffer resources are a device type: the host pass needs the kernel's name only
  constexpr int W = waves_of<RG>(), KG = W / RG, NB = 4 / KG;
  constexpr int OWN = kKeys / RG, PIECES = RG <= 4 ? 4 / RG : 1;      // rows, and KB of rope rows, that a wavefront fetches
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  typedef __attribute__((address_space(3))) float lds_f32;
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), rg = wave % RG, kg = wave / RG;

  // ---- this workgroup's part of the line of units --------------------------------------------------------------------
  int64_t u, u_end, base, total;      // base: the first unit of request req
  int req, run_base, groups;          // run_base: runs before request req; groups: parts that the line is cut into
  {
    __shared__ int64_t part[W], found_base;
    __shared__ int parts_runs[W], found[2];
    const int per = (p.n_req + 64 * W - 1) / (64 * W), r0 = min(tid * per, p.n_req), r1 = min(r0 + per, p.n_req);
    int64_t sum = 0;
    int runs = 0;
    for (int r = r0; r < r1; ++r) {
      int64_t b, n;
      run_units<RG>(p, r, b, n);
      sum += b * n;
      runs += (int)b;
    }
    int64_t scan = sum;
    int rscan = runs;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t a = __shfl_up(scan, d);
      const int b = __shfl_up(rscan, d);
      if (lane >= d) scan += a, rscan += b;
    }
    if (lane == 63) part[tid >> 6] = scan, parts_runs[tid >> 6] = rscan;
    __syncthreads();
    total = 0;
    int total_runs = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < (tid >> 6)) scan += part[w], rscan += parts_runs[w];
      total += part[w];
      total_runs += parts_runs[w];
    }
    if (tid == 0) {
      if (!by_run) ws.runs[blockIdx.x].parts = 0;
      if (blockIdx.x == 0) *ws.count = by_run ? total_runs : kGroups;
    }
    groups = (int)min((int64_t)kGroups, total);
    if ((int)blockIdx.x >= groups) return;
    u = (int64_t)blockIdx.x * total / groups;
    u_end = (int64_t)(blockIdx.x + 1) * total / groups;
    scan -= sum;
    rscan -= runs;
    if (sum > 0 && scan <= u && u < scan + sum) {
      for (int r = r0; r < r1; ++r) {
        int64_t b, n;
        run_units<RG>(p, r, b, n);
        if (u < scan + b * n) {
          found[0] = r;
          found[1] = rscan;
          found_base = scan;
          break;
        }
        scan += b * n;
        rscan += (int)b;
      }
    }
    __syncthreads();
    req = __builtin_amdgcn_readfirstlane(found[0]);
    run_base = __builtin_amdgcn_readfirstlane(found[1]);
    base = uniform64(found_base);
    total = uniform64(total);
    u = (int64_t)blockIdx.x * total / groups;
    u_end = (int64_t)(blockIdx.x + 1) * total / groups;
  }
  auto owner = [&](int64_t unit) { return (int)(((unit + 1) * groups - 1) / total); };      // the workgroup of a unit

  // ---- LDS places of operands ------------------------------------------------------------------------------------------
  lds_u8* const tiles = smem + kg * NB * kTile;
  lds_u8* const scale_area = smem + 4 * kTile + wave * kScaleArea;
  lds_f32* const stats = (lds_f32*)(smem + 4 * kTile + 8 * kScaleArea);
  // K, column block s of 32: chunk 4 s + grp of row col (+ 16); its low four bits change with s & 3
  const int zk = swizzle(col), zr = swizzle8(col), vrow = 4 * grp + (col >> 2);
  int ak[4], ar[2], av[8];
#pragma unroll
  for (int s = 0; s < 4; ++s) ak[s] = col * 1024 + (((4 * s + grp) ^ zk) << 4);
#pragma unroll
  for (int s = 0; s < 2; ++s) ar[s] = kTileL + col * 128 + (((4 * s + grp) ^ zr) << 4);
  // V^T, column block b of 16: chunks 2 b, 2 b + 1 of rows vrow (+ 16)
#pragma unroll
  for (int b = 0; b < 8; ++b) av[b] = vrow * 1024 + (((2 * b + ((col & 3) >> 1)) ^ swizzle(vrow)) << 4) + 8 * (col & 1);
  const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * 1.44269504088896341f;

  while (u < u_end) {
    // ---- the next run, or what of it is in this part ---------------------------------------------------------------------
    int64_t blocks, units;
    run_units<RG>(p, req, blocks, units);
    if (u >= base + blocks * units) {      // also requests without queries
      base += blocks * units;
      run_base += (int)blocks;
      ++req;
      continue;
    }
    const int block = __builtin_amdgcn_readfirstlane((int)((u - base) / units));
    const int64_t run0 = base + block * units;
    const int a0 = __builtin_amdgcn_readfirstlane((int)(u - run0)), a1 = __builtin_amdgcn_readfirstlane((int)min(units, u_end - run0));
    const bool whole = a0 == 0 && a1 == units;
    const int q0 = start_at(p.q_starts, req, p.n_tok), n = start_at(p.q_starts, req + 1, p.n_tok) - q0;
    const int keys = __builtin_amdgcn_readfirstlane(keys_of(p.kv_lens, req, p.max_blocks, p.block_shift));
    const int32_t* const table = p.table + (int64_t)req * p.table_stride;
    const int64_t row64 = (int64_t)block * (kRows * RG) + kRows * rg + col;
    const bool real = row64 < (int64_t)n * p.n_heads;
    const int row = (int)min(row64, (int64_t)n * p.n_heads - 1);
    int token = row / p.n_heads, head = row - token * p.n_heads;
    const int seen = !real ? 0 : p.causal ? max(0, min(keys, keys - n + token + 1)) : keys;
    // keys that any, and that all, of this wavefront's queries see
    int w_keys = seen, w_all = real ? seen : keys;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) {
      w_keys = max(w_keys, __shfl_xor(w_keys, d));
      w_all = min(w_all, __shfl_xor(w_all, d));
    }
    w_keys = __builtin_amdgcn_readfirstlane(w_keys);
    w_all = __builtin_amdgcn_readfirstlane(w_all);
    // keys that all queries of the run see, where some see more
    int some = INT_MAX;
    if (p.causal) {
      const int t0 = (int)((int64_t)block * (kRows * RG) / p.n_heads);
      const int t1 = (int)((min((int64_t)n * p.n_heads, (int64_t)(block + 1) * (kRows * RG)) - 1) / p.n_heads);
      if (t0 < t1) some = __builtin_amdgcn_readfirstlane(max(0, keys - n + t0 + 1));
    }

    s16x8 xq[18];
    {
      const uint16_t* src = p.q + (int64_t)(q0 + token) * p.q_stride + (int64_t)head * kQk + 8 * grp;
#pragma unroll
      for (int s = 0; s < 18; ++s) xq[s] = signed_query<T>(*reinterpret_cast<const s16x8*>(src + 32 * s), p.scale);
    }
    f32x4 o[32] = {};
    float m = -INFINITY, l = 0.f;

    // ---- fetching a tile ---------------------------------------------------------------------------------------------
    // Lanes r and r + 32 know the slot of row r of a tile, -1 where there is no key.
    auto slots_of = [&](int tile) {
      const int pos = tile * kKeys + (lane & 31);
      return pos >= 0 && pos < keys ? slot_of(table, pos, p.block_shift, p.n_blocks) : -1;
    };
    uint32_t codes[MX ? OWN : 1];
    mx_u32x4 ropes[MX ? PIECES : 1];
    // 16-bit rows: straight into LDS, a row for each copy; rows without a key come as zeros (a resource of no bytes), so that
    // 0 times them is 0.  Their rope rows do not matter: such keys' scores are replaced.
    auto fetch = [&](int slot, int buf) {
      typedef __attribute__((address_space(3))) void* lds_ptr;
      lds_u8* to = tiles + buf * kTile;
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const int r = rg * OWN + i, at = __builtin_amdgcn_readlane(slot, r);
        if constexpr (MX) {
          const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)(p.latent + (int64_t)max(at, 0) * (kLat / 2)), 0,
                                                            at < 0 ? 0 : kLat / 2, 0x00020000);
          codes[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * lane, 0, 0);
        } else {
          const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)(p.latent + (int64_t)max(at, 0) * p.latent_bytes), 0,
                                                            at < 0 ? 0 : 2 * kLat, 0x00020000);
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(to + r * 1024), 16, (lane ^ swizzle(r)) << 4, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if (rg * PIECES + i >= 4) break;
        const int r = 8 * (rg * PIECES + i) + (lane >> 3);
        const uint8_t* src = p.rope + (int64_t)max(__shfl(slot, r), 0) * p.rope_bytes + (((lane & 7) ^ swizzle8(r)) << 4);
        if constexpr (MX) ropes[i] = *reinterpret_cast<const mx_u32x4*>(src);
        else
          __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                           (lds_ptr)(to + kTileL + 1024 * (rg * PIECES + i)), 16, 0, 0);
      }
      if constexpr (MX) {
        const uint8_t* src = p.scales + (int64_t)max(__shfl(slot, rg * OWN + (lane & (OWN - 1))), 0) * (kLat / 32);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src, (lds_ptr)scale_area, 16, 0, 0);
      }
    };
    // MX rows, a tile later: 4-bit elements to 16-bit numbers, rounded where a scale takes them out of fp16's range.
    auto store = [&](uint32_t valid, int buf) {
      if constexpr (MX) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the scales' copy
        lds_u8* to = tiles + buf * kTile;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
          const int r = rg * OWN + i;
          const uint32_t s = scale_area[16 * i + (lane >> 2)];
          const float scale = s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s ? s << 23 : 0x400000u);
          mx_u32x4 v = mx_values8<T>(codes[i], scale);
          if (!(valid >> r & 1u)) v = mx_u32x4{0, 0, 0, 0};
          *(__attribute__((address_space(3))) mx_u32x4*)(to + r * 1024 + ((lane ^ swizzle(r)) << 4)) = v;
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          if (rg * PIECES + i < 4) *(__attribute__((address_space(3))) mx_u32x4*)(to + kTileL + 1024 * (rg * PIECES + i) + 16 * lane) = ropes[i];
      }
    };

    // ---- the products with a tile --------------------------------------------------------------------------------------
    auto use = [&](int j0, uint32_t valid, const lds_u8* at) __attribute__((always_inline)) {
      f32x4 s[2] = {};
#pragma unroll
      for (int k = 0; k < 18; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const s16x8 a = k < 16 ? lds_operand(at + ak[k & 3] + (k >> 2) * 256 + u * 16 * 1024)
                                 : lds_operand(at + ar[k & 1] + u * 16 * 128);
          s[u] = Mma<T>::mma(a, xq[k], s[u]);
        }
      if (valid != 0xFFFFFFFFu || j0 + kKeys > w_all) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 16 * u + 4 * grp + i;
            if (!(valid >> r & 1u) || j0 + r >= seen) s[u][i] = -INFINITY;
          }
      }
      float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])), fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      top = over_groups(top, [](float a, float b) { return fmaxf(a, b); }) * c;
      if (__any(top > m + kSlack)) {
        const float up = fmaxf(m, top), back = m == up ? 1.f : __builtin_amdgcn_exp2f(m - up);
#pragma unroll
        for (int b = 0; b < 32; ++b) o[b] *= back;
        l *= back;
        m = up;
      }
      const float ref = (m == -INFINITY ? 0.f : m) - Mma<T>::kLift;
      float e[8], sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(fmaf(s[i >> 2][i & 3], c, -ref));
        sum += e[i];
      }
      l += sum;
      const s16x8 w = Mma<T>::pack(e);
#pragma unroll
      for (int b = 0; b < 32; ++b) {
        const s16x4 lo = lds_transposed(at + av[b & 7] + (b >> 3) * 256);
        const s16x4 hi = lds_transposed(at + av[b & 7] + (b >> 3) * 256 + 16 * 1024);
        o[b] = Mma<T>::mma(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), w, o[b]);
      }
    };
    // A product takes the weight 0 of a key that a query does not see times its value, and NaN times 0 is NaN.  So where only some
    // of the run's queries see a key (j >= some), rows of a tile that are not finite are zeroed by the wavefront that fetched them, and
    // the queries that see such a key have NaN as their sum of weights.
    auto clear = [&](int j0, lds_u8* at) {
      uint32_t bad = 0;
      for (int r = max(rg * OWN, some - j0); r < (rg + 1) * OWN; ++r) {
        __attribute__((address_space(3))) mx_u32x4* row16 = (__attribute__((address_space(3))) mx_u32x4*)(at + r * 1024 + 16 * lane);
        const mx_u32x4 v = *row16;
        if (__any((not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w)) != 0)) {
          bad |= 1u << r;
          *row16 = mx_u32x4{0, 0, 0, 0};
        }
      }
      if constexpr (RG > 1) {
        __attribute__((address_space(3))) uint32_t* words = (__attribute__((address_space(3))) uint32_t*)(stats + 256);
        if (lane == 0) words[wave] = bad;
        tiles_ready();
        bad = 0;
#pragma unroll
        for (int g = 0; g < RG; ++g) bad |= words[kg * RG + g];
      }
      bad = __builtin_amdgcn_readfirstlane(bad);
      while (bad != 0) {
        const int r = __builtin_ctz(bad);
        bad &= bad - 1;
        if (j0 + r < seen) l = NAN;
      }
    };

    // ---- the tiles -----------------------------------------------------------------------------------------------------
    // valid: which rows of a tile hold keys.  A ballot's two halves are alike.
    int slot = slots_of(a0 * KG + kg);
    if constexpr (NB == 1) {
      if constexpr (MX) fetch(slot, 0);
      for (int i = a0; i < a1; ++i) {
        const uint32_t valid = (uint32_t)__ballot(slot >= 0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the tile before is read
        if constexpr (MX) store(valid, 0);
        else fetch(slot, 0);
        slot = i + 1 < a1 ? slots_of((i + 1) * KG + kg) : -1;
        if constexpr (MX) {
          if (i + 1 < a1) fetch(slot, 0);
        } else {
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        const int j0 = (i * KG + kg) * kKeys;
        if (j0 + kKeys > some) clear(j0, tiles);
        if (j0 < w_keys) use(j0, valid, tiles);
      }
    } else {
      uint32_t valid = (uint32_t)__ballot(slot >= 0);
      fetch(slot, 0);
      if constexpr (MX) store(valid, 0);
      slot = a0 + 1 < a1 ? slots_of((a0 + 1) * KG + kg) : -1;
      if constexpr (MX) {
        if (a0 + 1 < a1) fetch(slot, 0);
      }
      int buf = 0;
      for (int i = a0; i < a1; ++i) {
        tiles_ready();
        const uint32_t next = (uint32_t)__ballot(slot >= 0);
        const int j0 = (i * KG + kg) * kKeys;
        lds_u8* at = tiles + buf * kTile;
        buf ^= 1;
        if ((i + 1) * (KG * kKeys) > some) clear(j0, at);      // the same for all wavefronts
        if constexpr (MX) {
          if (j0 < w_keys) use(j0, valid, at);
          if (i + 1 < a1) {
            store(next, buf);
            slot = i + 2 < a1 ? slots_of((i + 2) * KG + kg) : -1;
            if (i + 2 < a1) fetch(slot, 0);
          }
        } else {
          if (i + 1 < a1) {
            fetch(slot, buf);
            slot = i + 2 < a1 ? slots_of((i + 2) * KG + kg) : -1;
          }
          if (j0 < w_keys) use(j0, valid, at);
        }
        valid = next;
      }
    }

    // ---- joining the key groups, and what leaves ---------------------------------------------------------------------------
    const int place = a0 == 0 ? 2 * (int)blockIdx.x + 1 : 2 * (int)blockIdx.x;
    int q_row = row;
    asm("" : "+v"(q_row));       // addresses of results are made here, not kept over the loop
    token = q_row / p.n_heads;
    head = q_row - token * p.n_heads;
    l = over_groups(l, [](float a, float b) { return a + b; });
    float top = m;
    if constexpr (KG > 1) {
      if (grp == 0) {
        stats[wave * 32 + col] = m;
        stats[wave * 32 + 16 + col] = l;
      }
      __syncthreads();
      float lsum = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) top = fmaxf(top, stats[(k * RG + rg) * 32 + col]);
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float mk = stats[(k * RG + rg) * 32 + col], lk = stats[(k * RG + rg) * 32 + 16 + col];
        lsum += mk == top ? lk : lk * __builtin_amdgcn_exp2f(mk - top);
      }
      l = lsum;
      const float back = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
      for (int b = 0; b < 32; ++b) o[b] *= back;
    }
    const float r = l == 0.f ? 0.f : 1.f / l;
    uint16_t* out = p.out + (int64_t)(q0 + token) * p.out_stride + (int64_t)head * kLat + 4 * grp;
    float* sums = ws.sums + ((int64_t)place * RG + rg) * (kRows * kLat) + 4 * lane;
    // columns 16 b + 4 grp .. of this lane's query
    auto leave = [&](int b, f32x4 v) {
      if (whole) {
        if (real) {
          mx_u32x2 h;
          h.x = (uint32_t)T::from_f32(v.x * r) | ((uint32_t)T::from_f32(v.y * r) << 16);
          h.y = (uint32_t)T::from_f32(v.z * r) | ((uint32_t)T::from_f32(v.w * r) << 16);
          *reinterpret_cast<mx_u32x2*>(out + 16 * b) = h;
        }
      } else {
        *reinterpret_cast<f32x4*>(sums + b * 256) = v;
      }
    };
    if constexpr (KG == 1) {
#pragma unroll
      for (int b = 0; b < 32; ++b) leave(b, o[b]);
    } else {
      // 128 KB at a time: all columns of four wavefronts or half of eight; each adds its share of its row group's blocks
      constexpr int STEP = 128 / W, MINE = STEP / KG;
#pragma unroll
      for (int t = 0; t < 32 / STEP; ++t) {
        __syncthreads();
#pragma unroll
        for (int b = 0; b < STEP; ++b) ((lds_f32x4*)smem)[(wave * STEP + b) * 64 + lane] = o[STEP * t + b];
        __syncthreads();
#pragma unroll
        for (int b = 0; b < MINE; ++b) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KG; ++k) v += ((const lds_f32x4*)smem)[((k * RG + rg) * STEP + kg * MINE + b) * 64 + lane];
          leave(STEP * t + kg * MINE + b, v);
        }
      }
    }
    if (kg == 0 && grp == 0) {
      if (whole) {
        if (real && p.lse)
          p.lse[(int64_t)(q0 + token) * p.n_heads + head] =
              l == 0.f ? -INFINITY : (top - Mma<T>::kLift + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
      } else {
        float* st = ws.stats + ((int64_t)place * RG + rg) * 32;
        st[col] = top;
        st[16 + col] = l;
      }
    }
    if (a0 == 0 && tid == 0) {
      const int first = (int)blockIdx.x;
      const int at = by_run ? run_base + block : first;
      if (at < kGroups)       // always, where q_starts ascends
        ws.runs[at] = Run{whole ? 0 : owner(run0 + units - 1) - first + 1, first, req, block};
    }
    u = run0 + a1;
    __syncthreads();          // the next run writes the tiles
  }
#endif
}

// The sums of a run that lies in several parts: a workgroup per row group and 64 columns, four quarters of the parts side by
// side.  Every sum goes in the order of the parts, so equal calls give equal bits.
template <typename T, int RG>
__global__ void __launch_bounds__(1024) latent_join_kernel(const LatentParams p, const Workspace ws) {
  __shared__ float weight[kGroups][kRows], most[64][kRows], sum[64][kRows];
  __shared__ f32x4 part[3][256];
  if ((int)blockIdx.x >= *ws.count) return;
  const Run run = ws.runs[blockIdx.x];
  if (run.parts <= 1) return;
  const int tid = threadIdx.x, rg = (int)blockIdx.y >> 3;
  auto place = [&](int k) { return (int64_t)(2 * (run.first + k) + (k == 0)) * RG + rg; };
  float top = -INFINITY;
  {
    const int row = tid & 15, k0 = tid >> 4;
    float l = 0.f;
    for (int k = k0; k < run.parts; k += 64) top = fmaxf(top, ws.stats[place(k) * 32 + row]);
    most[k0][row] = top;
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < 64; ++k) top = fmaxf(top, most[k][row]);
    for (int k = k0; k < run.parts; k += 64) {
      const float mk = ws.stats[place(k) * 32 + row], e = mk == top ? 1.f : __builtin_amdgcn_exp2f(mk - top);
      weight[k][row] = e;
      l += e * ws.stats[place(k) * 32 + 16 + row];
    }
    sum[k0][row] = l;
    __syncthreads();
  }
  // row tid % 16 is also the row of the lane's query
  const int lane = tid & 63, b = ((int)blockIdx.y & 7) * 4 + ((tid >> 6) & 3), quarter = tid >> 8, col = lane & 15, grp = lane >> 4;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const float* src = ws.sums + (b * 64 + lane) * 4;
#pragma unroll 4
  for (int k = quarter; k < run.parts; k += 4) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(src + place(k) * (kRows * kLat));
    acc += weight[k][col] * v;
  }
  if (quarter > 0) part[quarter - 1][tid & 255] = acc;
  __syncthreads();
  if (quarter > 0) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) acc += part[k][tid];
  float l = 0.f;
#pragma unroll 8
  for (int k = 0; k < 64; ++k) l += sum[k][col];
  const int q0 = start_at(p.q_starts, run.req, p.n_tok), n = start_at(p.q_starts, run.req + 1, p.n_tok) - q0;
  const int64_t row = (int64_t)run.block * (kRows * RG) + kRows * rg + col;
  if (row >= (int64_t)n * p.n_heads) return;
  const int token = (int)row / p.n_heads, head = (int)row - token * p.n_heads;
  const float r = l == 0.f ? 0.f : 1.f / l;
  mx_u32x2 h;
  h.x = (uint32_t)T::from_f32(acc.x * r) | ((uint32_t)T::from_f32(acc.y * r) << 16);
  h.y = (uint32_t)T::from_f32(acc.z * r) | ((uint32_t)T::from_f32(acc.w * r) << 16);
  *reinterpret_cast<mx_u32x2*>(p.out + (int64_t)(q0 + token) * p.out_stride + (int64_t)head * kLat + 16 * b + 4 * grp) = h;
  if (b == 0 && grp == 0 && p.lse)
    p.lse[(int64_t)(q0 + token) * p.n_heads + head] =
        l == 0.f ? -INFINITY : (top - Mma<T>::kLift + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

// Row groups of a workgroup: few rows leave key groups to the other wavefronts, many share each tile.
static int row_groups(int n_tok, int n_req, int n_heads) {
  const int64_t rows = ((int64_t)n_tok * n_heads + std::max(n_req, 1) - 1) / std::max(n_req, 1);
  return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 8;
}

constexpr size_t kHead = 256, kRunBytes = (kGroups * sizeof(Run) + 255) & ~(size_t)255;

size_t latent_workspace_bytes(int n_tok, int n_req, int n_heads) {
  return kHead + kRunBytes + (size_t)2 * kGroups * row_groups(n_tok, n_req, n_heads) * (128 + kSumBytes);
}

template <typename T, bool MX, int RG>
static hipError_t launch_latent(const LatentParams& p, void* mem, hipStream_t s) {
  uint8_t* at = (uint8_t*)mem;
  const Workspace ws = {(int32_t*)at, (Run*)(at + kHead), (float*)(at + kHead + kRunBytes),
                        (float*)(at + kHead + kRunBytes + (size_t)2 * kGroups * RG * 128)};
  // every request has at most one run more than its share of the rows
  const int64_t rows = (int64_t)p.n_tok * p.n_heads, runs = std::min(rows / (kRows * RG) + p.n_req, rows);
  const bool by_run = runs <= kGroups;
  hipError_t e = hipFuncSetAttribute((const void*)latent_kernel<T, MX, RG>, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(latent_kernel<T, MX, RG>), dim3(kGroups), dim3(64 * waves_of<RG>()), kLds, s, p, ws, by_run);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(latent_join_kernel<T, RG>), dim3((unsigned)std::min<int64_t>(runs, kGroups), 8 * RG), dim3(1024), 0, s,
                     p, ws);
  return hipGetLastError();
}

template <typename T, bool MX>
static hipError_t launch_rows(const LatentParams& p, void* ws, hipStream_t s) {
  const int rg = row_groups(p.n_tok, p.n_req, p.n_heads);
  return rg == 1   ? launch_latent<T, MX, 1>(p, ws, s)
         : rg == 2 ? launch_latent<T, MX, 2>(p, ws, s)
         : rg == 4 ? launch_latent<T, MX, 4>(p, ws, s)
                   : launch_latent<T, MX, 8>(p, ws, s);
}

hipError_t launch_latent_attention(const LatentParams& p, int dtype, int fmt, void* ws, hipStream_t s) {
  if (dtype == GALE_F16) return fmt ? launch_rows<F16, true>(p, ws, s) : launch_rows<F16, false>(p, ws, s);
  return fmt ? launch_rows<BF16, true>(p, ws, s) : launch_rows<BF16, false>(p, ws, s);
}

}  // namespace gale
