// Latent attention over a paged cache, absorbed form.
#include <climits>
#include <cmath>
#include <cstdint>

#include "gale_latent.h"

namespace gale {

// The queries of a request are its tokens' heads, token by token; a run is Q RG of them against all of the request's keys.
// A workgroup of four wavefronts has RG row groups of Q queries and KG = 4 / RG key groups: wavefront (rg, kg) walks every KG-th
// tile of keys with its own running maximum and sums, which are joined at the end of the run.  A wavefront keeps its queries
// and sums to itself, and a tile is read from LDS twice: as K by rows and, transposed by the read, as V.
//
// S^T = K Q^T and O^T = V^T P^T with the 16x16x32 MFMA: first operand: lane l holds row l % 16, columns 8 (l / 16) .. + 7, second
// alike; result register i of lane l: row 4 (l / 16) + i, column l % 16.  So a query is a lane's column in both, and the weights
// are an operand of the second product as they are, where V^T takes the keys in the same order.
//   Up to 16 rows: four key groups, tiles of 16 keys (V by the 16x16x16 MFMA), two for each wavefront, which no other one reads:
//     no barrier; bound by HBM (64 requests of 1 to 8192 keys, 16 heads: 70 us, 4.8 TB/s; 7.1 where it only fetches: the
//     rest is unequal parts and a part's start and end, 15 us).  4-bit rows are bound by their conversion and the products
//     after it (128 requests of 1 to 16384 keys: 176 us with the join; their bytes alone take 84).
//   Up to 32 and 64: tiles of 32 keys for two and four row groups of 16.  Each MFMA of 16 cycles takes a 1 KB operand from LDS, twice
//     its bandwidth, so the LDS is the bound once there are more rows than HBM's (32 requests of 1 to 4096 keys, 32 and 64 heads:
//     36 and 46 us; 4-bit rows 38 and 51).
//   More: eight wavefronts, two to a SIMD, four row groups of 32 queries: two MFMAs for each operand.  Queries (144 registers) and sums
//     (256) of 32 do not fit one wavefront (300 to 580 registers spilled, also with half of the queries in LDS and with 32x32x16
//     MFMAs), so two share them: each takes one half of the latent columns in both products, and they add their halves of the
//     scores through LDS.  One request of 131072 keys and 128 heads: 73 us, 495 TFLOP/s; bound by the barriers of each tile, with
//     two wavefronts to a SIMD, and by the sums that leave (64 MB, 18 us of join).
// Block ids of pages below 8 slots (16 for tiles of 32 keys) are vector loads, which return behind the copies in flight: 64 requests
// in pages of one slot take 79 us for 74, in 4 bits 68 for 61.
//
// All runs' tiles form one line, cut into up to kGroups equal parts, one for each workgroup (one to a CU): a run that lies in several
// parts leaves unnormalised sums in the workspace, two places to a workgroup (a run that began before its part, and one that goes
// on behind it), and latent_join_kernel adds them in the order of the parts.
constexpr int kGroups = 256, kLead = 4;

template <bool MX, int Q, int RG>
struct Shape {
  static constexpr int C = Q / 16, W = 4 * C;                        // wavefronts that share queries, and all of them
  static constexpr int KG = 4 / RG, KEYS = Q * RG == 16 ? 16 : 32;   // keys of a tile
  static constexpr int LATENTS = KEYS * 2 * kLat, TILE = LATENTS + KEYS * 2 * kRope;
  static constexpr int NB = 2;                                       // tiles in LDS of a key group
  static constexpr int F = W / KG, OWN = KEYS / F;                   // wavefronts that fetch a tile, rows of each,
  static constexpr int PIECES = KEYS / 8 >= F ? KEYS / 8 / F : 1;    // and KB of rope rows of each, of the first ones
  static constexpr int UNIT = KG * KEYS;
  static constexpr int ROWS = Q * RG;
  // MX, tiles of 16 keys: one of 16-bit numbers, and three of rows as they are in the cache: codes, rope rows, scales (64 places)
  static constexpr int RAW = KEYS * (kLat / 2) + KEYS * 2 * kRope + 1024, RING = 3;
  static constexpr int G = Q / 16, BLOCKS = 32 / C;                  // a wavefront's groups of 16 queries, and blocks of 16 columns
  static constexpr int SUMS = Q * kLat * 4;
};
// LDS: tiles; the halves of the scores, parts of the queries, (MX) scales; (MX, tiles of 16 keys) what Shape says; maxima and sums, a word of each wavefront
constexpr int kScores = 2 * 32 * 1152, kQueries = kScores + 32768, kScales = 4 * 32 * 1152, kStats = 155648, kWords = kStats + 1024, kLds = kWords + 64;
static_assert(4 * 16 * 1024 + 4 * 3 * Shape<true, 16, 1>::RAW <= kStats && kQueries + 2 * 16384 <= kScales && kScales + 8192 <= kStats && kQueries + 3 * 16384 <= kStats, "what lies in LDS");

struct Run {
  int32_t parts, first, req, block;      // 0 parts: nothing to join
};
struct Workspace {
  int32_t* count;                        // runs of the batch
  Run* runs;                             // by run if there are at most kGroups, else by the part that a run begins in
  float* stats;                          // [2 kGroups][RG][2][Q]: maxima (powers of two), sums of weights
  float* sums;                           // [2 kGroups][RG][2 Q][64 lanes] of 4: as a wavefront holds them
};

constexpr int min_of(int a, int b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {      // of numbers that are not negative
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Request r's runs: blocks of rows, and units of each.
template <typename Sh>
__device__ __forceinline__ void run_units(const LatentParams& p, int r, int& blocks, int& units) {
  const int64_t n = max(0, start_at(p.q_starts, r + 1, p.n_tok) - start_at(p.q_starts, r, p.n_tok));
  const int keys = keys_of(p.kv_lens, r, p.max_blocks, p.block_shift);
  blocks = (int)((n * p.n_heads + Sh::ROWS - 1) / Sh::ROWS);
  units = max(1, (int)(((int64_t)keys + Sh::UNIT - 1) / Sh::UNIT));
}

alignas(16) __device__ uint32_t zero_row[2 * kLat / 4];      // never written
static_assert(__alignof__(zero_row) >= 16, "16-byte copies read it");

// Which 32 columns a product with K takes together is free: four chunks of 8, one for each lane group.  The groups that the LDS serves
// at once, 0 and 1 or 2 and 3 with eight rows of each (all even and odd rows of four), must not meet where a chunk's bits
// and the row's swizzle cancel, so they differ in bit 2 of the chunk (bit 1 of the rope's), which the swizzle changes with bit 0 (1) of
// the row.  With consecutive chunks every read of K took twice as long (counters: a conflict cycle for each).
__device__ __forceinline__ int block_chunk(int s, int grp) {
  return (s & 3) | (grp & 1) << 2 | (s & 4) << 1 | (grp >> 1) << 4 | (s >> 3) << 5;
}
__device__ __forceinline__ int rope_chunk(int s, int grp) { return (grp & 1) << 1 | grp >> 1 | s << 2; }

template <typename T, bool MX, int Q, int RG>
__global__ void __launch_bounds__(16 * Q) __attribute__((amdgpu_waves_per_eu(Q / 16, Q / 16)))      // 64 W threads, C wavefronts to a SIMD
latent_kernel(const LatentParams p, const Workspace ws, bool by_run) {
#if defined(__HIP_DEVICE_COMPILE__)   // buffer resources are a device type: the host pass needs the kernel's name only
  typedef Shape<MX, Q, RG> Sh;
  constexpr int C = Sh::C, W = Sh::W, G = Sh::G, KG = Sh::KG, KEYS = Sh::KEYS, NB = Sh::NB, F = Sh::F, OWN = Sh::OWN;
  constexpr int PIECES = Sh::PIECES, BLOCKS = Sh::BLOCKS, QB = 18 / C, AHEAD = C == 1 ? 8 : 4, AHEAD_K = C == 1 ? 8 : 2;      // QB: blocks of 32 columns of the queries
  constexpr int QL = C == 1 ? 0 : MX ? 2 : 3;      // of them blocks 2, 5, 8 lie in LDS: as many as there is room for
  constexpr bool RAW = MX && KEYS == 16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  typedef __attribute__((address_space(3))) float lds_f32;
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  typedef __attribute__((address_space(3))) mx_u32x4 lds_u32x4;
  typedef __attribute__((address_space(3))) uint32_t lds_u32;
  typedef __attribute__((address_space(3))) void* lds_ptr;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), rg = wave % RG, kg = C == 1 ? wave / RG : 0;
  const int ch = C == 1 ? 0 : wave / RG, f = C == 1 ? rg : wave;      // half of the columns; place among those that fetch a tile

  // ---- this workgroup's part of the line of units --------------------------------------------------------------------
  int64_t u, u_end, base, part_units;      // base: the first unit of request req
  int req, run_base, lead;                 // run_base: runs before request req
  {
    int64_t* const part = (int64_t*)smem_raw;
    int* const runs_of = (int*)(smem_raw + 64);
    int* const found = (int*)(smem_raw + 128);
    const int per = (p.n_req + 64 * W - 1) / (64 * W), r0 = min(tid * per, p.n_req), r1 = min(r0 + per, p.n_req);
    int64_t sum = 0;
    int runs = 0, b = 0, n = 0;
    for (int r = r0; r < r1; ++r) {
      run_units<Sh>(p, r, b, n);
      sum += (int64_t)b * n;
      runs += b;
    }
    int64_t scan = sum;
    int rscan = runs;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t x = __shfl_up(scan, d);
      const int y = __shfl_up(rscan, d);
      if (lane >= d) scan += x, rscan += y;
    }
    if (lane == 63) part[wave] = scan, runs_of[wave] = rscan;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int64_t total = 0;
    int total_runs = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < wave) scan += part[w], rscan += runs_of[w];
      total += part[w];
      total_runs += runs_of[w];
    }
    if (tid == 0) {
      if (!by_run) ws.runs[blockIdx.x].parts = 0;
      if (blockIdx.x == 0) *ws.count = by_run ? total_runs : kGroups;
    }
    total = uniform64(total);
    // a run costs as much as `lead` units beside its own (its queries, the first tiles' latency, its sums): they stand in front of
    // it in the line, but where there are few units a workgroup takes one
    lead = total <= kGroups ? 0 : kLead;
    total += (int64_t)lead * total_runs;
    part_units = (total + kGroups - 1) / kGroups;
    u = (int64_t)blockIdx.x * part_units;
    u_end = min(total, u + part_units);
    if (u >= u_end) return;
    sum += (int64_t)lead * runs;
    scan += (int64_t)lead * rscan - sum;
    rscan -= runs;
    if (sum > 0 && scan <= u && u < scan + sum) {
      for (int r = r0; r < r1; ++r) {
        if (per > 1) run_units<Sh>(p, r, b, n);
        const int64_t mine = (int64_t)b * (n + lead);
        if (u < scan + mine) {
          found[0] = r;
          found[1] = rscan;
          *(int64_t*)(found + 2) = scan;
          break;
        }
        scan += mine;
        rscan += b;
      }
    }
    __syncthreads();
    req = __builtin_amdgcn_readfirstlane(found[0]);
    if (req < 0) return;      // only where q_starts does not ascend
    run_base = __builtin_amdgcn_readfirstlane(found[1]);
    base = uniform64(*(int64_t*)(found + 2));
    __syncthreads();      // the tiles take the place
  }

  // ---- LDS places of operands ------------------------------------------------------------------------------------------
  lds_u8* const tiles = RAW ? smem + wave * Sh::LATENTS : smem + kg * NB * Sh::TILE;
  lds_u8* const raw = smem + 4 * Sh::LATENTS + wave * Sh::RING * Sh::RAW;      // RAW only
  lds_u8* const scale_area = smem + kScales + wave * 1024;                      // MX without RAW
  lds_f32* const stats = (lds_f32*)(smem + kStats);
  const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * 1.44269504088896341f;

  for (;;) {
    // ---- the next run, or what of it is in this part ---------------------------------------------------------------------
    int blocks, units;
    run_units<Sh>(p, req, blocks, units);
    blocks = __builtin_amdgcn_readfirstlane(blocks);
    units = __builtin_amdgcn_readfirstlane(units) + lead;
    if (u >= base + (int64_t)blocks * units) {      // also requests without queries
      base += (int64_t)blocks * units;
      run_base += blocks;
      if (++req == p.n_req) return;      // likewise
      continue;
    }
    const int block = __builtin_amdgcn_readfirstlane((int)divide(u - base, units));
    const int64_t run0 = base + (int64_t)block * units;
    const int a0 = max(0, __builtin_amdgcn_readfirstlane((int)(u - run0)) - lead);
    const int a1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)units, u_end - run0)) - lead;
    if (a1 <= 0) break;      // the part ends in front of the run's first unit
    const bool whole = a0 == 0 && a1 == units - lead;
    const int q0 = start_at(p.q_starts, req, p.n_tok), n = start_at(p.q_starts, req + 1, p.n_tok) - q0;
    const int keys = __builtin_amdgcn_readfirstlane(keys_of(p.kv_lens, req, p.max_blocks, p.block_shift));
    const int32_t* const table = p.table + (int64_t)req * p.table_stride;
    const float lift = Mma<T>::lift(keys);

    // The blocks of the halves of unit i's tile (past the last key: the last key's; without a key: any number), each in one block where
    // those are large enough: scalar loads, ahead of their use, which no copy is waited for with.  In smaller blocks lane r of
    // KEYS lanes looks up row r's when it is needed.  slot_of_row: lane r's row of the cache, -1 where there is no key.
    const bool large = (2 << p.block_shift) >= KEYS;
    const int64_t blocks_of = uniform64((int64_t)(keys > 0 ? table : p.kv_lens));
    const uint32_t last_key = (uint32_t)max(keys, 1) - 1u;
    auto position = [&](int i) { return (i * KG + kg) * KEYS + here(lane & (KEYS - 1)); };
    auto look = [&](int i, int half) {
      const uint32_t pos = min((uint32_t)((i * KG + kg) * KEYS + half * (KEYS / 2)), last_key);
      return __builtin_amdgcn_readfirstlane(((const __attribute__((address_space(4))) int32_t*)blocks_of)[pos >> p.block_shift]);
    };
    auto slot_of_row = [&](int lower, int upper, int i) {
      const int pos = position(i);
      int id = pos & (KEYS / 2) ? upper : lower;
      if (!large) id = here(((const __attribute__((address_space(1))) int32_t*)blocks_of)[min((uint32_t)pos, last_key) >> p.block_shift]);
      return id >= 0 && id < p.n_blocks && (uint32_t)pos < (uint32_t)keys ? (id << p.block_shift) + (pos & ((1 << p.block_shift) - 1)) : -1;
    };
    constexpr uint32_t ALL = KEYS == 32 ? 0xFFFFFFFFu : 0xFFFFu;
    auto keys_in = [&](int slot) { return (uint32_t)__ballot(slot >= 0) & ALL; };
    int lower = look(a0, 0), upper = look(a0, 1), lower1 = look(a0 + 1, 0), upper1 = look(a0 + 1, 1);      // of the next tile, of the one behind

    // this lane's queries
    const int64_t rows = (int64_t)n * p.n_heads, row0 = (int64_t)block * Sh::ROWS + Q * rg + col;
    int w_keys = 0, w_all = keys;      // and the keys that any, and that all, of this wavefront's queries see
    lds_u8* const queries = smem + kQueries + wave * (2048 * QL) + 16 * lane;
    s16x8 xq[G][QB - QL];      // of the columns in both products, and of the rope part
    constexpr auto in_lds = [](int s) { return s % 3 == 2 && s / 3 < QL; };
    constexpr auto in_regs = [](int s) { return s - min_of(QL, (s + 1) / 3); };      // place of a block among those in registers
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const bool real = row0 + 16 * g < rows;
      const int row = (int)min(row0 + 16 * g, rows - 1), token = row / p.n_heads, head = row - token * p.n_heads;
      const int seen = p.causal ? max(0, min(keys, keys - n + token + 1)) : keys;
      w_keys = max(w_keys, real ? seen : 0);
      w_all = min(w_all, real ? seen : keys);
      const uint16_t* src = p.q + (int64_t)(q0 + token) * p.q_stride + (int64_t)head * kQk;
#pragma unroll
      for (int s = 0; s < QB; ++s) {
        const int at = s < 16 / C ? 8 * block_chunk(C == 1 ? s : 8 * ch + s, grp) : kLat + 8 * rope_chunk(C == 1 ? s - 16 : ch, grp);
        const s16x8 v = *reinterpret_cast<const s16x8*>(src + at);
        if (in_lds(s)) *(__attribute__((address_space(3))) s16x8*)(queries + (s / 3) * 2048 + g * 1024) = signed_query<T>(v, p.scale);
        else xq[g][in_regs(s)] = v;
      }
    }
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) {
      w_keys = max(w_keys, __shfl_xor(w_keys, d));
      w_all = min(w_all, __shfl_xor(w_all, d));
    }
    w_keys = __builtin_amdgcn_readfirstlane(w_keys);
    w_all = __builtin_amdgcn_readfirstlane(w_all);
    // C = 2: wavefronts meet within a tile, so all take the same ones
    if (C == 2) w_keys = keys;
    // keys that all queries of the run see, where there are more
    int some = INT_MAX;
    if (p.causal) {
      const int t0 = (int)((int64_t)block * Sh::ROWS / p.n_heads);
      if (t0 < n - 1) some = __builtin_amdgcn_readfirstlane(max(0, keys - n + t0 + 1));
    }

    // keys that this lane's query g sees: needed in the last tiles only, so it is not kept
    auto seen_of = [&](int g) {
      const int64_t q_row = (int64_t)block * Sh::ROWS + Q * rg + 16 * g + here(tid & 15);
      return q_row >= rows ? 0 : p.causal ? max(0, min(keys, keys - n + (int)q_row / p.n_heads + 1)) : keys;
    };

    f32x4 o[G][BLOCKS] = {};
    float m[G], l[G];
    int first_key = INT_MAX;      // that this wavefront has met
#pragma unroll
    for (int g = 0; g < G; ++g) m[g] = -INFINITY, l[g] = 0.f;

    // ---- fetching a tile ---------------------------------------------------------------------------------------------
    uint32_t codes[MX && !RAW ? OWN : 1];
    mx_u32x4 ropes[MX && !RAW ? PIECES : 1];
    // 16-bit rows: straight into LDS, a row for each copy; rows without a key come from a row of zeros, so that 0 times them is 0.
    // Their rope rows do not matter: such keys' scores are replaced.  Codes wait in registers, or in LDS.
    auto fetch = [&](int slot, lds_u8* to) __attribute__((always_inline)) {
      const int lane = here(tid & 63);
      typedef const __attribute__((address_space(1))) void* global_ptr;
      int at_codes[4], at_rope[PIECES], at_scale = 0;      // all exchanges first
      if constexpr (RAW) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at_codes[i] = max(__shfl(slot, 4 * i + (lane >> 4)), 0);
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) at_rope[i] = max(__shfl(slot, 8 * ((f * PIECES + i) % (KEYS / 8)) + (lane >> 3)), 0);
      if constexpr (MX) at_scale = max(__shfl(slot, f * OWN + (lane & (OWN - 1))), 0);
      if constexpr (RAW) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_global_load_lds((global_ptr)(p.latent + (int64_t)at_codes[i] * (kLat / 2) + 16 * (lane & 15)),
                                           (lds_ptr)(to + 1024 * i), 16, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
          const int r = f * OWN + i, at = __builtin_amdgcn_readlane(slot, r);
          if constexpr (MX) {
            codes[i] = *reinterpret_cast<const uint32_t*>(p.latent + (int64_t)max(at, 0) * (kLat / 2) + 4 * lane);
          } else {
            const uint8_t* row = at < 0 ? reinterpret_cast<const uint8_t*>(zero_row) : p.latent + (int64_t)at * p.latent_bytes;
            __builtin_amdgcn_global_load_lds((global_ptr)(row + ((lane ^ swizzle(r)) << 4)), (lds_ptr)(to + r * 1024), 16, 0, 0);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if (f * PIECES + i >= KEYS / 8) break;
        const int r = 8 * (f * PIECES + i) + (lane >> 3);
        const uint8_t* src = p.rope + (int64_t)at_rope[i] * p.rope_bytes + (((lane & 7) ^ swizzle8(r)) << 4);
        if constexpr (MX && !RAW) ropes[i] = *reinterpret_cast<const mx_u32x4*>(src);
        else
          __builtin_amdgcn_global_load_lds((global_ptr)src, (lds_ptr)(to + (RAW ? 4096 : Sh::LATENTS) + 1024 * (f * PIECES + i)), 16, 0, 0);
      }
      if constexpr (MX)
        __builtin_amdgcn_global_load_lds((global_ptr)(p.scales + (int64_t)at_scale * (kLat / 32)),
                                         RAW ? (lds_ptr)(to + 6144) : (lds_ptr)scale_area, 16, 0, 0);
    };
    constexpr int COPIES = RAW ? 7 : OWN + PIECES;      // of a fetch into LDS
    // MX rows, later: 4-bit elements to 16-bit numbers, rounded where a scale takes them out of fp16's range.
    auto store = [&](uint32_t valid, const lds_u8* from, lds_u8* to) __attribute__((always_inline)) {
      if constexpr (MX) {
        const lds_u8* scales = RAW ? from + 6144 : scale_area;
        const int lane = here(tid & 63);
        if constexpr (!RAW) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the scales' copy
        uint32_t scale[OWN], word[OWN];
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
          scale[i] = scales[16 * i + (lane >> 2)];
          word[i] = RAW ? *(const lds_u32*)(from + 256 * i + 4 * lane) : codes[RAW ? 0 : i];
        }
        __builtin_amdgcn_sched_barrier(0);      // all reads first
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
          const int r = f * OWN + i;
          const uint32_t keep = 0u - (valid >> r & 1u);      // rows without a key: 0 times 2^-127
          // 2^(s - 127): 0 is the subnormal 2^-127, 255 NaN
          const uint32_t x = max(scale[i] << 23 | (scale[i] + 1u) >> 8 << 22, 0x400000u);
          const mx_u32x4 v = mx_values8<T>(word[i] & keep, __uint_as_float(x & keep));
          *(lds_u32x4*)(to + r * 1024 + ((lane ^ swizzle(r)) << 4)) = v;
        }
        if constexpr (!RAW) {
#pragma unroll
          for (int i = 0; i < PIECES; ++i)
            if (f * PIECES + i < KEYS / 8) *(lds_u32x4*)(to + Sh::LATENTS + 1024 * (f * PIECES + i) + 16 * lane) = ropes[i];
        }
      }
    };

    // ---- the products with a tile: latents at `at`, rope rows at `rope` ----------------------------------------------------
    auto use = [&](int j0, uint32_t valid, const lds_u8* at, const lds_u8* rope) __attribute__((always_inline)) {
      at += 512 * ch;
      if (valid != 0) first_key = min(first_key, j0 + __builtin_ctz(valid));
      // operands are read AHEAD in front of their products; the scheduler by itself would read each right before
      constexpr int U = KEYS / 16, NK = QB * U;
      // LDS places of operands.  K, block s: the lane group's chunk (block_chunk) of row col (+ 16); V^T, column block b of 16: chunks
      // 2 b and 2 b + 1 of rows vrow (+ 16).  A row's swizzle and the block change the same bits 4 .. 7 of a place in a tile,
      // which starts at a multiple of 256: a block is one exclusive or away.
      const int lane = here(tid & 63), col = lane & 15, grp = lane >> 4, vrow = 4 * grp + (col >> 2);
      const int at_k = col * 1024 + (grp >> 1) * 256 + (((grp & 1) * 4 ^ swizzle(col)) << 4);
      const int at_r = col * 128 + ((rope_chunk(ch, grp) ^ swizzle8(col)) << 4);
      auto key = [&](int k) {
        const int u = k % U, s = k / U;
        return s < 16 / C ? lds_operand(at + (at_k ^ (((s & 3) | (s & 4) << 1) << 4)) + (s >> 3) * 512 + u * 16 * 1024)
                          : lds_operand(rope + (at_r ^ ((s & 1) << 6)) + u * 16 * 128);
      };
      f32x4 s[G][2] = {};      // U = 1: two chains, an MFMA takes longer than its issue
      {
        s16x8 a[AHEAD_K], x[G];      // x: the queries' next block from LDS
        const lds_u8* from = smem + kQueries + wave * (2048 * QL) + 16 * lane;
        if constexpr (QL > 0) {
#pragma unroll
          for (int g = 0; g < G; ++g) x[g] = lds_operand(from + g * 1024);
        }
#pragma unroll
        for (int k = 0; k < AHEAD_K; ++k) a[k] = key(k);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          __builtin_amdgcn_sched_barrier(0);
          const int b = k / U;
#pragma unroll
          for (int g = 0; g < G; ++g) s[g][k & 1] = Mma<T>::mma(a[k % AHEAD_K], in_lds(b) ? x[g] : xq[g][in_regs(b)], s[g][k & 1]);
          if (k + AHEAD_K < NK) a[k % AHEAD_K] = key(k + AHEAD_K);
          if (in_lds(b) && in_lds(b + 3) && k % U == U - 1) {
#pragma unroll
            for (int g = 0; g < G; ++g) x[g] = lds_operand(from + (b / 3 + 1) * 2048 + g * 1024);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const int at_v = vrow * 1024 + ((((col & 3) >> 1) ^ swizzle(vrow)) << 4) + 8 * (col & 1);
      if constexpr (C == 2) {      // the sum of both halves is the same in both wavefronts, bit for bit
        lds_f32x4* mine = (lds_f32x4*)(smem + kScores) + wave * 256 + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[64 * i] = s[i >> 1][i & 1];
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const lds_f32x4* other = mine + (ch ? -256 * RG : 256 * RG);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i >> 1][i & 1] += other[64 * i];
      }
      if constexpr (U == 1) {
#pragma unroll
        for (int g = 0; g < G; ++g) s[g][0] += s[g][1];
      }
      if (valid != ALL || j0 + KEYS > w_all) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int seen = seen_of(g);
#pragma unroll
          for (int i = 0; i < 4 * U; ++i) {
            const int r = 16 * (i >> 2) + 4 * grp + (i & 3);
            if (!(valid >> r & 1u) || j0 + r >= seen) s[g][i >> 2][i & 3] = -INFINITY;
          }
        }
      }
      float top[G];
      bool rise = false;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        top[g] = s[g][0][0];
#pragma unroll
        for (int i = 1; i < 4 * U; ++i) top[g] = fmaxf(top[g], s[g][i >> 2][i & 3]);
        top[g] = fmaxf(top[g], lane_xor<16>(top[g]));
        top[g] = fmaxf(top[g], lane_xor<32>(top[g])) * c;
        rise = rise || top[g] > m[g] + kSlack;
      }
      if (__any(rise)) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float up = fmaxf(m[g], top[g]), back = m[g] == up ? 1.f : __builtin_amdgcn_exp2f(m[g] - up);
#pragma unroll
          for (int b = 0; b < BLOCKS; ++b) o[g][b] *= back;
          l[g] *= back;
          m[g] = up;
        }
      }
      float e[G][4 * U];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float ref = (m[g] == -INFINITY ? 0.f : m[g]) - lift;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * U; ++i) {
          e[g][i] = __builtin_amdgcn_exp2f(fmaf(s[g][i >> 2][i & 3], c, -ref));
          sum += e[g][i];
        }
        l[g] += sum;
      }
      if constexpr (U == 1) {
        s16x4 w[G], a[AHEAD];
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = Mma<T>::pack4(e[g]);
        auto value = [&](int b) { return lds_transposed(at + (at_v ^ ((b & 7) << 5)) + (b >> 3) * 256); };
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) a[b] = value(b);
#pragma unroll
        for (int b = 0; b < 32; ++b) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int g = 0; g < G; ++g) o[g][b] = Mma<T>::mma4(a[b % AHEAD], w[g], o[g][b]);
          if (b + AHEAD < 32) a[b % AHEAD] = value(b + AHEAD);
        }
      } else {
        s16x8 w[G], a[AHEAD];
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = Mma<T>::pack(e[g]);
        auto value = [&](int b) {
          const lds_u8* from = at + (at_v ^ ((b & 7) << 5)) + (b >> 3) * 256;
          return __builtin_shufflevector(lds_transposed(from), lds_transposed(from + 16 * 1024), 0, 1, 2, 3, 4, 5, 6, 7);
        };
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) a[b] = value(b);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int g = 0; g < G; ++g) o[g][b] = Mma<T>::mma(a[b % AHEAD], w[g], o[g][b]);
          if (b + AHEAD < BLOCKS) a[b % AHEAD] = value(b + AHEAD);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // A product takes the weight 0 of a key that a query does not see times its value, and NaN times 0 is NaN.  So where not all
    // of the run's queries see a key (j >= some), rows of a tile that are not finite are zeroed by the wavefront that fetched them, and
    // the queries that see such a key have NaN as their sum of weights.
    auto clear = [&](int j0, lds_u8* at) __attribute__((always_inline)) {
      uint32_t bad = 0;
      for (int r = max(f * OWN, some - j0); r < (f + 1) * OWN; ++r) {
        lds_u32x4* row16 = (lds_u32x4*)(at + r * 1024 + 16 * lane);
        const mx_u32x4 v = *row16;
        if (__any((not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w)) != 0)) {
          bad |= 1u << r;
          *row16 = mx_u32x4{0, 0, 0, 0};
        }
      }
      if constexpr (F > 1) {
        lds_u32* words = (lds_u32*)(smem + kWords);
        if (lane == 0) words[wave] = bad;
        tiles_ready();
        bad = 0;
#pragma unroll
        for (int g = 0; g < F; ++g) bad |= words[kg * F + g];
      }
      bad = __builtin_amdgcn_readfirstlane(bad);
      while (bad != 0) {
        const int r = __builtin_ctz(bad);
        bad &= bad - 1;
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (j0 + r < seen_of(g)) l[g] = NAN;
      }
    };

    // ---- the tiles -----------------------------------------------------------------------------------------------------
    // A fetch and the use of another tile stand in one function with pointers that do not meet: the compiler, which does not see
    // how the places alternate, would otherwise wait for all copies in front of every transposing read.
    int slot = slot_of_row(lower, upper, a0);
    lower = lower1, upper = upper1;
    if constexpr (RAW) {
      // every wavefront by itself, three tiles' rows on the way: a fetch is 7 copies, and what is younger than a tile's is known
      lower1 = look(a0 + 2, 0), upper1 = look(a0 + 2, 1);
      uint32_t valid[3] = {keys_in(slot), 0, 0};
      fetch(slot, raw);
      if (a0 + 1 < a1) {
        slot = slot_of_row(lower, upper, a0 + 1);
        valid[1] = keys_in(slot);
        fetch(slot, raw + Sh::RAW);
      }
      lower = look(a0 + 3, 0), upper = look(a0 + 3, 1);
      if (a0 + 2 < a1) {
        slot = slot_of_row(lower1, upper1, a0 + 2);
        valid[2] = keys_in(slot);
        fetch(slot, raw + 2 * Sh::RAW);
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int s = 0; s < QB - QL; ++s) xq[g][s] = signed_query<T>(xq[g][s], p.scale);      // waited for behind the first copies
      auto step = [&](int i, lds_u8* __restrict rows, lds_u8* __restrict at) __attribute__((always_inline)) {
        const int j0 = (i * KG + kg) * KEYS;
        if (j0 < w_keys) {
          store(valid[0], rows, at);
          if (j0 + KEYS > some) clear(j0, at);
          use(j0, valid[0], at, rows + 4096);
        }
        valid[0] = valid[1];
        valid[1] = valid[2];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the tile is read
        slot = slot_of_row(lower, upper, i + 3);
        lower = look(i + 4, 0), upper = look(i + 4, 1);
        if (i + 3 < a1) {
          valid[2] = keys_in(slot);
          fetch(slot, rows);
        }
      };
      int buf = 0;
      for (int i = a0; i < a1; ++i) {
        if (i + 2 < a1) asm volatile("s_waitcnt vmcnt(14) lgkmcnt(0)" ::: "memory");
        else if (i + 1 < a1) asm volatile("s_waitcnt vmcnt(7) lgkmcnt(0)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        step(i, raw + buf * Sh::RAW, tiles);
        buf = buf == 2 ? 0 : buf + 1;
      }
    } else if constexpr (KEYS == 16) {
      // every wavefront by itself: the next tile's copies go out before this one's are waited for
      static_assert(COPIES == 18, "the wait below");
      uint32_t valid = keys_in(slot);
      fetch(slot, tiles);
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int s = 0; s < QB - QL; ++s) xq[g][s] = signed_query<T>(xq[g][s], p.scale);      // waited for behind the first copies
      auto step = [&](int i, lds_u8* __restrict to, lds_u8* __restrict at) __attribute__((always_inline)) {
        uint32_t next = 0;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the tile before is read
        slot = slot_of_row(lower, upper, i + 1);
        lower = look(i + 2, 0), upper = look(i + 2, 1);
        if (i + 1 < a1) {
          next = keys_in(slot);
          fetch(slot, to);
          asm volatile("s_waitcnt vmcnt(18)" ::: "memory");
        } else {
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        const int j0 = (i * KG + kg) * KEYS;
        if (j0 + KEYS > some) clear(j0, at);
        if (j0 < w_keys) use(j0, valid, at, at + Sh::LATENTS);
        valid = next;
      };
      int buf = 0;
      for (int i = a0; i < a1; ++i, buf ^= 1) step(i, tiles + (buf ^ 1) * Sh::TILE, tiles + buf * Sh::TILE);
    } else {
      uint32_t valid = keys_in(slot), next = 0;
      fetch(slot, tiles);
      if constexpr (MX) {
        store(valid, nullptr, tiles);
        slot = slot_of_row(lower, upper, a0 + 1);
        lower = look(a0 + 2, 0), upper = look(a0 + 2, 1);
        if (a0 + 1 < a1) {
          next = keys_in(slot);
          fetch(slot, nullptr);
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int s = 0; s < QB - QL; ++s) xq[g][s] = signed_query<T>(xq[g][s], p.scale);      // waited for behind the first copies
      auto step = [&](int i, lds_u8* __restrict to, lds_u8* __restrict at) __attribute__((always_inline)) {
        const int j0 = (i * KG + kg) * KEYS;
        if ((i + 1) * Sh::UNIT > some) clear(j0, at);      // the same for all wavefronts
        if constexpr (MX) {
          if (j0 < w_keys) use(j0, valid, at, at + Sh::LATENTS);
          valid = next;
          if (i + 1 < a1) store(next, nullptr, to);
          slot = slot_of_row(lower, upper, i + 2);
          lower = look(i + 3, 0), upper = look(i + 3, 1);
          if (i + 2 < a1) {
            next = keys_in(slot);
            fetch(slot, nullptr);
          }
        } else {
          slot = slot_of_row(lower, upper, i + 1);
          lower = look(i + 2, 0), upper = look(i + 2, 1);
          if (i + 1 < a1) {
            next = keys_in(slot);
            fetch(slot, to);
          }
          if (j0 < w_keys) use(j0, valid, at, at + Sh::LATENTS);
          valid = next;
        }
      };
      int buf = 0;
      for (int i = a0; i < a1; ++i, buf ^= 1) {
        tiles_ready();
        step(i, tiles + (buf ^ 1) * Sh::TILE, tiles + buf * Sh::TILE);
      }
    }

    // ---- joining the key groups, and what leaves ---------------------------------------------------------------------------
    const int place = a0 == 0 ? 2 * (int)blockIdx.x + 1 : 2 * (int)blockIdx.x;
    const int lane = here(tid & 63), col = lane & 15, grp = lane >> 4;
    float top[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      l[g] += lane_xor<16>(l[g]);
      l[g] += lane_xor<32>(l[g]);
      if (__any(m[g] == -INFINITY) && m[g] == -INFINITY && l[g] == 0.f && first_key < seen_of(g)) l[g] = kNoScore;
      top[g] = m[g];
    }
    if constexpr (KG > 1) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (grp == 0) {
          stats[wave * 2 * Q + 16 * g + col] = m[g];
          stats[wave * 2 * Q + Q + 16 * g + col] = l[g];
        }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const lds_f32* st = stats + 16 * g + col;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < KG; ++k) top[g] = fmaxf(top[g], st[(k * RG + rg) * 2 * Q]);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const float mk = st[(k * RG + rg) * 2 * Q], lk = st[(k * RG + rg) * 2 * Q + Q];
          sum += mk == top[g] ? lk : lk * __builtin_amdgcn_exp2f(mk - top[g]);
        }
        l[g] = sum;
        const float back = m[g] == top[g] ? 1.f : __builtin_amdgcn_exp2f(m[g] - top[g]);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) o[g][b] *= back;
      }
    }
    float* sums = ws.sums + ((int64_t)place * RG + rg) * (Q * kLat) + 4 * lane;
    float* st = ws.stats + ((int64_t)place * RG + rg) * 2 * Q + col;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t q_row = here(Q * rg + 16 * g + col) + (int64_t)block * Sh::ROWS;
      const bool real = q_row < rows;
      const int row = (int)min(q_row, rows - 1), token = row / p.n_heads, head = row - token * p.n_heads;
      const float r = normaliser(l[g]);
      uint16_t* out = p.out + (int64_t)(q0 + token) * p.out_stride + (int64_t)head * kLat + 4 * grp;
      auto leave = [&](int b, f32x4 v) {      // columns 16 b + 4 grp ..
        if (whole) {
          if (real) {
            mx_u32x2 h;
            h.x = (uint32_t)T::from_f32(v.x * r) | ((uint32_t)T::from_f32(v.y * r) << 16);
            h.y = (uint32_t)T::from_f32(v.z * r) | ((uint32_t)T::from_f32(v.w * r) << 16);
            *reinterpret_cast<mx_u32x2*>(out + 16 * b) = h;
          }
        } else {
          *reinterpret_cast<f32x4*>(sums + (32 * g + b) * 256) = v;
        }
      };
      if constexpr (KG == 1) {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) leave(16 * ch + b, o[g][b]);
      } else {
        // 32 KB of every wavefront; each adds its share of its row group's
        constexpr int MINE = 32 / KG;
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 32; ++b) ((lds_f32x4*)smem)[(wave * 32 + b) * 64 + lane] = o[g][b % BLOCKS];
        __syncthreads();
#pragma unroll
        for (int b = 0; b < MINE; ++b) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KG; ++k) v += ((const lds_f32x4*)smem)[((k * RG + rg) * 32 + kg * MINE + b) * 64 + lane];
          leave(kg * MINE + b, v);
        }
      }
      if (kg == 0 && ch == 0 && grp == 0) {
        if (!whole) {
          st[16 * g] = top[g];
          st[Q + 16 * g] = l[g];
        } else if (real && p.lse) {
          p.lse[(int64_t)(q0 + token) * p.n_heads + head] =
              l[g] == 0.f ? -INFINITY : (top[g] - lift + __builtin_amdgcn_logf(l[g])) * 0.693147180559945309f;
        }
      }
    }
    if (a0 == 0 && tid == 0) {
      const int first = (int)blockIdx.x, at = by_run ? run_base + block : first;
      if ((unsigned)at < kGroups)       // always, where q_starts ascends
        ws.runs[at] = Run{whole ? 0 : (int)divide(run0 + units - 1, part_units) - first + 1, first, req, block};
    }
    u = run0 + lead + a1;
    if (u >= u_end) break;
    __syncthreads();          // the next run writes the tiles
  }
#endif
}

// The sums of a run that lies in several parts: a workgroup per row group and four KB of sums, four quarters of the parts side by
// side, each in one pass with a running maximum, as the parts themselves are made: nothing is loaded twice, and the loads hang on
// the run's record only (latency: 16 parts of one query group in 4 us where maxima, weights and sums were three passes: 5).
// Every sum goes in the order of the parts, so equal calls give equal bits.
template <typename T, int Q, int RG>
__global__ void __launch_bounds__(1024) latent_join_kernel(const LatentParams p, const Workspace ws) {
  __shared__ f32x4 part[3][256];
  __shared__ float stats[3][256][2];
  const int count = *ws.count;
  const Run run = ws.runs[blockIdx.x];
  if ((int)blockIdx.x >= count || run.parts <= 1) return;      // past count the record is of an earlier call
  const int tid = threadIdx.x, rg = (int)blockIdx.y / (Q / 2);
  auto place = [&](int k) { return (int64_t)(2 * (run.first + k) + (k == 0)) * RG + rg; };
  const int lane = tid & 63, k1 = (int)blockIdx.y % (Q / 2) * 4 + ((tid >> 6) & 3), quarter = tid >> 8;
  const int b = k1 & 31, col = 16 * (k1 >> 5) + (lane & 15), grp = lane >> 4;      // part k1: columns 16 b + 4 grp .. of query col
  const float* const src = ws.sums + (k1 * 64 + lane) * 4;
  const float* const st = ws.stats + col;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  auto add = [&](float mk, float lk, f32x4 v) {
    const float up = fmaxf(m, mk), x = m == up ? 1.f : __builtin_amdgcn_exp2f(m - up), y = mk == up ? 1.f : __builtin_amdgcn_exp2f(mk - up);
    acc = x * acc + y * v;
    l = x * l + y * lk;
    m = up;
  };
#pragma unroll 4
  for (int k = quarter; k < run.parts; k += 4)
    add(st[place(k) * 2 * Q], st[place(k) * 2 * Q + Q], *reinterpret_cast<const f32x4*>(src + place(k) * (Q * kLat)));
  if (quarter > 0) {
    part[quarter - 1][tid & 255] = acc;
    stats[quarter - 1][tid & 255][0] = m;
    stats[quarter - 1][tid & 255][1] = l;
  }
  __syncthreads();
  if (quarter > 0) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) add(stats[k][tid][0], stats[k][tid][1], part[k][tid]);
  const int q0 = start_at(p.q_starts, run.req, p.n_tok), n = start_at(p.q_starts, run.req + 1, p.n_tok) - q0;
  const int64_t row = (int64_t)run.block * (Q * RG) + Q * rg + col;
  if (row >= (int64_t)n * p.n_heads) return;
  const int token = (int)row / p.n_heads, head = (int)row - token * p.n_heads;
  const float r = normaliser(l);
  mx_u32x2 h;
  h.x = (uint32_t)T::from_f32(acc.x * r) | ((uint32_t)T::from_f32(acc.y * r) << 16);
  h.y = (uint32_t)T::from_f32(acc.z * r) | ((uint32_t)T::from_f32(acc.w * r) << 16);
  *reinterpret_cast<mx_u32x2*>(p.out + (int64_t)(q0 + token) * p.out_stride + (int64_t)head * kLat + 16 * b + 4 * grp) = h;
  const float lift = Mma<T>::lift(keys_of(p.kv_lens, run.req, p.max_blocks, p.block_shift));
  if (b == 0 && grp == 0 && p.lse)
    p.lse[(int64_t)(q0 + token) * p.n_heads + head] =
        l == 0.f ? -INFINITY : (m - lift + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

// Rows of a run, by those of an average request, `rows`, and by the batch's units of 16 rows and 64 positions of the block table
// (a wider table than the lengths need counts as long contexts).  4-bit rows go by the same rule, which was not measured for
// them.  Few units: the most workgroups and the least time until the first
// product, though a tile is fetched by many; many: tiles that all rows of a run share.  us, bf16, 16-bit rows, 64-slot blocks:
//   units (requests x rows, positions)          runs of 16      32      64     128 rows
//     256 (4 x 32, 2048)                            20.3    24.7    27.4    37.4
//    1024 (4 x 128, 2048)                           26.6    26.6    26.2    44.8
//    2048 (16 x 32, 4096)                           36.8    33.1    38.0    56.8
//    4096 (32 x 32, 4096)                           60.7    44.7    53.2    79.8
//    8192 (32 x 64, 4096)                           108     66.5    59.9    80.1
//    8192 (16 x 128, 4096)                          83.7    64.0    59.3    61.9
//   16384 (32 x 128, 4096)                          195     112     96.4    84.1
//    2048 (32 x 16, 4096)                           38.5    41.9    53.0    80.7
static int run_rows(int n_tok, int n_req, int n_heads, int64_t positions) {
  const int64_t reqs = std::max(n_req, 1), rows = ((int64_t)n_tok * n_heads + reqs - 1) / reqs;
  const int64_t units = reqs * ((rows + 15) / 16) * std::min<int64_t>((positions + 63) / 64, 8193);
  if (rows <= 16 || units <= 1024) return 16;
  if (rows <= 32) return 32;
  return rows <= 64 || units <= 8192 ? 64 : 128;
}

constexpr size_t kHead = 256, kRunBytes = (kGroups * sizeof(Run) + 255) & ~(size_t)255;
static size_t stats_bytes(int rows) { return (size_t)2 * kGroups * rows * 2 * 4; }

size_t latent_workspace_bytes(int n_tok, int n_req, int n_heads) {
  const int rows = run_rows(n_tok, n_req, n_heads, INT64_MAX - 63);      // the most that a table can ask for
  return kHead + kRunBytes + stats_bytes(rows) + (size_t)2 * kGroups * rows * kLat * 4;
}

template <typename T, bool MX, int Q, int RG>
static hipError_t launch_latent(const LatentParams& p, void* mem, hipStream_t s) {
  uint8_t* at = (uint8_t*)mem;
  const Workspace ws = {(int32_t*)at, (Run*)(at + kHead), (float*)(at + kHead + kRunBytes),
                        (float*)(at + kHead + kRunBytes + stats_bytes(Q * RG))};
  // every request has at most one run more than its share of the rows
  const int64_t rows = (int64_t)p.n_tok * p.n_heads, runs = std::min(rows / (Q * RG) + p.n_req, rows);
  const bool by_run = runs <= kGroups;
  hipError_t e = hipFuncSetAttribute((const void*)latent_kernel<T, MX, Q, RG>, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(latent_kernel<T, MX, Q, RG>), dim3(kGroups), dim3(64 * Shape<MX, Q, RG>::W), kLds, s, p, ws, by_run);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(latent_join_kernel<T, Q, RG>), dim3((unsigned)std::min<int64_t>(runs, kGroups), Q / 2 * RG), dim3(1024),
                     0, s, p, ws);
  return hipGetLastError();
}

template <typename T, bool MX>
static hipError_t launch_rows(const LatentParams& p, void* ws, hipStream_t s) {
  const int rows = run_rows(p.n_tok, p.n_req, p.n_heads, (int64_t)p.max_blocks << p.block_shift);
  return rows == 16   ? launch_latent<T, MX, 16, 1>(p, ws, s)
         : rows == 32 ? launch_latent<T, MX, 16, 2>(p, ws, s)
         : rows == 64 ? launch_latent<T, MX, 16, 4>(p, ws, s)
                      : launch_latent<T, MX, 32, 4>(p, ws, s);
}

hipError_t launch_latent_attention(const LatentParams& p, int dtype, int fmt, void* ws, hipStream_t s) {
  if (dtype == GALE_F16) return fmt ? launch_rows<F16, true>(p, ws, s) : launch_rows<F16, false>(p, ws, s);
  return fmt ? launch_rows<BF16, true>(p, ws, s) : launch_rows<BF16, false>(p, ws, s);
}

}  // namespace gale
