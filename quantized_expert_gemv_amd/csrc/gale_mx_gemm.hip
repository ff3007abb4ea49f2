// Products of MX numbers: y = A . W^T (+ add), A in 4 or 8 bits, W in 4 bits, on the scaled MFMA.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128 columns and applies one power-of-two scale per
// row and 32 columns: an MX block is exactly one lane's share of an operand, and its scale byte that lane's scale.
// Operand layouts (measured with one-hot operands): lane l serves row l % 16; with g = l / 16, 4-bit elements are
// columns 32 g .. 32 g + 31, 8-bit ones columns 16 g .. 16 g + 15 and 64 + 16 g .. 64 + 16 g + 15; the scale of lane group g
// is that of columns 32 g .. 32 g + 31 for either width.  Result register r of lane l is (row 4 g + r of the first
// operand, row l % 16 of the second).  W is the first operand, so a lane holds four consecutive columns of y.
//
// The sums inside the instruction, measured on gfx950 with constructed operands: the products of each eight
// consecutive columns are cut (towards zero) to multiples of 2^(e - 13), e the largest sum of two elements' exponents (without
// the carry of the mantissas' product: 3.75 x 6 = 22.5 has e = 1 + 2); the sums of the eights, scaled, and the accumulator
// add like fp32 numbers.  Products of two 4-bit elements are multiples of 2^-2 with e <= 4 and never cut.  Those of an 8-bit and a
// 4-bit element go from 2^-10 to 448 x 6 with e = 10 and are: so the 8-bit operand is split at magnitude 4 into two,
// which are multiplied one after the other.  The upper part's products are multiples of 2^-2 with e <= 10 (cut at 2^-3), the
// lower part's multiples of 2^-10 with e <= 3 (cut at 2^-10): both whole.
//
// Buffer loads: the range check covers the vector and the scalar offset together (measured inside one allocation), and a
// load past the range gives zeros, in registers and in LDS.  So rows behind the last one need no masks.
#include "gale_mx.h"

namespace gale {

typedef int v8i __attribute__((ext_vector_type(8)));

struct MxGemmParams {
  int m, n, groups;          // groups: 128-column groups of a row
  const uint8_t* a;
  const uint8_t* as;
  const uint8_t* w;
  const uint8_t* ws;
  const void* add;           // NULL: none
  int64_t add_stride;
  void* y;
  int64_t y_stride;
  bool wide, wide8;          // rows of y and add are aligned for four columns, for 16 bytes at a time
};

// Format codes of the MFMA: 0 for E4M3, 4 for E2M1.

// The elements of an 8-bit operand of magnitude 4 and more (codes from 0x48), and the others; zero elsewhere.
__device__ __forceinline__ void mx_split8(const v8i& v, v8i& hi, v8i& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = (uint32_t)v[i];
    const uint32_t ge = (((x & 0x7F7F7F7Fu) + 0x38383838u) >> 7) & 0x01010101u;   // 1 in each byte from 0x48
    const uint32_t mask = (ge << 8) - ge;                                         // 255 in those bytes
    hi[i] = (int)(x & mask);
    lo[i] = (int)(x & ~mask);
  }
}

// acc += (16 rows of W) . (16 rows of A)^T over one group of 128 columns.
template <int FMT>
__device__ __forceinline__ f32x4 mx_mfma(const v8i& w, int w_scale, const v8i& a, int a_scale, f32x4 acc) {
  if constexpr (FMT == GALE_MX_E2M1) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc, 4, 4, 0, w_scale, 0, a_scale);
  } else {
    v8i hi, lo;
    mx_split8(a, hi, lo);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, lo, acc, 4, 0, 0, w_scale, 0, a_scale);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, hi, acc, 4, 0, 0, w_scale, 0, a_scale);
  }
}

// Four consecutive columns n0 .. n0 + 3 of row i of y, as far as they exist.  p.wide: y and add take them in one access.
template <typename T>
__device__ __forceinline__ void mx_store4(const MxGemmParams& p, int i, int n0, float a0, float a1, float a2, float a3) {
  typedef typename T::bits bits;
  typedef bits bits4 __attribute__((ext_vector_type(4)));
  float v[4] = {a0, a1, a2, a3};
  bits* y = (bits*)p.y + (int64_t)i * p.y_stride + n0;
  const bits* c = (const bits*)p.add + (int64_t)i * p.add_stride + n0;
  if (p.wide && n0 + 4 <= p.n) {
    if (p.add) {
      const bits4 u = *reinterpret_cast<const bits4*>(c);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += T::to_f32(u[r]);
    }
    bits4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = T::from_f32(v[r]);
    *reinterpret_cast<bits4*>(y) = o;
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n0 + r < p.n) y[r] = T::from_f32(p.add ? v[r] + T::to_f32(c[r]) : v[r]);
  }
}

// ---------------------------------------------------------------------------
// Streaming kernel, for few rows of A
// ---------------------------------------------------------------------------
// Bound by reading W once.  A workgroup owns 16 rows of W (16 columns of y) and up to 16 MT rows of A; its wavefronts split
// the row's 128-column groups into consecutive runs and take them four at a time: the loads of four groups (of W from
// HBM, of A from the caches) and their scales (16 bytes of a row: one load) are issued a turn ahead of their products.
// The partial sums meet in LDS in wavefront order.
constexpr int kFar = 0x7FFFFFF0;      // an offset past every buffer: such a load gives 0 and reads nothing

template <int FMT, int MT>
struct StreamTurn {
  mx_u32x4 w[4], a[4][MT][FMT == GALE_MX_E2M1 ? 1 : 2], ws, as[MT];
};

template <typename T, int FMT, int MT>
__global__ void __launch_bounds__(512) mx_gemm_stream_kernel(const MxGemmParams p, int per_wave) {
#if defined(__HIP_DEVICE_COMPILE__)   // buffer resources are a device type: the host pass needs the kernel's name only
  __shared__ f32x4 part[8][MT][64];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), waves = (int)blockDim.x >> 6;
  const int n0 = (int)blockIdx.x * 16, m0 = (int)blockIdx.y * 16 * MT;
  const int a_pitch = p.groups * (FMT == GALE_MX_E2M1 ? 64 : 128), w_pitch = p.groups * 64, s_pitch = p.groups * 4;
  const int am = min(16 * MT, p.m - m0), wn = min(16, p.n - n0);        // rows that exist: others read as zero
  const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + (size_t)m0 * a_pitch), 0, am * a_pitch, 0x00020000);
  const auto rw = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + (size_t)n0 * w_pitch), 0, wn * w_pitch, 0x00020000);
  const auto rsa = __builtin_amdgcn_make_buffer_rsrc((void*)(p.as + (size_t)m0 * s_pitch), 0, am * s_pitch, 0x00020000);
  const auto rsw = __builtin_amdgcn_make_buffer_rsrc((void*)(p.ws + (size_t)n0 * s_pitch), 0, wn * s_pitch, 0x00020000);
  const int g0 = wave * per_wave, g1 = min(p.groups, g0 + per_wave);
  const int va = r * a_pitch + 16 * g, vw = r * w_pitch + 16 * g, vs = r * s_pitch;
  auto load = [&](int k, StreamTurn<FMT, MT>& t) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = k + j < g1;      // groups behind the run read as zero, whatever lies there
      t.w[j] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? vw : kFar, (k + j) * 64, 0);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if constexpr (FMT == GALE_MX_E2M1) {
          t.a[j][i][0] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? va + i * 16 * a_pitch : kFar, (k + j) * 64, 0);
        } else {
          t.a[j][i][0] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? va + i * 16 * a_pitch : kFar, (k + j) * 128, 0);
          t.a[j][i][1] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? va + i * 16 * a_pitch + 64 : kFar, (k + j) * 128, 0);
        }
    }
    t.ws = __builtin_amdgcn_raw_buffer_load_b128(rsw, vs, k * 4, 0);
#pragma unroll
    for (int i = 0; i < MT; ++i) t.as[i] = __builtin_amdgcn_raw_buffer_load_b128(rsa, vs + i * 16 * s_pitch, k * 4, 0);
  };
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  StreamTurn<FMT, MT> cur;
  load(g0, cur);
  for (int k = g0; k < g1; k += 4) {
    StreamTurn<FMT, MT> next;
    load(k + 4, next);                 // behind the run: nothing is read
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const v8i w = {(int)cur.w[j].x, (int)cur.w[j].y, (int)cur.w[j].z, (int)cur.w[j].w, 0, 0, 0, 0};
      const bool in = k + j < g1;      // the scales of the next run's groups, or of the next row, do not count
      const int sw = in ? (int)(cur.ws[j] >> (8 * g)) : 0;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int sa = in ? (int)(cur.as[i][j] >> (8 * g)) : 0;
        v8i a = {(int)cur.a[j][i][0].x, (int)cur.a[j][i][0].y, (int)cur.a[j][i][0].z, (int)cur.a[j][i][0].w, 0, 0, 0, 0};
        if constexpr (FMT == GALE_MX_E4M3) {
          a[4] = (int)cur.a[j][i][1].x;
          a[5] = (int)cur.a[j][i][1].y;
          a[6] = (int)cur.a[j][i][1].z;
          a[7] = (int)cur.a[j][i][1].w;
        }
        acc[i] = mx_mfma<FMT>(w, sw, a, sa, acc[i]);
      }
    }
    cur = next;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int x = (int)threadIdx.x; x < MT * 64; x += (int)blockDim.x) {
    const int i = x >> 6, l = x & 63;
    f32x4 v = part[0][i][l];
    for (int o = 1; o < waves; ++o) v += part[o][i][l];
    const int row = m0 + 16 * i + (l & 15), col = n0 + 4 * (l >> 4);
    if (row < p.m && col < p.n) mx_store4<T>(p, row, col, v[0], v[1], v[2], v[3]);
  }
#endif
}

template <typename T, int FMT, int MT>
static hipError_t launch_stream(const MxGemmParams& p, hipStream_t s) {
  // a wavefront gets at least one turn of four groups
  const int waves = std::min(8, (p.groups + 3) / 4);
  hipLaunchKernelGGL(HIP_KERNEL_NAME(mx_gemm_stream_kernel<T, FMT, MT>), dim3((p.n + 15) / 16, (p.m + 16 * MT - 1) / (16 * MT)),
                     dim3(64 * waves), 0, s, p, (p.groups + waves - 1) / waves);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tile kernel
// ---------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_byte;

// A stage of the tile kernel is 256 columns: 8 blocks per row, four v_mfma_scale_f32_32x32x64 steps.  Lane l of a step serves
// row l % 32 and half h = l / 32: its 4-bit elements are one block, its 8-bit ones 16 columns of either of the
// instruction's two blocks.  Which 64 columns a step takes is free as long as both operands agree: step s takes blocks s and
// 4 + s, so the four scales of a lane's steps are four neighbouring bytes, 4 h + s, one register per row and
// stage whose byte s the instruction selects.

// Rows of a stage in LDS are 128 (4-bit) or 256 bytes, in 16-byte chunks.  A ds_read_b128 serves 16 lanes at a time from
// 64 banks (256 bytes), here the same chunk c of 16 rows: it sits at place c ^ (r / 2 % 8) of row r (two rows span the
// banks), or at c ^ (r % 16) of an 8-bit row, and the 16 places are apart.  (With c ^ (r % 8) the counters showed
// a conflict in every read.)
template <int FMT>
__device__ __forceinline__ int stage_swizzle(int row) { return FMT == GALE_MX_E2M1 ? (row >> 1) & 7 : row & 15; }

template <int FMT>
__device__ __forceinline__ v8i stage_operand(const lds_byte* row, int swz, int h, int s) {
  if constexpr (FMT == GALE_MX_E2M1) {
    const mx_u32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) mx_u32x4*>(row + 16 * ((4 * h + s) ^ swz));
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  } else {
    const mx_u32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) mx_u32x4*>(row + 16 * ((2 * s + h) ^ swz));
    const mx_u32x4 u = *reinterpret_cast<const __attribute__((address_space(3))) mx_u32x4*>(row + 16 * ((8 + 2 * s + h) ^ swz));
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, (int)u.x, (int)u.y, (int)u.z, (int)u.w};
  }
}

template <int FMT, int S>
__device__ __forceinline__ f32x16 stage_mfma(const v8i& w, int w_scale, const v8i& a, int a_scale, f32x16 acc) {
  if constexpr (FMT == GALE_MX_E2M1) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, acc, 4, 4, S, w_scale, S, a_scale);
  } else {
    v8i hi, lo;
    mx_split8(a, hi, lo);
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, lo, acc, 4, 0, S, w_scale, S, a_scale);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, hi, acc, 4, 0, S, w_scale, S, a_scale);
  }
}

template <int FMT, int WM, int WN, int TM, int TN>
struct TileShape {
  static constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN, WAVES = WM * WN;
  static constexpr int AB = FMT == GALE_MX_E2M1 ? 128 : 256;     // bytes of a stage's row of A
  static constexpr int IA = BM * AB / 1024 / WAVES, IW = BN * 128 / 1024 / WAVES;  // 1 KB copies per wavefront and stage
  static constexpr int STAGE = BM * AB + BN * 128;
  static constexpr int SCALES = (BM + BN) * 32;        // scale bytes of four stages
  static constexpr int LDS = 2 * STAGE + 2 * SCALES;
  static constexpr int READS = TM * (AB / 128) + TN, MFMAS = TM * TN;   // ds_read_b128 and MFMA of a step
  static constexpr int RPM = READS > MFMAS ? 2 : 1, MPR = READS > MFMAS ? 1 : MFMAS / READS;   // how they alternate
};

// WM x WN wavefronts, each TM x TN tiles of 32 x 32.
template <typename T, int FMT, int WM, int WN, int TM, int TN>
__global__ void __launch_bounds__(64 * WM * WN, 1) mx_gemm_tile_kernel(const MxGemmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)   // buffer resources are a device type: the host pass needs the kernel's name only
  typedef TileShape<FMT, WM, WN, TM, TN> Sh;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem_raw[];
  lds_byte* smem = (lds_byte*)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;

  // Workgroup -> tile.  Workgroups go round robin over the 8 XCDs: each XCD gets a contiguous run of tiles, and a run
  // walks panels of four tile rows column by column, so the ~32 tiles that an XCD works on at once share few
  // rows of A and W in its L2.
  const int mt = (p.m + Sh::BM - 1) / Sh::BM, nt = (p.n + Sh::BN - 1) / Sh::BN;
  const int total = mt * nt, per = total >> 3, rest = total & 7;
  const int xcd = blockIdx.x & 7, in = blockIdx.x >> 3;
  const int t = xcd * per + min(xcd, rest) + in;
  const int panel = t / (4 * nt), left = t - panel * 4 * nt;
  const int ph = min(4, mt - 4 * panel);
  const int tn = left / ph, tm = 4 * panel + left - tn * ph;
  const int m0 = tm * Sh::BM, n0 = tn * Sh::BN;

  const int a_pitch = p.groups * (FMT == GALE_MX_E2M1 ? 64 : 128), w_pitch = p.groups * 64, s_pitch = p.groups * 4;
  const int am = min(Sh::BM, p.m - m0), wnr = min(Sh::BN, p.n - n0);   // rows that exist: others read as zero
  const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + (size_t)m0 * a_pitch), 0, am * a_pitch, 0x00020000);
  const auto rw = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + (size_t)n0 * w_pitch), 0, wnr * w_pitch, 0x00020000);
  const auto rsa = __builtin_amdgcn_make_buffer_rsrc((void*)(p.as + (size_t)m0 * s_pitch), 0, am * s_pitch, 0x00020000);
  const auto rsw = __builtin_amdgcn_make_buffer_rsrc((void*)(p.ws + (size_t)n0 * s_pitch), 0, wnr * s_pitch, 0x00020000);

  // copies: 1 KB of consecutive LDS places, lane l the place 16 l
  constexpr int AC = Sh::AB / 16, AR = 64 / AC;      // chunks per row of A, rows per copy
  constexpr int AV = 16 / AR;                        // copies until the swizzle of rows repeats
  static_assert(Sh::IA % AV == 0 && Sh::IW % 2 == 0, "a wavefront's copies start where the swizzle starts");
  int va[AV], vw[2];
#pragma unroll
  for (int o = 0; o < AV; ++o)
    va[o] = (lane / AC) * a_pitch + 16 * ((lane % AC) ^ stage_swizzle<FMT>(lane / AC + AR * o));
#pragma unroll
  for (int o = 0; o < 2; ++o)
    vw[o] = (lane >> 3) * w_pitch + 16 * ((lane & 7) ^ stage_swizzle<GALE_MX_E2M1>((lane >> 3) + 8 * o));
  // chunks behind the row's last group (the second half of an odd last stage) come from nowhere: the next row's codes
  // could be NaN
  bool ha[AV], hw[2];
#pragma unroll
  for (int o = 0; o < AV; ++o) ha[o] = ((lane % AC) ^ stage_swizzle<FMT>(lane / AC + AR * o)) >= AC / 2;
#pragma unroll
  for (int o = 0; o < 2; ++o) hw[o] = ((lane & 7) ^ stage_swizzle<GALE_MX_E2M1>((lane >> 3) + 8 * o)) >= 4;
  auto copy_stage = [&](int stage, int buf) {
    const bool half = 2 * stage + 1 == p.groups;
    lds_byte* la = smem + buf * Sh::STAGE + wave * Sh::IA * 1024;
    lds_byte* lw = smem + buf * Sh::STAGE + Sh::BM * Sh::AB + wave * Sh::IW * 1024;
#pragma unroll
    for (int i = 0; i < Sh::IA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (__attribute__((address_space(3))) void*)(la + i * 1024), 16,
                                               half && ha[i % AV] ? kFar : va[i % AV],
                                               stage * Sh::AB + (wave * Sh::IA + i) * AR * a_pitch, 0, 0);
#pragma unroll
    for (int i = 0; i < Sh::IW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (__attribute__((address_space(3))) void*)(lw + i * 1024), 16,
                                               half && hw[i & 1] ? kFar : vw[i & 1],
                                               stage * 128 + (wave * Sh::IW + i) * 8 * w_pitch, 0, 0);
  };
  // Scales, 32 bytes per row for four stages, also through LDS: from the registers' side every wavefront would ask the
  // L1 for all its rows, 40 such loads of 32 lines each per workgroup and four stages (128 x 256) where 12 do, next to 256
  // copies of 8 lines.
  const int stages = (p.groups + 1) >> 1;
  const int vs = (lane >> 1) * s_pitch + 16 * (lane & 1);
  auto copy_scales = [&](int four, int half) {
    lds_byte* ls = smem + 2 * Sh::STAGE + half * Sh::SCALES;
#pragma unroll
    for (int k = 0; k < (Sh::BM / 32 + Sh::WAVES - 1) / Sh::WAVES; ++k) {
      const int i = (wave + k * Sh::WAVES) % (Sh::BM / 32);       // too many wavefronts copy some rows twice
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (__attribute__((address_space(3))) void*)(ls + i * 1024), 16, vs,
                                               four * 32 + i * 32 * s_pitch, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < (Sh::BN / 32 + Sh::WAVES - 1) / Sh::WAVES; ++k) {
      const int i = (wave + k * Sh::WAVES) % (Sh::BN / 32);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsw, (__attribute__((address_space(3))) void*)(ls + Sh::BM * 32 + i * 1024), 16,
                                               vs, four * 32 + i * 32 * s_pitch, 0, 0);
    }
  };
  int sa[TM], sw[TN], sa_next[TM], sw_next[TN];      // of this stage and the next
  auto read_scales = [&](int half, int u) {
    const lds_byte* la = smem + 2 * Sh::STAGE + half * Sh::SCALES + (wm * 32 * TM + r) * 32 + 8 * u + 4 * h;
    const lds_byte* lw = smem + 2 * Sh::STAGE + half * Sh::SCALES + Sh::BM * 32 + (wn * 32 * TN + r) * 32 + 8 * u + 4 * h;
#pragma unroll
    for (int i = 0; i < TM; ++i) sa_next[i] = *reinterpret_cast<const __attribute__((address_space(3))) int*>(la + i * 1024);
#pragma unroll
    for (int i = 0; i < TN; ++i) sw_next[i] = *reinterpret_cast<const __attribute__((address_space(3))) int*>(lw + i * 1024);
  };
  // What lies behind the row's last block gets scales of 0 (2^-127) on both sides, which make its products vanish: the
  // second half of a last stage of 128 columns, and the stages that fill up the last four.
  auto take_scales = [&](int stage) {
    const bool there = 2 * stage + h < p.groups;
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = there ? sa_next[i] : 0;
#pragma unroll
    for (int i = 0; i < TN; ++i) sw[i] = there ? sw_next[i] : 0;
  };
  const int swz_a = stage_swizzle<FMT>(r), swz_w = stage_swizzle<GALE_MX_E2M1>(r);
  auto read_step = [&](int buf, int s, v8i a[TM], v8i w[TN]) {
    const lds_byte* la = smem + buf * Sh::STAGE + (wm * 32 * TM + r) * Sh::AB;
    const lds_byte* lw = smem + buf * Sh::STAGE + Sh::BM * Sh::AB + (wn * 32 * TN + r) * 128;
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = stage_operand<FMT>(la + i * 32 * Sh::AB, swz_a, h, s);
#pragma unroll
    for (int i = 0; i < TN; ++i) w[i] = stage_operand<GALE_MX_E2M1>(lw + i * 32 * 128, swz_w, h, s);
  };

  copy_stage(0, 0);
  copy_scales(0, 0);
  copy_stage(min(1, stages - 1), 1);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;

  v8i a0[TM], w0[TN], a1[TM], w1[TN];
#define MX_STEP(S, A, W)                                                                                       \
  _Pragma("unroll") for (int i = 0; i < TM; ++i) _Pragma("unroll") for (int j = 0; j < TN; ++j) acc[i][j] =    \
      stage_mfma<FMT, S>(W[j], sw[j], A[i], sa[i], acc[i][j]);
#define MX_SPREAD                                                                                  \
  _Pragma("unroll") for (int i = 0; i < Sh::READS / Sh::RPM; ++i) {                                \
    __builtin_amdgcn_sched_group_barrier(0x100, Sh::RPM, 0);                                       \
    __builtin_amdgcn_sched_group_barrier(0x008, Sh::MPR, 0);                                       \
  }                                                                                                \
  __builtin_amdgcn_sched_barrier(0)

  static_assert(Sh::IA + Sh::IW <= 15, "the wait counts below");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (Sh::IA + Sh::IW));   // all but the second stage's copies have landed
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  read_scales(0, 0);
  read_step(0, 0, a0, w0);
  // The operands of a step are read from LDS during the products of the step before it; the fences keep the steps
  // apart and the groups spread each step's reads over its products.
  // Four stages per turn, without a branch: MFMAs are free to sink past one, and the schedule with them.
  for (int four = 0; 4 * four < stages; ++four) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int buf = u & 1;
      if (u == 2) copy_scales(four + 1, (four + 1) & 1);   // past the end: bytes that nothing takes
      take_scales(4 * four + u);
      __builtin_amdgcn_sched_barrier(0);
      read_step(buf, 1, a1, w1);
      MX_STEP(0, a0, w0);
      MX_SPREAD;
      read_step(buf, 2, a0, w0);
      MX_STEP(1, a1, w1);
      MX_SPREAD;
      read_step(buf, 3, a1, w1);
      MX_STEP(2, a0, w0);
      MX_SPREAD;
      // every wavefront has read its share of this stage, and its copies of the next one have landed
      __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      read_scales(u == 3 ? (four + 1) & 1 : four & 1, (u + 1) & 3);
      read_step(buf ^ 1, 0, a0, w0);
      copy_stage(min(4 * four + u + 2, stages - 1), buf);   // past the end: the last stage again
      MX_STEP(3, a1, w1);
#pragma unroll
      for (int i = 0; i < Sh::MFMAS / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, (2 * (Sh::READS + TM + TN) + Sh::MFMAS - 1) / Sh::MFMAS, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < Sh::MFMAS / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x020, 2 * (Sh::IA + Sh::IW) / Sh::MFMAS, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);     // no copy is in flight when the workgroup's LDS goes
#undef MX_STEP
#undef MX_SPREAD

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));   // no MFMA moves into the branches below
  // Out through LDS, 16 rows of the wavefront at a time, so that eight columns of a row leave in one or two 16-byte
  // stores and 4 rows fill whole lines.  (Straight from the registers a store touches 32 rows with 16 bytes each.)
  __syncthreads();
  constexpr int OC = 32 * TN, OP = OC * 4 + 16;     // columns and padded bytes of a row
  lds_byte* lo = smem + wave * 16 * OP;
  const int lpr = OC / 8;                           // lanes per row on the way out
  const int orow = lane / lpr, oc = lane % lpr * 8;
#pragma unroll
  for (int i = 0; i < 2 * TM; ++i) {
    if ((r >> 4) == (i & 1)) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x16& c = acc[i >> 1][j];
          *reinterpret_cast<__attribute__((address_space(3))) f32x4*>(lo + (r & 15) * OP + (32 * j + 8 * k + 4 * h) * 4) =
              f32x4{c[4 * k], c[4 * k + 1], c[4 * k + 2], c[4 * k + 3]};
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int o = 0; o < 16 * lpr / 64; ++o) {
      const int row16 = o * (64 / lpr) + orow;
      const int row = m0 + wm * 32 * TM + i * 16 + row16, col = n0 + wn * 32 * TN + oc;
      float v[8];
      const f32x4 v0 = *reinterpret_cast<const __attribute__((address_space(3))) f32x4*>(lo + row16 * OP + oc * 4);
      const f32x4 v1 = *reinterpret_cast<const __attribute__((address_space(3))) f32x4*>(lo + row16 * OP + oc * 4 + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = v0[e];
        v[4 + e] = v1[e];
      }
      if (row < p.m && col < p.n) {
        typedef typename T::bits bits;
        if (p.add) {
          float c[8];
          load8<T>((const bits*)p.add + (int64_t)row * p.add_stride, col, p.n, p.wide8, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += c[e];
        }
        store8<T>((bits*)p.y + (int64_t)row * p.y_stride, col, p.n, p.wide8, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
#endif
}

template <typename T, int FMT, int WM, int WN, int TM, int TN>
static hipError_t launch_tile(const MxGemmParams& p, hipStream_t s) {
  typedef TileShape<FMT, WM, WN, TM, TN> Sh;
  const int64_t tiles = (int64_t)((p.m + Sh::BM - 1) / Sh::BM) * ((p.n + Sh::BN - 1) / Sh::BN);
  auto kern = mx_gemm_tile_kernel<T, FMT, WM, WN, TM, TN>;
  const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, Sh::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(64 * Sh::WAVES), Sh::LDS, s, p);
  return hipGetLastError();
}

// Time of a tile shape in microseconds, fitted to K = 4096 (16 stages) and N = 4096 at M = 64 .. 4096: about 6 to start and
// end a round of resident tiles; per tile and 16 stages 4.5e-4 per result (12e-4 with 8-bit A in its two parts) and
// 0.02 per 128 bytes of its rows.  With it, M = 128 / 512 / 1024 / 2048 / 4096 in 4 bits take 8 / 11 / 16 / 30 / 45 us, against
// 28 / 31 / 33 / 37 / 47 us in 256 x 256 tiles throughout and 8 / 11 / 22 / 43 / 84 us in 64 x 64.
template <int FMT, int WM, int WN, int TM, int TN>
static float tile_cost(const MxGemmParams& p, int cus) {
  typedef TileShape<FMT, WM, WN, TM, TN> Sh;
  const int64_t tiles = (int64_t)((p.m + Sh::BM - 1) / Sh::BM) * ((p.n + Sh::BN - 1) / Sh::BN);
  const int resident = std::min(3, (160 * 1024) / Sh::LDS);
  const float per_result = FMT == GALE_MX_E2M1 ? 4.5e-4f : 12e-4f;
  const float turns = (float)((p.groups + 7) / 8) / 4;       // of 16 stages: whole turns of four
  const float tile = turns * (per_result * Sh::BM * Sh::BN + 0.02f * (Sh::BM * Sh::AB / 128 + Sh::BN));
  const int64_t per_cu = (tiles + cus - 1) / cus;
  return 6.f * (float)((per_cu + resident - 1) / resident) + tile * (float)per_cu;
}

template <typename T, int FMT>
static hipError_t launch_best_tile(const MxGemmParams& p, hipStream_t s) {
  const int cus = device_cu_count();
  float best = 1e30f;
  hipError_t (*run)(const MxGemmParams&, hipStream_t) = nullptr;
  auto offer = [&](float cost, hipError_t (*f)(const MxGemmParams&, hipStream_t)) {
    if (cost < best) {
      best = cost;
      run = f;
    }
  };
  if constexpr (FMT == GALE_MX_E2M1) {
    offer(tile_cost<FMT, 4, 2, 2, 4>(p, cus), launch_tile<T, FMT, 4, 2, 2, 4>);   // 256 x 256
    offer(tile_cost<FMT, 2, 2, 2, 4>(p, cus), launch_tile<T, FMT, 2, 2, 2, 4>);   // 128 x 256
  } else {
    offer(tile_cost<FMT, 4, 2, 1, 4>(p, cus), launch_tile<T, FMT, 4, 2, 1, 4>);   // 128 x 256
  }
  offer(tile_cost<FMT, 2, 2, 2, 2>(p, cus), launch_tile<T, FMT, 2, 2, 2, 2>);     // 128 x 128
  offer(tile_cost<FMT, 2, 2, 1, 2>(p, cus), launch_tile<T, FMT, 2, 2, 1, 2>);     // 64 x 128
  offer(tile_cost<FMT, 2, 2, 1, 1>(p, cus), launch_tile<T, FMT, 2, 2, 1, 1>);     // 64 x 64
  return run(p, s);
}

template <typename T, int FMT>
static hipError_t mx_gemm_t(const MxGemmParams& p, hipStream_t s) {
  // 2^19 rows per launch, so that a launch's tiles stay far below a grid's limit
  for (int m0 = 0; m0 < p.m; m0 += 1 << 19) {
    MxGemmParams q = p;
    q.m = std::min(p.m - m0, 1 << 19);
    q.a = p.a + (size_t)m0 * p.groups * (FMT == GALE_MX_E2M1 ? 64 : 128);
    q.as = p.as + (size_t)m0 * p.groups * 4;
    q.y = (typename T::bits*)p.y + m0 * p.y_stride;
    if (p.add) q.add = (const typename T::bits*)p.add + m0 * p.add_stride;
    const hipError_t e = q.m > 32   ? launch_best_tile<T, FMT>(q, s)
                         : q.m > 16 ? launch_stream<T, FMT, 2>(q, s)
                                    : launch_stream<T, FMT, 1>(q, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_gemm(int m, int n, int k, const uint8_t* a, const uint8_t* as, int a_fmt, const uint8_t* w,
                          const uint8_t* ws, const void* add, int64_t add_stride, void* y, int y_dtype,
                          int64_t y_stride, hipStream_t s) {
  const int es = y_dtype == GALE_F32 ? 4 : 2;
  auto four_wide = [es](const void* q, int64_t stride) { return (uintptr_t)q % (4 * es) == 0 && stride % 4 == 0; };
  MxGemmParams p = {m, n, mx_groups(k), a, as, w, ws, add, add_stride, y, y_stride,
                    four_wide(y, y_stride) && (!add || four_wide(add, add_stride)),
                    rows_wide(y, y_stride, es) && (!add || rows_wide(add, add_stride, es))};
  const bool four = a_fmt == GALE_MX_E2M1;
  if (y_dtype == GALE_F16) return four ? mx_gemm_t<F16, GALE_MX_E2M1>(p, s) : mx_gemm_t<F16, GALE_MX_E4M3>(p, s);
  if (y_dtype == GALE_BF16) return four ? mx_gemm_t<BF16, GALE_MX_E2M1>(p, s) : mx_gemm_t<BF16, GALE_MX_E4M3>(p, s);
  return four ? mx_gemm_t<F32, GALE_MX_E2M1>(p, s) : mx_gemm_t<F32, GALE_MX_E4M3>(p, s);
}

}  // namespace gale
