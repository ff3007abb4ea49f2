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
// consecutive columns are cut (towards zero) to multiples of 2^(e - 13), e the exponent of the largest of them; the
// sums of the eights, scaled, and the accumulator add like fp32 numbers.  Products of two 4-bit elements span 2^-2 ..
// 2^5 and are never cut.  Those of an 8-bit and a 4-bit element span 2^-10 .. 2^11 and are: so the 8-bit operand is
// split at magnitude 4 into two, which are multiplied one after the other.  The upper part's products are multiples of
// 2^-2 below 2^12 (cut at 2^(10 - 13)), the lower part's multiples of 2^-10 below 2^5 (cut at 2^(3 - 13)): both whole.
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
};

// Format codes of the MFMA: 0 for E4M3, 4 for E2M1.

template <int FMT>
__device__ __forceinline__ v8i mx_operand(const uint8_t* row, int grp, int g) {
  if constexpr (FMT == GALE_MX_E2M1) {
    const mx_u32x4 v = *reinterpret_cast<const mx_u32x4*>(row + 64 * (size_t)grp + 16 * g);
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  } else {
    const mx_u32x4 v = *reinterpret_cast<const mx_u32x4*>(row + 128 * (size_t)grp + 16 * g);
    const mx_u32x4 u = *reinterpret_cast<const mx_u32x4*>(row + 128 * (size_t)grp + 64 + 16 * g);
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, (int)u.x, (int)u.y, (int)u.z, (int)u.w};
  }
}

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

// Four consecutive columns n0 .. n0 + 3 of row i of y, as far as they exist.
template <typename T>
__device__ __forceinline__ void mx_store4(const MxGemmParams& p, int i, int n0, const f32x4& acc) {
  typedef typename T::bits bits;
  bits* y = (bits*)p.y + (int64_t)i * p.y_stride + n0;
  const bits* c = (const bits*)p.add + (int64_t)i * p.add_stride + n0;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n0 + r < p.n) y[r] = T::from_f32(p.add ? acc[r] + T::to_f32(c[r]) : acc[r]);
}

// One wavefront per 16 x 16 tile of y.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) mx_gemm_simple_kernel(const MxGemmParams p) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int n0 = ((int)blockIdx.x * 4 + ((int)threadIdx.x >> 6)) * 16, m0 = (int)blockIdx.y * 16;
  if (n0 >= p.n) return;
  const int wr = min(n0 + r, p.n - 1), ar = min(m0 + r, p.m - 1);
  const uint8_t* w = p.w + (size_t)wr * p.groups * 64;
  const uint8_t* a = p.a + (size_t)ar * p.groups * (FMT == GALE_MX_E2M1 ? 64 : 128);
  const uint8_t* ws = p.ws + (size_t)wr * p.groups * 4 + g;
  const uint8_t* as = p.as + (size_t)ar * p.groups * 4 + g;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < p.groups; ++k)
    acc = mx_mfma<FMT>(mx_operand<GALE_MX_E2M1>(w, k, g), (int)ws[4 * k], mx_operand<FMT>(a, k, g), (int)as[4 * k], acc);
  // the products stay outside the branch below: an MFMA reads the registers of every lane
  asm volatile("" : "+v"(acc));
  if (m0 + r < p.m) mx_store4<T>(p, m0 + r, n0 + 4 * g, acc);
}

template <typename T, int FMT>
static hipError_t mx_gemm_t(const MxGemmParams& p, hipStream_t s) {
  // at most 2^16 rows of tiles per launch
  for (int m0 = 0; m0 < p.m; m0 += 1 << 19) {
    MxGemmParams q = p;
    q.m = std::min(p.m - m0, 1 << 19);
    q.a = p.a + (size_t)m0 * p.groups * (FMT == GALE_MX_E2M1 ? 64 : 128);
    q.as = p.as + (size_t)m0 * p.groups * 4;
    q.y = (typename T::bits*)p.y + m0 * p.y_stride;
    if (p.add) q.add = (const typename T::bits*)p.add + m0 * p.add_stride;
    hipLaunchKernelGGL(HIP_KERNEL_NAME(mx_gemm_simple_kernel<T, FMT>), dim3((p.n + 63) / 64, (q.m + 15) / 16), dim3(256), 0,
                       s, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_gemm(int m, int n, int k, const uint8_t* a, const uint8_t* as, int a_fmt, const uint8_t* w,
                          const uint8_t* ws, const void* add, int64_t add_stride, void* y, int y_dtype,
                          int64_t y_stride, hipStream_t s) {
  MxGemmParams p = {m, n, mx_groups(k), a, as, w, ws, add, add_stride, y, y_stride};
  const bool four = a_fmt == GALE_MX_E2M1;
  if (y_dtype == GALE_F16) return four ? mx_gemm_t<F16, GALE_MX_E2M1>(p, s) : mx_gemm_t<F16, GALE_MX_E4M3>(p, s);
  if (y_dtype == GALE_BF16) return four ? mx_gemm_t<BF16, GALE_MX_E2M1>(p, s) : mx_gemm_t<BF16, GALE_MX_E4M3>(p, s);
  return four ? mx_gemm_t<F32, GALE_MX_E2M1>(p, s) : mx_gemm_t<F32, GALE_MX_E4M3>(p, s);
}

}  // namespace gale
