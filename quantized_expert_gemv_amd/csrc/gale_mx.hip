// MX (microscaled) numbers: quantisation, its SwiGLU form, and the numbers that MX rows stand for.
//
// A thread takes units of eight columns, so a block of 32 is a quad of lanes and its amax two DPP steps.
// All three kernels are bound by HBM: 2 + 17/32 bytes per fp16 number to 4 bits.
#include "gale_mx.h"

namespace gale {

// g sigmoid(g), within a few ulp where the result is a normal number.  With e = e^(-|g| / 2), sigmoid is 1 / (1 + e^2), or e^2 /
// (1 + e^2) for negative g: multiplied as (g e) (e / (1 + e^2)), no factor underflows before the result does.  The exponent
// -|g| log2(e) / 2 is taken with the rounding of its product (x + lo), since the hardware's 2^x turns an absolute error of
// x into a relative one.  With the library's exponential and division the arithmetic bounds the kernel
// (4096 x 2048 fp16 into 8 bits: 12.2 us against 10.2 with two units per thread).  The codes are made those of 64-bit arithmetic: where the result
// lies so near a border of the rounding that its error matters, one element in 16,000, it is computed in 64 bits
// (together 11.1 us, one unit per thread).  So are the results that 32 bits hold with fewer bits: subnormal products, and those
// of a silu below 2^-120 (g under -87 or next to 0) and an up value above 1, which may bring it back among the normal numbers.
__device__ __forceinline__ float silu(float g) {
  const float a = fabsf(g), kHi = 0.72134752044448170f, kLo = 9.62981496e-9f;   // log2(e) / 2 = kHi + kLo
  const float x = -a * kHi;
  const float lo = fmaf(-a, kHi, -x) - a * kLo;
  float e = __builtin_amdgcn_exp2f(x);
  e = fmaf(e, lo * 0.693147180559945309f, e);
  const float r = __builtin_amdgcn_rcpf(fmaf(e, e, 1.0f));
  return g < 0.f ? (g * e) * (e * r) : g * r;
}

// silu(g) u in 64 bits, rounded to odd in 32.
__device__ __forceinline__ float swiglu_odd(float g, float u) {
  return f32_to_odd((double)g * (1.0 / (1.0 + exp(-(double)g))) * (double)u);
}

// Units (8 columns, padded rows) of a launch are numbered row by row; the host keeps their count below 2^31.
template <typename T, int FMT, bool SWIGLU, int U>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const typename T::bits* __restrict__ x, int64_t x_stride,
                                                          uint32_t n_units, int cols, int row_units, bool wide,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  // U units per thread, 256 apart, all loads first.  n_units is a multiple of 16: no quad is split.
  float v[U][8], up[U][8];
  uint32_t row[U];
  int u[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = min(blockIdx.x * (256u * U) + 256u * k + threadIdx.x, n_units - 1u);
    row[k] = i / (uint32_t)row_units;
    u[k] = (int)(i - row[k] * (uint32_t)row_units);
    const typename T::bits* xr = x + (int64_t)row[k] * x_stride;
    load8<T>(xr, 8 * u[k], cols, wide, v[k]);
    if constexpr (SWIGLU) load8<T>(xr + cols, 8 * u[k], cols, wide, up[k]);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (blockIdx.x * (256u * U) + 256u * k + threadIdx.x >= n_units) return;
    if constexpr (SWIGLU) {
      float g[8], a[8], least = INFINITY;
      uint32_t near = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = v[k][j];
        a[j] = silu(g[j]);
        v[k][j] = a[j] * up[k][j];
        least = fminf(least, fminf(fabsf(a[j]), fabsf(v[k][j])));
        // off by less than 16 of its last place; borders between elements and between scales end in 19 zero bits
        near |= ((__float_as_uint(v[k][j]) + 16u) & 0x7FFFFu) <= 32u && v[k][j] != 0.f ? 1u << j : 0u;
      }
      if (least < 0x1p-120f) {         // zeros do not count
        least = INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          least = fminf(least, fminf(fabsf(g[j]), fabsf(up[k][j])) == 0.f ? 1.f : fminf(fabsf(a[j]), fabsf(v[k][j])));
      }
      if (least < 0x1p-120f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // below g = -200 no up value brings the product back; a product rounded to zero lies far below half of the
          // smallest element, 2^-137
          const bool lost = fabsf(a[j]) < 0x1p-120f && g[j] > -200.f && g[j] != 0.f && fabsf(up[k][j]) > 1.f;
          near |= lost || (v[k][j] != 0.f && fabsf(v[k][j]) < 0x1p-126f) ? 1u << j : 0u;
        }
      }
      while (near != 0) {
        const int n = __builtin_ctz(near);
        near &= near - 1;
        float gn = g[0], un = up[k][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
          gn = j == n ? g[j] : gn;
          un = j == n ? up[k][j] : un;
        }
        const float y = swiglu_odd(gn, un);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = j == n ? y : v[k][j];
      }
    }
    uint32_t words[2];
    const uint32_t s = mx_encode8<FMT>(v[k], words);
    mx_store8<FMT>(codes + (size_t)row[k] * row_units * (FMT == GALE_MX_E2M1 ? 4 : 8),
                   scales + (size_t)row[k] * (row_units >> 2), u[k], s, words);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int fmt,
                                                            uint32_t n_units, int cols, int row_units, bool wide,
                                                            typename T::bits* __restrict__ y, int64_t y_stride) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n_units) return;
  const uint32_t row = i / (uint32_t)row_units;
  const int u = (int)(i - row * (uint32_t)row_units);
  const uint32_t s = scales[(size_t)row * (row_units >> 2) + (u >> 2)];
  // 2^(s - 127): s = 0 is the subnormal 2^-127, 255 NaN
  const float scale = s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s ? s << 23 : 0x400000u);
  float v[8];
  if (fmt == GALE_MX_E2M1) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[(size_t)i];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = (w >> (4 * j)) & 15u;
      // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: exponent c / 2, mantissa bit c % 2, subnormal below 2
      const uint32_t e = (c >> 1) & 3u, m = c & 1u;
      const float a = e == 0 ? 0.5f * (float)m : __uint_as_float(((e + 126u) << 23) | (m << 22));
      v[j] = (c & 8u ? -a : a) * scale;
    }
  } else {
    const mx_u32x2 w = reinterpret_cast<const mx_u32x2*>(codes)[(size_t)i];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v[4 * j + 0] = __builtin_amdgcn_cvt_f32_fp8((int)w[j], 0) * scale;
      v[4 * j + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[j], 1) * scale;
      v[4 * j + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[j], 2) * scale;
      v[4 * j + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[j], 3) * scale;
    }
  }
  if (8 * u < cols) store8<T>(y + (int64_t)row * y_stride, 8 * u, cols, wide, v);
}

// Rows of one launch: their units stay below 2^31.
static int64_t slab_rows(int row_units) { return std::max<int64_t>(1, ((int64_t)1 << 31) / row_units - 1); }

template <typename T, int FMT, bool SWIGLU>
static hipError_t quantize_t(const void* x, int64_t x_stride, int64_t rows, int cols, uint8_t* codes, uint8_t* scales,
                             hipStream_t s) {
  const int ru = mx_groups(cols) * (GALE_MX_GROUP / 8);
  constexpr int es = sizeof(typename T::bits);
  // the up half starts at column cols: its units are wide only when cols keeps the alignment
  const bool wide = rows_wide(x, x_stride, es) && (!SWIGLU || cols * es % 16 == 0);
  constexpr int U = SWIGLU ? 1 : 2;      // the 64-bit way of a SwiGLU takes the registers of a second unit
  const int64_t slab = slab_rows(ru);
  for (int64_t r = 0; r < rows; r += slab) {
    const int64_t n = std::min(slab, rows - r);
    const uint32_t units = (uint32_t)(n * ru);
    hipLaunchKernelGGL(HIP_KERNEL_NAME(mx_quantize_kernel<T, FMT, SWIGLU, U>), dim3((units + 256 * U - 1) / (256 * U)), dim3(256), 0, s,
                       (const typename T::bits*)x + r * x_stride, x_stride, units, cols, ru, wide,
                       codes + (size_t)r * mx_code_row(FMT, cols), scales + (size_t)r * mx_scale_row(cols));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
static hipError_t quantize_d(const void* x, int64_t x_stride, int64_t rows, int cols, int fmt, bool swiglu,
                             uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (fmt == GALE_MX_E2M1)
    return swiglu ? quantize_t<T, GALE_MX_E2M1, true>(x, x_stride, rows, cols, codes, scales, s)
                  : quantize_t<T, GALE_MX_E2M1, false>(x, x_stride, rows, cols, codes, scales, s);
  return swiglu ? quantize_t<T, GALE_MX_E4M3, true>(x, x_stride, rows, cols, codes, scales, s)
                : quantize_t<T, GALE_MX_E4M3, false>(x, x_stride, rows, cols, codes, scales, s);
}

hipError_t launch_mx_quantize(const void* x, int x_dtype, int64_t x_stride, int64_t rows, int cols, int fmt,
                              bool swiglu, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (x_dtype == GALE_F16) return quantize_d<F16>(x, x_stride, rows, cols, fmt, swiglu, codes, scales, s);
  if (x_dtype == GALE_BF16) return quantize_d<BF16>(x, x_stride, rows, cols, fmt, swiglu, codes, scales, s);
  return quantize_d<F32>(x, x_stride, rows, cols, fmt, swiglu, codes, scales, s);
}

template <typename T>
static hipError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t rows, int cols, void* y,
                               int64_t y_stride, hipStream_t s) {
  const int ru = mx_groups(cols) * (GALE_MX_GROUP / 8);
  const bool wide = rows_wide(y, y_stride, sizeof(typename T::bits));
  const int64_t slab = slab_rows(ru);
  for (int64_t r = 0; r < rows; r += slab) {
    const int64_t n = std::min(slab, rows - r);
    const uint32_t units = (uint32_t)(n * ru);
    hipLaunchKernelGGL(HIP_KERNEL_NAME(mx_dequantize_kernel<T>), dim3((units + 255) / 256), dim3(256), 0, s,
                       codes + (size_t)r * mx_code_row(fmt, cols), scales + (size_t)r * mx_scale_row(cols), fmt, units,
                       cols, ru, wide, (typename T::bits*)y + r * y_stride, y_stride);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t rows, int cols, void* y,
                                int y_dtype, int64_t y_stride, hipStream_t s) {
  if (y_dtype == GALE_F16) return dequantize_t<F16>(codes, scales, fmt, rows, cols, y, y_stride, s);
  if (y_dtype == GALE_BF16) return dequantize_t<BF16>(codes, scales, fmt, rows, cols, y, y_stride, s);
  return dequantize_t<F32>(codes, scales, fmt, rows, cols, y, y_stride, s);
}

}  // namespace gale
