// Residual addition and RMS norm, with an optional MX output.
//
// s = x + r (rounded to the rows' type), y = s / sqrt(mean(s^2) + eps) * w.  One pass over memory: a workgroup
// holds its row in registers between the sum of squares and the outputs.
//
// The 8- or 4-bit form of y is that of the exact number (to a few 2^-45): with plain 32-bit arithmetic a few elements in a million
// took the neighbouring code and two blocks in a million the other of two scales, as the last bit of y fell.  The squares are
// added in 64 bits (in 32 by eights, one element in ten million was on the wrong side of a border, at the same time: 112 us
// for 16,384 x 4,096 bf16 with an 8-bit output), 1 / rms is held as two floats ih + il, and s w as p + q: y = p ih + t,
// t = p il + q ih, is rounded once.  A second rounding, to the element, differs from that of the exact number only where y
// fell on a border: halfway between two elements, or the largest number at a scale.  All borders end in 19 zero bits, which
// one element in 2^19 does: for those the rest p ih + t - y pushes y off the border, to the side it came from.  (With y in 64
// bits too the arithmetic, not HBM, bounds the kernel: 123 us.)  Rows whose sum or rms is near the ends of 32 bits are computed in
// 64, and so are eights of columns with such a product or result.
#include "gale_mx.h"
#include "gale_lanes.h"

namespace gale {

struct NormParams {
  const void* x;
  const void* res;           // NULL: none
  int64_t x_stride, res_stride;
  const void* w;             // NULL: ones
  int w_dtype;
  int cols, row_units;       // row_units: 8-column units, whole 128-column groups when MX is written
  float eps;
  void* sum;                 // NULL: not wanted
  void* y;                   // NULL: not wanted
  int y_dtype;
  uint8_t* codes;
  uint8_t* scales;
  bool wide_x, wide_res, wide_w, wide_sum, wide_y;
};

template <int M>
__device__ __forceinline__ double xor_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = lane_xor_u32<M>((uint32_t)b), hi = lane_xor_u32<M>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the workgroup, in an order fixed by its size: lanes first, then wavefronts.
__device__ __forceinline__ double block_sum(double v, double* s_wave) {
  v += xor_f64<1>(v);
  v += xor_f64<2>(v);
  v += xor_f64<4>(v);
  v += xor_f64<8>(v);
  v += xor_f64<16>(v);
  v += xor_f64<32>(v);
  const int nw = (int)blockDim.x >> 6;
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < nw; ++i) t += s_wave[i];
  return t;
}

// FMT 0: no MX output.  U: units per thread, U * blockDim.x >= row_units.
template <typename T, int FMT, int U>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormParams p) {
  __shared__ double s_wave[16];
  typedef typename T::bits bits;
  const int64_t row = blockIdx.x;
  const bits* xr = (const bits*)p.x + row * p.x_stride;
  const bits* rr = (const bits*)p.res + row * p.res_stride;
  float v[U][8];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int c = 8 * (int)(threadIdx.x + k * blockDim.x);
    load8<T>(xr, c, p.cols, p.wide_x, v[k]);
  }
  if (p.res) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int c = 8 * (int)(threadIdx.x + k * blockDim.x);
      float r[8];
      load8<T>(rr, c, p.cols, p.wide_res, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = T::to_f32(T::from_f32(v[k][i] + r[i]));
    }
  }
  double sq = 0.0;
#pragma unroll
  for (int k = 0; k < U; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fma((double)v[k][i], (double)v[k][i], sq);
  }
  sq = block_sum(sq, s_wave);
  // the same for the whole workgroup: p, ih and il are far from the ends of 32 bits, or rows without a finite sum
  const bool ordinary = sq > 1e-20 && sq < 1e35;
  const double ms = sq / p.cols + (double)p.eps;
  // 1 / sqrt(ms): the hardware's estimate and one Newton step, or as written for rows out of the ordinary
  double inv = __builtin_amdgcn_rsq(ms);
  inv = fma(inv * 0.5, fma(-ms * inv, inv, 1.0), inv);
  if (!ordinary) inv = 1.0 / sqrt(ms);
  const float ih = (float)inv, il = (float)(inv - (double)ih);
  const float tiny = 0x1p-100f * fmaxf(1.f, 1.f / ih);    // |p| from here on has p and p / rms above 2^-100
  const bool by_32 = ordinary || (sq == 0.0 && p.eps > 0.f);      // also rows of zeros
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int u = (int)(threadIdx.x + k * blockDim.x), c = 8 * u;
    if (u >= p.row_units) continue;   // row_units is a multiple of 4 when FMT: no quad is split
    if (p.sum && c < p.cols) store8<T>((bits*)p.sum + row * p.cols, c, p.cols, p.wide_sum, v[k]);
    float w[8];
    if (p.w) load8_dt(p.w, p.w_dtype, c, p.cols, p.wide_w, w);
    if (!p.w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    }
    float y[8];
    uint32_t low = 0xFFFFFFFFu;
    bool far = !by_32;
    if (by_32) {
      float least = INFINITY, most = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float pr = v[k][i] * w[i], q = fmaf(v[k][i], w[i], -pr);
        y[i] = fmaf(pr, ih, fmaf(pr, il, q * ih));
        least = fminf(least, fabsf(pr));
        most = fmaxf(most, fabsf(pr));
        if constexpr (FMT != 0) low = min(low, __float_as_uint(y[i]) & 0x7FFFFu);
      }
      // Products and results near the ends of 32 bits, where p + q or t are not whole, go by 64.  Those of a zero factor
      // need not: y is the product, with its sign.
      if (least < tiny || most > 0x1p126f) {
        least = INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float pr = v[k][i] * w[i];
          const bool zero = fminf(fabsf(v[k][i]), fabsf(w[i])) == 0.f;
          least = fminf(least, zero ? 1.f : fabsf(pr));
          y[i] = zero ? pr : y[i];
        }
        far = least < tiny || most > 0x1p126f;
      }
    }
    uint32_t odd = 0;                 // two bits per column: the step of its rounding to odd, and one
    if (far) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = v[k][i];
        asm volatile("" : "+v"(x));            // not the 64-bit numbers of the squares: they would stay in registers
        const double d = (double)x * inv * (double)w[i];
        y[i] = (float)d;
        if constexpr (FMT != 0) odd |= (uint32_t)(odd_step(d, y[i]) + 1) << (2 * i);
        __builtin_amdgcn_sched_barrier(0);     // one after the other: registers for eight at once would cost occupancy
      }
    }
    if (p.y && c < p.cols) {
      const int es = p.y_dtype == GALE_F32 ? 4 : 2;
      store8_dt((char*)p.y + row * p.cols * es, p.y_dtype, c, p.cols, p.wide_y, y);
    }
    if constexpr (FMT != 0) {
      if (far) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(__float_as_uint(y[i]) + ((odd >> (2 * i)) & 3u) - 1u);
      } else if (low == 0 && ordinary) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float pr = v[k][i] * w[i], q = fmaf(v[k][i], w[i], -pr);
          const float rest = fmaf(pr, ih, -y[i]) + fmaf(pr, il, q * ih);
          const uint32_t b = __float_as_uint(y[i]);
          // infinity is no border: it stays, and makes its block NaN
          const bool border = (b & 0x7FFFFu) == 0 && rest != 0.f && y[i] != 0.f && fabsf(y[i]) < INFINITY;
          y[i] = border ? __uint_as_float(b + ((rest > 0.f) == (y[i] > 0.f) ? 1 : -1)) : y[i];
        }
      }
      if (c + 8 > p.cols) {
        // columns behind the row are zero also where 1 / rms is infinite
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = c + i < p.cols ? y[i] : 0.f;
      }
      uint32_t words[2];
      const uint32_t s = mx_encode8<FMT>(y, words);
      mx_store8<FMT>(p.codes + row * mx_code_row(FMT, p.cols), p.scales + row * mx_scale_row(p.cols), u, s, words);
    }
  }
}

template <typename T, int FMT>
static hipError_t launch_norm_t(const NormParams& p, int64_t rows, hipStream_t s) {
  const int ru = p.row_units;
  // Few rows: one unit per thread, the shortest way through a row.  More rows than the card holds at once: two per thread,
  // which keeps more rows in flight per CU (16,384 x 4,096 bf16: see above; 317 rows take either the same).
  if (ru <= 512 && rows <= 2 * device_cu_count()) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(add_rms_norm_kernel<T, FMT, 1>), dim3((unsigned)rows), dim3((ru + 63) / 64 * 64), 0, s, p);
  } else {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(add_rms_norm_kernel<T, FMT, 2>), dim3((unsigned)rows),
                       dim3((ru + 127) / 128 * 64), 0, s, p);
  }
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_norm_f(const NormParams& p, int fmt, int64_t rows, hipStream_t s) {
  if (fmt == GALE_MX_E2M1) return launch_norm_t<T, GALE_MX_E2M1>(p, rows, s);
  if (fmt == GALE_MX_E4M3) return launch_norm_t<T, GALE_MX_E4M3>(p, rows, s);
  return launch_norm_t<T, 0>(p, rows, s);
}

hipError_t launch_add_rms_norm(const void* x, int64_t x_stride, const void* res, int64_t res_stride, int dtype,
                               int64_t rows, int cols, const void* w, int w_dtype, float eps, void* sum, void* y,
                               int y_dtype, int fmt, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int es = dtype == GALE_F32 ? 4 : 2, ys = y_dtype == GALE_F32 ? 4 : 2;
  NormParams p;
  p.x_stride = x_stride;
  p.res_stride = res_stride;
  p.w = w;
  p.w_dtype = w_dtype;
  p.cols = cols;
  p.row_units = codes ? mx_groups(cols) * (GALE_MX_GROUP / 8) : (cols + 7) / 8;
  p.eps = eps;
  p.y_dtype = y_dtype;
  p.wide_x = rows_wide(x, x_stride, es);
  p.wide_res = rows_wide(res, res_stride, es);
  p.wide_w = rows_wide(w, 0, 1);
  p.wide_sum = rows_wide(sum, cols, es);
  p.wide_y = rows_wide(y, cols, ys);
  const int f = codes ? fmt : 0;
  // a grid has fewer than 2^32 threads: a million rows per launch
  for (int64_t r = 0; r < rows; r += (1 << 20)) {
    const int64_t n = std::min<int64_t>(rows - r, 1 << 20);
    p.x = (const char*)x + r * x_stride * es;
    p.res = res ? (const char*)res + r * res_stride * es : nullptr;
    p.sum = sum ? (char*)sum + r * cols * es : nullptr;
    p.y = y ? (char*)y + r * cols * ys : nullptr;
    p.codes = codes ? codes + r * mx_code_row(fmt, cols) : nullptr;
    p.scales = codes ? scales + r * mx_scale_row(cols) : nullptr;
    const hipError_t e = dtype == GALE_F16    ? launch_norm_f<F16>(p, f, n, s)
                         : dtype == GALE_BF16 ? launch_norm_f<BF16>(p, f, n, s)
                                              : launch_norm_f<F32>(p, f, n, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gale
