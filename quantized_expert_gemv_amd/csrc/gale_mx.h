// Device pieces shared by the kernels that read and write MX (microscaled) numbers and 16- or 32-bit
// rows: eight-column loads and stores of any dtype, and the encoding of an MX block.
#pragma once
#include "gale_internal.h"

namespace gale {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mx_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mx_u32x2 __attribute__((ext_vector_type(2)));

// Storage types of the rows: bit patterns and their fp32 values.
struct F16 {
  typedef uint16_t bits;
  static __device__ __forceinline__ float to_f32(uint16_t b) {
    __half_raw r;
    r.x = b;
    return __half2float(__half(r));
  }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return __half_as_ushort(__float2half_rn(v)); }
};
struct BF16 {
  typedef uint16_t bits;
  static __device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  // to nearest even; a NaN stays one (its payload may round to infinity otherwise)
  static __device__ __forceinline__ uint16_t from_f32(float v) {
    const __bf16 b = (__bf16)v;
    return __builtin_bit_cast(uint16_t, b);
  }
};
struct F32 {
  typedef float bits;
  static __device__ __forceinline__ float to_f32(float b) { return b; }
  static __device__ __forceinline__ float from_f32(float v) { return v; }
};

// Eight columns c .. c + 7 of a row, zero behind column cols.  wide: the row starts on a 16-byte
// boundary and c is a multiple of 8, so a whole unit is one or two 16-byte loads.
template <typename T>
__device__ __forceinline__ void load8(const typename T::bits* row, int c, int cols, bool wide, float v[8]) {
  if (wide && c + 8 <= cols) {
    if constexpr (sizeof(typename T::bits) == 2) {
      const mx_u32x4 r = *reinterpret_cast<const mx_u32x4*>(row + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = T::to_f32((uint16_t)(r[i] & 0xFFFFu));
        v[2 * i + 1] = T::to_f32((uint16_t)(r[i] >> 16));
      }
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(row + c);
      const f32x4 b = *reinterpret_cast<const f32x4*>(row + c + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? T::to_f32(row[c + i]) : 0.f;
  }
}

// Whether every row starts on a 16-byte boundary (es: bytes per element).
inline bool rows_wide(const void* p, int64_t stride, int es) { return ((uintptr_t)p & 15) == 0 && stride * es % 16 == 0; }

// Stores columns c .. c + 7 below cols, rounded to T; wide as in load8.
template <typename T>
__device__ __forceinline__ void store8(typename T::bits* row, int c, int cols, bool wide, const float v[8]) {
  if (wide && c + 8 <= cols) {
    if constexpr (sizeof(typename T::bits) == 2) {
      mx_u32x4 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = (uint32_t)T::from_f32(v[2 * i]) | ((uint32_t)T::from_f32(v[2 * i + 1]) << 16);
      *reinterpret_cast<mx_u32x4*>(row + c) = r;
    } else {
      *reinterpret_cast<f32x4*>(row + c) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = T::from_f32(v[i]);
  }
}

// The same for a dtype known at run time (uniform over the launch).
__device__ __forceinline__ void load8_dt(const void* row, int dtype, int c, int cols, bool wide, float v[8]) {
  if (dtype == GALE_F16) load8<F16>((const uint16_t*)row, c, cols, wide, v);
  else if (dtype == GALE_BF16) load8<BF16>((const uint16_t*)row, c, cols, wide, v);
  else load8<F32>((const float*)row, c, cols, wide, v);
}
__device__ __forceinline__ void store8_dt(void* row, int dtype, int c, int cols, bool wide, const float v[8]) {
  if (dtype == GALE_F16) store8<F16>((uint16_t*)row, c, cols, wide, v);
  else if (dtype == GALE_BF16) store8<BF16>((uint16_t*)row, c, cols, wide, v);
  else store8<F32>((float*)row, c, cols, wide, v);
}

// Row sizes in memory: whole groups of 128 columns.
__host__ __device__ inline int mx_groups(int cols) { return (cols + GALE_MX_GROUP - 1) / GALE_MX_GROUP; }
__host__ __device__ inline int mx_code_row(int fmt, int cols) { return mx_groups(cols) * (fmt == GALE_MX_E2M1 ? 64 : 128); }
__host__ __device__ inline int mx_scale_row(int cols) { return mx_groups(cols) * 4; }

// Encodes an MX block spread over four consecutive lanes (a quad), eight columns each.  Every lane of the
// quad gets the block's scale byte; words gets the lane's eight elements (one word of 4-bit, two of 8-bit).
//
// With amax = 1.m 2^(f - 127) and the format's largest number 1.M 2^E, the smallest scale 2^(s - 127) with
// amax <= 1.M 2^E 2^(s - 127) is s = f - E when m <= M, one more otherwise, and at least 0.  Magnitudes
// compare as their bit patterns, where infinities and NaNs are larger than every number.
// x 2^(127 - s) is exact (or so far below half the smallest element that it rounds to zero either way), so
// the conversion's rounding to nearest even is the only one.
template <int FMT>
__device__ __forceinline__ uint32_t mx_encode8(const float v[8], uint32_t words[2]) {
  constexpr int E = FMT == GALE_MX_E2M1 ? 2 : 8;
  constexpr uint32_t M = FMT == GALE_MX_E2M1 ? 0x400000u : 0x600000u;   // 6 = 1.5 2^2, 448 = 1.75 2^8
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  const int s = max(0, (int)(top >> 23) - E + ((top & 0x7FFFFFu) > M ? 1 : 0));
  const bool nan = top >= 0x7F800000u;
  const float mul = __uint_as_float((uint32_t)(254 - s) << 23);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * mul;
  if constexpr (FMT == GALE_MX_E2M1) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
    words[0] = nan ? 0u : w;
  } else {
    int a = 0, b = 0;
    a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
    words[0] = nan ? 0u : (uint32_t)a;
    words[1] = nan ? 0u : (uint32_t)b;
  }
  return nan ? 255u : (uint32_t)s;
}

// A 64-bit number is rounded to odd in 32: a second rounding then goes as it would from the number itself.  odd_step: what
// that adds to the bits of f, d rounded to nearest.  What 32 bits do not hold stays infinite, and makes its block NaN.
__device__ __forceinline__ int odd_step(double d, float f) {
  if (!(fabsf(f) < INFINITY) || (double)f == d || (__float_as_uint(f) & 1u)) return 0;
  return fabs(d) > fabs((double)f) ? 1 : -1;
}
__device__ __forceinline__ float f32_to_odd(double d) {
  const float f = (float)d;
  return __uint_as_float(__float_as_uint(f) + odd_step(d, f));
}

// Stores a lane's part of an encoded block: unit u = column / 8 of the row; the quad's first lane stores the
// scale.
template <int FMT>
__device__ __forceinline__ void mx_store8(uint8_t* code_row, uint8_t* scale_row, int u, uint32_t scale,
                                          const uint32_t words[2]) {
  if constexpr (FMT == GALE_MX_E2M1)
    *reinterpret_cast<uint32_t*>(code_row + 4 * (size_t)u) = words[0];
  else
    *reinterpret_cast<mx_u32x2*>(code_row + 8 * (size_t)u) = mx_u32x2{words[0], words[1]};
  if ((u & 3) == 0) scale_row[u >> 2] = (uint8_t)scale;
}

}  // namespace gale
