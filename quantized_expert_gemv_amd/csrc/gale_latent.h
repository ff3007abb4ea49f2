// Device pieces shared by the kernels of latent attention.
#pragma once
#include "gale_lanes.h"
#include "gale_mx.h"

namespace gale {

// A value that the compiler takes as new here: what is made of it is not kept in registers over a loop.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

constexpr int kLat = GALE_LATENT_DIM, kRope = GALE_LATENT_ROPE, kQk = kLat + kRope;

// Entry r of an ascending array of starts, within [0, n].
__device__ __forceinline__ int start_at(const int32_t* starts, int r, int n) { return min(max(starts[r], 0), n); }

// Keys of request r.
__device__ __forceinline__ int keys_of(const int32_t* kv_lens, int r, int max_blocks, int shift) {
  return (int)min((int64_t)max(kv_lens[r], 0), (int64_t)max_blocks << shift);
}

// ---------------------------------------------------------------------------
// Matrix-core pieces.  Both forms compute S^T = K Q^T and O^T = V^T P^T with the 32x32x16 MFMA, 32 queries to a wavefront:
//   first operand: lane l holds row l % 32, columns 8 (l / 32) .. + 7; second operand alike with its rows as columns;
//   result register i of lane l: row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32 (measured with one-hot operands).
// A query is a lane's column in both products, so its maximum, sum and scale are one register per lane, and eight
// registers of S^T become an operand of the second product as they are: the order of the keys inside a product of 16 is free
// as long as V^T has the same one (0-3 and 8-11 for the lower lanes, 4-7 and 12-15 for the upper).  V lies in LDS as rows of keys;
// ds_read_b64_tr_b16 gives each lane four keys of one column: lane i of 16 addresses 8 bytes, (key i / 4, columns 4 (i % 4) ..),
// and receives column i of the four keys.
//
// The second product takes the weights in the values' type: in fp32 its rate would be a sixteenth, and in two parts (a rounded
// weight and what it leaves) the product would be twice as long.  Their sums and the sum of weights are fp32.  Against 64 bits, relative,
// the rounding is not seen where values have a mean (absorbed, 1.7e-3 in bf16 and 2.1e-4 in fp16, as without it); where they have
// none, it adds to the result's own (expanded form, random values: 2.3e-3 for 1.7e-3 in bf16, 2.5e-4 for 2.0e-4 in fp16).
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <typename T>
struct Mma;
template <>
struct Mma<F16> {
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  typedef _Float16 v4 __attribute__((ext_vector_type(4)));
  // weights are 2^(s - m + lift) for a score s and the maximum m that is in use, at most kSlack below the true one; 2^7 puts the
  // smallest subnormal of fp16 at 2^-31 of the largest weight, and the largest at 2^15
  static __device__ __forceinline__ float lift(int) { return 7.f; }
  static __device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma4(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(v4, a), __builtin_bit_cast(v4, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ s16x4 pack4(const float* v) {
    v4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (_Float16)v[i];
    return __builtin_bit_cast(s16x4, r);
  }
  static __device__ __forceinline__ s16x8 pack(const float* v) {
    v8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
    return __builtin_bit_cast(s16x8, r);
  }
};
template <>
struct Mma<BF16> {
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  typedef __bf16 v4 __attribute__((ext_vector_type(4)));
  // weights of at most 1 / (2 keys), keys taken up to a power of two: sums of values, which may lie at the end of fp32's range, reach
  // no further than the largest one (the 2 is for what rounding adds).  The price is at the other end: with 2^17 keys, products
  // of values below 2^-100 leave fp32's normal range.
  static __device__ __forceinline__ float lift(int keys) { return keys > 1 ? (float)(__builtin_clz(keys - 1) - 32 - 9) : -9.f; }
  static __device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma4(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ s16x4 pack4(const float* v) {
    v4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (__bf16)v[i];
    return __builtin_bit_cast(s16x4, r);
  }
  static __device__ __forceinline__ s16x8 pack(const float* v) {
    v8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
    return __builtin_bit_cast(s16x8, r);
  }
};
constexpr float kSlack = 8.f;     // sums are rescaled when the maximum has risen by more than 2^8

// Where a row's 16-byte chunk lies: chunk ^ swizzle(row).  Rows are multiples of 256 bytes, so eight rows of one chunk (an
// operand of K) and four rows of two or four chunks (an operand of V^T) have to part by the swizzle: bits 0-2 differ over eight
// rows, bits 0-3 over 16, bits 1-2 and 2-3 over four.
__device__ __forceinline__ int swizzle(int row) {
  return ((row >> 2) & 1) | (row & 2) | ((row & 1) << 2) | ((((row >> 1) ^ (row >> 3)) & 1) << 3);
}
// The same for rows of 128 bytes (eight chunks): eight rows differ, and 16 with the row's place in 256 bytes.
__device__ __forceinline__ int swizzle8(int row) {
  return ((row >> 2) & 1) | (row & 2) | (((row ^ (row >> 3)) & 1) << 2);
}

__device__ __forceinline__ s16x8 lds_operand(const lds_u8* p) { return *(const __attribute__((address_space(3))) s16x8*)p; }
__device__ __forceinline__ s16x4 lds_transposed(const lds_u8* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// A query's sum of weights: 0 where it sees no key, and kNoScore (in sums: below 0) where it sees some, but all of their scores are
// -infinity, which the maximum does not tell apart.  Its result is 0 or the formula's 0 / 0; what its sums are multiplied by:
constexpr float kNoScore = -1.f;
__device__ __forceinline__ float normaliser(float l) { return l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN; }

// The other half's value of a lane's column.
__device__ __forceinline__ float other_half(float v) { return lane_xor<32>(v); }

// Copies into LDS that a wavefront has issued have landed, its reads are done, and so are the others'.
__device__ __forceinline__ void tiles_ready() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Bits that are set where one of a word's two 16-bit numbers is an infinity or a NaN.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t kExp = __is_same(T, F16) ? 0x7C007C00u : 0x7F807F80u, kOne = __is_same(T, F16) ? 0x04000400u : 0x00800080u;
  return ((w & kExp) + kOne) & 0x80008000u;
}
// The same numbers with zeros in those places.
template <typename T>
__device__ __forceinline__ s16x8 finite_only(s16x8 v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = not_finite<T>(w[i]);
    w[i] &= ~((b - (b >> 15)) | b);            // 0x8000 -> 0xFFFF in each half
  }
  return __builtin_bit_cast(s16x8, w);
}

// Eight 16-bit numbers times the sign of a scale, or times 0: with it, scores are scaled by |scale| (1 for 0).
template <typename T>
__device__ __forceinline__ s16x8 signed_query(s16x8 v, float scale) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 w = __builtin_bit_cast(u32x4, v);
  const uint32_t sign = scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t odd = not_finite<T>(w[i]);
    w[i] = scale == 0.f ? odd - (odd >> 15) : w[i] ^ sign;      // 0 times infinity or NaN: 0x7FFF, a NaN
  }
  return __builtin_bit_cast(s16x8, w);
}

// Eight 4-bit elements (the low nibble of the low byte first) times a scale, as 16-bit numbers.
template <typename T>
__device__ __forceinline__ mx_u32x4 mx_values8(uint32_t w, float scale) {
  mx_u32x4 v;
  if constexpr (__is_same(T, F16)) {
    v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0));
    v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1));
    v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2));
    v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3));
  } else {
    v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
  return v;
}

}  // namespace gale
