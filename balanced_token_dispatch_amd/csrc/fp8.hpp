// Shared pieces of the 8-bit path: block exponents, scale-row pitch, conversions (gfx950 only).
//
// A block of 128 values (a row's columns, or 128 x 128 weights) is stored as v * 2^-e in an
// 8-bit format, with e the least exponent that brings the block's largest finite magnitude
// within the format's largest value, 0.875 * 2^TOP.  Scales are powers of two because the
// matrix instructions take one exponent byte (2^(byte - 127)) per row and 32 values of the
// contraction for nothing, and because scaling by them rounds nothing.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kBlock = 128;       // values per scale
constexpr int kUnitScale = 127;   // the byte of 2^0: zero blocks and padding

typedef __attribute__((ext_vector_type(8))) int32_t i32x8;

// Bytes per row of scales for n columns: 16 for each 2048 columns begun, so every row of
// scales starts 16-byte aligned.
__host__ __device__ inline long long scale_pitch(long long n) { return (n + 2047) / 2048 * 16; }

// Largest value 0.875 * 2^TOP: 448 (e4m3), 57344 (e5m2).
template <int FMT>
constexpr int kTop = FMT == MOE_E5M2 ? 16 : 9;

// Bits of |v| for the block maximum: non-finite values do not count.
__device__ inline uint32_t finite_mag(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// Exponent of a block whose largest finite magnitude has bits `mag`: with mag = m 2^x, m in
// [0.5, 1), the least e with mag <= 0.875 2^(TOP + e) is x - TOP, or one more when m > 0.875.
// At least -127 (the smallest scale), 0 for a block of zeros.  The largest finite fp32 gives
// e = 128 - TOP <= 119.
template <int FMT>
__device__ inline int block_exponent(uint32_t mag) {
  if (mag == 0) return 0;
  const int x = (int)(mag >> 23) - 126;  // (subnormal: far below the clamp)
  const int e = x - kTop<FMT> + ((mag & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// 2^e as the conversions below take it (a scale byte's value: 2^-127 is the subnormal).
__device__ inline float exponent_scale(int e) {
  return __builtin_bit_cast(float, e == -127 ? 0x00400000u : (uint32_t)(e + 127) << 23);
}

typedef __attribute__((ext_vector_type(2))) short i16x2;

// Four values divided by `scale` (a power of two) as 8-bit bytes, rounded to nearest even; a NaN stays
// NaN, an infinity becomes NaN in e4m3, which has none.
template <int FMT>
__device__ inline uint32_t pack_fp8x4(float a, float b, float c, float d, float scale) {
  i16x2 r = {0, 0};
  if constexpr (FMT == MOE_E5M2) {
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c, d, scale, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}

// The same from two words of two bf16 values.
template <int FMT>
__device__ inline uint32_t pack_fp8x4(uint32_t ab, uint32_t cd, float scale) {
  i16x2 r = {0, 0};
  const bf16x2 lo = __builtin_bit_cast(bf16x2, ab), hi = __builtin_bit_cast(bf16x2, cd);
  if constexpr (FMT == MOE_E5M2) {
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, lo, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, hi, scale, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, lo, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, hi, scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}

typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;

// The larger magnitude of each half of two words of bf16 values.
__device__ inline uint32_t mag_max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b & 0x7FFF7FFFu)));
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace moe
