// Rows of logits shared by the lanes of a wave (L lanes a token): reductions, loads and scores.
#pragma once

#include "common.hpp"

namespace moe {

// The value of the lane N places on, around a row of 16 lanes.
template <int CTRL>
__device__ inline uint32_t rotated(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;
// Keys whose unsigned order is the values' order: -0 and 0 are equal, a NaN is above all.
// No key is 0 (0 marks a taken expert).
__device__ inline uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline unsigned long long order_key(double v) {
  if (v != v) return ~0ull;
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}

// The value of a key of fp32 order (the largest logit, from its key).
__device__ inline float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <bool BF16>
__device__ inline float load_logit(const void *p, long long i) {
  if constexpr (BF16)
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
  else
    return ((const float *)p)[i];
}

// The logistic of x over exp(m), m at most 0: exp(x) / (1 + exp(x)) below 0 and 1 / (1 + exp(-x)) above it share
// the denominator 1 + exp(-|x|), which never overflows.  With m the token's largest chosen logit (0 where that is
// positive) the scores that are added reach 1/2, however low all of them are, and exp(m) leaves their ratios.
__device__ inline float logistic_over(float x, float m) {
  if (x == -__builtin_inff()) return 0.0f;
  const float e = expf(-fabsf(x));
  float n = x >= 0.0f ? 1.0f : e;
  if (m < 0.0f) n = expf(x - m);  // x is at most m then
  return n / (1.0f + e);
}

// Maximum and sum over the L lanes of a token, the same in all of them: rotations within 16 lanes,
// then rows and halves of the wave swapped.
template <int L>
__device__ inline uint32_t token_max(uint32_t v) {
  v = max(v, rotated<kRor8>(v));
  v = max(v, rotated<kRor4>(v));
  v = max(v, rotated<kRor2>(v));
  v = max(v, rotated<kRor1>(v));
  if (L >= 32) {
    const auto w = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(w[0], w[1]);
  }
  if (L >= 64) {
    const auto w = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(w[0], w[1]);
  }
  return v;
}
template <int L>
__device__ inline unsigned long long token_max(unsigned long long v) {
  // the high words' maximum, then the low words' among the lanes that have it
  const uint32_t hi = token_max<L>((uint32_t)(v >> 32));
  return (unsigned long long)hi << 32 | token_max<L>((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
template <int L>
__device__ inline float token_sum(float v) {
  auto at = [](uint32_t x) { return __builtin_bit_cast(float, x); };
  v += at(rotated<kRor8>(__builtin_bit_cast(uint32_t, v)));
  v += at(rotated<kRor4>(__builtin_bit_cast(uint32_t, v)));
  v += at(rotated<kRor2>(__builtin_bit_cast(uint32_t, v)));
  v += at(rotated<kRor1>(__builtin_bit_cast(uint32_t, v)));
  if (L >= 32) {
    const auto w = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = at(w[0]) + at(w[1]);
  }
  if (L >= 64) {
    const auto w = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = at(w[0]) + at(w[1]);
  }
  return v;
}
template <int L>
__device__ inline double token_sum(double v) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// 4 logits from element i, of which n are in the row (the others: -inf).  vec: the row is aligned to 4 values
// and n is 4 or at most 0.
template <bool BF16>
__device__ inline f32x4 load_4(const void *p, long long i, int n, bool vec) {
  const float ninf = -__builtin_inff();
  f32x4 v = {ninf, ninf, ninf, ninf};
  if (vec) {
    if (n <= 0) return v;
    if constexpr (BF16) {
      const uint2 q = *(const uint2 *)((const uint16_t *)p + i);
      v = (f32x4){bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
    } else {
      v = *(const f32x4 *)((const float *)p + i);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) v[j] = load_logit<BF16>(p, i + j);
  }
  return v;
}

}  // namespace moe
