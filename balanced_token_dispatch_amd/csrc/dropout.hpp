// The dropout mask from a counter: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011), 16 bits for each
// element.  With 32 bits an element the ten rounds (two 32 x 32 products each, at a quarter of the rate of
// an addition) would be needed for every 4 elements instead of 8; p is met to 2^-17 and the scale belongs
// to the p that is met, so that no mean shifts.
#pragma once

#include "vectors.hpp"

namespace moe {

struct Drop {
  const int64_t *rng;  // seed, offset
  unsigned long long offset;
  uint32_t below;  // of 65536: dropped where the 16 bits are below it; 0: no dropout
  uint32_t last;   // 65536 below - 1
  float scale;     // of the others
};

// p in [0, 1]
inline Drop make_drop(double p, const int64_t *rng, int64_t offset) {
  Drop d;
  d.rng = rng;
  d.offset = (unsigned long long)offset;
  d.below = (uint32_t)(65536.0 * p + 0.5);
  d.last = (d.below << 16) - 1;  // all bits for 65536
  d.scale = d.below < 65536 ? 65536.0f / (float)(65536 - d.below) : 0.0f;
  return d;
}

inline bool drop_ok(double p, const int64_t *rng) {
  return p >= 0.0 && p <= 1.0 && (uintptr_t)rng % 8 == 0 && (rng || p == 0.0);
}

// Key and upper counter of a call, the same in every lane.
struct DropKey {
  uint32_t k0, k1, c2, c3;
};

__device__ inline DropKey drop_key(const Drop &d) {
  const unsigned long long seed = d.rng[0], at = (unsigned long long)d.rng[1] + d.offset;
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)at, (uint32_t)(at >> 32)};
}

__device__ inline uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }

// The 128 bits of the eight elements from 8 * block on.
__device__ inline u32x4 philox(unsigned long long block, DropKey k) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = k.c2, c3 = k.c3;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const unsigned long long p0 = (unsigned long long)c0 * 0xD2511F53u, p1 = (unsigned long long)c2 * 0xCD9E8D57u;
    c0 = xor3((uint32_t)(p1 >> 32), c1, k.k0);
    c1 = (uint32_t)p1;
    c2 = xor3((uint32_t)(p0 >> 32), c3, k.k1);
    c3 = (uint32_t)p0;
    k.k0 += 0x9E3779B9u, k.k1 += 0xBB67AE85u;
  }
  return (u32x4){c0, c1, c2, c3};
}

// The bits of eight elements from any element on: of two blocks where it is not the first of one.
__device__ inline u32x4 drop_bits(unsigned long long element, DropKey k) {
  const unsigned long long block = element >> 3;
  const int s = (int)(element & 7);
  u32x4 a = philox(block, k);
  if (s == 0) return a;
  const u32x4 b = philox(block + 1, k);
  uint32_t w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  if (s & 4)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (s & 2)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if (s & 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] >> 16 | w[i + 1] << 16;
  return (u32x4){w[0], w[1], w[2], w[3]};
}

// v = r + drop(v) of eight values.  A half is compared as the upper half of a word, whatever is below it.
__device__ inline void drop_8(u32x4 bits, const Drop &d, float (&v)[8], const float (&r)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = j & 1 ? bits[j >> 1] : bits[j >> 1] << 16;
    v[j] = fmaf(u <= d.last ? 0.0f : v[j], d.scale, r[j]);
  }
}
__device__ inline void drop_8(u32x4 bits, const Drop &d, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = j & 1 ? bits[j >> 1] : bits[j >> 1] << 16;
    v[j] = (u <= d.last ? 0.0f : v[j]) * d.scale;
  }
}

}  // namespace moe
