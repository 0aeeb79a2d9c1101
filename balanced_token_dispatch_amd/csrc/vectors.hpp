// Runs of eight values as a thread's step, at any alignment, and checks of what a call's tensors share.
#pragma once

#include "common.hpp"

namespace moe {

// n (1 to 8) values of a tensor from element i, as fp32; the rest 0.  Eight are read in vectors at any
// alignment of the element.
template <bool BF16>
__device__ inline void load_8(const void *p, long long i, int n, float (&v)[8]) {
  if constexpr (BF16) {
    const uint16_t *q = (const uint16_t *)p + i;
    if (n >= 8) {
      u32x4 t;
      __builtin_memcpy(&t, q, 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(t[j]), v[2 * j + 1] = bf16_hi(t[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? __builtin_bit_cast(float, (uint32_t)q[j] << 16) : 0.0f;
    }
  } else {
    const float *q = (const float *)p + i;
    if (n >= 8) {
      f32x4 t[2];
      __builtin_memcpy(t, q, 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = t[j >> 2][j & 3];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? q[j] : 0.0f;
    }
  }
}

// The first n of eight values to a tensor from element i on, rounded to its type.
template <bool BF16>
__device__ inline void store_8(void *p, long long i, int n, const float (&v)[8]) {
  if constexpr (BF16) {
    uint16_t *q = (uint16_t *)p + i;
    u32x4 t;
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    if (n >= 8) {
      __builtin_memcpy(q, &t, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = (uint16_t)(j & 1 ? t[j >> 1] >> 16 : t[j >> 1]);
    }
  } else {
    float *q = (float *)p + i;
    if (n >= 8) {
      const f32x4 t[2] = {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
      __builtin_memcpy(q, t, 32);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = v[j];
    }
  }
}

// Bytes of i values.  A row's place as a pointer that is the same in all lanes and 32 bits of offset in it spares the
// lanes 64-bit sums.
template <bool BF16>
__device__ inline long long bytes_of(long long i) { return i * (BF16 ? 2 : 4); }

// Eight values as they lie in memory, at any alignment of the element: the values from `at` on of a row.
// STREAM: past the caches (see kStreamBytes).
template <bool BF16>
struct Raw;

template <>
struct Raw<true> {
  u32x4 t;
  typedef u32x4 __attribute__((aligned(2))) Any;
  template <bool STREAM>
  __device__ inline void load(const void *row, uint32_t at) {
    const Any *p = (const Any *)((const char *)row + 2 * at);
    if constexpr (STREAM) t = __builtin_nontemporal_load(p); else t = *p;
  }
  template <bool STREAM>
  __device__ inline void store(void *row, uint32_t at) const {
    Any *p = (Any *)((char *)row + 2 * at);
    if constexpr (STREAM) __builtin_nontemporal_store(t, p); else *p = t;
  }
  __device__ inline Raw() {}
  __device__ inline Raw(const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  }
  __device__ inline void values(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(t[j]), v[2 * j + 1] = bf16_hi(t[j]);
  }
};

template <>
struct Raw<false> {
  f32x4 t[2];
  typedef f32x4 __attribute__((aligned(4))) Any;
  template <bool STREAM>
  __device__ inline void load(const void *row, uint32_t at) {
    const Any *p = (const Any *)((const char *)row + 4 * at);
    if constexpr (STREAM)
      t[0] = __builtin_nontemporal_load(p), t[1] = __builtin_nontemporal_load(p + 1);
    else
      t[0] = p[0], t[1] = p[1];
  }
  template <bool STREAM>
  __device__ inline void store(void *row, uint32_t at) const {
    Any *p = (Any *)((char *)row + 4 * at);
    if constexpr (STREAM)
      __builtin_nontemporal_store(t[0], p), __builtin_nontemporal_store(t[1], p + 1);
    else
      p[0] = t[0], p[1] = t[1];
  }
  __device__ inline Raw() {}
  __device__ inline Raw(const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j >> 2][j & 3] = v[j];
  }
  __device__ inline void values(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = t[j >> 2][j & 3];
  }
};

// The row of a tensor that begins `bytes` into it.
__device__ inline const char *row_at(const void *p, long long bytes) { return (const char *)p + bytes; }
__device__ inline char *row_at(void *p, long long bytes) { return (char *)p + bytes; }

// Bytes moved from which a kernel's loads and stores ask the caches to keep nothing: whoever reads what was written finds
// little of it in the memory-side cache (256 MB) then, and evictions cost.  A kernel and one that reads its results
// after it, us with / without: norm of 7168 columns with its sum written, 235 MB 60.8 / 58.8, 470 MB 118 / 123, 940 MB
// 231 / 248; dropout 84 MB 22.2 / 21.7, 252 MB 57.5 / 58.9, 504 MB 111 / 117.  Alone, the norm of 470 MB takes 79.0 / 81.8,
// the dropout of 352 MB 55.4 / 62.3.  Norm rows of up to 512 and above 16384 columns and the balance loss do not ask (not
// measured for them).
constexpr int64_t kStreamBytes = 256 << 20;

// Whether two ranges share memory.  Ranges that are the same one are told apart by `same`.
inline bool shares(const void *a, size_t an, const void *b, size_t bn, bool same) {
  if (!a || !b || !an || !bn) return false;
  if (same && a == b) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + bn && y < x + an;
}

// Whether output o (bytes long) shares memory with none of n ranges but, where it may take a place, with all of one that
// may be taken.
struct Range {
  const void *p;
  size_t bytes;
  bool place = false;  // an output may take its place
};
inline bool stands_alone(const void *o, size_t bytes, const Range *r, int n, bool takes_place = false) {
  for (int i = 0; i < n; ++i)
    if (shares(o, bytes, r[i].p, r[i].bytes, takes_place && r[i].place)) return false;
  return true;
}

}  // namespace moe
