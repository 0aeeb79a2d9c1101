// moe_quant_rows, moe_quant_weight: rows and expert weights into 8 bits with a power-of-two
// scale for each block of 128 (1 x 128 of a row, 128 x 128 of a weight matrix).
//
// Both read each value once and write each byte once: HBM-bound.  32768 rows of 7168 gathered from 16384
// (0.91 GB with the 16-bit copy) take 174 us, 5.2 TB/s; 68 weights of 2048 x 1408 (0.78 GB) 147 us,
// 5.3 TB/s; torch's copy of 4 GiB moves 4.8.
#include "fp8.hpp"

namespace moe {

constexpr int kQuantMaxThreads = 1024;
constexpr int kQuantPer = 16;  // values per thread
constexpr int kQuantLanes = kBlock / kQuantPer;  // threads per block of 128
constexpr int kQuantMaxGridX = 1 << 20;

// A thread's 16 values of a row: 8 from column 8 l of the block (l = its place among the block's 8
// threads) and 8 from column 64 + 8 l, so that each load and store of a wave covers whole runs of 64
// values.  bf16 values stay packed as loaded; Row<false> holds fp32 (an fp32 row, or a weighted one).
template <bool PACKED>
struct Row;

template <>
struct Row<true> {
  u32x4 t[2];
  __device__ inline void zero() { t[0] = t[1] = (u32x4){0, 0, 0, 0}; }
  // Bits of the largest finite magnitude, as fp32 bits.
  __device__ inline uint32_t mag() const {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 4; ++q) m = mag_max2(m, t[h][q]);
    m = max(m << 16, m & 0xFFFF0000u);
    if (m >= 0x7F800000u) {  // an infinity or NaN among them: value by value
      m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) m = max(m, max(finite_mag(bf16_lo(t[h][q])), finite_mag(bf16_hi(t[h][q]))));
    }
    return m;
  }
  template <int FMT>
  __device__ inline uint2 pack(int h, float scale) const {
    uint2 o;
    o.x = pack_fp8x4<FMT>(t[h][0], t[h][1], scale);
    o.y = pack_fp8x4<FMT>(t[h][2], t[h][3], scale);
    return o;
  }
  __device__ inline u32x4 bf16(int h) const { return t[h]; }
};

template <>
struct Row<false> {
  float v[16];
  __device__ inline void zero() {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.0f;
  }
  __device__ inline uint32_t mag() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, finite_mag(v[e]));
    return m;
  }
  template <int FMT>
  __device__ inline uint2 pack(int h, float scale) const {
    uint2 o;
    o.x = pack_fp8x4<FMT>(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3], scale);
    o.y = pack_fp8x4<FMT>(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7], scale);
    return o;
  }
  __device__ inline u32x4 bf16(int h) const {
    u32x4 t;
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = pack_bf16x2(v[8 * h + 2 * e], v[8 * h + 2 * e + 1]);
    return t;
  }
};

// 8 values from index i of the source, as part h of a row.
template <bool BF16>
__device__ inline void load_part(Row<true> &r, int h, const void *x, long long i, float) {
  r.t[h] = *(const u32x4 *)((const uint16_t *)x + i);
}

template <bool BF16>
__device__ inline void load_part(Row<false> &r, int h, const void *x, long long i, float w) {
  if constexpr (BF16) {
    const u32x4 t = *(const u32x4 *)((const uint16_t *)x + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      r.v[8 * h + 2 * q] = w * bf16_lo(t[q]);
      r.v[8 * h + 2 * q + 1] = w * bf16_hi(t[q]);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f32x4 t = *(const f32x4 *)((const float *)x + i + 4 * p);
#pragma unroll
      for (int q = 0; q < 4; ++q) r.v[8 * h + 4 * p + q] = w * t[q];
    }
  }
}

// One row per grid x step.
template <bool BF16, int FMT, bool WEIGHTED>
__global__ __launch_bounds__(kQuantMaxThreads) void k_quant_rows(
    const void *__restrict__ x, long long src_rows, const int32_t *__restrict__ gather, int div,
    const float *__restrict__ row_scale, uint8_t *__restrict__ q, uint8_t *__restrict__ scale,
    void *__restrict__ copy, long long rows, int width, int pitch) {
  const int nblk = (width + kBlock - 1) / kBlock;
  for (long long i = blockIdx.x; i < rows; i += gridDim.x) {
    long long src = i;
    float w = 1.0f;
    if (gather) {
      const int c = gather[i];
      src = c < 0 ? -1 : c / div;
      if (src >= src_rows) src = -1;
      if (WEIGHTED && src >= 0) w = row_scale[c];
    } else if (WEIGHTED) {
      w = row_scale[i];
    }
    for (int u = blockIdx.y * blockDim.x + threadIdx.x; u < nblk * kQuantLanes; u += gridDim.y * blockDim.x) {
      const int b = u / kQuantLanes, c0 = b * kBlock + u % kQuantLanes * 8;
      Row<BF16 && !WEIGHTED> r;
      r.zero();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (src >= 0 && c0 + 64 * h < width) load_part<BF16>(r, h, x, src * width + c0 + 64 * h, w);
      uint32_t mag = r.mag();
#pragma unroll
      for (int off = 1; off < kQuantLanes; off <<= 1) mag = max(mag, (uint32_t)__shfl_xor((int)mag, off, kWave));
      const int ex = block_exponent<FMT>(mag);
      const float es = exponent_scale(ex);
      if (u % kQuantLanes == 0) scale[i * pitch + b] = (uint8_t)(ex + 127);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const long long at = i * width + c0 + 64 * h;
        if (c0 + 64 * h >= width) continue;
        const unsigned long long bytes = __builtin_bit_cast(unsigned long long, r.template pack<FMT>(h, es));
        // q past the caches or not, the copy past them, as measured (32768 rows gathered from 16384, of 7168, us; q
        // through / past): bf16 rows with a copy 168 / 191 (193 with neither past), weighted 207 / 186, fp32 345 / 339;
        // 32768 fp32 rows of 2048 without a copy 58 / 50.  At other shapes the two lie within a tenth of each other,
        // either way: weighted bf16 rows of 2048 with a copy 52 / 56, of 7168 without one 138 / 128.
        if constexpr (BF16 && !WEIGHTED)
          *(unsigned long long *)(q + at) = bytes;
        else
          __builtin_nontemporal_store(bytes, (unsigned long long *)(q + at));
        if (!copy) continue;
        if constexpr (BF16) {
          __builtin_nontemporal_store(r.bf16(h), (u32x4 *)((uint16_t *)copy + at));
        } else {
          f32x4 *d = (f32x4 *)((float *)copy + at);
#pragma unroll
          for (int p = 0; p < 2; ++p)
            __builtin_nontemporal_store((f32x4){r.v[8 * h + 4 * p], r.v[8 * h + 4 * p + 1],
                                                r.v[8 * h + 4 * p + 2], r.v[8 * h + 4 * p + 3]}, d + p);
        }
      }
    }
    if (blockIdx.y == 0)
      for (int b = nblk + threadIdx.x; b < pitch; b += blockDim.x) scale[i * pitch + b] = kUnitScale;
  }
}

// N consecutive values from index i of a bf16 or fp32 array, widened.
template <bool BF16, int N>
__device__ inline void load_values(const void *p, long long i, float (&v)[N]) {
  if constexpr (BF16) {
    const u32x4 *s = (const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
    for (int h = 0; h < N / 8; ++h) {
      const u32x4 t = s[h];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[8 * h + 2 * q] = bf16_lo(t[q]);
        v[8 * h + 2 * q + 1] = bf16_hi(t[q]);
      }
    }
  } else {
    const f32x4 *s = (const f32x4 *)((const float *)p + i);
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
      const f32x4 t = s[h];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[4 * h + q] = t[q];
    }
  }
}

// One 128 x 128 block of one expert per workgroup: 256 threads of 4 x 16 values.  q keeps the
// weights' own order, qt is transposed (through LDS), both with the block's one exponent.
constexpr int kWtThreads = 256;
constexpr int kWtLd = 132;  // LDS bytes per transposed row

template <bool BF16>
__global__ __launch_bounds__(kWtThreads) void k_quant_weight(
    const void *__restrict__ w, uint8_t *__restrict__ q, uint8_t *__restrict__ q_scale,
    uint8_t *__restrict__ qt, uint8_t *__restrict__ qt_scale, int Kd, int N, int kb_n, int nb_n,
    long long blocks) {
  __shared__ uint32_t wave_mag[kWtThreads / kWave];
  __shared__ uint8_t tile[kBlock * kWtLd];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int r0 = tid >> 3, c0 = (tid & 7) * 16;
  const int pq = (int)scale_pitch(N), pt = (int)scale_pitch(Kd);
  for (long long t = blockIdx.x; t < blocks; t += gridDim.x) {
    const int nb = (int)(t % nb_n), kb = (int)(t / nb_n % kb_n);
    const long long g = t / nb_n / kb_n;
    const int k0 = kb * kBlock, n0 = nb * kBlock;
    float v[4][16];
    uint32_t mag = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int k = k0 + r0 + 32 * p, n = n0 + c0;
#pragma unroll
      for (int e = 0; e < 16; ++e) v[p][e] = 0.0f;
      if (k < Kd && n < N) load_values<BF16>(w, (g * Kd + k) * N + n, v[p]);
#pragma unroll
      for (int e = 0; e < 16; ++e) mag = max(mag, finite_mag(v[p][e]));
    }
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) mag = max(mag, (uint32_t)__shfl_xor((int)mag, off, kWave));
    if (lane == 0) wave_mag[wid] = mag;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWtThreads / kWave; ++i) mag = max(mag, wave_mag[i]);
    const int ex = block_exponent<MOE_E4M3>(mag);
    const float es = exponent_scale(ex);
    // each block writes its own byte; the last one of a row of scales pads the row
    if (q_scale) {
      uint8_t *s = q_scale + (g * kb_n + kb) * pq;
      if (tid == 0) s[nb] = (uint8_t)(ex + 127);
      if (nb == nb_n - 1)
        for (int i = nb_n + tid; i < pq; i += kWtThreads) s[i] = kUnitScale;
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = r0 + 32 * p, k = k0 + r;
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_fp8x4<MOE_E4M3>(v[p][4 * e], v[p][4 * e + 1], v[p][4 * e + 2], v[p][4 * e + 3], es);
      if (q && k < Kd && n0 + c0 < N) *(u32x4 *)(q + (g * Kd + k) * N + n0 + c0) = o;
#pragma unroll
      for (int e = 0; e < 16; ++e) tile[(c0 + e) * kWtLd + r] = (uint8_t)(o[e >> 2] >> (8 * (e & 3)));
    }
    __syncthreads();
    if (qt) {
      const int n = n0 + (tid >> 1), kk = (tid & 1) * 64;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (n >= N || k0 + kk + 16 * e >= Kd) continue;
        u32x4 o;
#pragma unroll
        for (int h = 0; h < 4; ++h) o[h] = *(const uint32_t *)(tile + (tid >> 1) * kWtLd + kk + 16 * e + 4 * h);
        *(u32x4 *)(qt + (g * N + n) * Kd + k0 + kk + 16 * e) = o;
      }
    }
    if (qt_scale) {
      uint8_t *s = qt_scale + (g * nb_n + nb) * pt;
      if (tid == 0) s[kb] = (uint8_t)(ex + 127);
      if (kb == kb_n - 1)
        for (int i = kb_n + tid; i < pt; i += kWtThreads) s[i] = kUnitScale;
    }
    __syncthreads();
  }
}

template <bool BF16, int FMT>
static void launch_quant_rows(dim3 grid, int threads, hipStream_t stream, const void *x,
                              int64_t src_rows, const int32_t *gather, int div,
                              const float *row_scale, void *q, void *scale, void *copy, int64_t rows,
                              int64_t width, int pitch) {
  if (row_scale)
    hipLaunchKernelGGL((k_quant_rows<BF16, FMT, true>), grid, dim3(threads), 0, stream, x, src_rows,
                       gather, div, row_scale, (uint8_t *)q, (uint8_t *)scale, copy, rows, (int)width,
                       pitch);
  else
    hipLaunchKernelGGL((k_quant_rows<BF16, FMT, false>), grid, dim3(threads), 0, stream, x, src_rows,
                       gather, div, row_scale, (uint8_t *)q, (uint8_t *)scale, copy, rows, (int)width,
                       pitch);
}

}  // namespace moe

using namespace moe;

constexpr int64_t kMaxWidth = 1 << 22;

extern "C" size_t moe_scale_row_bytes(int64_t n) { return n < 1 ? 0 : (size_t)scale_pitch(n); }

extern "C" moe_status_t moe_quant_rows(moe_dtype dtype, moe_fp8 fmt, int64_t rows, int64_t width,
                                       const void *x, int64_t src_rows, const int32_t *gather,
                                       int32_t gather_div, const float *row_scale, void *q,
                                       void *scale, void *copy, hipStream_t stream) {
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_EINVAL;
  if (fmt != MOE_E4M3 && fmt != MOE_E5M2) return MOE_EINVAL;
  if (rows < 0 || rows >= (1LL << 31) || width < 16 || width % 16 || width > kMaxWidth) return MOE_EINVAL;
  if (src_rows < 0 || src_rows >= (1LL << 31) || gather_div < 1) return MOE_EINVAL;
  if (!gather && rows > src_rows) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (src_rows == 0) return MOE_EINVAL;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q) || !aligned16(scale) || !aligned16(copy) ||
      (uintptr_t)gather % 4 || (uintptr_t)row_scale % 4)
    return MOE_EINVAL;
  const int pitch = (int)scale_pitch(width);
  const int units = ceil_div(width, kBlock) * kQuantLanes;  // threads of one row
  const int threads = units < kQuantMaxThreads ? (units + kWave - 1) / kWave * kWave : kQuantMaxThreads;
  const dim3 grid((unsigned)(rows < kQuantMaxGridX ? rows : kQuantMaxGridX),
                  (unsigned)ceil_div(units, threads));
  const auto launch = dtype == MOE_BF16
                          ? (fmt == MOE_E4M3 ? launch_quant_rows<true, MOE_E4M3> : launch_quant_rows<true, MOE_E5M2>)
                          : (fmt == MOE_E4M3 ? launch_quant_rows<false, MOE_E4M3> : launch_quant_rows<false, MOE_E5M2>);
  launch(grid, threads, stream, x, src_rows, gather, gather_div, row_scale, q, scale, copy, rows, width, pitch);
  return launch_status();
}

extern "C" moe_status_t moe_quant_weight(moe_dtype dtype, int32_t G, int32_t Kd, int32_t N,
                                         const void *w, void *q, void *q_scale, void *qt,
                                         void *qt_scale, hipStream_t stream) {
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_EINVAL;
  if (G < 1 || Kd < 16 || N < 16 || Kd % 16 || N % 16 || Kd > kMaxWidth || N > kMaxWidth) return MOE_EINVAL;
  if (!w || (!q && !qt) || !q != !q_scale || !qt != !qt_scale) return MOE_EINVAL;
  if (!aligned16(w) || !aligned16(q) || !aligned16(q_scale) || !aligned16(qt) || !aligned16(qt_scale))
    return MOE_EINVAL;
  const int kb_n = ceil_div(Kd, kBlock), nb_n = ceil_div(N, kBlock);
  const long long blocks = (long long)G * kb_n * nb_n;
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22)));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_quant_weight<true>, grid, dim3(kWtThreads), 0, stream, w, (uint8_t *)q,
                       (uint8_t *)q_scale, (uint8_t *)qt, (uint8_t *)qt_scale, Kd, N, kb_n, nb_n,
                       blocks);
  else
    hipLaunchKernelGGL(k_quant_weight<false>, grid, dim3(kWtThreads), 0, stream, w, (uint8_t *)q,
                       (uint8_t *)q_scale, (uint8_t *)qt, (uint8_t *)qt_scale, Kd, N, kb_n, nb_n,
                       blocks);
  return launch_status();
}
