// moe_quant_rows, moe_quant_weight: rows and expert weights into 8 bits with a power-of-two
// scale for each block of 128 (1 x 128 of a row, 128 x 128 of a weight matrix).
//
// Both read each value once and write each byte once: HBM-bound.
#include "fp8.hpp"

namespace moe {

constexpr int kQuantMaxThreads = 1024;
constexpr int kQuantPer = 16;  // values per thread: one 16-byte store of 8-bit values
constexpr int kQuantLanes = kBlock / kQuantPer;  // threads per block of 128
constexpr int kQuantMaxGridX = 1 << 20;

// This thread's 16 values of a row (bf16 or fp32), widened.
template <bool BF16>
__device__ inline void load16(const void *p, long long i, float (&v)[kQuantPer]) {
  if constexpr (BF16) {
    const u32x4 *s = (const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
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
    for (int h = 0; h < 4; ++h) {
      const f32x4 t = s[h];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[4 * h + q] = t[q];
    }
  }
}

// One row per grid x step, kQuantPer values per thread, 8 threads per block of 128.
template <bool BF16, int FMT>
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
      if (row_scale && src >= 0) w = row_scale[c];
    } else if (row_scale) {
      w = row_scale[i];
    }
    for (int u = blockIdx.y * blockDim.x + threadIdx.x; u < pitch * kQuantLanes;
         u += gridDim.y * blockDim.x) {
      const int b = u / kQuantLanes, c0 = u * kQuantPer;
      float v[kQuantPer] = {};
      if (src >= 0 && c0 < width) {
        load16<BF16>(x, src * width + c0, v);
        if (row_scale) {
#pragma unroll
          for (int e = 0; e < kQuantPer; ++e) v[e] *= w;
        }
      }
      uint32_t mag = 0;
#pragma unroll
      for (int e = 0; e < kQuantPer; ++e) mag = max(mag, finite_mag(v[e]));
#pragma unroll
      for (int off = 1; off < kQuantLanes; off <<= 1) mag = max(mag, (uint32_t)__shfl_xor((int)mag, off, kWave));
      const int ex = block_exponent<FMT>(mag);
      if (u % kQuantLanes == 0)
        scale[i * pitch + b] = (uint8_t)(b < nblk ? ex + 127 : kUnitScale);
      if (c0 >= width) continue;
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_fp8x4<FMT>(ldexpf(v[4 * e], -ex), ldexpf(v[4 * e + 1], -ex),
                               ldexpf(v[4 * e + 2], -ex), ldexpf(v[4 * e + 3], -ex));
      *(u32x4 *)(q + i * width + c0) = o;
      if (copy) {
        if constexpr (BF16) {
          u32x4 *d = (u32x4 *)((uint16_t *)copy + i * width + c0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u32x4 t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = pack_bf16x2(v[8 * h + 2 * e], v[8 * h + 2 * e + 1]);
            d[h] = t;
          }
        } else {
          f32x4 *d = (f32x4 *)((float *)copy + i * width + c0);
#pragma unroll
          for (int h = 0; h < 4; ++h) d[h] = (f32x4){v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        }
      }
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
      if (k < Kd && n < N) load16<BF16>(w, (g * Kd + k) * N + n, v[p]);
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
        o[e] = pack_fp8x4<MOE_E4M3>(ldexpf(v[p][4 * e], -ex), ldexpf(v[p][4 * e + 1], -ex),
                                    ldexpf(v[p][4 * e + 2], -ex), ldexpf(v[p][4 * e + 3], -ex));
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

template <bool BF16>
static void launch_quant_rows(moe_fp8 fmt, dim3 grid, int threads, hipStream_t stream,
                              const void *x, int64_t src_rows, const int32_t *gather, int div,
                              const float *row_scale, void *q, void *scale, void *copy,
                              int64_t rows, int64_t width, int pitch) {
  if (fmt == MOE_E5M2)
    hipLaunchKernelGGL((k_quant_rows<BF16, MOE_E5M2>), grid, dim3(threads), 0, stream, x, src_rows,
                       gather, div, row_scale, (uint8_t *)q, (uint8_t *)scale, copy, rows,
                       (int)width, pitch);
  else
    hipLaunchKernelGGL((k_quant_rows<BF16, MOE_E4M3>), grid, dim3(threads), 0, stream, x, src_rows,
                       gather, div, row_scale, (uint8_t *)q, (uint8_t *)scale, copy, rows,
                       (int)width, pitch);
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
  if (src_rows < 1 || src_rows >= (1LL << 31) || gather_div < 1) return MOE_EINVAL;
  if (!gather && rows > src_rows) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q) || !aligned16(scale) || !aligned16(copy))
    return MOE_EINVAL;
  const int pitch = (int)scale_pitch(width);
  const int units = pitch * kQuantLanes;  // threads of one row, the padding of its scales included
  const int threads = units < kQuantMaxThreads ? units : kQuantMaxThreads;
  const dim3 grid((unsigned)(rows < kQuantMaxGridX ? rows : kQuantMaxGridX),
                  (unsigned)ceil_div(units, threads));
  if (dtype == MOE_BF16)
    launch_quant_rows<true>(fmt, grid, threads, stream, x, src_rows, gather, gather_div, row_scale,
                            q, scale, copy, rows, width, pitch);
  else
    launch_quant_rows<false>(fmt, grid, threads, stream, x, src_rows, gather, gather_div, row_scale,
                             q, scale, copy, rows, width, pitch);
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
