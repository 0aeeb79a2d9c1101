// moe_group_gemm_scaled: the grouped GEMM with both operands in 8 bits and a power-of-two
// scale for each block of 128 (1 x 128 of the rows, 128 x 128 of the weights):
//
//   out[m, n] = sum over blocks kb of 2^(sa[m, kb] + sb[g, n / 128, kb] - 254)
//               * sum over k in block kb of a[m, k] b[g, n, k],     m in segment g.
//
// Both operands are contiguous along the contraction (FWD takes the transposed weights of
// moe_quant_weight, DGRAD the ones in their own order), so one kernel serves both.  The scales
// go into the matrix instruction (v_mfma_scale_f32_*_f8f6f4): one byte per row and 32 values of
// the contraction, so a block of 128 passes the same byte four times, and the fp32 accumulators
// hold the scaled sum throughout.
//
// What the matrix unit rounds (measured on gfx950, the same in the unscaled 8-bit instructions):
// it lines up the 8 products of 8 neighbouring k's at the largest one's exponent E and cuts each
// off below 2^(E - 13), then adds the groups and the accumulator in fp32.  Against the operands'
// own rounding to 8 bits (2^-4 of each value) that is nothing: 4e-5 of the result's norm on
// operands of random bytes, where rounding the result to bf16 costs 1.7e-3.  It is why there is no
// fp32 output here.
#include "fp8.hpp"

namespace moe {

constexpr int kScMaxDim = 1 << 22;  // largest Kd and N (offsets within a tile stay in 32 bits)
constexpr int kScMaxG = 1088;

// ---- Few rows -----------------------------------------------------------------------------
// 16 rows of one segment x 16 output columns per workgroup of 4 waves; wave w takes the blocks
// kb = w, w + 4, ... of the contraction, straight from memory into v_mfma_scale_f32_16x16x128,
// and the four sums are added in wave order through LDS.
constexpr int kFewRows = 16, kFewCols = 16, kFewWaves = 4, kFewThreads = 64 * kFewWaves;

// Segment table in LDS: sCu (clamped to [0, M_total]) and sStart[rho] = first tile of `tile`
// rows of segment rho; returns the number of tiles.
template <int THREADS>
__device__ inline int sc_build_tiles(const int32_t *cu, int G, int M_total, int tile, int *sCu,
                                     int *sStart) {
  __shared__ int tmp[THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  for (int i = tid; i <= G; i += THREADS) sCu[i] = min(max(cu[i], 0), M_total);
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < G; base += THREADS) {
    const int rho = base + tid;
    int v = 0;
    if (rho < G) v = max(sCu[rho + 1] - sCu[rho] + tile - 1, 0) / tile;
    int x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off, 64);
      if (lane >= off) x += y;
    }
    if (lane == 63) tmp[wid] = x;
    __syncthreads();
    int before = carry, tot = carry;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
      before += w < wid ? tmp[w] : 0;
      tot += tmp[w];
    }
    if (rho < G) sStart[rho] = before + x - v;
    carry = tot;
    __syncthreads();
  }
  if (tid == 0) sStart[G] = carry;
  __syncthreads();
  return carry;
}

// last rho with sStart[rho] <= t: the segment owning tile t
__device__ inline int sc_find_seg(const int *sStart, int G, int t) {
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sStart[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ inline i32x8 join(u32x4 a, u32x4 b) {
  return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

template <int FMT>
__global__ __launch_bounds__(kFewThreads) void k_scaled_few(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ a_scale,
    const uint8_t *__restrict__ b, const uint8_t *__restrict__ b_scale,
    const int32_t *__restrict__ cu, uint16_t *__restrict__ out, int G, int M_total, int K, int N) {
  __shared__ int sCu[kScMaxG + 1], sStart[kScMaxG + 1];
  __shared__ f32x4 part[kFewWaves][64];
  const int n_rt = sc_build_tiles<kFewThreads>(cu, G, M_total, kFewRows, sCu, sStart);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int n_ct = (N + kFewCols - 1) / kFewCols, nblk = (K + kBlock - 1) / kBlock;
  const long long pitch = scale_pitch(K), total = (long long)n_rt * n_ct;
  const int nnb = (N + kBlock - 1) / kBlock;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const int rt = (int)(t / n_ct), ct = (int)(t % n_ct);
    const int g = sc_find_seg(sStart, G, rt);
    const int m0 = sCu[g] + (rt - sStart[g]) * kFewRows, n0 = ct * kFewCols;
    const int m = m0 + (lane & 15), n = n0 + (lane & 15);
    const bool mok = m < sCu[g + 1], nok = n < N;
    const uint8_t *ar = a + (long long)m * K, *br = b + ((long long)g * N + n) * K;
    const uint8_t *as = a_scale + m * pitch;
    const uint8_t *bs = b_scale + ((long long)g * nnb + n0 / kBlock) * pitch;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int kb = wid; kb < nblk; kb += kFewWaves) {
      const int k = kb * kBlock + 32 * (lane >> 4);
      const u32x4 z = {0, 0, 0, 0};
      const u32x4 a0 = mok && k < K ? *(const u32x4 *)(ar + k) : z;
      const u32x4 a1 = mok && k + 16 < K ? *(const u32x4 *)(ar + k + 16) : z;
      const u32x4 b0 = nok && k < K ? *(const u32x4 *)(br + k) : z;
      const u32x4 b1 = nok && k + 16 < K ? *(const u32x4 *)(br + k + 16) : z;
      const int sa = mok ? as[kb] : kUnitScale, sb = bs[kb];
      // weights as the first operand: each lane ends with 4 consecutive columns of one row
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b0, b1), join(a0, a1), acc, 0,
                                                             FMT == MOE_E5M2 ? 1 : 0, 0, sb, 0, sa);
    }
    part[wid][lane] = acc;
    __syncthreads();
    if (wid == 0) {
      f32x4 v = part[0][lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) v += part[w][lane];
      const int c = n0 + 4 * (lane >> 4);
      if (mok && c < N) {
        uint2 o;
        o.x = pack_bf16x2(v[0], v[1]);
        o.y = pack_bf16x2(v[2], v[3]);
        *(uint2 *)(out + (long long)m * N + c) = o;
      }
    }
    __syncthreads();
  }
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_group_gemm_scaled_workspace_bytes(void) { return 0; }

extern "C" moe_status_t moe_group_gemm_scaled(moe_gemm_op op, moe_fp8 a_fmt, int32_t G, int32_t M_total, int32_t Kd, int32_t N,
                                              const void *a, const void *a_scale, const void *b,
                                              const void *b_scale, const int32_t *cu_seqlens,
                                              void *out, void *ws, size_t ws_bytes,
                                              hipStream_t stream) {
  if (op != MOE_GEMM_FWD && op != MOE_GEMM_DGRAD) return MOE_EINVAL;
  if (a_fmt != MOE_E4M3 && a_fmt != MOE_E5M2) return MOE_EINVAL;
  if (G < 1 || G > kScMaxG || M_total < 0 || Kd < 16 || N < 16 || Kd % 16 || N % 16) return MOE_EINVAL;
  if (Kd > kScMaxDim || N > kScMaxDim) return MOE_EINVAL;
  if (ws && ws_bytes < moe_group_gemm_scaled_workspace_bytes()) return MOE_ENOSPACE;
  if (M_total == 0) return MOE_OK;
  if (!a || !a_scale || !b || !b_scale || !cu_seqlens || !out) return MOE_EINVAL;
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(b) || !aligned16(b_scale) ||
      !aligned16(out) || !aligned16(ws) || ((uintptr_t)cu_seqlens & 3))
    return MOE_EINVAL;
  // both operands end contiguous along the contraction: FWD contracts Kd, DGRAD contracts N
  const int K = op == MOE_GEMM_FWD ? Kd : N, C = op == MOE_GEMM_FWD ? N : Kd;
  const dim3 grid(device_cu_count() * 8), block(kFewThreads);
  const uint8_t *a8 = (const uint8_t *)a, *b8 = (const uint8_t *)b;
  const uint8_t *as = (const uint8_t *)a_scale, *bs = (const uint8_t *)b_scale;
  if (a_fmt == MOE_E4M3)
    hipLaunchKernelGGL(k_scaled_few<MOE_E4M3>, grid, block, 0, stream, a8, as, b8, bs, cu_seqlens,
                       (uint16_t *)out, G, M_total, K, C);
  else
    hipLaunchKernelGGL(k_scaled_few<MOE_E5M2>, grid, block, 0, stream, a8, as, b8, bs, cu_seqlens,
                       (uint16_t *)out, G, M_total, K, C);
  return launch_status();
}
