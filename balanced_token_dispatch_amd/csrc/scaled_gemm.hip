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
#include <type_traits>

#include "fp8.hpp"

namespace moe {

constexpr int kScMaxDim = 1 << 21;  // largest Kd and N (offsets within a tile stay in 32 bits)
constexpr int kScMaxG = 1088;
constexpr long long kScMaxTiles = 1LL << 30;

// ---- Few rows -----------------------------------------------------------------------------
// 16 rows of one segment x 16 CT output columns per workgroup of W waves; wave w takes the blocks
// kb = w, w + W, ... of the contraction, D of them in flight, straight from memory into
// v_mfma_scale_f32_16x16x128 (every weight byte is used once per 16 rows, so staging it in LDS would
// gain nothing), and the W sums are added in wave order through LDS.
//
// Bound by the weights' bytes: 512 rows on 264 experts of 7168 x 2048 read 3.27 GB in 531 to 560 us, 6.2 to 5.8
// TB/s, where torch's copy of 4 GiB moves 4.8 TB/s.  With few weights, by the launch and two trips to memory:
// 6 rows on 6 experts of 2048 x 1408 (17 MB, 3 us at that rate) take 7.7 us.
constexpr int kFewRows = 16, kFewCols = 16;

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
    if (rho < G && sCu[rho + 1] > sCu[rho])
      v = (sCu[rho + 1] - sCu[rho] - 1) / tile + 1;  // (adding tile - 1 first would pass 2^31)
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

// last rho with sStart[rho] <= t: the segment owning tile t, by the whole wave (t the same in all lanes):
// every lane looks at one of 64 places, then at one of those between two.  Halving the range took 7 to
// 10 reads of LDS one after the other.
__device__ inline int sc_find_seg(const int *sStart, int G, int t) {
  const int lane = threadIdx.x & 63, step = (G + kWave - 1) / kWave;  // at most 17
  const int i = lane * step;
  const int base = (__popcll(__ballot(i < G && sStart[min(i, G)] <= t)) - 1) * step;
  const int j = base + lane;
  return base + __popcll(__ballot(lane < step && j < G && sStart[min(j, G)] <= t)) - 1;
}

__device__ inline i32x8 join(u32x4 a, u32x4 b) {
  return (i32x8){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

constexpr int kOutside = 0x7FFFFFF0;  // an offset past every buffer: the load returns zero

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void *base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, 0x00020000);
}

template <int FMT, int W, int CT, int D>
__global__ __launch_bounds__(64 * W) void k_scaled_few(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ a_scale,
    const uint8_t *__restrict__ b, const uint8_t *__restrict__ b_scale,
    const int32_t *__restrict__ cu, uint16_t *__restrict__ out, int G, int M_total, int K, int N) {
  __shared__ int sCu[kScMaxG + 1], sStart[kScMaxG + 1];
  __shared__ f32x4 part[W][CT][64];
  const int n_rt = sc_build_tiles<64 * W>(cu, G, M_total, kFewRows, sCu, sStart);
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_ct = (N + kFewCols * CT - 1) / (kFewCols * CT), nblk = (K + kBlock - 1) / kBlock;
  const int pitch = (int)scale_pitch(K), nnb = (N + kBlock - 1) / kBlock;
  const int total = (int)min((long long)n_rt * n_ct, kScMaxTiles);
  // lane l holds bytes 16 (l / 16) .. + 16 and 64 more on of row l % 16: each load takes whole
  // half lines of 16 rows, and the order of the contraction is the same for both operands
  const int r = lane & 15, kq = 16 * (lane >> 4), off = r * K + kq;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int rt = t / n_ct, n0 = t % n_ct * kFewCols * CT;
    const int g = sc_find_seg(sStart, G, rt);
    const int m0 = __builtin_amdgcn_readfirstlane(sCu[g] + (rt - sStart[g]) * kFewRows);
    const int rows = __builtin_amdgcn_readfirstlane(min(kFewRows, sCu[g + 1] - m0));
    const int cols = min(kFewCols * CT, N - n0);
    // rows past the segment and weights past N lie past their buffers
    const __amdgpu_buffer_rsrc_t ra = buffer_of(a + (long long)m0 * K, rows * K);
    const __amdgpu_buffer_rsrc_t rb = buffer_of(b + ((long long)g * N + n0) * K, cols * K);
    const __amdgpu_buffer_rsrc_t rsa = buffer_of(a_scale + (long long)m0 * pitch, rows * pitch);
    const __amdgpu_buffer_rsrc_t rsb = buffer_of(b_scale + ((long long)g * nnb + n0 / kBlock) * pitch, pitch);
    f32x4 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int k0 = wid; k0 < nblk; k0 += W * D) {
      u32x4 x[D][2 + 2 * CT];
      int sa[D], sb[D];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int kb = k0 + d * W, k = kb * kBlock;
        const bool in0 = k + kq < K, in1 = k + kq + 64 < K;
        const int so = kb < nblk ? k : 0;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int oc = off + c * kFewCols * K;
          x[d][2 + 2 * c] = __builtin_amdgcn_raw_buffer_load_b128(rb, in0 ? oc : kOutside, so, 0);
          x[d][3 + 2 * c] = __builtin_amdgcn_raw_buffer_load_b128(rb, in1 ? oc + 64 : kOutside, so, 0);
        }
        x[d][0] = __builtin_amdgcn_raw_buffer_load_b128(ra, in0 ? off : kOutside, so, 0);
        x[d][1] = __builtin_amdgcn_raw_buffer_load_b128(ra, in1 ? off + 64 : kOutside, so, 0);
        sa[d] = __builtin_amdgcn_raw_buffer_load_b8(rsa, kb < nblk ? r * pitch + kb : kOutside, 0, 0);
        sb[d] = __builtin_amdgcn_raw_buffer_load_b8(rsb, kb < nblk ? kb : kOutside, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);  // all of them in flight before the first is used
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int c = 0; c < CT; ++c)
          // weights as the first operand: each lane ends with 4 consecutive columns of one row
          acc[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              join(x[d][2 + 2 * c], x[d][3 + 2 * c]), join(x[d][0], x[d][1]), acc[c], 0,
              FMT == MOE_E5M2 ? 1 : 0, 0, sb[d], 0, sa[d]);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) part[wid][c][lane] = acc[c];
    __syncthreads();
    if (wid < CT) {
      f32x4 v = part[0][wid][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v += part[w][wid][lane];
      const int c = wid * kFewCols + 4 * (lane >> 4);
      if (r < rows && c < cols) {
        uint2 o;
        o.x = pack_bf16x2(v[0], v[1]);
        o.y = pack_bf16x2(v[2], v[3]);
        *(uint2 *)(out + (long long)(m0 + r) * N + n0 + c) = o;
      }
    }
    __syncthreads();
  }
}

// ---- Many rows ------------------------------------------------------------------------------
// Output tiles of 64 TM x 64 TN on a persistent grid, 4 waves (one per SIMD) of 32 TM x 32 TN each
// in v_mfma_scale_f32_32x32x64 blocks.  A stage is 128 of the contraction (one scale block): whole
// 128-byte lines of each operand's rows, loaded straight into LDS (buffer_load .. lds), in a ring of
// R stages.
//
// What bounds it.  32768 rows on 264 experts of 7168 x 2048 (4.24 GB) take 829 us, 5.1 TB/s: memory.
// With one expert (32768 x 7168 x 2048, 256 x 256 tiles) 372 to 390 us, 2.6 to 2.5 PFLOP/s, for normal
// and for random bytes, where torch's library product takes 310 to 325 and the bare matrix
// instructions reach 4.7-5.0: the chip's power sets the clock there (1.75 GHz; 303 us on zeros, the
// library 229), and the matrix units are busy 61% of the cycles.  Between them, with 1408 of
// contraction (24576 rows, 68 experts, 128 x 256 tiles: 107 us, floor 56), what costs is the tiles' last
// rows (15% more than the rows there are), the last round of tiles (8 for 7.1) and 11 stages a tile
// against one start of the ring and one store of the results.
constexpr int kTileThreads = 256, kTileWaves = 4;
// Scales come in pieces of 16 stages: 16 bytes of each of the tile's rows and then of its column
// blocks, in three buffers in turn (a tile's last piece may be too short a time to fetch the next
// tile's first in, so that one is fetched during the piece before).
constexpr int kScaleStages = 16, kScaleBufs = 3;
constexpr int kGroupRows = 8, kXcdCount = 8;

template <int TM_, int TN_, int R_>
struct Tile {
  static constexpr int TM = TM_, TN = TN_, R = R_;
  static constexpr int rows = 64 * TM, cols = 64 * TN;
  static constexpr int a_bytes = rows * kBlock, stage = (rows + cols) * kBlock;
  static constexpr int a_loads = 2 * TM, b_loads = 2 * TN;  // 1-KB loads per wave and stage
  static constexpr int scale_bytes = rows * 16 + 256;       // of one piece
  static constexpr int ring = R * stage;
  static constexpr bool whole = TM * TN <= 4;
  static constexpr int stores = 2 * TM * TN;                // of one wave's part of the tile
};

typedef __attribute__((address_space(3))) void *lds_ptr;
typedef __attribute__((ext_vector_type(16))) float f32x16;

__device__ inline uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)(lds_ptr)p; }

// 16 bytes per lane from buffer offset off + soff to LDS at m0 + 16 * lane.  Written as asm so that
// the compiler does not track it (its alias analysis cannot tell the ring's stages apart and would
// drain every load at each barrier): no register result, so nothing in flight can overwrite a
// register, and completion is ordered by the explicit waits and barriers of the stage loop alone.
// One wait state separates the write of M0 from its use.
__device__ inline void load_to_lds(int off, __amdgpu_buffer_rsrc_t rs, int soff, uint32_t m0) {
  asm volatile(
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off),
      "s"(rs), "s"(soff), "{m0}"(m0)
      : "memory");
}

// Every wave's LDS reads are done and every wave is here.  Not __syncthreads: that also waits for the
// stores of the tile before.
__device__ inline void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int N>
__device__ inline void wait_loads() {  // at most N vector-memory operations in flight
  static_assert(N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// An operand's rows of K bytes go out 32 a round of loads: load u of wave w covers rows
// 32 u + 8 w .. + 8, 8 lanes a row.  The 16-byte chunk k (0..7) of row r lies at position
// k ^ ((r >> 1) & 7) of its LDS row, which keeps the fragment reads free of bank conflicts.  The byte
// offsets hold for both operands and every stage: a stage moves the scalar offset by 128, which
// the buffer's range check does not look at, so rows past the operand read as zeros.  RAGGED: so does
// what lies past K in the last stage.
template <int LOADS>
struct Offsets {
  int off[LOADS];  // of load u
  int k;           // this lane's contraction index within a stage
};

template <int LOADS>
__device__ inline Offsets<LOADS> offsets(int K) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, r = wid * 8 + (lane >> 3);
  Offsets<LOADS> o;
  o.k = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
#pragma unroll
  for (int u = 0; u < LOADS; ++u) o.off[u] = (r + 32 * u) * K + o.k;
  return o;
}

template <bool RAGGED, int LOADS>
__device__ inline void op_load(const Offsets<LOADS> &o, __amdgpu_buffer_rsrc_t rs, int s, int K,
                               uint32_t lds, int u) {
  int off = o.off[u];
  if (RAGGED) off = s * kBlock + o.k < K ? off : kOutside;
  load_to_lds(off, rs, s * kBlock, lds + u * kTileWaves * 1024);
}

// As load_to_lds where `skip` is 0; a branch inside the asm, because a branch of the compiler's would cut the
// stage in two blocks of code, and it moves the matrix instructions of the first behind the cut.
__device__ inline void load_to_lds_unless(int skip, int off, __amdgpu_buffer_rsrc_t rs, int soff, uint32_t m0) {
  asm volatile(
      "s_cmp_lg_u32 %3, 0\n\t"
      "s_cbranch_scc1 .Lskip%=\n\t"
      "buffer_load_dwordx4 %0, %1, %2 offen lds\n"
      ".Lskip%=:" ::"v"(off),
      "s"(rs), "s"(soff), "s"(skip), "{m0}"(m0)
      : "memory", "scc");
}

// 4 bytes per lane, the same way.
__device__ inline void load4_to_lds_unless(int skip, int off, __amdgpu_buffer_rsrc_t rs, int soff,
                                           uint32_t m0) {
  asm volatile(
      "s_cmp_lg_u32 %3, 0\n\t"
      "s_cbranch_scc1 .Lskip%=\n\t"
      "buffer_load_dword %0, %1, %2 offen lds\n"
      ".Lskip%=:" ::"v"(off),
      "s"(rs), "s"(soff), "s"(skip), "{m0}"(m0)
      : "memory", "scc");
}

// At most N operations in flight, or MORE more where `few` is 0.
template <int N, int MORE>
__device__ inline void wait_loads_or(int few) {
  static_assert(N + MORE < 64, "vmcnt range");
  asm volatile(
      "s_cmp_lg_u32 %0, 0\n\t"
      "s_cbranch_scc1 .Lfew%=\n\t"
      "s_waitcnt vmcnt(%1)\n\t"
      "s_branch .Ldone%=\n"
      ".Lfew%=:\n\t"
      "s_waitcnt vmcnt(%2)\n"
      ".Ldone%=:" ::"s"(few),
      "n"(N + MORE), "n"(N)
      : "memory", "scc");
}

// Fragment of 32 rows (first row `row`) for sub-step ks of a stage: 32 bytes per lane, chunks
// 4 ks + h and 4 ks + 2 + h of half-wave h.  Both operands use the same chunks, and a scale spans
// the stage, so which 64 of the contraction a sub-step takes does not matter.
__device__ inline i32x8 read_fragment(const uint8_t *op, int row, int lane, int ks) {
  const int r = row + (lane & 31), h = lane >> 5, x = (r >> 1) & 7;
  const u32x4 lo = *(const u32x4 *)(op + r * kBlock + ((4 * ks + h) ^ x) * 16);
  const u32x4 hi = *(const u32x4 *)(op + r * kBlock + ((4 * ks + 2 + h) ^ x) * 16);
  return join(lo, hi);
}

template <class T>
struct Fragments {
  i32x8 a[T::TM], b[T::TN];
  // item i of the fragments of sub-step ks: b's first, as every matrix instruction order needs them
  __device__ inline void read(int i, const uint8_t *stage, int wi, int wj, int lane, int ks) {
    if (i < T::TN)
      b[i] = read_fragment(stage + T::a_bytes, wj + 32 * i, lane, ks);
    else
      a[i - T::TN] = read_fragment(stage, wi + 32 * (i - T::TN), lane, ks);
  }
};

template <int FMT>
__device__ inline f32x16 mma(i32x8 b, i32x8 a, f32x16 c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, FMT == MOE_E5M2 ? 1 : 0, 0, sb, 0,
                                                         sa);
}

// The tile as bf16, straight from the accumulators: of each 32 x 32 block a lane holds 4 consecutive
// columns of one row in 4 groups; swapping half-waves between two groups leaves it 8 consecutive
// ones, so a store writes 32 bytes of each of 32 rows.  Every store is issued (a lane past the tile's
// rows or columns has an offset past the buffer), because the waits of the next tile count them.
// cols is a multiple of 16.
template <class T>
__device__ inline void tile_out(const f32x16 (&acc)[T::TM][T::TN], uint16_t *out, int ld, int rows,
                                int cols) {
  const int wid = threadIdx.x >> 6;
  int lane = threadIdx.x & 63;
  // the offsets are worked out per tile, not kept across the stages
  asm volatile("" : "+v"(lane));
  asm volatile("" : "+s"(ld));
  const int wi = (wid >> 1) * 32 * T::TM + (lane & 31), wj = (wid & 1) * 32 * T::TN + (lane >> 5) * 8;
  const __amdgpu_buffer_rsrc_t rs = buffer_of(out, ((rows - 1) * ld + cols) * 2);
  const int off = (wi * ld + wj) * 2;
#pragma unroll
  for (int tm = 0; tm < T::TM; ++tm)
#pragma unroll
    for (int tn = 0; tn < T::TN; ++tn) {
      f32x16 v = acc[tm][tn];
      asm volatile("" : "+a"(v));  // out of its accumulators here, not all blocks at once
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        u32x4 o;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto w = __builtin_amdgcn_permlane32_swap(
              pack_bf16x2(v[8 * g + 2 * h], v[8 * g + 2 * h + 1]),
              pack_bf16x2(v[8 * g + 4 + 2 * h], v[8 * g + 4 + 2 * h + 1]), false, false);
          o[h] = w[0];
          o[2 + h] = w[1];
        }
        const bool in = wi + tm * 32 < rows && wj + tn * 32 + g * 16 < cols;
        __builtin_amdgcn_raw_buffer_store_b128(o, rs, in ? off : kOutside,
                                               (tm * 32 * ld + tn * 32 + g * 16) * 2, 0);
        __builtin_amdgcn_sched_barrier(0);  // one store's registers at a time
      }
    }
}

// Where a tile lies; all in scalar registers.
struct Place {
  const uint8_t *a, *b, *sa, *sb;  // first byte of its rows, weights and their scales
  int m0, rows, j0, cols;          // first row, rows (0: no tile), first column, columns
};

template <class T, int FMT, bool RAGGED>
__global__ __launch_bounds__(kTileThreads) void k_scaled_tiles(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ a_scale,
    const uint8_t *__restrict__ b, const uint8_t *__restrict__ b_scale,
    const int32_t *__restrict__ cu, uint16_t *__restrict__ out, int G, int M_total, int K, int N) {
  constexpr int TM = T::TM, TN = T::TN, R = T::R, NM = TM * TN, H = NM / 2, NF = TM + TN;
  __shared__ __attribute__((aligned(16))) uint8_t ring[T::ring];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kScaleBufs * T::scale_bytes];
  __shared__ int sCu[kScMaxG + 1], sStart[kScMaxG + 1];
  const int n_rt =
      __builtin_amdgcn_readfirstlane(sc_build_tiles<kTileThreads>(cu, G, M_total, T::rows, sCu, sStart));
  const int n_ct = (N + T::cols - 1) / T::cols;
  const int nnb = (N + kBlock - 1) / kBlock, pitch = (int)scale_pitch(K);
  const int total = (int)min((long long)n_rt * n_ct, kScMaxTiles);
  // each XCD takes neighbouring tiles, walked in groups of 8 row tiles: shared panels in its L2
  const int grid = gridDim.x;
  const int lb = grid % kXcdCount ? blockIdx.x : blockIdx.x % kXcdCount * (grid / kXcdCount) + blockIdx.x / kXcdCount;
  auto place = [&](int t) {
    Place p = {a, b, a_scale, b_scale, 0, 0, 0, 0};
    if (t >= total) return p;
    const int per = kGroupRows * n_ct, grp = t / per, r = t - grp * per;
    const int gm = min(kGroupRows, n_rt - grp * kGroupRows);
    const int rt = grp * kGroupRows + r % gm;
    // read from LDS, so uniform only to us: the operands' buffers need them in scalar registers
    const int g = sc_find_seg(sStart, G, rt);
    p.m0 = __builtin_amdgcn_readfirstlane(sCu[g] + (rt - sStart[g]) * T::rows);
    p.rows = __builtin_amdgcn_readfirstlane(min(T::rows, sCu[g + 1] - p.m0));
    p.j0 = r / gm * T::cols;
    p.cols = min(T::cols, N - p.j0);
    p.a = a + (long long)p.m0 * K;
    p.b = b + ((long long)g * N + p.j0) * K;
    p.sa = a_scale + (long long)p.m0 * pitch;
    p.sb = b_scale + ((long long)g * nnb + p.j0 / kBlock) * pitch;
    return p;
  };
  int t = lb;
  if (t >= total) return;
  Place at = place(t), next = place(t + grid);

  // The workgroup's tiles are one stream of stages, nk a tile, in ring slots 0, 1, .. R - 1, 0, ..:
  // near a tile's end the loads that run ahead are the next tile's, so its first stages arrive while
  // the last ones are multiplied and the results stored.  (nk is at least R, so that loads never run
  // past the next tile; stages past the contraction load zeros.)
  //
  // A stage s is two sub-steps of TM TN matrix instructions; behind each the wave issues a few memory
  // operations for later.  R > 2:
  //   sub-step 0: reads the fragments of sub-step 1 and the scales of stage s + 1; issues b's loads of
  //     stage s + R - 1; asks for the next piece of scales;
  //   wait until only the loads of stages s + 2 .. s + R - 1 are in flight (stage s + 1 has landed),
  //   barrier (every wave has read all of stage s);
  //   sub-step 1: reads the fragments of stage s + 1's sub-step 0; issues a's loads of stage s + R into slot
  //     s % R.
  // R = 2 (kDeep), where a stage's slot has to be free early for its loads to have the time they need:
  //   barrier (every wave has read all of stage s, both sub-steps, into registers);
  //   sub-step 0: issues the first two thirds of the loads of stage s + 2 into slot s % 2;
  //   wait until only those are in flight (stage s + 1 has landed), barrier;
  //   sub-step 1: issues the other loads; reads all fragments and the scales of stage s + 1, those of its
  //     sub-step 1 into registers that alternate from stage to stage; asks for the next piece of scales.
  // (32768 x 1 x 7168 x 2048, all in one run: 381 us; loads over one sub-step 403, over both 384.)
  // Loads and stores complete in order, so where the stores of the tile before came after the loads
  // waited for (stage 0), they are counted in; the loads of the scales only make a wait stricter.
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wi = (wid >> 1) * 32 * TM, wj = (wid & 1) * 32 * TN;
  const uint32_t wave_lds = __builtin_amdgcn_readfirstlane(wid) * 1024;
  const uint32_t ring_lds = lds_addr(ring) + wave_lds, scales_lds = lds_addr(scales);
  const int kblocks = (K + kBlock - 1) / kBlock, nk = max(kblocks, R);
  constexpr int kAhead = (R - 2) * (T::a_loads + T::b_loads);
  constexpr int kAll = T::a_loads + T::b_loads;
  constexpr bool kDeep = R == 2;
  constexpr int kSpan = 3 * NM / 2;  // matrix instructions over which a stage's loads go out (kDeep)
  static_assert(!(kDeep && T::whole), "whole stages need a ring of more than 2");
  // b's loads go out in sub-step 0, one stage later than a's
  constexpr bool kSplit = !kDeep && !T::whole;
  constexpr int kLoads = T::a_loads > T::b_loads ? T::a_loads : T::b_loads;
  const Offsets<kLoads> lo = offsets<kLoads>(K);

  // The piece of a tile's scales from byte `at` on into LDS buffer `buf`, where `skip` is 0: wave
  // w < TM loads a's rows 64 w .. + 64, and wave 0 the rows of b's column blocks.
  const int w = __builtin_amdgcn_readfirstlane(wid), scale_off = (lane + 64 * (w / TM ? 0 : w)) * pitch;
  const int block_off = (lane >> 2) * pitch + (lane & 3) * 4;
  auto load_scales = [&](int skip, const Place &p, int at, int buf) {
    const uint32_t to = scales_lds + buf * T::scale_bytes;
    load_to_lds_unless(skip | w / TM, scale_off, buffer_of(p.sa, p.rows * pitch), at, to + w * 1024);
    load4_to_lds_unless(skip | w, block_off, buffer_of(p.sb, (p.cols + kBlock - 1) / kBlock * pitch),
                        at, to + T::rows * 16);
  };
  // What to fetch at stage s (q: its place in its piece, in buffer buf).  At the start of a piece, the
  // piece after it: the tile's own, or after its last one the next tile's first.  A last piece of
  // fewer than R stages is over before a load then issued is sure to have landed; what follows it is
  // fetched from stage kSecond of the piece before, into the buffer after next.
  constexpr int kSecond = T::whole ? 8 : 14;
  struct Fetch {
    int skip, at, to;  // 0: fetch; first byte of the rows of scales; LDS buffer
    bool own;
  };
  auto next_scales = [&](int s, int q, int nk, int buf) {
    const int rest = nk - (s + kScaleStages - q);  // stages of the tile after this piece
    // each 0 where it holds (as numbers: truth values would go through vector registers): a piece
    // starts that is not a short last one; place kSecond, and the piece after this one is a short last
    const int first = q | max(R - (nk - s), 0);
    const int second = (q ^ kSecond) | max(rest - R + 1, 0) | max(1 - rest, 0);
    Fetch f;
    f.own = q == 0 && rest > 0;
    f.skip = first * second;
    f.at = f.own ? s + kScaleStages : 0;
    const int to = buf + (second == 0 ? 2 : 1);
    f.to = to >= kScaleBufs ? to - kScaleBufs : to;
    if constexpr (!T::whole)  // worked out where it is called, some matrix instructions ahead of its use
      asm volatile("" : "+s"(f.skip), "+s"(f.at), "+s"(f.to));
    return f;
  };
  load_scales(0, at, 0, 0);
#pragma unroll
  for (int s = 0; s < R; ++s) {
    const __amdgpu_buffer_rsrc_t ra = buffer_of(at.a, s < kblocks ? at.rows * K : 0);
    const __amdgpu_buffer_rsrc_t rb = buffer_of(at.b, s < kblocks ? at.cols * K : 0);
#pragma unroll
    for (int u = 0; u < T::a_loads; ++u) op_load<RAGGED>(lo, ra, s, K, ring_lds + s * T::stage, u);
    if (kSplit && s == R - 1) break;
#pragma unroll
    for (int u = 0; u < T::b_loads; ++u)
      op_load<RAGGED>(lo, rb, s, K, ring_lds + s * T::stage + T::a_bytes, u);
  }
  wait_loads<kAhead + T::a_loads + (kSplit ? 0 : T::b_loads)>();
  lds_barrier();
  Fragments<T> f[2], g[2];  // of sub-steps 0 and 1
#pragma unroll
  for (int i = 0; i < (kSplit ? 1 : 2) * NF; ++i) f[i / NF].read(i % NF, ring, wi, wj, lane, i / NF);
  // scale bytes of this lane's rows and of the wave's column block: stage q of the piece in buffer buf
  auto scale_at = [&](int buf, int q, int row) -> int { return scales[buf * T::scale_bytes + row * 16 + q]; };
  int sa[TM], sb, buf = 0;
#pragma unroll
  for (int i = 0; i < TM; ++i) sa[i] = scale_at(0, 0, wi + 32 * i + (lane & 31));
  sb = scale_at(0, 0, T::rows + (wj >> 7));
  int cur = 0;         // ring slot of stage s
  int settled = 1;     // 0: the stores of the tile before may be in flight
  for (;;) {
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < NM; ++i) acc[i / TN][i % TN] = (f32x16){};
    if constexpr (T::whole) {
      auto stage = [&](int s, Fragments<T> (&f)[2], Fragments<T> (&g)[2], auto inner) __attribute__((always_inline)) {
        constexpr bool kInner = decltype(inner)::value;
        const int nxt = cur + 1 == R ? 0 : cur + 1;
        const uint8_t *ns = ring + nxt * T::stage;
        const int q = s % kScaleStages;
        const bool turn = q == kScaleStages - 1 || (!kInner && s == nk - 1);
        const int nbuf = !turn ? buf : buf + 1 == kScaleBufs ? 0 : buf + 1, nq = turn ? 0 : q + 1;
        const int mask = kInner || s == nk - 1 || s + 1 < kblocks ? 255 : 0;  // as below
        const int ls = kInner ? s + R : s + R - nk;
        const Place &lp = kInner ? at : next;
        const __amdgpu_buffer_rsrc_t ra = buffer_of(lp.a, kInner || ls < kblocks ? lp.rows * K : 0);
        const __amdgpu_buffer_rsrc_t rb = buffer_of(lp.b, kInner || ls < kblocks ? lp.cols * K : 0);
        wait_loads_or<kAhead, T::stores>(s | settled);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        int na[TM];
#pragma unroll
        for (int j = 0; j < 2 * NF; ++j) g[j / NF].read(j % NF, ns, wi, wj, lane, j / NF);
#pragma unroll
        for (int j = 0; j < TM; ++j) na[j] = scale_at(nbuf, nq, wi + 32 * j + (lane & 31));
        const int nb = scale_at(nbuf, nq, T::rows + (wj >> 7));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2 * NM; ++i) {
          const int tm = i % NM / TN, tn = i % TN;
          acc[tm][tn] = mma<FMT>(f[i / NM].b[tn], f[i / NM].a[tm], acc[tm][tn], sb, sa[tm]);
#pragma unroll
          for (int u = 0; u < T::a_loads + T::b_loads; ++u)
            if (u * 2 * NM / (T::a_loads + T::b_loads) == i) {
              if (u < T::a_loads)
                op_load<RAGGED>(lo, ra, ls, K, ring_lds + cur * T::stage, u);
              else
                op_load<RAGGED>(lo, rb, ls, K, ring_lds + cur * T::stage + T::a_bytes, u - T::a_loads);
            }
          if (i == NM) {
            const Fetch fe = next_scales(s, q, nk, buf);
            load_scales(fe.skip, fe.own ? at : next, fe.at, fe.to);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = na[i] & mask;
        sb = nb & mask;
        buf = nbuf;
        cur = nxt;
      };
      int s = 0;
#pragma clang loop unroll(disable)
      for (; s + 1 + R < nk; s += 2) {
        stage(s, f, g, std::true_type{});
        stage(s + 1, g, f, std::true_type{});
      }
      if (s + R < nk) {
        stage(s++, f, g, std::true_type{});
#pragma unroll
        for (int h = 0; h < 2; ++h) f[h] = g[h];
      }
#pragma clang loop unroll(disable)
      for (; s + 2 <= nk; s += 2) {
        stage(s, f, g, std::false_type{});
        stage(s + 1, g, f, std::false_type{});
      }
      if (s < nk) {
        stage(s, f, g, std::false_type{});
#pragma unroll
        for (int h = 0; h < 2; ++h) f[h] = g[h];
      }
    } else {
    // inner: the stages whose loads that run ahead are this tile's.  f0, f1: the fragments of the sub-steps;
    // to1: where the next stage's sub-step 1 goes.
    auto stage = [&](int s, Fragments<T> &f0, Fragments<T> &f1, Fragments<T> &to1, auto inner) __attribute__((always_inline)) {
      constexpr bool kInner = decltype(inner)::value;
      const int nxt = cur + 1 == R ? 0 : cur + 1, prv = cur == 0 ? R - 1 : cur - 1;
      const uint8_t *cs = ring + cur * T::stage, *ns = ring + nxt * T::stage;
      int na[TM], nb = 0;
      const int q = s % kScaleStages;
      // the next piece: this tile's next 16 stages, or the next tile's first
      const bool turn = q == kScaleStages - 1 || (!kInner && s == nk - 1);
      const int nbuf = !turn ? buf : buf + 1 == kScaleBufs ? 0 : buf + 1, nq = turn ? 0 : q + 1;
      // 0 for a stage past the contraction, whose scale bytes may be anything (2^-127 times zeros).  Applied at
      // the stage's end: next to the read it would wait for it, five times a stage
      const int mask = kInner || s == nk - 1 || s + 1 < kblocks ? 255 : 0;
      // loads of stage s + R (b's of s + R - 1 where they are split): this tile's or, past its end,
      // the next one's.  (nk is more than the contraction's blocks only where it is R: no inner stages then.)
      const int as = kInner ? s + R : s + R - nk;
      const Place &ap = kInner ? at : next;
      const __amdgpu_buffer_rsrc_t ra = buffer_of(ap.a, kInner || as < kblocks ? ap.rows * K : 0);
      const int bn = s + R - (kSplit ? 1 : 0), bs = kInner || bn < nk ? bn : bn - nk;
      const Place &bp = kInner || bn < nk ? at : next;
      const __amdgpu_buffer_rsrc_t rb = buffer_of(bp.b, kInner || bs < kblocks ? bp.cols * K : 0);
      const uint32_t to_a = ring_lds + cur * T::stage, to_b = ring_lds + (kSplit ? prv : cur) * T::stage + T::a_bytes;
      __builtin_amdgcn_sched_barrier(0);
      Fetch fe;
      // matrix instruction i of the stage's 2 NM, and what is issued behind it
      auto slot = [&](int i) __attribute__((always_inline)) {
        const int tm = i % NM / TN, tn = i % TN;
        acc[tm][tn] = mma<FMT>(i < NM ? f0.b[tn] : f1.b[tn], i < NM ? f0.a[tm] : f1.a[tm], acc[tm][tn], sb, sa[tm]);
        if constexpr (kDeep) {
#pragma unroll
          for (int j = 0; j < 2 * NF; ++j)
            if (NM + j * NM / (2 * NF) == i) (j < NF ? f0 : to1).read(j % NF, ns, wi, wj, lane, j / NF);
        } else {
#pragma unroll
          for (int j = 0; j < NF; ++j)
            if (j * H / NF == i % NM) (i < NM ? f1 : f0).read(j, i < NM ? cs : ns, wi, wj, lane, i < NM);
        }
        constexpr int kScale = kDeep ? NM : H;
#pragma unroll
        for (int j = 0; j < TM; ++j)
          if (kScale + j * (NM - H) / TM == i) na[j] = scale_at(nbuf, nq, wi + 32 * j + (lane & 31));
        if (i == kScale + NM - H - 1) nb = scale_at(nbuf, nq, T::rows + (wj >> 7));
#pragma unroll
        for (int u = 0; u < T::a_loads; ++u)
          if ((kSplit ? NM + u * NM / T::a_loads : u * kSpan / kAll) == i) op_load<RAGGED>(lo, ra, as, K, to_a, u);
#pragma unroll
        for (int u = 0; u < T::b_loads; ++u)
          if ((kSplit ? u * NM / T::b_loads : (T::a_loads + u) * kSpan / kAll) == i)
            op_load<RAGGED>(lo, rb, bs, K, to_b, u);
        if (i == (kDeep ? NM : 0) + H / 2) fe = next_scales(s, q, nk, buf);
        if (i == (kDeep ? NM : 0) + H) load_scales(fe.skip, fe.own ? at : next, fe.at, fe.to);
        __builtin_amdgcn_sched_barrier(0);
      };
      if constexpr (kDeep) {
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < NM; ++i) slot(i);
      wait_loads_or<kDeep ? (NM * kAll + kSpan - 1) / kSpan : kAhead, T::stores>(s | settled);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = NM; i < 2 * NM; ++i) slot(i);
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = na[i] & mask;
      sb = nb & mask;
      buf = nbuf;
      cur = nxt;
    };
    int s = 0;
    if constexpr (kDeep) {
#pragma clang loop unroll(disable)
      for (; s + 1 + R < nk; s += 2) {
        stage(s, f[0], f[1], g[1], std::true_type{});
        stage(s + 1, f[0], g[1], f[1], std::true_type{});
      }
      if (s + R < nk) {
        stage(s++, f[0], f[1], g[1], std::true_type{});
        f[1] = g[1];
      }
      stage(s, f[0], f[1], g[1], std::false_type{});
      stage(s + 1, f[0], g[1], f[1], std::false_type{});
    } else {
#pragma clang loop unroll(disable)
      for (; s + R < nk; ++s) stage(s, f[0], f[1], f[1], std::true_type{});
#pragma clang loop unroll(disable)
      for (; s < nk; ++s) stage(s, f[0], f[1], f[1], std::false_type{});
    }
    }
    tile_out<T>(acc, out + (long long)at.m0 * N + at.j0, N, at.rows, at.cols);
    __builtin_amdgcn_sched_barrier(0);
    settled = 0;
    t += grid;
    if (t >= total) break;
    at = next;
    next = place(t + grid);
  }
  wait_loads<0>();  // the loads past the last tile write this workgroup's LDS
}

template <class T, int FMT>
static void launch_tiles(const uint8_t *a, const uint8_t *as, const uint8_t *b,
                         const uint8_t *bs, const int32_t *cu, uint16_t *out, int G, int M_total, int K,
                         int N, hipStream_t stream) {
  const dim3 grid(device_cu_count()), block(kTileThreads);
  if (K % kBlock)
    hipLaunchKernelGGL((k_scaled_tiles<T, FMT, true>), grid, block, 0, stream, a, as, b, bs, cu, out, G,
                       M_total, K, N);
  else
    hipLaunchKernelGGL((k_scaled_tiles<T, FMT, false>), grid, block, 0, stream, a, as, b, bs, cu, out, G,
                       M_total, K, N);
}

// Which kernel: by the rows a segment has on average and by how many tiles of a size there are
// likely to be (a full tile for each of its rows, and half a tile more for each segment), since the
// segments themselves are only known on the device.  Measured, us a launch in a graph (rows, segments,
// contraction x columns; few rows / 64 x 64 / 64 x 128 / 128 x 256 / 256 x 256 tiles; * the rule's):
//   6, 68, 2048x1408         *7.7 / 10.1 / 12.0 / 17.7 / 24
//   16, 1, 7168x7168         * 17 /   22 /   28 /   45 / 68
//   512, 264, 7168x2048      *560 /  525 /  527 /  529 / 566
//   256, 1, 4096x4096          53 /*15.6 / 17.7 / 32.3 / 45
//   1000, 16, 1024x1024        18 / 11.8 /  8.8*/ 14.0 / 17.7
//   1024, 68, 2048x1408        49 /   41 /   34*/   38 / 44
//   4096, 264, 7168x2048      954 /  649 /  658*/  671 / 717
//   5003, 18, 1408x2064         - /   61 /   37 /  *31 / 26
//   24576, 68, 1408x2048        - /  245 /  156 / *107 / 103
//   32768, 264, 7168x2048       - / 1433 / 1111 / *831 / 848
//   2000, 1, 7168x7168       1206 /  241 /  148 /  101 / 89*
//   32768, 1, 7168x2048         - / 1097 /  713 /  440 / 375*
// The rows of these lie on all of their segments.  Where most segments are empty, as in a rank's layout (its
// E / R home experts and its slots of E + B segments), the average is far below what a segment with rows has,
// and the rule takes a kernel for shorter ones; the host knows no better from these arguments (rows on 9 segments):
//   2048 on 9 of 264, 7168x2048  *362 / 93 / 64 / 52 / 81
//   32768 on 9 of 264, 7168x2048    - / 1112 / 734 / *470 / 424
//   1536 on 9 of 68, 2048x1408     58 / 23 / *18 / 20 / 29
//   24576 on 9 of 68, 2048x1408     - / 210 / 124 / *83 / 83
template <int FMT>
static void launch_scaled(const uint8_t *a, const uint8_t *as, const uint8_t *b, const uint8_t *bs,
                          const int32_t *cu, uint16_t *out, int G, int M_total, int K, int N,
                          hipStream_t stream) {
  const long long cus = device_cu_count(), segs = G < M_total ? G : M_total;
  auto tiles = [&](int rows, int cols) {
    return ((long long)M_total * 2 / rows + segs + 1) / 2 * ((N + cols - 1) / cols);
  };
  if (M_total <= kFewRows || M_total <= 8LL * G) {
    const long long most = (segs + M_total / kFewRows) * ceil_div(N, kFewCols * 2);
    hipLaunchKernelGGL((k_scaled_few<FMT, 4, 2, 2>), dim3((unsigned)(most < cus * 8 ? most : cus * 8)),
                       dim3(256), 0, stream, a, as, b, bs, cu, out, G, M_total, K, N);
  } else if (M_total >= 512LL * G && tiles(256, 256) * 4 >= cus * 3) {
    launch_tiles<Tile<4, 4, 2>, FMT>(a, as, b, bs, cu, out, G, M_total, K, N, stream);
  } else if (M_total > 64LL * G && tiles(128, 256) * 4 >= cus * 3) {
    launch_tiles<Tile<2, 4, 3>, FMT>(a, as, b, bs, cu, out, G, M_total, K, N, stream);
  } else if (tiles(64, 64) * 4 <= cus * 5) {  // about one tile a compute unit
    launch_tiles<Tile<1, 1, 8>, FMT>(a, as, b, bs, cu, out, G, M_total, K, N, stream);
  } else {
    launch_tiles<Tile<1, 2, 6>, FMT>(a, as, b, bs, cu, out, G, M_total, K, N, stream);
  }
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_group_gemm_scaled(moe_gemm_op op, moe_fp8 a_fmt, int32_t G, int32_t M_total, int32_t Kd, int32_t N,
                                              const void *a, const void *a_scale, const void *b,
                                              const void *b_scale, const int32_t *cu_seqlens,
                                              void *out, hipStream_t stream) {
  if (op != MOE_GEMM_FWD && op != MOE_GEMM_DGRAD) return MOE_EINVAL;
  if (a_fmt != MOE_E4M3 && a_fmt != MOE_E5M2) return MOE_EINVAL;
  if (G < 1 || G > kScMaxG || M_total < 0 || Kd < 16 || N < 16 || Kd % 16 || N % 16) return MOE_EINVAL;
  if (Kd > kScMaxDim || N > kScMaxDim) return MOE_EINVAL;
  // tiles are counted in 32 bits, with room for the grid beyond the last (the smallest are 16 x 32)
  if ((M_total / kFewRows + (int64_t)G) * ceil_div(op == MOE_GEMM_FWD ? N : Kd, kFewCols * 2) >= kScMaxTiles)
    return MOE_EINVAL;
  if (M_total == 0) return MOE_OK;
  if (!a || !a_scale || !b || !b_scale || !cu_seqlens || !out) return MOE_EINVAL;
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(b) || !aligned16(b_scale) ||
      !aligned16(out) || ((uintptr_t)cu_seqlens & 3))
    return MOE_EINVAL;
  // both operands end contiguous along the contraction: FWD contracts Kd, DGRAD contracts N
  const int K = op == MOE_GEMM_FWD ? Kd : N, C = op == MOE_GEMM_FWD ? N : Kd;
  const uint8_t *a8 = (const uint8_t *)a, *b8 = (const uint8_t *)b;
  const uint8_t *as = (const uint8_t *)a_scale, *bs = (const uint8_t *)b_scale;
  if (a_fmt == MOE_E4M3)
    launch_scaled<MOE_E4M3>(a8, as, b8, bs, cu_seqlens, (uint16_t *)out, G, M_total, K, C, stream);
  else
    launch_scaled<MOE_E5M2>(a8, as, b8, bs, cu_seqlens, (uint16_t *)out, G, M_total, K, C, stream);
  return launch_status();
}
