// moe_layer_norm, moe_layer_norm_backward: rows normalised on the way into the layer, the residual sum and
// the dropout of the branch before it taken along, and their gradients.
//
// A row is read once and kept in registers (eight consecutive values a thread and step) while its mean and
// then the mean of its squared differences are summed: both in fp32, the second from the differences, so
// that a mean far from 0 costs no digits.  Rows wider than the registers of a workgroup are read again.
//
// HBM-bound, with dropout nearly as much by the ten rounds of its counter: bf16 rows of 7168 with residual, median kernel
// times over three sets of inputs: 32768 rms rows (1.9 GB) 325 us, 5.8 TB/s; 4096 with dropout and statistics (235 MB) 44 to
// 45, 5.3 TB/s; the gradient of 8192 with dropout and the residual's gradient (587 MB) 108 and 5 for the sums of columns,
// 5.2 TB/s; a gradient of 2^24 values (2048 rows, 117 MB) 32 with them, 3.6 TB/s.  One row 3.4 us.  The best copy reaches
// 5.9.  With one row a workgroup and no loads ahead these took 381, 68 and 157 + 12.  Rows above 16384 columns, read two or
// three times: 2.1 to 3.4 TB/s of what they would have to move.
#include <type_traits>

#include "dropout.hpp"
#include "lanes.hpp"

namespace moe {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxWaves = kNormMaxThreads / kWave;
constexpr int kNormParts = 1024; // at most as many sums of columns a backward call makes, then adds up
constexpr int kColParts = 64;    // the same of rows that are read again
constexpr int kNormLanesThreads = 256;  // where several rows share a workgroup

// The threads of a row: LANES of a wave, or (LANES 0) a workgroup.  Sums are the same in all of them, in a fixed order.
template <int LANES>
struct RowThreads {
  int t, count;  // this thread's place, threads a row
  long long row, step;
  float (*part)[kNormMaxWaves];  // two places, a third where sum_again() is called
  int slot = 0;
  // groups: workgroups that walk the rows (0: the grid's)
  __device__ inline RowThreads(float (*p)[kNormMaxWaves], int groups = 0) : part(p) {
    const unsigned all = groups ? groups : gridDim.x;
    if constexpr (LANES > 0) {
      constexpr int ROWS = kNormLanesThreads / LANES;
      t = threadIdx.x % LANES, count = LANES;
      row = (long long)blockIdx.x * ROWS + threadIdx.x / LANES, step = (long long)all * ROWS;
    } else {
      t = threadIdx.x, count = blockDim.x;
      row = blockIdx.x, step = all;
    }
  }
  __device__ inline float sum(float v) {
    if constexpr (LANES > 0) {
      return token_sum<LANES>(v);
    } else {
      v = token_sum<kWave>(v);
      if (blockDim.x == kWave) return v;
      // two places in turn: who writes one again has passed the barrier behind the other's reads
      float *p = part[slot ^= 1];
      if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
      __syncthreads();
      const int w = threadIdx.x & 15;
      return token_sum<16>(w < (int)(blockDim.x >> 6) ? p[w] : 0.0f);
    }
  }
  // One more sum of a row that needs it, at most one between two of sum(), whose barriers keep its place's uses apart.
  __device__ inline float sum_again(float v) {
    if constexpr (LANES > 0) {
      return token_sum<LANES>(v);
    } else {
      v = token_sum<kWave>(v);
      if (blockDim.x == kWave) return v;
      float *p = part[2];
      if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
      __syncthreads();
      const int w = threadIdx.x & 15;
      return token_sum<16>(w < (int)(blockDim.x >> 6) ? p[w] : 0.0f);
    }
  }
};

// Where a step's eight columns begin, and how many of them an earlier thread has already: the last run of a row whose
// width is no multiple of 8 is moved back to end with the row (a thread without columns has the row's last eight, all
// of them others').  So every load is whole, and what two threads write is the same.
struct Run {
  int at, skip;
  __device__ inline Run(int t, int count, int i, int W) {
    const int c = 8 * (t + i * count);
    at = min(c, W - 8);
    skip = min(c - at, 8);
  }
};

// Sum of f(j) over the columns of a run that are this thread's.
template <class F>
__device__ inline float run_sum(const Run &r, F f) {
  float s = 0.0f;
  if (r.skip == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s += f(j);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) s += j >= r.skip ? f(j) : 0.0f;
  }
  return s;
}

// The same of the squares of v scale.  Fused by hand: left to the compiler, which of the products are rounded before they are
// added differed from one use to the next, and a row's last bits with it.
__device__ inline float run_squares(const Run &r, const float (&v)[8], float scale = 1.0f) {
  float s = 0.0f;
  if (r.skip == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[j] * scale, v[j] * scale, s);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) s = j >= r.skip ? fmaf(v[j] * scale, v[j] * scale, s) : s;
  }
  return s;
}

// 1 / sqrt(v), within one step; the instruction takes numbers below 2^-126 for 0.
__device__ inline float inverse_root(float v) {
  const bool tiny = v < 0x1p-100f;
  return __builtin_amdgcn_rsqf(tiny ? v * 0x1p60f : v) * (tiny ? 0x1p30f : 1.0f);
}

// Where the sum of a row's squares is more than fp32 holds (values from 2^53 on at the widest row), the squares are summed
// again of the values scaled by this: below 2^105, which a row's own sum still holds, they fit at any width.
constexpr float kLargeScale = 0x1p-80f;
__device__ inline float inverse_root_large(float v, float eps) {
  return inverse_root(v + eps * kLargeScale * kLargeScale) * kLargeScale;
}

__device__ inline void load_w(const void *w, bool bf16, long long i, int n, float (&v)[8]) {
  bf16 ? load_8<true>(w, i, n, v) : load_8<false>(w, i, n, v);
}

struct NormArgs {
  const void *x, *residual, *weight, *bias;
  void *total, *y;
  float *mean, *rstd;
  long long rows;
  int width;
  bool w_bf16, late;  // late: the next row's residual is fetched only behind a row's sums
  float eps;
  Drop drop;
};

// Rows of 8 to 8 CHUNKS threads columns.  The next row's loads are under way while a row is summed and written; two
// rows ahead gained nothing.  A thread has one run up to 8192 columns: with two in half the threads the dropout of
// 4096 x 7168 took 48 to 52 us against 46 (fewer waves, more registers).
template <bool BF16, bool RMS, bool DROP, bool STREAM, int LANES, int CHUNKS>
__global__ __launch_bounds__(LANES ? kNormLanesThreads : kNormMaxThreads) void k_norm(NormArgs a) {
  __shared__ float part[3][kNormMaxWaves];
  RowThreads<LANES> me(part);
  const int W = a.width;
  DropKey key{};
  if (DROP) key = drop_key(a.drop);
  float w[CHUNKS][8], b[CHUNKS][8];
  Raw<BF16> x[CHUNKS], r[CHUNKS];
  auto fetch = [&](Raw<BF16> *to, const void *from, long long row) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
      to[i].template load<STREAM>(row_at(from, bytes_of<BF16>(row * W)), Run(me.t, me.count, i, W).at);
  };
  const bool early = a.residual && !a.late, late = a.residual && a.late;
  // The row's dropout, worked out between the sums of the row before, while the row is on its way: at the use of the values
  // it took 46 or 50 us (4096 x 7168), as the compiler placed it, right behind the fetch 51, at the row's end 48, here 46.
  u32x4 bits[CHUNKS];
  auto draw = [&](long long row) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i)
      bits[i] = drop_bits((unsigned long long)(row * W + Run(me.t, me.count, i, W).at), key);
  };
  if (me.row < a.rows) {
    fetch(x, a.x, me.row);
    if (a.residual) fetch(r, a.residual, me.row);
    if (DROP) draw(me.row);
  }
  auto weights = [&](int i) {
    const Run u(me.t, me.count, i, W);
    load_w(a.weight, a.w_bf16, u.at, 8, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
    if (a.bias) load_w(a.bias, a.w_bf16, u.at, 8, b[i]);
  };
  constexpr bool KEEP = CHUNKS == 1;
  if (KEEP) weights(0);
  const float rw = 1.0f / W;
  for (long long row = me.row; row < a.rows; row += me.step) {
    const long long base = row * W;
    float h[CHUNKS][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const Run u(me.t, me.count, i, W);
      x[i].values(h[i]);
      if (DROP) {
        float v[8] = {};
        if (a.residual) r[i].values(v);
        drop_8(bits[i], a.drop, h[i], v);
      } else if (a.residual) {
        float v[8];
        r[i].values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += v[j];
      }
      sum += RMS ? run_squares(u, h[i]) : run_sum(u, [&](int j) { return h[i][j]; });
    }
    const bool more = row + me.step < a.rows;
    if (more) fetch(x, a.x, row + me.step);
    if (more && early) fetch(r, a.residual, row + me.step);
    sum = me.sum(sum) * rw;
    // from here on every thread has its columns: an output may take their place
    if (a.total)
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const Run u(me.t, me.count, i, W);
        if (u.skip < 8) Raw<BF16>(h[i]).template store<STREAM>(row_at(a.total, bytes_of<BF16>(base)), u.at);
      }
    if (DROP && more) draw(row + me.step);
    const float mean = RMS ? 0.0f : sum;
    float var = sum;
    if (!RMS) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] -= mean;
        sq += run_squares(Run(me.t, me.count, i, W), h[i]);
      }
      var = me.sum(sq) * rw;
    }
    float rstd = inverse_root(var + a.eps);
    if (__builtin_expect(__any(var == __builtin_inff()), 0)) {  // of the waves of a workgroup that share a row: all or none
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) sq += run_squares(Run(me.t, me.count, i, W), h[i], kLargeScale);
      sq = me.sum_again(sq) * rw;
      if (var == __builtin_inff()) rstd = inverse_root_large(sq, a.eps);
    }
    if (more && late) {
      // vmcnt(0): behind the next x, not beside it (rms, us beside / behind: 32768 x 7168 bf16 325 / 320, 8192 x 7168 fp32
      // 189 / 177, 32768 x 6144 bf16 282 / 287; layer norm the same within 1%)
      __builtin_amdgcn_s_waitcnt(0x0F70);
      fetch(r, a.residual, row + me.step);
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const Run u(me.t, me.count, i, W);
      if (u.skip == 8) continue;
      if (!KEEP) weights(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = fmaf(h[i][j] * rstd, w[i][j], b[i][j]);
      Raw<BF16>(h[i]).template store<STREAM>(row_at(a.y, bytes_of<BF16>(base)), u.at);
    }
    if (me.t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Rows of any width, read again for each sum.
template <bool BF16, bool RMS, bool DROP>
__global__ __launch_bounds__(kNormMaxThreads) void k_norm_any(NormArgs a) {
  __shared__ float part[2][kNormMaxWaves];
  RowThreads<0> me(part);
  const int W = a.width;
  DropKey key{};
  if (DROP) key = drop_key(a.drop);
  for (long long row = me.row; row < a.rows; row += me.step) {
    const long long base = row * W;
    auto read = [&](int at, int n, float (&v)[8]) {
      load_8<BF16>(a.x, base + at, n, v);
      if (DROP) drop_8(drop_bits((unsigned long long)(base + at), key), a.drop, v);
      if (a.residual) {
        float r[8];
        load_8<BF16>(a.residual, base + at, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
      }
    };
    float mean = 0.0f, sum = 0.0f;
    if (!RMS) {
      for (int at = 8 * me.t; at < W; at += 8 * me.count) {
        float v[8];
        read(at, W - at, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += at + j < W ? v[j] : 0.0f;
      }
      mean = me.sum(sum) / W;
    }
    float scale = 1.0f, var;
    for (;; scale = kLargeScale) {
      float sq = 0.0f;
      for (int at = 8 * me.t; at < W; at += 8 * me.count) {
        float v[8];
        read(at, W - at, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = at + j < W ? (v[j] - mean) * scale : 0.0f;
          sq = fmaf(d, d, sq);
        }
      }
      var = me.sum(sq) / W;
      if (var != __builtin_inff() || scale != 1.0f) break;
    }
    const float rstd = scale / sqrtf(var + a.eps * scale * scale);
    for (int at = 8 * me.t; at < W; at += 8 * me.count) {
      const int n = W - at;
      float v[8], w[8], b[8] = {};
      read(at, n, v);
      load_w(a.weight, a.w_bf16, at, n, w);
      if (a.bias) load_w(a.bias, a.w_bf16, at, n, b);
      if (a.total) store_8<BF16>(a.total, base + at, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf((v[j] - mean) * rstd, w[j], b[j]);
      store_8<BF16>(a.y, base + at, n, v);
    }
    if (me.t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

struct NormBwdArgs {
  const void *total, *weight, *dy, *dtotal;
  const float *mean, *rstd;
  void *dx, *dresidual;
  float *parts;  // [groups][2][width]: sums of dy xh and of dy; NULL: not wanted, or written by column groups
  float *dweight, *dbias;  // what column groups write
  long long rows;
  int width, groups;  // groups: workgroups that walk the rows; those behind them take kGroupColumns columns each
  bool w_bf16, accumulate;
  Drop drop;
};

template <bool BF16>
__device__ inline float value_at(const void *p, long long i) {
  return BF16 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16) : ((const float *)p)[i];
}

// dweight and dbias of kGroupColumns columns, of all rows: what a workgroup behind the rows' own does in a short call, beside
// them, instead of a second launch behind them.  The rows are read once more, out of the caches.  A wave takes 16
// columns of 4 rows.
constexpr int kGroupColumns = 16;
template <bool BF16, bool RMS>
__device__ inline void column_sums(const NormBwdArgs &a) {
  __shared__ float part[2][kNormMaxWaves][kGroupColumns];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = blockDim.x >> 6, W = a.width;
  const int c = ((int)blockIdx.x - a.groups) * kGroupColumns + (lane & 15), at = min(c, W - 1);
  constexpr int FLIGHT = 8;
  float dw = 0.0f, db = 0.0f;
  for (long long r0 = 4 * w + (lane >> 4); r0 < a.rows; r0 += 4LL * waves * FLIGHT) {
    float h[FLIGHT], d[FLIGHT], m[FLIGHT], s[FLIGHT];
#pragma unroll
    for (int k = 0; k < FLIGHT; ++k) {
      const long long r = min(r0 + 4LL * waves * k, a.rows - 1);
      h[k] = value_at<BF16>(a.total, r * W + at);
      d[k] = value_at<BF16>(a.dy, r * W + at);
      m[k] = RMS ? 0.0f : a.mean[r];
      s[k] = a.rstd[r];
    }
#pragma unroll
    for (int k = 0; k < FLIGHT; ++k) {
      if (r0 + 4LL * waves * k >= a.rows) break;
      dw = fmaf(d[k], (h[k] - m[k]) * s[k], dw);
      db += d[k];
    }
  }
#pragma unroll
  for (int off = 16; off < kWave; off <<= 1) dw += __shfl_xor(dw, off, kWave), db += __shfl_xor(db, off, kWave);
  if (lane < 16) part[0][w][lane] = dw, part[1][w][lane] = db;
  __syncthreads();
  if (threadIdx.x >= 16 || c >= W) return;
  dw = db = 0.0f;
  for (int i = 0; i < waves; ++i) dw += part[0][i][lane], db += part[1][i][lane];
  if (a.dweight) a.dweight[c] = a.accumulate ? a.dweight[c] + dw : dw;
  if (a.dbias) a.dbias[c] = a.accumulate ? a.dbias[c] + db : db;
}

// The gradient of rows as k_norm has them.  Each workgroup adds up its rows' dy xh and dy column by column, in registers,
// and k_norm_parts adds the workgroups' sums; the sum's gradient is fetched with the row (fetched when the row is
// begun, 16384 x 4096 took 116 us against 98 on one workgroup per CU).
template <bool BF16, bool RMS, bool DROP, bool STREAM, int LANES, int CHUNKS>
__global__ __launch_bounds__(LANES ? kNormLanesThreads : kNormMaxThreads) void k_norm_bwd(NormBwdArgs a) {
  if ((int)blockIdx.x >= a.groups) {
    column_sums<BF16, RMS>(a);
    return;
  }
  __shared__ float part[2][kNormMaxWaves];
  RowThreads<LANES> me(part, a.groups);
  const int W = a.width;
  DropKey key{};
  if (DROP) key = drop_key(a.drop);
  // With two runs a thread the registers of 1024 threads do not hold it all (spilled, 4096 x 16384 bf16 took 212 us; as it is,
  // 12 of the 16 variants still keep 8 to 80 bytes a thread in scratch, the most in fp32 with dropout: 2730 x 12288 fp32 171
  // us with dropout and the residual's gradient, 122 without).  The
  // sums of the columns go to LDS then (each thread its own), dtotal is fetched when its row is begun, and the weights of
  // fp32 rows are read again for each row (4 x 2^25 values in 12288 columns 125 us, 128 kept; bf16 67, 60 kept).
  constexpr bool LDS = CHUNKS > 1, KEEP = !LDS || BF16;
  __shared__ f32x4 held[LDS ? CHUNKS * 4 : 1][LDS ? kNormMaxThreads : 1];
  float w[CHUNKS][8], dw[LDS ? 1 : CHUNKS][8], db[LDS ? 1 : CHUNKS][8];
  Raw<BF16> t[CHUNKS], d[CHUNKS], q[CHUNKS];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](long long row) {
    const long long bytes = bytes_of<BF16>(row * W);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const Run u(me.t, me.count, i, W);
      t[i].template load<STREAM>(row_at(a.total, bytes), u.at);
      d[i].template load<STREAM>(row_at(a.dy, bytes), u.at);
      if (!LDS && a.dtotal) q[i].template load<STREAM>(row_at(a.dtotal, bytes), u.at);
    }
    if (!RMS) mean = a.mean[row];
    rstd = a.rstd[row];
  };
  if (me.row < a.rows) fetch(me.row);
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    if (KEEP) load_w(a.weight, a.w_bf16, Run(me.t, me.count, i, W).at, 8, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[LDS ? 0 : i][j] = db[LDS ? 0 : i][j] = 0.0f;
    if (LDS)
#pragma unroll
      for (int k = 0; k < 4; ++k) held[4 * i + k][threadIdx.x] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  const float rw = 1.0f / W;
  for (long long row = me.row; row < a.rows; row += me.step) {
    const long long base = row * W;
    const float rs = rstd;
    if (LDS && a.dtotal)
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i)
        q[i].template load<STREAM>(row_at(a.dtotal, bytes_of<BF16>(base)), Run(me.t, me.count, i, W).at);
    float xh[CHUNKS][8], g[CHUNKS][8], sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const Run u(me.t, me.count, i, W);
      if (!KEEP) load_w(a.weight, a.w_bf16, u.at, 8, w[i]);
      float v[8];
      t[i].values(xh[i]);
      d[i].values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = (xh[i][j] - mean) * rs;
        g[i][j] = v[j] * w[i][j];
        if (!LDS) dw[i][j] = fmaf(v[j], xh[i][j], dw[i][j]), db[i][j] += v[j];
      }
      if (LDS)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f32x4 s = held[4 * i + k][threadIdx.x];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * (k & 1) + j;
            s[j] = k < 2 ? fmaf(v[e], xh[i][e], s[j]) : s[j] + v[e];
          }
          held[4 * i + k][threadIdx.x] = s;
        }
      if (!RMS) sg += run_sum(u, [&](int j) { return g[i][j]; });
      sgx += run_sum(u, [&](int j) { return g[i][j] * xh[i][j]; });
      if (!LDS && a.dtotal) q[i].values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = fmaf(rs, g[i][j], !LDS && a.dtotal ? v[j] : 0.0f);
    }
    if (row + me.step < a.rows) fetch(row + me.step);
    if (!RMS) sg = me.sum(sg) * rw * rs;
    sgx = me.sum(sgx) * rw * rs;
    // an output may take its columns' place from here on: every thread's loads of them stand before the sums, those of dtotal
    // too where their values are used only below (a wave's memory accesses keep their order, and the sums' barrier the waves')
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const Run u(me.t, me.count, i, W);
      if (u.skip == 8) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[i][j] = fmaf(-xh[i][j], sgx, g[i][j]);
        if (!RMS) g[i][j] -= sg;
      }
      if (LDS && a.dtotal) {
        float v[8];
        q[i].values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] += v[j];
      }
      if (a.dresidual) Raw<BF16>(g[i]).template store<STREAM>(row_at(a.dresidual, bytes_of<BF16>(base)), u.at);
      if (DROP) drop_8(drop_bits((unsigned long long)(base + u.at), key), a.drop, g[i]);
      Raw<BF16>(g[i]).template store<STREAM>(row_at(a.dx, bytes_of<BF16>(base)), u.at);
    }
  }
  if (!a.parts) return;
  float *p = a.parts + (long long)blockIdx.x * 2 * W;
  auto keep = [&](const Run &u, const float (&v)[8], const float (&s)[8]) {
    if (u.skip == 0) {
      store_8<false>(p, u.at, 8, v);
      store_8<false>(p + W, u.at, 8, s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= u.skip) p[u.at + j] = v[j], p[W + u.at + j] = s[j];
    }
  };
  if constexpr (LANES == 0) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      if (LDS)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[0][j] = held[4 * i + (j >> 2)][threadIdx.x][j & 3];
          db[0][j] = held[4 * i + 2 + (j >> 2)][threadIdx.x][j & 3];
        }
      keep(Run(me.t, me.count, i, W), dw[LDS ? 0 : i], db[LDS ? 0 : i]);
    }
  } else {
    static_assert(CHUNKS == 1, "a lane's one run");
    __shared__ float sums[kNormLanesThreads][16];
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[threadIdx.x][j] = dw[0][j], sums[threadIdx.x][8 + j] = db[0][j];
    __syncthreads();
    if ((int)threadIdx.x >= LANES) return;
    for (int k = 1; k < kNormLanesThreads / LANES; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[0][j] += sums[k * LANES + threadIdx.x][j];
        db[0][j] += sums[k * LANES + threadIdx.x][8 + j];
      }
    keep(Run(me.t, me.count, 0, W), dw[0], db[0]);
  }
}

// dx and dresidual of rows of any width, read again for the result.
template <bool BF16, bool RMS, bool DROP>
__global__ __launch_bounds__(kNormMaxThreads) void k_norm_bwd_any(NormBwdArgs a) {
  __shared__ float part[2][kNormMaxWaves];
  RowThreads<0> me(part);
  const int W = a.width;
  DropKey key{};
  if (DROP) key = drop_key(a.drop);
  for (long long row = me.row; row < a.rows; row += me.step) {
    const long long base = row * W;
    const float mean = RMS ? 0.0f : a.mean[row], rstd = a.rstd[row];
    auto read = [&](int at, int n, float (&xh)[8], float (&g)[8]) {
      float w[8];
      load_8<BF16>(a.total, base + at, n, xh);
      load_8<BF16>(a.dy, base + at, n, g);
      load_w(a.weight, a.w_bf16, at, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) xh[j] = (xh[j] - mean) * rstd, g[j] *= w[j];  // g is 0 behind the row
    };
    float sg = 0.0f, sgx = 0.0f;
    for (int at = 8 * me.t; at < W; at += 8 * me.count) {
      float xh[8], g[8];
      read(at, W - at, xh, g);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < W) sg += g[j], sgx = fmaf(g[j], xh[j], sgx);
    }
    if (!RMS) sg = me.sum(sg) / W;
    sgx = me.sum(sgx) / W;
    for (int at = 8 * me.t; at < W; at += 8 * me.count) {
      const int n = W - at;
      float xh[8], g[8], q[8] = {};
      read(at, n, xh, g);
      if (a.dtotal) load_8<BF16>(a.dtotal, base + at, n, q);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = fmaf(rstd, g[j] - (RMS ? 0.0f : sg) - xh[j] * sgx, q[j]);
      if (a.dresidual) store_8<BF16>(a.dresidual, base + at, n, g);
      if (DROP) drop_8(drop_bits((unsigned long long)(base + at), key), a.drop, g);
      store_8<BF16>(a.dx, base + at, n, g);
    }
  }
}

// The columns' sums of rows too wide for k_norm_bwd to keep: a workgroup takes 256 columns of every
// gridDim.y-th row.
constexpr int kColThreads = 256;
template <bool BF16, bool RMS>
__global__ __launch_bounds__(kColThreads) void k_norm_cols(NormBwdArgs a) {
  const int c = blockIdx.x * kColThreads + threadIdx.x, W = a.width;
  if (c >= W) return;
  float dw = 0.0f, db = 0.0f;
  for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float h = value_at<BF16>(a.total, row * W + c), d = value_at<BF16>(a.dy, row * W + c);
    dw += d * ((h - (RMS ? 0.0f : a.mean[row])) * a.rstd[row]);
    db += d;
  }
  float *p = a.parts + (long long)blockIdx.y * 2 * W;
  p[c] = dw;
  p[W + c] = db;
}

// dweight and dbias from n parts: kPartsColumns columns of one of them a workgroup, its threads over the parts.
constexpr int kPartsThreads = 1024, kPartsColumns = 32;
__global__ __launch_bounds__(kPartsThreads) void k_norm_parts(const float *__restrict__ parts, int n, int W,
                                                             float *dweight, float *dbias, int accumulate) {
  constexpr int LINES = kPartsThreads / kPartsColumns;
  __shared__ float s[LINES][kPartsColumns];
  float *out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int t = threadIdx.x % kPartsColumns, w = threadIdx.x / kPartsColumns, c = blockIdx.x * kPartsColumns + t;
  float v = 0.0f;
  if (c < W) {
    // the loads of a thread under way together: the parts come from other caches
    const float *p = parts + (long long)blockIdx.y * W + c;
    constexpr int FLIGHT = 16;
    for (int i0 = w; i0 < n; i0 += LINES * FLIGHT) {
      float t[FLIGHT];
#pragma unroll
      for (int k = 0; k < FLIGHT; ++k) {
        const int i = i0 + LINES * k;
        t[k] = i < n ? p[(long long)i * 2 * W] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < FLIGHT; ++k) v += t[k];
    }
  }
  s[w][t] = v;
  __syncthreads();
  if (w || c >= W) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < LINES; ++i) v += s[i][t];
  out[c] = accumulate ? out[c] + v : v;
}

// Widths that a row's threads keep in registers; others go through the kernels that read a row again.
constexpr int kNormNarrowest = 8;
constexpr int kNormWidest = 16 * kNormMaxThreads;
constexpr int kNormMaxWidth = 1 << 22;

static bool row_kept(int64_t width) { return width >= kNormNarrowest && width <= kNormWidest; }

// Calls f with whether a call that moves so many bytes streams them, the lanes of a row (0: a workgroup), the steps of a
// thread, the workgroup's threads and its rows.
template <class F>
static void with_row(int W, int64_t moved, F f) {
  using std::false_type;
  using std::integral_constant;
  using std::true_type;
#define MOE_ROW(s, l, c, threads, rows) f(s, integral_constant<int, l>{}, integral_constant<int, c>{}, threads, rows)
  auto waves = [&](int chunks) { return ceil_div(W, 8 * chunks * kWave) * kWave; };
  const bool stream = moved >= kStreamBytes;
  if (W <= 128) MOE_ROW(false_type{}, 16, 1, kNormLanesThreads, 16);
  else if (W <= 256) MOE_ROW(false_type{}, 32, 1, kNormLanesThreads, 8);
  else if (W <= 512) MOE_ROW(false_type{}, 64, 1, kNormLanesThreads, 4);
  else if (W <= 8 * kNormMaxThreads && stream) MOE_ROW(true_type{}, 0, 1, waves(1), 1);
  else if (W <= 8 * kNormMaxThreads) MOE_ROW(false_type{}, 0, 1, waves(1), 1);
  else if (stream) MOE_ROW(true_type{}, 0, 2, waves(2), 1);
  else MOE_ROW(false_type{}, 0, 2, waves(2), 1);
#undef MOE_ROW
}

// Workgroups per CU that walk the rows, from the bytes each has under way (the next row's loads): enough for the memory's
// latency and no more, since more of them only spread the accesses.  32768 x 4096 bf16 rms with residual (16 KB under way
// in each) take 181 us with 1 and 199 with 2, 65536 x 2048 (8 KB) 253, 180 and 206 with 1, 2 and 4; without residual
// 32768 x 7168 (14 KB) 221 and 187 with 1 and 2; the gradient of 16384 x 2048 (12 KB) 71, 55, 57 and 62 with 1 to 4.
static int per_cu(int64_t under_way, int64_t wanted) {
  const int64_t n = (wanted + under_way - 1) / under_way;
  return (int)(n > 8 ? 8 : n);
}
constexpr int64_t kNormUnderWay = 16 << 10, kNormBwdUnderWay = 20 << 10;

// A backward call of so many values, and of so many rows for each wave of a workgroup, has its columns summed by workgroups
// beside the rows' own (us, so / in two launches: 292 x 7168 bf16 11.0 / 16.4, 585 x 7168 19.1 / 16.2, 512 x 4096 9.6 / 13.6,
// 1024 x 4096 17.9 / 16.3; 512 x 64 fp32, 128 rows a wave, 7.7 / 8.8).
constexpr int64_t kBesideValues = 1 << 21;
constexpr int kBesideRows = 128;

static int norm_parts(int64_t rows, int64_t width, int64_t bytes) {
  int64_t groups = rows, most = kColParts;
  if (row_kept(width))
    with_row((int)width, 0, [&](auto, auto, auto, int threads, int per) {
      groups = (rows + per - 1) / per;
      most = (int64_t)device_cu_count() * per_cu(bytes * per * width, kNormBwdUnderWay);
    });
  if (most > kNormParts) most = kNormParts;
  return (int)(groups < most ? groups : most);
}

// Threads of the kernels that read a row again, and their largest grid (2^32 threads are too many for a launch).
constexpr int64_t kAnyMaxGrid = 1 << 20;
static int any_threads(int64_t width) { return width >= 8 * kNormMaxThreads ? kNormMaxThreads : ceil_div(width, 8 * kWave) * kWave; }

static bool norm_args_ok(moe_dtype dtype, moe_norm_kind kind, moe_dtype w_dtype, int64_t rows, int64_t width) {
  if ((dtype != MOE_BF16 && dtype != MOE_F32) || (w_dtype != MOE_BF16 && w_dtype != MOE_F32)) return false;
  if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return false;
  return rows >= 0 && rows < (1LL << 31) && width >= 1 && width <= kNormMaxWidth;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_layer_norm(moe_dtype dtype, moe_norm_kind kind, moe_dtype w_dtype,
                                       int64_t rows, int64_t width, const void *x, const void *residual,
                                       const void *weight, const void *bias, double eps, double p,
                                       const int64_t *rng, int64_t offset, void *total, void *y,
                                       float *mean, float *rstd, hipStream_t stream) {
  if (!norm_args_ok(dtype, kind, w_dtype, rows, width) || !drop_ok(p, rng)) return MOE_EINVAL;
  if (!(eps >= 0.0) || eps - eps != 0.0 || (kind == MOE_NORM_RMS && mean)) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (!x || !weight || !y || (!total && (residual || p > 0.0))) return MOE_EINVAL;
  const size_t size = dtype == MOE_BF16 ? 2 : 4, w_size = w_dtype == MOE_BF16 ? 2 : 4;
  if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)total | (uintptr_t)y) % size ||
      ((uintptr_t)weight | (uintptr_t)bias) % w_size || ((uintptr_t)mean | (uintptr_t)rstd) % 4)
    return MOE_EINVAL;
  const size_t bytes = (size_t)rows * width * size, w_bytes = width * w_size, s_bytes = rows * 4;
  const Range in[] = {{x, bytes, true}, {residual, bytes, true}, {weight, w_bytes}, {bias, w_bytes},
                      {rng, 16}, {total, bytes}, {mean, s_bytes}, {rstd, s_bytes}};
  if (!stands_alone(y, bytes, in, 8, true) || !stands_alone(total, bytes, in, 5, true) || !stands_alone(mean, s_bytes, in, 6) ||
      !stands_alone(rstd, s_bytes, in, 7))
    return MOE_EINVAL;
  NormArgs a{x, residual, weight, bias, total, y, mean, rstd, rows, (int)width, w_dtype == MOE_BF16, false, (float)eps,
             make_drop(p, rng, offset)};
  auto go = [&](auto bf16, auto rms, auto drop) {
    if (!row_kept(width)) {
      hipLaunchKernelGGL((k_norm_any<bf16.value, rms.value, drop.value>), dim3((unsigned)(rows < kAnyMaxGrid ? rows : kAnyMaxGrid)),
                         dim3(any_threads(width)), 0, stream, a);
      return;
    }
    with_row((int)width, (int64_t)bytes * (2 + (residual ? 1 : 0) + (total ? 1 : 0)), [&](auto st, auto l, auto c, int threads, int per) {
      const int64_t groups = (rows + per - 1) / per, one = (int64_t)size * per * width;
      // a residual that would double what is under way beyond that waits (32768 x 7168: 359 us, 324 with it late)
      a.late = 2 * one > kNormUnderWay + kNormUnderWay / 4;
      const int64_t most = (int64_t)device_cu_count() * per_cu(residual ? 2 * one : one, kNormUnderWay);
      hipLaunchKernelGGL((k_norm<bf16.value, rms.value, drop.value, st.value, l.value, c.value>),
                         dim3((unsigned)(groups < most ? groups : most)), dim3(threads), 0, stream, a);
    });
  };
  auto pick = [&](auto bf16, auto rms) { a.drop.below ? go(bf16, rms, std::true_type{}) : go(bf16, rms, std::false_type{}); };
  auto kinds = [&](auto bf16) { kind == MOE_NORM_RMS ? pick(bf16, std::true_type{}) : pick(bf16, std::false_type{}); };
  dtype == MOE_BF16 ? kinds(std::true_type{}) : kinds(std::false_type{});
  return launch_status();
}

extern "C" size_t moe_layer_norm_backward_workspace_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || rows >= (1LL << 31) || width < 1 || width > kNormMaxWidth) return 0;
  return (size_t)norm_parts(rows, width, 4) * 2 * width * sizeof(float);  // of two bf16 tensors: most parts
}

extern "C" moe_status_t moe_layer_norm_backward(moe_dtype dtype, moe_norm_kind kind, moe_dtype w_dtype,
                                                int64_t rows, int64_t width, const void *total,
                                                const void *weight, const float *mean, const float *rstd,
                                                const void *dy, const void *dtotal, double p,
                                                const int64_t *rng, int64_t offset, void *dx,
                                                void *dresidual, float *dweight, float *dbias,
                                                int32_t accumulate, void *ws, size_t ws_bytes,
                                                hipStream_t stream) {
  if (!norm_args_ok(dtype, kind, w_dtype, rows, width) || !drop_ok(p, rng)) return MOE_EINVAL;
  if ((accumulate != 0 && accumulate != 1) || (kind == MOE_NORM_RMS && mean)) return MOE_EINVAL;
  const bool sums = dweight || dbias;
  if (rows && (!total || !weight || !rstd || !dy || !dx || (kind == MOE_NORM_LAYER && !mean))) return MOE_EINVAL;
  if (!rows && !sums) return MOE_OK;
  const size_t size = dtype == MOE_BF16 ? 2 : 4, w_size = w_dtype == MOE_BF16 ? 2 : 4;
  if (((uintptr_t)total | (uintptr_t)dy | (uintptr_t)dtotal | (uintptr_t)dx | (uintptr_t)dresidual) % size ||
      (uintptr_t)weight % w_size || ((uintptr_t)mean | (uintptr_t)rstd | (uintptr_t)dweight | (uintptr_t)dbias) % 4)
    return MOE_EINVAL;
  const size_t need = moe_layer_norm_backward_workspace_bytes(rows, width);
  if (sums && rows) {
    if (!ws || (uintptr_t)ws % 16) return MOE_EINVAL;
    if (ws_bytes < need) return MOE_ENOSPACE;
  }
  const size_t bytes = (size_t)rows * width * size, w_bytes = width * w_size, s_bytes = rows * 4, d_bytes = width * 4;
  const Range in[] = {{dy, bytes, true},        {dtotal, bytes, true},       {total, bytes},   {weight, w_bytes},
                      {mean, s_bytes},   {rstd, s_bytes},      {rng, 16},        {ws, sums ? need : 0},
                      {dweight, d_bytes}, {dbias, d_bytes},    {dresidual, bytes}};
  if (!stands_alone(dx, bytes, in, 11, true) || !stands_alone(dresidual, bytes, in, 10, true)) return MOE_EINVAL;
  if (sums && (!stands_alone(dweight, d_bytes, in, 8) || !stands_alone(dbias, d_bytes, in, 9) ||
               !stands_alone(ws, need, in, 7)))
    return MOE_EINVAL;
  const int parts = norm_parts(rows, width, (int64_t)size * (dtotal ? 3 : 2));
  NormBwdArgs a{total, weight, dy, dtotal, mean, rstd, dx, dresidual, sums ? (float *)ws : nullptr, dweight, dbias, rows,
                (int)width, parts, w_dtype == MOE_BF16, accumulate != 0, make_drop(p, rng, offset)};
  // dy is read beside the rows' work only where that does not write over it
  bool beside = sums && rows && row_kept(width) && rows * width <= kBesideValues && dx != dy && dresidual != dy;
  auto go = [&](auto bf16, auto rms, auto drop) {
    if (!row_kept(width)) {
      if (sums)  // before dx, which may take dy's place
        hipLaunchKernelGGL((k_norm_cols<bf16.value, rms.value>), dim3(ceil_div(width, kColThreads), parts),
                           dim3(kColThreads), 0, stream, a);
      hipLaunchKernelGGL((k_norm_bwd_any<bf16.value, rms.value, drop.value>), dim3((unsigned)(rows < kAnyMaxGrid ? rows : kAnyMaxGrid)),
                         dim3(any_threads(width)), 0, stream, a);
      return;
    }
    with_row((int)width, (int64_t)bytes * (3 + (dtotal ? 1 : 0) + (dresidual ? 1 : 0)), [&](auto st, auto l, auto c, int threads, int) {
      beside = beside && c.value == 1 && rows <= kBesideRows * (threads / kWave);
      if (beside) a.parts = nullptr;
      hipLaunchKernelGGL((k_norm_bwd<bf16.value, rms.value, drop.value, st.value, l.value, c.value>),
                         dim3(parts + (beside ? ceil_div(width, kGroupColumns) : 0)), dim3(threads), 0, stream, a);
    });
  };
  auto pick = [&](auto bf16, auto rms) { a.drop.below ? go(bf16, rms, std::true_type{}) : go(bf16, rms, std::false_type{}); };
  auto kinds = [&](auto bf16) { kind == MOE_NORM_RMS ? pick(bf16, std::true_type{}) : pick(bf16, std::false_type{}); };
  if (rows) dtype == MOE_BF16 ? kinds(std::true_type{}) : kinds(std::false_type{});
  if (sums && !beside)
    hipLaunchKernelGGL(k_norm_parts, dim3(ceil_div(width, kPartsColumns), 2), dim3(kPartsThreads), 0, stream,
                       (const float *)ws, parts, (int)width, dweight, dbias, accumulate);
  return launch_status();
}
