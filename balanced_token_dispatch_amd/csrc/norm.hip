// moe_layer_norm, moe_layer_norm_backward: rows normalised on the way into the layer, the residual sum and
// the dropout of the branch before it taken along, and their gradients.
//
// A row is read once and kept in registers (eight consecutive values a thread and step) while its mean and
// then the mean of its squared differences are summed: both in fp32, the second from the differences, so
// that a mean far from 0 costs no digits.  Rows wider than the registers of a workgroup are read again.
#include <type_traits>

#include "dropout.hpp"

namespace moe {

constexpr int kNormMaxWaves = 16;

// Sum over the WAVES waves of a row, the same in all its threads, in a fixed order.
template <int WAVES>
__device__ inline float row_sum(float v, float *part) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
  if constexpr (WAVES > 1) {
    __syncthreads();  // the sums before are read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[w];
  }
  return v;
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
  bool w_bf16;
  float eps;
  Drop drop;
};

// WAVES waves a row, CHUNKS steps of 8 values a thread (0: as many as the row has, read again for each sum).
template <bool BF16, bool RMS, bool DROP, int WAVES, int CHUNKS>
__global__ __launch_bounds__(WAVES * kWave) void k_norm(NormArgs a) {
  constexpr int T = WAVES * kWave, KEEP = CHUNKS ? CHUNKS : 1;
  __shared__ float part[WAVES];
  const int W = a.width, steps = CHUNKS ? CHUNKS : (W + 8 * T - 1) / (8 * T);
  DropKey key{};
  if (DROP) key = drop_key(a.drop);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const long long base = row * W;
    float kept[KEEP][8];
    // h of step i (of which n > 0 columns are in the row)
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
    auto h = [&](int i, int at, int n, float (&v)[8]) {
      if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = kept[i][j];
      } else {
        read(at, n, v);
      }
    };
    float sum = 0.0f;
#pragma unroll KEEP
    for (int i = 0; i < steps; ++i) {
      const int at = 8 * (threadIdx.x + i * T), n = W - at;
      float v[8] = {};
      if (n > 0) read(at, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) sum += v[j];
        if (CHUNKS > 0) kept[i][j] = v[j];
      }
    }
    float mean = 0.0f;
    if (!RMS) mean = row_sum<WAVES>(sum, part) / W;
    float sq = 0.0f;
#pragma unroll KEEP
    for (int i = 0; i < steps; ++i) {
      const int at = 8 * (threadIdx.x + i * T), n = W - at;
      if (n <= 0) continue;
      float v[8];
      h(i, at, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) sq += (v[j] - mean) * (v[j] - mean);
    }
    const float rstd = 1.0f / sqrtf(row_sum<WAVES>(sq, part) / W + a.eps);
#pragma unroll KEEP
    for (int i = 0; i < steps; ++i) {
      const int at = 8 * (threadIdx.x + i * T), n = W - at;
      if (n <= 0) continue;
      float v[8], w[8], b[8] = {};
      h(i, at, n, v);
      load_w(a.weight, a.w_bf16, at, n, w);
      if (a.bias) load_w(a.bias, a.w_bf16, at, n, b);
      if (a.total) store_8<BF16>(a.total, base + at, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (v[j] - mean) * rstd * w[j] + b[j];
      store_8<BF16>(a.y, base + at, n, v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

struct NormBwdArgs {
  const void *total, *weight, *dy, *dtotal;
  const float *mean, *rstd;
  void *dx, *dresidual;
  float *parts;  // [gridDim.x][2][width]: sums of dy xh and of dy; NULL: not wanted
  long long rows;
  int width;
  bool w_bf16;
  Drop drop;
};

template <bool BF16, bool RMS, bool DROP, int WAVES, int CHUNKS>
__global__ __launch_bounds__(WAVES * kWave) void k_norm_bwd(NormBwdArgs a) {
  constexpr int T = WAVES * kWave, KEEP = CHUNKS ? CHUNKS : 1;
  __shared__ float part[WAVES];
  const int W = a.width, steps = CHUNKS ? CHUNKS : (W + 8 * T - 1) / (8 * T);
  DropKey key{};
  if (DROP) key = drop_key(a.drop);
  float dw[KEEP][8] = {}, db[KEEP][8] = {};
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const long long base = row * W;
    const float mean = RMS ? 0.0f : a.mean[row], rstd = a.rstd[row];
    float kept_h[KEEP][8], kept_g[KEEP][8];
    // xh and g of a step
    auto read = [&](int at, int n, float (&xh)[8], float (&g)[8], float (&d)[8]) {
      float w[8];
      load_8<BF16>(a.total, base + at, n, xh);
      load_8<BF16>(a.dy, base + at, n, d);
      load_w(a.weight, a.w_bf16, at, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) xh[j] = (xh[j] - mean) * rstd, g[j] = d[j] * w[j];
    };
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll KEEP
    for (int i = 0; i < steps; ++i) {
      const int at = 8 * (threadIdx.x + i * T), n = W - at;
      float xh[8] = {}, g[8] = {}, d[8] = {};
      if (n > 0) read(at, n, xh, g, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          sg += g[j];
          sgx += g[j] * xh[j];
        }
        if (CHUNKS > 0) {
          kept_h[i][j] = xh[j], kept_g[i][j] = g[j];
          if (j < n) dw[i][j] += d[j] * xh[j], db[i][j] += d[j];
        }
      }
    }
    if (!RMS) sg = row_sum<WAVES>(sg, part) / W;
    sgx = row_sum<WAVES>(sgx, part) / W;
#pragma unroll KEEP
    for (int i = 0; i < steps; ++i) {
      const int at = 8 * (threadIdx.x + i * T), n = W - at;
      if (n <= 0) continue;
      float xh[8], g[8], d[8];
      if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) xh[j] = kept_h[i][j], g[j] = kept_g[i][j];
      } else {
        read(at, n, xh, g, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * (g[j] - (RMS ? 0.0f : sg) - xh[j] * sgx);
      if (a.dtotal) {
        float t[8];
        load_8<BF16>(a.dtotal, base + at, n, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += t[j];
      }
      if (a.dresidual) store_8<BF16>(a.dresidual, base + at, n, d);
      if (DROP) drop_8(drop_bits((unsigned long long)(base + at), key), a.drop, d);
      store_8<BF16>(a.dx, base + at, n, d);
    }
  }
  if constexpr (CHUNKS > 0) {
    if (!a.parts) return;
    float *p = a.parts + (long long)blockIdx.x * 2 * W;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int at = 8 * (threadIdx.x + i * T), n = W - at;
      if (n <= 0) continue;
      store_8<false>(p, at, n, dw[i]);
      store_8<false>(p + W, at, n, db[i]);
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
    float h, d;
    if constexpr (BF16) {
      h = __builtin_bit_cast(float, (uint32_t)((const uint16_t *)a.total)[row * W + c] << 16);
      d = __builtin_bit_cast(float, (uint32_t)((const uint16_t *)a.dy)[row * W + c] << 16);
    } else {
      h = ((const float *)a.total)[row * W + c];
      d = ((const float *)a.dy)[row * W + c];
    }
    dw += d * ((h - (RMS ? 0.0f : a.mean[row])) * a.rstd[row]);
    db += d;
  }
  float *p = a.parts + (long long)blockIdx.y * 2 * W;
  p[c] = dw;
  p[W + c] = db;
}

// dweight and dbias from n parts: 64 columns of one of them a workgroup, its waves over the parts.
constexpr int kPartsThreads = 1024;
__global__ __launch_bounds__(kPartsThreads) void k_norm_parts(const float *__restrict__ parts, int n, int W,
                                                             float *dweight, float *dbias, int accumulate) {
  constexpr int WAVES = kPartsThreads / kWave;
  __shared__ float s[WAVES][kWave];
  float *out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = blockIdx.x * kWave + lane;
  float v = 0.0f;
  if (c < W)
    for (int i = w; i < n; i += WAVES) v += parts[((long long)i * 2 + blockIdx.y) * W + c];
  s[w][lane] = v;
  __syncthreads();
  if (w || c >= W) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) v += s[i][lane];
  out[c] = accumulate ? out[c] + v : v;
}

// Calls f with the waves a row and the steps a thread for a width.
template <class F>
static void with_row(int W, F f) {
  auto of = [&](auto w, auto c) { return f(w, c); };
  using std::integral_constant;
#define MOE_ROW(w, c) of(integral_constant<int, w>{}, integral_constant<int, c>{})
  if (W <= 512) MOE_ROW(1, 1);
  else if (W <= 1024) MOE_ROW(1, 2);
  else if (W <= 2048) MOE_ROW(2, 2);
  else if (W <= 4096) MOE_ROW(4, 2);
  else if (W <= 8192) MOE_ROW(8, 2);
  else if (W <= 16384) MOE_ROW(16, 2);
  else MOE_ROW(16, 0);
#undef MOE_ROW
}

constexpr int kNormWidest = 16384;       // kept in registers
constexpr int kNormMaxWidth = 1 << 22;
constexpr int kNormParts = 512;          // sums of columns that a backward call makes, then adds up
constexpr int kColParts = 64;            // the same for wider rows

static int norm_parts(int64_t rows, int64_t width) {
  const int most = width > kNormWidest ? kColParts : kNormParts;
  return (int)(rows < most ? rows : most);
}

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
  const Range in[] = {{x, bytes, true}, {residual, bytes, true}, {weight, w_bytes, false}, {bias, w_bytes, false},
                      {rng, 16, false}, {total, bytes, false}, {mean, s_bytes, false}, {rstd, s_bytes, false}};
  if (!stands_alone(y, bytes, in, 8) || !stands_alone(total, bytes, in, 5) || !stands_alone(mean, s_bytes, in, 6) ||
      !stands_alone(rstd, s_bytes, in, 7))
    return MOE_EINVAL;
  NormArgs a{x, residual, weight, bias, total, y, mean, rstd, rows, (int)width, w_dtype == MOE_BF16, (float)eps,
             make_drop(p, rng, offset)};
  auto go = [&](auto bf16, auto rms, auto drop) {
    with_row((int)width, [&](auto w, auto c) {
      hipLaunchKernelGGL((k_norm<bf16.value, rms.value, drop.value, w.value, c.value>),
                         dim3((unsigned)(rows < (1 << 22) ? rows : 1 << 22)), dim3(w.value * kWave), 0, stream, a);
    });
  };
  auto pick = [&](auto bf16, auto rms) { a.drop.below ? go(bf16, rms, std::true_type{}) : go(bf16, rms, std::false_type{}); };
  auto kinds = [&](auto bf16) { kind == MOE_NORM_RMS ? pick(bf16, std::true_type{}) : pick(bf16, std::false_type{}); };
  dtype == MOE_BF16 ? kinds(std::true_type{}) : kinds(std::false_type{});
  return launch_status();
}

extern "C" size_t moe_layer_norm_backward_workspace_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || rows >= (1LL << 31) || width < 1 || width > kNormMaxWidth) return 0;
  return (size_t)norm_parts(rows, width) * 2 * width * sizeof(float);
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
  const Range in[] = {{dy, bytes, true},        {dtotal, bytes, true},       {total, bytes, false},   {weight, w_bytes, false},
                      {mean, s_bytes, false},   {rstd, s_bytes, false},      {rng, 16, false},        {ws, sums ? need : 0, false},
                      {dweight, d_bytes, false}, {dbias, d_bytes, false},    {dresidual, bytes, false}};
  if (!stands_alone(dx, bytes, in, 11) || !stands_alone(dresidual, bytes, in, 10)) return MOE_EINVAL;
  if (sums && (!stands_alone(dweight, d_bytes, in, 8) || !stands_alone(dbias, d_bytes, in, 9) ||
               !stands_alone(ws, need, in, 7)))
    return MOE_EINVAL;
  NormBwdArgs a{total, weight, dy, dtotal, mean, rstd, dx, dresidual, sums ? (float *)ws : nullptr, rows, (int)width,
                w_dtype == MOE_BF16, make_drop(p, rng, offset)};
  const int parts = norm_parts(rows, width);
  auto go = [&](auto bf16, auto rms, auto drop) {
    if (sums && width > kNormWidest)  // before dx, which may take dy's place
      hipLaunchKernelGGL((k_norm_cols<bf16.value, rms.value>), dim3(ceil_div(width, kColThreads), parts),
                         dim3(kColThreads), 0, stream, a);
    with_row((int)width, [&](auto w, auto c) {
      const int64_t most = c.value ? kNormParts : 1 << 22;
      hipLaunchKernelGGL((k_norm_bwd<bf16.value, rms.value, drop.value, w.value, c.value>),
                         dim3((unsigned)(rows < most ? rows : most)), dim3(w.value * kWave), 0, stream, a);
    });
  };
  auto pick = [&](auto bf16, auto rms) { a.drop.below ? go(bf16, rms, std::true_type{}) : go(bf16, rms, std::false_type{}); };
  auto kinds = [&](auto bf16) { kind == MOE_NORM_RMS ? pick(bf16, std::true_type{}) : pick(bf16, std::false_type{}); };
  if (rows) dtype == MOE_BF16 ? kinds(std::true_type{}) : kinds(std::false_type{});
  if (sums)
    hipLaunchKernelGGL(k_norm_parts, dim3(ceil_div(width, kWave), 2), dim3(kPartsThreads), 0, stream,
                       (const float *)ws, parts, (int)width, dweight, dbias, accumulate);
  return launch_status();
}
