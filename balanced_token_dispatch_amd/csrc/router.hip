// moe_router_topk, moe_router_backward: the K experts of each token and their weights from the
// gate's logits, and the logits' gradient from the weights'.
//
// One wave per token.  Lane l holds the V consecutive experts l V .. l V + V - 1, so of equal
// values the lowest expert is the first set bit of a ballot's lowest lane.
#include <type_traits>

#include "common.hpp"

namespace moe {

constexpr int kRtThreads = 256;
constexpr int kRtMaxE = 1024;

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
  return v;
}
__device__ inline double wave_max(double v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v = fmax(v, __shfl_xor(v, off, kWave));
  return v;
}
__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
  return v;
}
__device__ inline uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, kWave));
  return v;
}
__device__ inline unsigned long long wave_max(unsigned long long v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const unsigned long long o = __shfl_xor(v, off, kWave);
    v = v > o ? v : o;
  }
  return v;
}

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

template <bool BF16>
__device__ inline float load_logit(const void *p, long long i) {
  if constexpr (BF16)
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
  else
    return ((const float *)p)[i];
}

// 1 / (1 + exp(-x)); exp's overflow to infinity gives the right zero
__device__ inline float logistic(float x) { return 1.0f / (1.0f + expf(-x)); }

template <int V, bool BF16, int SCORE, bool BIAS>
__global__ __launch_bounds__(kRtThreads) void k_router_topk(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ idx,
    float *__restrict__ w, long long T, int E, int K, float factor) {
  const int lane = threadIdx.x & 63;
  const long long waves = (long long)gridDim.x * (kRtThreads / kWave);
  for (long long t = (long long)blockIdx.x * (kRtThreads / kWave) + (threadIdx.x >> 6); t < T;
       t += waves) {
    using Key = std::conditional_t<BIAS, unsigned long long, uint32_t>;
    float x[V];
    Key key[V];
    int rank[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane * V + j;
      x[j] = e < E ? load_logit<BF16>(logits, t * E + e) : -__builtin_inff();
      rank[j] = -1;
    }
    float top = -__builtin_inff();  // of all experts
    if (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
      top = wave_max(top);
    }
    if constexpr (BIAS) {
      // selection by score + bias: near ties decide which experts run, so in 64 bits
      double s[V], sum = 0.0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[j] = x[j];
        if (SCORE == MOE_SCORE_SIGMOID) s[j] = 1.0 / (1.0 + exp(-s[j]));
        if (SCORE == MOE_SCORE_SOFTMAX) sum += s[j] = exp(s[j] - (double)top);
      }
      if (SCORE == MOE_SCORE_SOFTMAX) sum = wave_sum(sum);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = lane * V + j;
        if (SCORE == MOE_SCORE_SOFTMAX) s[j] /= sum;
        key[j] = e < E ? order_key(s[j] + (double)bias[e]) : 0;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = lane * V + j < E ? order_key(x[j]) : 0;
    }
    for (int r = 0; r < K; ++r) {
      Key best = 0;
      int bj = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (key[j] > best) best = key[j], bj = j;
      const Key most = wave_max(best);
      const int owner = __ffsll((unsigned long long)__ballot(best == most)) - 1;
      if (lane == owner) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j == bj) key[j] = 0, rank[j] = r;
        idx[t * K + r] = lane * V + bj;
      }
    }
    // weights of the chosen: score / sum, 0 where the sum is 0
    float m = top, sum = 0.0f, s[V];
    if (SCORE == MOE_SCORE_SOFTMAX_TOPK) {
#pragma unroll
      for (int j = 0; j < V; ++j) m = rank[j] >= 0 ? fmaxf(m, x[j]) : m;
      m = wave_max(m);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool in = SCORE == MOE_SCORE_SOFTMAX ? lane * V + j < E : rank[j] >= 0;
      s[j] = SCORE == MOE_SCORE_SIGMOID ? logistic(x[j]) : x[j] == -__builtin_inff() ? 0.0f : expf(x[j] - m);
      sum += in ? s[j] : 0.0f;
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (rank[j] >= 0) w[t * K + rank[j]] = sum == 0.0f ? 0.0f : factor * (s[j] / sum);
  }
}

// dlogits of one token per wave.  Each chosen entry's gradient is worked out by one lane, 64
// entries at a time, and added in entry order into the lanes that hold the experts (the same
// expert twice adds twice).
template <int V, bool BF16, int SCORE>
__global__ __launch_bounds__(kRtThreads) void k_router_bwd(
    const void *__restrict__ logits, const int32_t *__restrict__ idx,
    const float *__restrict__ dw, void *__restrict__ dlogits, long long T, int E, int K,
    float factor) {
  const int lane = threadIdx.x & 63;
  const long long waves = (long long)gridDim.x * (kRtThreads / kWave);
  const float ninf = -__builtin_inff();
  for (long long t = (long long)blockIdx.x * (kRtThreads / kWave) + (threadIdx.x >> 6); t < T;
       t += waves) {
    float x[V];
    float m = ninf, sum = 0.0f, inner = 0.0f;
    if (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = lane * V + j;
        x[j] = e < E ? load_logit<BF16>(logits, t * E + e) : ninf;
        m = fmaxf(m, x[j]);
      }
      m = wave_max(m);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[j] = x[j] == ninf ? 0.0f : expf(x[j] - m);
        sum += x[j];
      }
    }
    // entry r of this token: its expert (-1: none), logit and weight's gradient
    auto entry = [&](int r, int &e, float &c, float &d) {
      e = -1, c = ninf, d = 0.0f;
      if (r < K) {
        e = idx[t * K + r];
        if (e < 0 || e >= E) e = -1;
        if (e >= 0) c = load_logit<BF16>(logits, t * E + e), d = factor * dw[t * K + r];
      }
    };
    int e;
    float c, d;
    if (SCORE == MOE_SCORE_SOFTMAX_TOPK) {
      for (int r = lane; r < K; r += kWave) entry(r, e, c, d), m = fmaxf(m, c);
      m = wave_max(m);
    }
    auto score = [&](float v) {
      return SCORE == MOE_SCORE_SIGMOID ? logistic(v) : v == ninf ? 0.0f : expf(v - m);
    };
    for (int r = lane; r < K; r += kWave) {
      entry(r, e, c, d);
      const float s = score(c);
      if (SCORE != MOE_SCORE_SOFTMAX) sum += e >= 0 ? s : 0.0f;
      inner += d * s;
    }
    sum = wave_sum(sum);
    const float rs = sum == 0.0f ? 0.0f : 1.0f / sum;
    inner = wave_sum(inner) * rs;
    float out[V];
#pragma unroll
    for (int j = 0; j < V; ++j) out[j] = SCORE == MOE_SCORE_SOFTMAX ? -inner * (x[j] * rs) : 0.0f;
    for (int r0 = 0; r0 < K; r0 += kWave) {
      entry(r0 + lane, e, c, d);
      const float wgt = score(c) * rs;
      float gr = 0.0f;
      if (e >= 0) {
        if (SCORE == MOE_SCORE_SOFTMAX) gr = wgt * d;
        if (SCORE == MOE_SCORE_SOFTMAX_TOPK) gr = wgt * (d - inner);
        if (SCORE == MOE_SCORE_SIGMOID) gr = wgt * (d - inner) / (1.0f + expf(c));
      }
      for (int r = 0; r < min(K - r0, kWave); ++r) {
        const int er = __shfl(e, r, kWave);
        const float g = __shfl(gr, r, kWave);
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] += er == lane * V + j ? g : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int n = lane * V + j;
      if (n >= E) continue;
      if constexpr (BF16)
        ((uint16_t *)dlogits)[t * E + n] = (uint16_t)pack_bf16x2(out[j], 0.0f);
      else
        ((float *)dlogits)[t * E + n] = out[j];
    }
  }
}

template <int V, bool BF16, int SCORE>
static void launch_topk(dim3 grid, hipStream_t stream, const void *logits, const float *bias,
                        int32_t *idx, float *w, int64_t T, int E, int K, float factor) {
  if (bias)
    hipLaunchKernelGGL((k_router_topk<V, BF16, SCORE, true>), grid, dim3(kRtThreads), 0, stream,
                       logits, bias, idx, w, T, E, K, factor);
  else
    hipLaunchKernelGGL((k_router_topk<V, BF16, SCORE, false>), grid, dim3(kRtThreads), 0, stream,
                       logits, bias, idx, w, T, E, K, factor);
}

template <int V, bool BF16>
struct Router {
  static void topk(int score, dim3 grid, hipStream_t stream, const void *logits, const float *bias,
                   int32_t *idx, float *w, int64_t T, int E, int K, float factor) {
    if (score == MOE_SCORE_SOFTMAX_TOPK)
      launch_topk<V, BF16, MOE_SCORE_SOFTMAX_TOPK>(grid, stream, logits, bias, idx, w, T, E, K, factor);
    else if (score == MOE_SCORE_SOFTMAX)
      launch_topk<V, BF16, MOE_SCORE_SOFTMAX>(grid, stream, logits, bias, idx, w, T, E, K, factor);
    else
      launch_topk<V, BF16, MOE_SCORE_SIGMOID>(grid, stream, logits, bias, idx, w, T, E, K, factor);
  }
  static void bwd(int score, dim3 grid, hipStream_t stream, const void *logits, const int32_t *idx,
                  const float *dw, void *dlogits, int64_t T, int E, int K, float factor) {
    if (score == MOE_SCORE_SOFTMAX_TOPK)
      hipLaunchKernelGGL((k_router_bwd<V, BF16, MOE_SCORE_SOFTMAX_TOPK>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor);
    else if (score == MOE_SCORE_SOFTMAX)
      hipLaunchKernelGGL((k_router_bwd<V, BF16, MOE_SCORE_SOFTMAX>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor);
    else
      hipLaunchKernelGGL((k_router_bwd<V, BF16, MOE_SCORE_SIGMOID>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor);
  }
};

// The V of E experts: the least of 1, 4, 8, 16 with 64 V >= E.
template <class F>
static void with_v(int E, bool bf16, F f) {
  if (E <= 64) bf16 ? f(Router<1, true>{}) : f(Router<1, false>{});
  else if (E <= 256) bf16 ? f(Router<4, true>{}) : f(Router<4, false>{});
  else if (E <= 512) bf16 ? f(Router<8, true>{}) : f(Router<8, false>{});
  else bf16 ? f(Router<16, true>{}) : f(Router<16, false>{});
}

static bool router_args_ok(moe_dtype dtype, moe_score score, int64_t T, int32_t E, int32_t K,
                           float factor) {
  if (dtype != MOE_BF16 && dtype != MOE_F32) return false;
  if (score != MOE_SCORE_SOFTMAX_TOPK && score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return false;
  if (T < 0 || T >= (1LL << 31) || E < 1 || E > kRtMaxE || K < 1 || K > E) return false;
  return factor == factor && factor - factor == 0.0f;  // finite
}

static dim3 router_grid(int64_t T) {
  const int64_t b = (T + kRtThreads / kWave - 1) / (kRtThreads / kWave);
  return dim3((unsigned)(b < (1 << 22) ? b : (1 << 22)));
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_router_topk(moe_dtype dtype, moe_score score, int64_t T, int32_t E,
                                        int32_t K, const void *logits, const float *bias,
                                        float factor, int32_t *topk_idx, float *topk_w,
                                        hipStream_t stream) {
  if (!router_args_ok(dtype, score, T, E, K, factor)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_EINVAL;
  with_v(E, dtype == MOE_BF16, [&](auto r) {
    r.topk(score, router_grid(T), stream, logits, bias, topk_idx, topk_w, T, E, K, factor);
  });
  return launch_status();
}

extern "C" moe_status_t moe_router_backward(moe_dtype dtype, moe_score score, int64_t T, int32_t E,
                                            int32_t K, const void *logits, const int32_t *topk_idx,
                                            const float *dtopk_w, float factor, void *dlogits,
                                            hipStream_t stream) {
  if (!router_args_ok(dtype, score, T, E, K, factor)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !dtopk_w || !dlogits || logits == dlogits) return MOE_EINVAL;
  with_v(E, dtype == MOE_BF16, [&](auto r) {
    r.bwd(score, router_grid(T), stream, logits, topk_idx, dtopk_w, dlogits, T, E, K, factor);
  });
  return launch_status();
}
