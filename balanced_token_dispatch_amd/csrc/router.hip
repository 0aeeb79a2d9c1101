// moe_router_topk, moe_router_backward: the K experts of each token and their weights from the
// gate's logits, and the logits' gradient from the weights'.
//
// One wave per token.  Expert e sits in chunk c = e / (64 P), lane e / P % 64, place e % P of the lane
// (P = 4, 16 bytes of fp32 a lane, so that a row moves as contiguous vectors; P = 1 up to 64
// experts), so of equal values the lowest expert is in the first chunk, lowest lane, first place.
//
// Latency-bound at small T, and by the K rounds of selection (a lane-local maximum, six data-parallel
// steps across the wave, one ballot) at large: 4096 x 256 fp32 logits, K = 8, in 5.6 us, launch included,
// where reading them takes 0.8 us; the gradient of 8192 x 384 bf16 logits (6.3 MB written) in 7.
#include <type_traits>

#include "common.hpp"

namespace moe {

constexpr int kRtThreads = 256;
constexpr int kRtMaxE = 1024;

// Wave-wide maximum and sum without LDS: each step combines a lane with one a power of two away (row
// shifts within 16 lanes, then the last lane of a row into the next rows); lane 63 ends with all.
template <int CTRL, int ROWS>
__device__ inline uint32_t dpp_step(uint32_t keep, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)keep, (int)v, CTRL, ROWS, 0xF, false);
}
constexpr int kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118, kBcast15 = 0x142, kBcast31 = 0x143;

__device__ inline uint32_t wave_max(uint32_t v) {
  v = max(v, dpp_step<kShr1, 0xF>(0, v));
  v = max(v, dpp_step<kShr2, 0xF>(0, v));
  v = max(v, dpp_step<kShr4, 0xF>(0, v));
  v = max(v, dpp_step<kShr8, 0xF>(0, v));
  v = max(v, dpp_step<kBcast15, 0xA>(0, v));
  v = max(v, dpp_step<kBcast31, 0xC>(0, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ inline float wave_sum(float v) {
  auto at = [](uint32_t x) { return __builtin_bit_cast(float, x); };
  v += at(dpp_step<kShr1, 0xF>(0, __builtin_bit_cast(uint32_t, v)));
  v += at(dpp_step<kShr2, 0xF>(0, __builtin_bit_cast(uint32_t, v)));
  v += at(dpp_step<kShr4, 0xF>(0, __builtin_bit_cast(uint32_t, v)));
  v += at(dpp_step<kShr8, 0xF>(0, __builtin_bit_cast(uint32_t, v)));
  v += at(dpp_step<kBcast15, 0xA>(0, __builtin_bit_cast(uint32_t, v)));
  v += at(dpp_step<kBcast31, 0xC>(0, __builtin_bit_cast(uint32_t, v)));
  return at((uint32_t)__builtin_amdgcn_readlane((int)__builtin_bit_cast(uint32_t, v), 63));
}

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
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

// The value of a key of fp32 order (the largest logit, from its key).
__device__ inline float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ inline uint32_t wave_max_hi(unsigned long long v, uint32_t *lo) {
  // the high words' maximum, then the low words' among the lanes that have it
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  *lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return hi;
}
__device__ inline unsigned long long wave_max(unsigned long long v) {
  uint32_t lo;
  const uint32_t hi = wave_max_hi(v, &lo);
  return (unsigned long long)hi << 32 | lo;
}

template <bool BF16>
__device__ inline float load_logit(const void *p, long long i) {
  if constexpr (BF16)
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
  else
    return ((const float *)p)[i];
}

// Where lane `lane` holds place v of its C P values.
template <int P>
__device__ inline int expert_of(int lane, int v) {
  return v / P * (64 * P) + lane * P + v % P;
}

// This lane's values of the row that starts at element i, -inf past E.  vec: whole rows are aligned to
// a lane's 4 values and E is a multiple of them.
template <int C, int P, bool BF16>
__device__ inline void load_row(const void *p, long long i, int E, bool vec, float (&x)[C * P]) {
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_inff();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = expert_of<P>(lane, c * P);
    if (P == 4 && vec) {
      if (e >= E) {
#pragma unroll
        for (int j = 0; j < P; ++j) x[c * P + j] = ninf;
      } else if constexpr (BF16) {
        const uint2 t = *(const uint2 *)((const uint16_t *)p + i + e);
        x[c * P] = bf16_lo(t.x);
        x[c * P + 1 % P] = bf16_hi(t.x);
        x[c * P + 2 % P] = bf16_lo(t.y);
        x[c * P + 3 % P] = bf16_hi(t.y);
      } else {
        const f32x4 t = *(const f32x4 *)((const float *)p + i + e);
#pragma unroll
        for (int j = 0; j < P; ++j) x[c * P + j] = t[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < P; ++j) x[c * P + j] = e + j < E ? load_logit<BF16>(p, i + e + j) : ninf;
    }
  }
}

// 1 / (1 + exp(-x)); exp's overflow to infinity gives the right zero
__device__ inline float logistic(float x) { return 1.0f / (1.0f + expf(-x)); }

template <int C, int P, bool BF16, int SCORE, bool BIAS>
__global__ __launch_bounds__(kRtThreads) void k_router_topk(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ idx,
    float *__restrict__ w, long long T, int E, int K, float factor, int vec) {
  constexpr int V = C * P;
  using Key = std::conditional_t<BIAS, unsigned long long, uint32_t>;
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_inff();
  const long long waves = (long long)gridDim.x * (kRtThreads / kWave);
  for (long long t = (long long)blockIdx.x * (kRtThreads / kWave) + (threadIdx.x >> 6); t < T;
       t += waves) {
    float x[V];
    Key key[V];
    int rank[V];
    load_row<C, P, BF16>(logits, t * E, E, vec, x);
    float top = ninf;  // of all experts
    if (SCORE == MOE_SCORE_SOFTMAX) {
      uint32_t k = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) k = max(k, x[j] == x[j] ? order_key(x[j]) : 0u);
      k = wave_max(k);
      top = k ? key_value(k) : ninf;
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
        const int e = expert_of<P>(lane, j);
        if (SCORE == MOE_SCORE_SOFTMAX) s[j] /= sum;
        key[j] = e < E ? order_key(s[j] + (double)bias[e]) : 0;
        rank[j] = -1;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = expert_of<P>(lane, j) < E ? order_key(x[j]) : 0, rank[j] = -1;
    }
    for (int r = 0; r < K; ++r) {
      Key best = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) best = max(best, key[j]);
      const Key most = wave_max(best);
      // the first chunk that has it, its lowest lane, that lane's first place
      bool open = true;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        bool here = false;
#pragma unroll
        for (int j = 0; j < P; ++j) here |= key[c * P + j] == most;
        const unsigned long long who = __ballot(open && here);
        if (open && who) {
          open = false;
          bool mine = lane == __ffsll(who) - 1;
#pragma unroll
          for (int j = 0; j < P; ++j)
            if (mine && key[c * P + j] == most) key[c * P + j] = 0, rank[c * P + j] = r, mine = false;
        }
      }
    }
    // weights of the chosen: score / sum, 0 where the sum is 0
    float m = top, sum = 0.0f, s[V];
    if (SCORE == MOE_SCORE_SOFTMAX_TOPK) {
      uint32_t k = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) k = max(k, rank[j] >= 0 && x[j] == x[j] ? order_key(x[j]) : 0u);
      k = wave_max(k);
      m = k ? key_value(k) : ninf;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool in = SCORE == MOE_SCORE_SOFTMAX ? expert_of<P>(lane, j) < E : rank[j] >= 0;
      s[j] = SCORE == MOE_SCORE_SIGMOID ? logistic(x[j]) : x[j] == ninf ? 0.0f : expf(x[j] - m);
      sum += in ? s[j] : 0.0f;
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (rank[j] >= 0) {
        idx[t * K + rank[j]] = expert_of<P>(lane, j);
        w[t * K + rank[j]] = sum == 0.0f ? 0.0f : factor * (s[j] / sum);
      }
  }
}

// dlogits of one token per wave.  Each chosen entry's gradient is worked out by one lane, 64
// entries at a time, and added in entry order into the lanes that hold the experts (the same
// expert twice adds twice).
template <int C, int P, bool BF16, int SCORE>
__global__ __launch_bounds__(kRtThreads) void k_router_bwd(
    const void *__restrict__ logits, const int32_t *__restrict__ idx,
    const float *__restrict__ dw, void *__restrict__ dlogits, long long T, int E, int K,
    float factor, int vec) {
  constexpr int V = C * P;
  const int lane = threadIdx.x & 63;
  const long long waves = (long long)gridDim.x * (kRtThreads / kWave);
  const float ninf = -__builtin_inff();
  auto largest = [&](float a, float b) { return b > a ? b : a; };  // of numbers; a NaN passes by
  for (long long t = (long long)blockIdx.x * (kRtThreads / kWave) + (threadIdx.x >> 6); t < T;
       t += waves) {
    float x[V];
    float m = ninf, sum = 0.0f, inner = 0.0f;
    auto all_lanes = [&]() {
      const uint32_t k = wave_max(m == ninf ? 0u : order_key(m));
      m = k ? key_value(k) : ninf;
    };
    if (SCORE == MOE_SCORE_SOFTMAX) {
      load_row<C, P, BF16>(logits, t * E, E, vec, x);
#pragma unroll
      for (int j = 0; j < V; ++j) m = largest(m, x[j]);
      all_lanes();
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
      for (int r = lane; r < K; r += kWave) entry(r, e, c, d), m = largest(m, c);
      all_lanes();
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
        const int er = __builtin_amdgcn_readlane(e, r);
        const float g = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, gr), r));
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] += er == expert_of<P>(lane, j) ? g : 0.0f;
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int n = expert_of<P>(lane, c * P);
      if (P == 4 && vec) {
        if (n >= E) continue;
        if constexpr (BF16) {
          uint2 o;
          o.x = pack_bf16x2(out[c * P], out[c * P + 1 % P]);
          o.y = pack_bf16x2(out[c * P + 2 % P], out[c * P + 3 % P]);
          *(uint2 *)((uint16_t *)dlogits + t * E + n) = o;
        } else {
          *(f32x4 *)((float *)dlogits + t * E + n) =
              (f32x4){out[c * P], out[c * P + 1 % P], out[c * P + 2 % P], out[c * P + 3 % P]};
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (n + j >= E) continue;
        if constexpr (BF16)
          ((uint16_t *)dlogits)[t * E + n + j] = (uint16_t)pack_bf16x2(out[c * P + j], 0.0f);
        else
          ((float *)dlogits)[t * E + n + j] = out[c * P + j];
      }
    }
  }
}

template <int C, int P, bool BF16, int SCORE>
static void launch_topk(dim3 grid, hipStream_t stream, const void *logits, const float *bias,
                        int32_t *idx, float *w, int64_t T, int E, int K, float factor, int vec) {
  if (bias)
    hipLaunchKernelGGL((k_router_topk<C, P, BF16, SCORE, true>), grid, dim3(kRtThreads), 0, stream,
                       logits, bias, idx, w, T, E, K, factor, vec);
  else
    hipLaunchKernelGGL((k_router_topk<C, P, BF16, SCORE, false>), grid, dim3(kRtThreads), 0, stream,
                       logits, bias, idx, w, T, E, K, factor, vec);
}

template <int C, int P, bool BF16>
struct Router {
  static void topk(int score, dim3 grid, hipStream_t stream, const void *logits, const float *bias,
                   int32_t *idx, float *w, int64_t T, int E, int K, float factor, int vec) {
    if (score == MOE_SCORE_SOFTMAX_TOPK)
      launch_topk<C, P, BF16, MOE_SCORE_SOFTMAX_TOPK>(grid, stream, logits, bias, idx, w, T, E, K, factor, vec);
    else if (score == MOE_SCORE_SOFTMAX)
      launch_topk<C, P, BF16, MOE_SCORE_SOFTMAX>(grid, stream, logits, bias, idx, w, T, E, K, factor, vec);
    else
      launch_topk<C, P, BF16, MOE_SCORE_SIGMOID>(grid, stream, logits, bias, idx, w, T, E, K, factor, vec);
  }
  static void bwd(int score, dim3 grid, hipStream_t stream, const void *logits, const int32_t *idx,
                  const float *dw, void *dlogits, int64_t T, int E, int K, float factor, int vec) {
    if (score == MOE_SCORE_SOFTMAX_TOPK)
      hipLaunchKernelGGL((k_router_bwd<C, P, BF16, MOE_SCORE_SOFTMAX_TOPK>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor, vec);
    else if (score == MOE_SCORE_SOFTMAX)
      hipLaunchKernelGGL((k_router_bwd<C, P, BF16, MOE_SCORE_SOFTMAX>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor, vec);
    else
      hipLaunchKernelGGL((k_router_bwd<C, P, BF16, MOE_SCORE_SIGMOID>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor, vec);
  }
};

// The fewest values per lane that hold E experts.
template <class F>
static void with_shape(int E, bool bf16, F f) {
  if (E <= 64) bf16 ? f(Router<1, 1, true>{}) : f(Router<1, 1, false>{});
  else if (E <= 256) bf16 ? f(Router<1, 4, true>{}) : f(Router<1, 4, false>{});
  else if (E <= 512) bf16 ? f(Router<2, 4, true>{}) : f(Router<2, 4, false>{});
  else bf16 ? f(Router<4, 4, true>{}) : f(Router<4, 4, false>{});
}

// Whether every row of p can be read and written as vectors of 4 values.
static bool rows_of_4(moe_dtype dtype, int E, const void *p) {
  return E % 4 == 0 && (uintptr_t)p % (dtype == MOE_BF16 ? 8 : 16) == 0;
}

static bool router_args_ok(moe_dtype dtype, moe_score score, int64_t T, int32_t E, int32_t K,
                           float factor) {
  if (dtype != MOE_BF16 && dtype != MOE_F32) return false;
  if (score != MOE_SCORE_SOFTMAX_TOPK && score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return false;
  if (T < 0 || T >= (1LL << 31) || E < 1 || E > kRtMaxE || K < 1 || K > E) return false;
  return factor == factor && factor - factor == 0.0f;  // finite
}

static bool misaligned(const void *p, size_t n) { return (uintptr_t)p % n != 0; }

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
  if (misaligned(logits, dtype == MOE_BF16 ? 2 : 4) || misaligned(bias, 4) || misaligned(topk_idx, 4) ||
      misaligned(topk_w, 4))
    return MOE_EINVAL;
  with_shape(E, dtype == MOE_BF16, [&](auto r) {
    r.topk(score, router_grid(T), stream, logits, bias, topk_idx, topk_w, T, E, K, factor,
           rows_of_4(dtype, E, logits));
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
  const size_t size = dtype == MOE_BF16 ? 2 : 4;
  if (misaligned(logits, size) || misaligned(dlogits, size) || misaligned(topk_idx, 4) ||
      misaligned(dtopk_w, 4))
    return MOE_EINVAL;
  with_shape(E, dtype == MOE_BF16, [&](auto r) {
    r.bwd(score, router_grid(T), stream, logits, topk_idx, dtopk_w, dlogits, T, E, K, factor,
          rows_of_4(dtype, E, logits) && rows_of_4(dtype, E, dlogits));
  });
  return launch_status();
}
