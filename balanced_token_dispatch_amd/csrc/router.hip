// moe_router_topk, moe_router_backward: the K experts of each token and their weights from the
// gate's logits, and the logits' gradient from the weights'.
//
// Several tokens share a wave (16 lanes each up to 256 experts) where there are enough of them.
//
// Latency-bound at small T (one token of 256 experts, K = 8: 3.4 us, launch included), and by the K rounds of
// selection at large: 4096 x 256 fp32 logits 4.9 us where reading them takes 0.8, 65536 x 256 20 us where
// it takes 11.  With a bias, by a 64-bit exponential and division for each expert and 64-bit keys: 65536 x 256 take
// 52 us on the logits themselves, 56 on the logistic, 59 on the softmax over all; 4096 x 256 7.4, 7.6, 9.3.  The
// gradient of 8192 x 384 bf16 logits (6.3 MB written) takes 4.6 us (logistic 4.9), of 65536 x 256 fp32 ones (67 MB)
// 17.5: every row goes through LDS, also where all but K of its entries are 0.
#include <type_traits>

#include "lanes.hpp"

namespace moe {

constexpr int kRtThreads = 256;
constexpr int kRtMaxE = 1024;

// L lanes per token, V = 4 G consecutive experts each, so that of equal values the lowest expert is in
// the lowest lane, first place.  The keys lie in LDS, and a lane keeps the largest of each group of 4:
// a round of the selection is a maximum over those and over the token's lanes, and only the lane that
// has it goes back to the 4 keys of one group.  (Keys all in registers, looked through by every lane
// each round, took 2 to 3 times as long: one token per wave, 43 us at 65536 x 256.)
template <int L, int V, bool BF16, int SCORE, bool BIAS>
__global__ __launch_bounds__(kRtThreads) void k_router_topk(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ idx,
    float *__restrict__ w, long long T, int E, int K, float factor, int vec) {
  constexpr int G = V / 4, kTokens = kWave / L;  // tokens per wave
  using Key = std::conditional_t<BIAS, unsigned long long, uint32_t>;
  typedef __attribute__((ext_vector_type(4))) Key Keys;
  __shared__ Keys keys[kRtThreads][G];
  __shared__ uint16_t chosen[kRtThreads * V];
  const int lane = threadIdx.x & 63, l = lane % L, e0 = l * V;
  const float ninf = -__builtin_inff();
  Keys *own = keys[threadIdx.x];
  uint16_t *list = chosen + (threadIdx.x - l) * V;
  for (long long t0 = ((long long)blockIdx.x * kRtThreads + (threadIdx.x & ~63)) / L; t0 < T;
       t0 += (long long)gridDim.x * (kRtThreads / L)) {
    const long long t = t0 + lane / L;
    float x[V];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const f32x4 q = load_4<BF16>(logits, t * E + e0 + 4 * g, t < T ? E - e0 - 4 * g : 0, vec);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * g + j] = q[j];
    }
    float top = ninf;  // of all experts
    if (SCORE == MOE_SCORE_SOFTMAX) {
      uint32_t k = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) k = max(k, x[j] == x[j] ? order_key(x[j]) : 0u);
      k = token_max<L>(k);
      top = k ? key_value(k) : ninf;
    }
    Key most_of[G];
    if constexpr (BIAS) {
      // selection by score + bias: near ties decide which experts run, so in 64 bits
      double s[V], sum = 0.0;
      const double base = top == ninf ? 0.0 : (double)top;  // with every logit -inf, scores of 0, not NaN
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[j] = x[j];
        if (SCORE == MOE_SCORE_SIGMOID) s[j] = 1.0 / (1.0 + exp(-s[j]));
        if (SCORE == MOE_SCORE_SOFTMAX) sum += s[j] = exp(s[j] - base);
      }
      if (SCORE == MOE_SCORE_SOFTMAX) sum = token_sum<L>(sum);
      if (sum == 0.0) sum = 1.0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        Keys k;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          double v = s[4 * g + j];
          if (SCORE == MOE_SCORE_SOFTMAX) v /= sum;
          k[j] = e0 + 4 * g + j < E ? order_key(v + (double)bias[e0 + 4 * g + j]) : 0;
        }
        own[g] = k;
        most_of[g] = max(max(k[0], k[1]), max(k[2], k[3]));
      }
    } else {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        Keys k;
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = e0 + 4 * g + j < E ? order_key(x[4 * g + j]) : 0;
        own[g] = k;
        most_of[g] = max(max(k[0], k[1]), max(k[2], k[3]));
      }
    }
    float sum = 0.0f;
    if (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < V; ++j) sum += e0 + j < E && x[j] != ninf ? expf(x[j] - top) : 0.0f;
      sum = token_sum<L>(sum);
    }
    Key first = 0;  // the largest key
    for (int r = 0; r < K; ++r) {
      Key best = most_of[0];
#pragma unroll
      for (int g = 1; g < G; ++g) best = max(best, most_of[g]);
      const Key most = token_max<L>(best);
      first = max(first, most);
      const unsigned long long who = __ballot(best == most) >> (lane - l);
      if (l == __ffsll(who) - 1) {  // the token's lowest lane that has it
        int g = 0;
#pragma unroll
        for (int i = G - 1; i > 0; --i) g = most_of[i] == most ? i : g;
        if (G > 1) g = most_of[0] == most ? 0 : g;
        Keys k = own[g];
        int p = 3;
#pragma unroll
        for (int j = 2; j >= 0; --j) p = k[j] == most ? j : p;
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = j == p ? 0 : k[j];
        own[g] = k;
        const Key rest = max(max(k[0], k[1]), max(k[2], k[3]));
#pragma unroll
        for (int i = 0; i < G; ++i) most_of[i] = i == g ? rest : most_of[i];
        list[r] = (uint16_t)(e0 + 4 * g + p);
      }
    }
    asm volatile("" ::: "memory");  // the list is read by other lanes of this wave, after its writes
    // weights of the chosen: score / sum, 0 where the sum is 0
    float m = top;
    auto logit = [&](int r) { return t < T && r < K ? load_logit<BF16>(logits, t * E + list[r]) : ninf; };
    if (SCORE == MOE_SCORE_SOFTMAX_TOPK || (SCORE == MOE_SCORE_SIGMOID && BIAS)) {
      uint32_t k = 0;
      for (int r = l; r < K; r += L) {
        const float c = logit(r);
        k = max(k, c == c ? order_key(c) : 0u);
      }
      k = token_max<L>(k);
      m = k ? key_value(k) : ninf;
    }
    // without a bias the first chosen is the largest (where it is NaN, so are the weights)
    if (SCORE == MOE_SCORE_SIGMOID) m = fminf(BIAS ? m : key_value((uint32_t)first), 0.0f);
    auto score = [&](float c) {
      return SCORE == MOE_SCORE_SIGMOID ? logistic_over(c, m) : c == ninf ? 0.0f : expf(c - m);
    };
    const float mine = score(logit(l));  // of the lane's first entry: the only one up to L
    if (SCORE != MOE_SCORE_SOFTMAX) {
      sum = l < K ? mine : 0.0f;
      for (int r = l + L; r < K; r += L) sum += score(logit(r));
      sum = token_sum<L>(sum);
    }
    for (int r = l; r < K; r += L)
      if (t < T) {
        idx[t * K + r] = list[r];
        w[t * K + r] = sum == 0.0f ? 0.0f : factor * ((r == l ? mine : score(logit(r))) / sum);
      }
  }
}

// dlogits, L lanes per token and V = 4 G experts each: group i of lane l starts at expert 4 (l + L i), so
// that a row moves as contiguous vectors.  The row is put together in LDS: first what every expert gets,
// then each chosen entry's gradient, worked out by one lane, L entries at a time.  Entries of the same
// expert are added by the first of them, in their order.  (One token per wave, every lane looking for its
// experts among the entries, took 27 us at 65536 x 64 and 35 at 65536 x 256.)
template <int L, int V, bool BF16, int SCORE>
__global__ __launch_bounds__(kRtThreads) void k_router_bwd(
    const void *__restrict__ logits, const int32_t *__restrict__ idx,
    const float *__restrict__ dw, void *__restrict__ dlogits, long long T, int E, int K,
    float factor, int vec) {
  constexpr int G = V / 4;
  __shared__ f32x4 rows[kRtThreads * G];
  const int lane = threadIdx.x & 63, l = lane % L;
  f32x4 *row = rows + (threadIdx.x - l) * G;
  float *at = (float *)row;
  const float ninf = -__builtin_inff();
  auto largest = [&](float a, float b) { return b > a ? b : a; };  // of numbers; a NaN passes by
  for (long long t0 = ((long long)blockIdx.x * kRtThreads + (threadIdx.x & ~63)) / L; t0 < T;
       t0 += (long long)gridDim.x * (kRtThreads / L)) {
    const long long t = t0 + lane / L;
    float m = ninf, sum = 0.0f, inner = 0.0f;
    auto all_lanes = [&]() {
      const uint32_t k = token_max<L>(m == ninf ? 0u : order_key(m));
      m = k ? key_value(k) : ninf;
    };
    f32x4 x[G];
    if (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int e = 4 * (l + L * i);
        x[i] = load_4<BF16>(logits, t * E + e, t < T ? E - e : 0, vec);
#pragma unroll
        for (int j = 0; j < 4; ++j) m = largest(m, x[i][j]);
      }
      all_lanes();
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = x[i][j] == ninf ? 0.0f : expf(x[i][j] - m);
          sum += x[i][j];
        }
    }
    // entry r of this token: its expert (-1: none), logit and weight's gradient; the lane's first one (the only
    // one up to L) is loaded once
    auto load_entry = [&](int r, int &e, float &c, float &d) {
      e = -1, c = ninf, d = 0.0f;
      if (t < T && r < K) {
        e = idx[t * K + r];
        if (e < 0 || e >= E) e = -1;
        if (e >= 0) c = load_logit<BF16>(logits, t * E + e), d = factor * dw[t * K + r];
      }
    };
    int e, e1;
    float c, d, c1, d1;
    load_entry(l, e1, c1, d1);
    auto entry = [&](int r, int &e, float &c, float &d) {
      if (r == l)
        e = e1, c = c1, d = d1;
      else
        load_entry(r, e, c, d);
    };
    if (SCORE != MOE_SCORE_SOFTMAX) {
      for (int r = l; r < K; r += L) entry(r, e, c, d), m = largest(m, c);
      all_lanes();
    }
    if (SCORE == MOE_SCORE_SIGMOID) m = fminf(m, 0.0f);
    auto score = [&](float v) {
      return SCORE == MOE_SCORE_SIGMOID ? logistic_over(v, m) : v == ninf ? 0.0f : expf(v - m);
    };
    const float s1 = score(c1);
    if (l < K) {
      if (SCORE != MOE_SCORE_SOFTMAX) sum += e1 >= 0 ? s1 : 0.0f;
      inner += d1 * s1;
    }
    for (int r = l + L; r < K; r += L) {
      entry(r, e, c, d);
      const float s = score(c);
      if (SCORE != MOE_SCORE_SOFTMAX) sum += e >= 0 ? s : 0.0f;
      inner += d * s;
    }
    sum = token_sum<L>(sum);
    const float rs = sum == 0.0f ? 0.0f : 1.0f / sum;
    inner = token_sum<L>(inner) * rs;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (SCORE == MOE_SCORE_SOFTMAX)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = -inner * (x[i][j] * rs);
      row[l + L * i] = v;
    }
    for (int r0 = 0; r0 < K; r0 += L) {
      entry(r0 + l, e, c, d);
      const float wgt = (r0 == 0 ? s1 : score(c)) * rs;
      float gr = 0.0f;
      if (e >= 0) {
        if (SCORE == MOE_SCORE_SOFTMAX) gr = wgt * d;
        if (SCORE == MOE_SCORE_SOFTMAX_TOPK) gr = wgt * (d - inner);
        if (SCORE == MOE_SCORE_SIGMOID) gr = wgt * (d - inner) / (1.0f + expf(c));
      }
      float total = 0.0f;
      bool first = e >= 0;
      for (int r = 0; r < min(K - r0, L); ++r) {
        const int er = __shfl(e, lane - l + r, kWave);
        const float g = __shfl(gr, lane - l + r, kWave);
        total += er == e ? g : 0.0f;
        first = first && (er != e || r >= l);
      }
      asm volatile("" ::: "memory");  // the row's entries were written by other lanes of this wave
      if (first) at[e] += total;
    }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int n = 4 * (l + L * i);
      if (t >= T || n >= E) continue;
      const f32x4 v = row[l + L * i];
      if (vec) {
        if constexpr (BF16) {
          uint2 o;
          o.x = pack_bf16x2(v[0], v[1]);
          o.y = pack_bf16x2(v[2], v[3]);
          *(uint2 *)((uint16_t *)dlogits + t * E + n) = o;
        } else {
          *(f32x4 *)((float *)dlogits + t * E + n) = v;
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (n + j >= E) continue;
        if constexpr (BF16)
          ((uint16_t *)dlogits)[t * E + n + j] = (uint16_t)pack_bf16x2(v[j], 0.0f);
        else
          ((float *)dlogits)[t * E + n + j] = v[j];
      }
    }
  }
}

template <int L, int V, bool BF16, int SCORE>
static void launch_topk(dim3 grid, hipStream_t stream, const void *logits, const float *bias,
                        int32_t *idx, float *w, int64_t T, int E, int K, float factor, int vec) {
  if (bias)
    hipLaunchKernelGGL((k_router_topk<L, V, BF16, SCORE, true>), grid, dim3(kRtThreads), 0, stream,
                       logits, bias, idx, w, T, E, K, factor, vec);
  else
    hipLaunchKernelGGL((k_router_topk<L, V, BF16, SCORE, false>), grid, dim3(kRtThreads), 0, stream,
                       logits, bias, idx, w, T, E, K, factor, vec);
}

template <int L_, int V, bool BF16>
struct Router {
  static constexpr int L = L_;
  static void topk(int score, dim3 grid, hipStream_t stream, const void *logits, const float *bias,
                   int32_t *idx, float *w, int64_t T, int E, int K, float factor, int vec) {
    if (score == MOE_SCORE_SOFTMAX_TOPK)
      launch_topk<L, V, BF16, MOE_SCORE_SOFTMAX_TOPK>(grid, stream, logits, bias, idx, w, T, E, K, factor, vec);
    else if (score == MOE_SCORE_SOFTMAX)
      launch_topk<L, V, BF16, MOE_SCORE_SOFTMAX>(grid, stream, logits, bias, idx, w, T, E, K, factor, vec);
    else
      launch_topk<L, V, BF16, MOE_SCORE_SIGMOID>(grid, stream, logits, bias, idx, w, T, E, K, factor, vec);
  }
  static void backward(int score, dim3 grid, hipStream_t stream, const void *logits, const int32_t *idx,
                       const float *dw, void *dlogits, int64_t T, int E, int K, float factor, int vec) {
    if (score == MOE_SCORE_SOFTMAX_TOPK)
      hipLaunchKernelGGL((k_router_bwd<L, V, BF16, MOE_SCORE_SOFTMAX_TOPK>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor, vec);
    else if (score == MOE_SCORE_SOFTMAX)
      hipLaunchKernelGGL((k_router_bwd<L, V, BF16, MOE_SCORE_SOFTMAX>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor, vec);
    else
      hipLaunchKernelGGL((k_router_bwd<L, V, BF16, MOE_SCORE_SIGMOID>), grid, dim3(kRtThreads), 0,
                         stream, logits, idx, dw, dlogits, T, E, K, factor, vec);
  }
};

// Lanes and experts per lane.  Few lanes share the wave's instructions among more tokens; all 64 make a
// token's own time shortest, which is what counts while there are not two tokens for each SIMD.
// moe_router_topk of fp32 logits, K = 8, us a launch (16 lanes / 64 lanes): 1 x 256 4.3 / 3.3, 1024 x 256
// 4.9 / 4.0, 4096 x 256 4.9 / 5.2, 65536 x 256 21 / 40; K = 6: 1 x 64 2.8 / 3.0, 65536 x 64 11 / 34.
// More experts a lane cost: 65536 x 1024, K = 16, with 32 lanes of 32 111 / 64 lanes of 16 106, 65536 x 64 with 8 a
// lane 13 / with 4 10.
template <bool BF16, class F>
static void with_shape(int E, int64_t T, F f) {
  const bool few = T <= 8LL * device_cu_count();
  if (E <= 64) f(Router<16, 4, BF16>{});
  else if (E <= 128 && !few) f(Router<16, 8, BF16>{});
  else if (E <= 256 && !few) f(Router<16, 16, BF16>{});
  else if (E <= 256) f(Router<64, 4, BF16>{});
  else if (E <= 512 && !few) f(Router<32, 16, BF16>{});
  else if (E <= 512) f(Router<64, 8, BF16>{});
  else f(Router<64, 16, BF16>{});
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

// Workgroups for T tokens of `lanes` lanes.
static dim3 router_grid(int64_t T, int lanes) {
  const int64_t per = kRtThreads / lanes, b = (T + per - 1) / per;
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
  auto launch = [&](auto r) {
    r.topk(score, router_grid(T, r.L), stream, logits, bias, topk_idx, topk_w, T, E, K, factor,
          rows_of_4(dtype, E, logits));
  };
  dtype == MOE_BF16 ? with_shape<true>(E, T, launch) : with_shape<false>(E, T, launch);
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
  auto launch = [&](auto r) {
    r.backward(score, router_grid(T, r.L), stream, logits, topk_idx, dtopk_w, dlogits, T, E, K, factor,
          rows_of_4(dtype, E, logits) && rows_of_4(dtype, E, dlogits));
  };
  dtype == MOE_BF16 ? with_shape<true>(E, T, launch) : with_shape<false>(E, T, launch);
  return launch_status();
}
