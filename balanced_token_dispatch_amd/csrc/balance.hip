// moe_expert_counts, moe_balance_loss, moe_balance_loss_backward: what the gate's losses take from the ids
// and the logits, sequence by sequence, and the logits' gradient.
//
// balance[b] = E / sum(c) * mean_s sum_e c_e P[s, e] needs no mean of P: the counts are known before the
// logits are read, so each token's sum over its experts stays in its lanes, and the tokens' sums are
// added up in chunks of kTokens.  A chunk's tokens of one sequence give one partial sum, at place (chunk +
// sequence): along the tokens one of the two grows with each new partial sum, so no place is taken twice.
#include <type_traits>

#include "lanes.hpp"
#include "vectors.hpp"

namespace moe {

constexpr int kBalThreads = 256;
constexpr int kBalMaxE = 1024;
constexpr int kTokens = 16;          // tokens per chunk
constexpr int kCountTokens = 2048;   // tokens per workgroup of the counts

struct Sequences {
  const int32_t *cu;  // NULL: one of all T tokens
  int n, T;
};

// The sequence of token t: -1 before the first one, n behind the last.  Whatever cu holds, a sequence b in
// [0, n) has cu[b] <= t < cu[b + 1].
__device__ inline int sequence_of(const Sequences &s, int t) {
  if (!s.cu) return 0;
  if (t < s.cu[0]) return -1;
  if (t >= s.cu[s.n]) return s.n;
  int lo = 0, hi = s.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Tokens [first, last) of sequence b, within [0, T].
__device__ inline int first_token(const Sequences &s, int b) { return s.cu ? min(max(s.cu[b], 0), s.T) : 0; }
__device__ inline int last_token(const Sequences &s, int b) { return s.cu ? min(max(s.cu[b + 1], 0), s.T) : s.T; }

// ---- counts ------------------------------------------------------------------------------------

__global__ __launch_bounds__(kBalThreads) void k_count_zero(int32_t *__restrict__ counts, long long n) {
  for (long long i = (long long)blockIdx.x * kBalThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kBalThreads)
    counts[i] = 0;
}

// Adds the ids of kCountTokens tokens, sequence by sequence, in LDS and then to counts (whole numbers: their
// order changes nothing).
__global__ __launch_bounds__(kBalThreads) void k_expert_counts(const int32_t *__restrict__ idx, Sequences s, int E,
                                                              int K, int32_t *__restrict__ counts) {
  __shared__ int32_t bins[kBalMaxE];
  int t = (int)min((long long)blockIdx.x * kCountTokens, (long long)s.T);
  const int end = (int)min((long long)t + kCountTokens, (long long)s.T);
  while (t < end) {
    const int b = sequence_of(s, t);
    if (b >= s.n) break;
    const int stop = !s.cu ? end : min(end, b < 0 ? s.cu[0] : s.cu[b + 1]);  // above t
    if (b >= 0) {
      for (int e = threadIdx.x; e < E; e += kBalThreads) bins[e] = 0;
      __syncthreads();
      for (long long i = (long long)t * K + threadIdx.x; i < (long long)stop * K; i += kBalThreads) {
        const int e = idx[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&bins[e], 1);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < E; e += kBalThreads)
        if (bins[e]) atomicAdd(&counts[(long long)b * E + e], bins[e]);
      __syncthreads();
    }
    t = stop;
  }
}

// ---- rows of logits ----------------------------------------------------------------------------

// Group i of lane l of a token's L lanes: 4 experts from 4 (l + L i) on; -inf behind the last expert.
template <bool BF16>
__device__ inline f32x4 experts_4(const void *p, long long row, int E, int e) {
  const float ninf = -__builtin_inff();
  f32x4 v = {ninf, ninf, ninf, ninf};
  const long long i = row * E + e;
  const int n = E - e;
  if (n >= 4) {
    if constexpr (BF16) {
      uint2 q;
      __builtin_memcpy(&q, (const uint16_t *)p + i, 8);
      v = (f32x4){bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
    } else {
      __builtin_memcpy(&v, (const float *)p + i, 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) v[j] = load_logit<BF16>(p, i + j);
  }
  return v;
}

// Largest value of a token's lanes; a NaN passes by (it comes back through the sums).
template <int L>
__device__ inline float lanes_max(float m) {
  const uint32_t k = token_max<L>(m == -__builtin_inff() ? 0u : order_key(m));
  return k ? key_value(k) : -__builtin_inff();
}

// A token's logits as numerators of its probabilities: p over sp for the balance loss, and the maximum m and sum sz
// of exp(x - m) for the z loss.  With softmax scores the two are one.
template <int L, int G, bool SIGMOID>
struct TokenRow {
  f32x4 x[G], p[G];
  float m, sp, sz;
  template <bool BF16>
  __device__ inline void read(const void *logits, long long t, int E, int l, bool z) {
    const float ninf = -__builtin_inff();
    m = ninf;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      x[i] = experts_4<BF16>(logits, t, E, 4 * (l + L * i));
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, x[i][j]);
    }
    m = lanes_max<L>(m);
    sp = sz = 0.0f;
    const float base = fminf(m, 0.0f);
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = x[i][j];
        if (SIGMOID) {
          p[i][j] = logistic_over(v, base);
          if (z) sz += v == ninf ? 0.0f : expf(v - m);
        } else {
          p[i][j] = v == ninf ? 0.0f : expf(v - m);
        }
        sp += p[i][j];
      }
    sp = token_sum<L>(sp);
    sz = SIGMOID ? (z ? token_sum<L>(sz) : 0.0f) : sp;
  }
  // log of the sum of exp(logits); 0 where all are -inf
  __device__ inline float lse() const { return sz == 0.0f ? 0.0f : m + logf(sz); }
};

// Counts of sequence b as this lane's experts have them; 0 behind the last expert.
template <int L, int G>
__device__ inline void read_counts(const int32_t *counts, int b, int E, int l, f32x4 (&c)[G]) {
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * (l + L * i) + j;
      c[i][j] = e < E ? (float)counts[(long long)b * E + e] : 0.0f;
    }
}

// A workgroup per chunk of tokens: parts[chunk + sequence] = sums of sum_e c_e P_e and of lse^2.
template <int L, int V, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kBalThreads) void k_balance_rows(const void *__restrict__ logits, Sequences s,
                                                             const int32_t *__restrict__ counts, int E, bool z,
                                                             float2 *__restrict__ parts) {
  constexpr int G = V / 4, GROUPS = kBalThreads / L;
  __shared__ float2 sum_of[kTokens];
  __shared__ int seq_of[kTokens];
  const int l = threadIdx.x % L;
  for (int i = threadIdx.x / L; i < kTokens; i += GROUPS) {
    const long long t = (long long)blockIdx.x * kTokens + i;
    const int b = t < s.T ? sequence_of(s, (int)t) : s.n;
    float2 v = {0.0f, 0.0f};
    if (b >= 0 && b < s.n) {
      TokenRow<L, G, SIGMOID> r;
      r.template read<BF16>(logits, t, E, l, z);
      f32x4 c[G];
      read_counts<L, G>(counts, b, E, l, c);
      float d = 0.0f;
#pragma unroll
      for (int q = 0; q < G; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) d += c[q][j] * r.p[q][j];
      d = token_sum<L>(d);
      v.x = r.sp == 0.0f ? 0.0f : d / r.sp;
      v.y = r.lse() * r.lse();
    }
    if (l == 0) sum_of[i] = v, seq_of[i] = b;
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i >= kTokens) return;
  const int b = seq_of[i];
  if (b < 0 || b >= s.n || (i > 0 && seq_of[i - 1] == b)) return;
  float2 v = {0.0f, 0.0f};
  for (int k = i; k < kTokens && seq_of[k] == b; ++k) v.x += sum_of[k].x, v.y += sum_of[k].y;
  parts[(long long)blockIdx.x + b] = v;
}

// Sum of one value per thread, the same in every thread, in a fixed order.
__device__ inline double block_total(double v) {
  __shared__ double part[kBalThreads / kWave];
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < kBalThreads / kWave; ++w) sum += part[w];
  return sum;
}

// A workgroup per sequence: its partial sums added up, in 64 bits (there may be millions of tokens).
__global__ __launch_bounds__(kBalThreads) void k_balance_total(const float2 *__restrict__ parts, Sequences s,
                                                              const int32_t *__restrict__ counts, int E,
                                                              float *__restrict__ balance, float *__restrict__ zloss) {
  const int b = blockIdx.x, lo = first_token(s, b), hi = last_token(s, b);
  double d = 0.0, z = 0.0, c = 0.0;
  if (lo < hi) {
    for (int i = lo / kTokens + threadIdx.x; i <= (hi - 1) / kTokens; i += kBalThreads) {
      const float2 v = parts[(long long)i + b];
      d += v.x, z += v.y;
    }
    for (int e = threadIdx.x; e < E; e += kBalThreads) c += counts[(long long)b * E + e];
  }
  d = block_total(d);
  z = block_total(z);
  c = block_total(c);
  if (threadIdx.x == 0) {
    const double n = max(hi - lo, 1);
    balance[b] = c > 0.0 ? (float)(d * E / (c * n)) : 0.0f;
    if (zloss) zloss[b] = (float)(z / n);
  }
}

// dlogits of a token, with f_e = E c_e / sum(c) and D = sum_e f_e P_e:
//   dbalance / n * P_e (f_e - D) [* (1 - logistic(x_e))]  +  2 dzloss / n * lse * softmax_e
template <int L, int V, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kBalThreads) void k_balance_bwd(const void *__restrict__ logits, Sequences s,
                                                            const int32_t *__restrict__ counts, int E,
                                                            const float *__restrict__ dbalance,
                                                            const float *__restrict__ dzloss, const void *add,
                                                            void *dlogits) {
  constexpr int G = V / 4, GROUPS = kBalThreads / L;
  const int l = threadIdx.x % L;
  const float ninf = -__builtin_inff();
  for (long long t = (long long)blockIdx.x * GROUPS + threadIdx.x / L; t < s.T; t += (long long)gridDim.x * GROUPS) {
    const int b = sequence_of(s, (int)t);
    if (b < 0 || b >= s.n) continue;
    TokenRow<L, G, SIGMOID> r;
    r.template read<BF16>(logits, t, E, l, dzloss != nullptr);
    f32x4 c[G];
    read_counts<L, G>(counts, b, E, l, c);
    float d = 0.0f, total = 0.0f;
#pragma unroll
    for (int q = 0; q < G; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) d += c[q][j] * r.p[q][j], total += c[q][j];
    d = token_sum<L>(d);
    total = token_sum<L>(total);
    const float n = (float)max(last_token(s, b) - first_token(s, b), 1);
    const float rs = r.sp == 0.0f ? 0.0f : 1.0f / r.sp;
    const float db = dbalance && total > 0.0f ? dbalance[b] / n * ((float)E / total) * rs : 0.0f;
    const float dz = dzloss && r.sz != 0.0f ? 2.0f * dzloss[b] / n * r.lse() / r.sz : 0.0f;
    d *= rs;
#pragma unroll
    for (int q = 0; q < G; ++q) {
      const int e = 4 * (l + L * q);
      if (e >= E) continue;
      f32x4 g;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = r.x[q][j];
        g[j] = db * r.p[q][j] * (c[q][j] - d);
        if (SIGMOID) {
          g[j] = x == ninf ? 0.0f : g[j] / (1.0f + expf(x));
          if (dzloss) g[j] += x == ninf ? 0.0f : dz * expf(x - r.m);
        } else {
          g[j] += dz * r.p[q][j];
        }
      }
      if (add) {
        const f32x4 a = experts_4<BF16>(add, t, E, e);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] += a[j];
      }
      const long long at = t * E + e;
      if (e + 4 <= E) {
        if constexpr (BF16) {
          const uint2 o = {pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
          __builtin_memcpy((uint16_t *)dlogits + at, &o, 8);
        } else {
          __builtin_memcpy((float *)dlogits + at, &g, 16);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (e + j >= E) continue;
          if constexpr (BF16)
            ((uint16_t *)dlogits)[at + j] = (uint16_t)pack_bf16x2(g[j], 0.0f);
          else
            ((float *)dlogits)[at + j] = g[j];
        }
      }
    }
  }
}

// Calls f with the lanes a token and the experts a lane.
template <class F>
static void with_lanes(int E, F f) {
  using std::integral_constant;
#define MOE_LANES(l, v) f(integral_constant<int, l>{}, integral_constant<int, v>{})
  if (E <= 64) MOE_LANES(16, 4);
  else if (E <= 128) MOE_LANES(16, 8);
  else if (E <= 256) MOE_LANES(16, 16);
  else if (E <= 512) MOE_LANES(32, 16);
  else MOE_LANES(64, 16);
#undef MOE_LANES
}

static bool sequences_ok(int64_t T, int32_t E, int32_t n_seq, const int32_t *cu) {
  return T >= 0 && T < (1LL << 31) && E >= 1 && E <= kBalMaxE && n_seq >= 1 && n_seq <= (1 << 20) &&
         (cu || n_seq == 1) && (uintptr_t)cu % 4 == 0;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_expert_counts(int64_t T, int32_t E, int32_t K, const int32_t *topk_idx,
                                          int32_t n_seq, const int32_t *cu_tokens, int32_t *counts,
                                          hipStream_t stream) {
  if (!sequences_ok(T, E, n_seq, cu_tokens) || K < 1 || K > E || T * K >= (1LL << 31)) return MOE_EINVAL;
  if (!counts || (T && !topk_idx) || ((uintptr_t)counts | (uintptr_t)topk_idx) % 4) return MOE_EINVAL;
  const size_t c_bytes = (size_t)n_seq * E * 4;
  if (shares(counts, c_bytes, topk_idx, (size_t)T * K * 4, false) ||
      shares(counts, c_bytes, cu_tokens, ((size_t)n_seq + 1) * 4, false))
    return MOE_EINVAL;
  const Sequences s{cu_tokens, n_seq, (int)T};
  const int64_t n = (int64_t)n_seq * E, fill = (n + kBalThreads - 1) / kBalThreads;
  hipLaunchKernelGGL(k_count_zero, dim3((unsigned)(fill < 4096 ? fill : 4096)), dim3(kBalThreads), 0, stream, counts, n);
  if (T)
    hipLaunchKernelGGL(k_expert_counts, dim3(ceil_div(T, kCountTokens)), dim3(kBalThreads), 0, stream, topk_idx, s, E, K,
                       counts);
  return launch_status();
}

extern "C" size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t n_seq) {
  if (T < 0 || T >= (1LL << 31) || n_seq < 1) return 0;
  return ((size_t)ceil_div(T, kTokens) + n_seq) * sizeof(float2);
}

extern "C" moe_status_t moe_balance_loss(moe_dtype dtype, moe_score score, int64_t T, int32_t E,
                                         const void *logits, int32_t n_seq, const int32_t *cu_tokens,
                                         const int32_t *counts, float *balance, float *zloss, void *ws,
                                         size_t ws_bytes, hipStream_t stream) {
  if ((dtype != MOE_BF16 && dtype != MOE_F32) || !sequences_ok(T, E, n_seq, cu_tokens)) return MOE_EINVAL;
  if (score != MOE_SCORE_SOFTMAX_TOPK && score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if ((T && !logits) || !counts || !balance || !ws || (uintptr_t)ws % 8) return MOE_EINVAL;
  const size_t size = dtype == MOE_BF16 ? 2 : 4, need = moe_balance_loss_workspace_bytes(T, n_seq);
  if ((uintptr_t)logits % size || ((uintptr_t)counts | (uintptr_t)balance | (uintptr_t)zloss) % 4) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_ENOSPACE;
  const size_t o_bytes = (size_t)n_seq * 4;
  const Range in[] = {{logits, (size_t)T * E * size}, {counts, o_bytes * E},
                      {cu_tokens, o_bytes + 4}, {ws, need}, {zloss, o_bytes}};
  if (!stands_alone(balance, o_bytes, in, 5) || !stands_alone(zloss, o_bytes, in, 4) || !stands_alone(ws, need, in, 3))
    return MOE_EINVAL;
  const Sequences s{cu_tokens, n_seq, (int)T};
  float2 *parts = (float2 *)ws;
  auto go = [&](auto bf16, auto sigmoid) {
    with_lanes(E, [&](auto l, auto v) {
      hipLaunchKernelGGL((k_balance_rows<l.value, v.value, bf16.value, sigmoid.value>), dim3(ceil_div(T, kTokens)),
                         dim3(kBalThreads), 0, stream, logits, s, counts, E, zloss != nullptr, parts);
    });
  };
  auto scores = [&](auto bf16) { score == MOE_SCORE_SIGMOID ? go(bf16, std::true_type{}) : go(bf16, std::false_type{}); };
  if (T) dtype == MOE_BF16 ? scores(std::true_type{}) : scores(std::false_type{});
  hipLaunchKernelGGL(k_balance_total, dim3(n_seq), dim3(kBalThreads), 0, stream, (const float2 *)parts, s, counts, E,
                     balance, zloss);
  return launch_status();
}

extern "C" moe_status_t moe_balance_loss_backward(moe_dtype dtype, moe_score score, int64_t T, int32_t E,
                                                  const void *logits, int32_t n_seq,
                                                  const int32_t *cu_tokens, const int32_t *counts,
                                                  const float *dbalance, const float *dzloss,
                                                  const void *add, void *dlogits, hipStream_t stream) {
  if ((dtype != MOE_BF16 && dtype != MOE_F32) || !sequences_ok(T, E, n_seq, cu_tokens)) return MOE_EINVAL;
  if (score != MOE_SCORE_SOFTMAX_TOPK && score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !dlogits) return MOE_EINVAL;
  const size_t size = dtype == MOE_BF16 ? 2 : 4, bytes = (size_t)T * E * size, o_bytes = (size_t)n_seq * 4;
  if (((uintptr_t)logits | (uintptr_t)add | (uintptr_t)dlogits) % size ||
      ((uintptr_t)counts | (uintptr_t)dbalance | (uintptr_t)dzloss) % 4)
    return MOE_EINVAL;
  const Range in[] = {{add, bytes, true}, {logits, bytes}, {counts, o_bytes * E},
                      {cu_tokens, o_bytes + 4}, {dbalance, o_bytes}, {dzloss, o_bytes}};
  if (!stands_alone(dlogits, bytes, in, 6, true)) return MOE_EINVAL;
  const Sequences s{cu_tokens, n_seq, (int)T};
  auto go = [&](auto bf16, auto sigmoid) {
    with_lanes(E, [&](auto l, auto v) {
      const int64_t groups = kBalThreads / l.value, blocks = (T + groups - 1) / groups;
      hipLaunchKernelGGL((k_balance_bwd<l.value, v.value, bf16.value, sigmoid.value>),
                         dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(kBalThreads), 0, stream, logits, s,
                         counts, E, dbalance, dzloss, add, dlogits);
    });
  };
  auto scores = [&](auto bf16) { score == MOE_SCORE_SIGMOID ? go(bf16, std::true_type{}) : go(bf16, std::false_type{}); };
  dtype == MOE_BF16 ? scores(std::true_type{}) : scores(std::false_type{});
  return launch_status();
}
