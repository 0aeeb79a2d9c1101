// moe_expert_counts, moe_balance_loss, moe_balance_loss_backward: what the gate's losses take from the ids
// and the logits, sequence by sequence, and the logits' gradient.
//
// balance[b] = E / sum(c) * mean_s sum_e c_e P[s, e] needs no mean of P: the counts are known before the
// logits are read, so each token's sum over its experts stays in its lanes, and the tokens' sums are
// added up in chunks of tokens.  A chunk's tokens of one sequence give one partial sum, at place (chunk +
// sequence): along the tokens one of the two grows with each new partial sum, so no place is taken twice.
//
// Latency-bound at usual sizes, by the exponentials at many tokens and by HBM at many experts; calls in a graph over three
// sets of inputs, us:
//   tokens x experts, sequences      counts (K = 8)   losses   gradient (added to the router's)
//   64 x 64 fp32, 1 (K = 6)           4.4              4.8      4.3
//   8192 x 384 fp32, 4                5.3              10.7     11.6
//   32768 x 256 bf16 logistic, 61     9.1              16.1     17.9   (17 MB and 50 MB move in 3 and 8.5)
//   32768 x 256 bf16 softmax, 61      9.4              14.1     14.6
//   65536 x 1024 fp32, 16             8.5              59.5     162    (4.5 and 5.0 TB/s)
//   65536 x 64 bf16, 128 (K = 6)      11.5             14.1     13.1   (in one sequence 8.9, 11.4, 10.9)
//   65536 x 64 bf16, 4096 (K = 6)     68               21.8     16.7   (bins cleared and flushed for each piece of a sequence)
#include <type_traits>

#include "lanes.hpp"
#include "vectors.hpp"

namespace moe {

constexpr int kBalThreads = 256;
constexpr int kBalMaxE = 1024;
constexpr int kMinTokens = 4, kMaxTokens = 256;  // tokens per chunk

struct Sequences {
  const int32_t *cu;  // NULL: one of all T tokens
  int n, T;
};

// The sequences that hold tokens first and last, by one wave: -1 before the first one, n behind the last.  Whatever cu
// holds, a sequence b in [0, n) that comes out has cu[b] <= t < cu[b + 1].  Each step looks at 64 bounds.
__device__ inline int2 sequences_of(const Sequences &s, int first, int last) {
  if (!s.cu) return {0, 0};
  const int lane = threadIdx.x & 63;
  int lo[2] = {0, 0}, hi[2] = {s.n, s.n}, t[2] = {first, last};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    // cu[lo] <= t < cu[hi] from the first step on
    bool open = true;
    int step = (s.n + kWave - 1) / kWave;
    while (open) {
      const int i = min(lo[k] + lane * step, hi[k]);
      const unsigned long long at = __ballot(s.cu[i] <= t[k]);
      if (at == 0) {
        lo[k] = -1;
        break;
      }
      const int l = 63 - __clzll(at), from = __shfl(i, l, kWave);
      if (from == s.n || (hi[k] == s.n && s.cu[s.n] <= t[k])) {
        lo[k] = s.n;
        break;
      }
      hi[k] = min(from + step, hi[k]);
      lo[k] = from;
      open = step > 1;
      step = (hi[k] - lo[k] + kWave - 1) / kWave;
    }
    if (k == 0 && first == last) return {lo[0], lo[0]};
  }
  return {lo[0], lo[1]};
}

// The sequence of token t, which lies between two tokens of sequences lo and hi (as sequences_of gives them).
__device__ inline int sequence_between(const Sequences &s, int t, int2 at) {
  int lo = at.x, hi = at.y;
  if (lo == hi) return lo;
  if (lo < 0) {
    if (t < s.cu[0]) return -1;
    lo = 0;
  }
  if (hi >= s.n) {
    if (t >= s.cu[s.n]) return s.n;
    hi = s.n - 1;
  }
  ++hi;  // cu[lo] <= t < cu[hi]
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

constexpr int kCountThreads = 1024;
constexpr int kCountCopies = 4;      // of the bins, lanes taking turns: a popular expert's ids meet in one place less often
constexpr int kCountIds = 2048;      // about as many ids a workgroup
constexpr int kCountAlone = 32768;   // ids of a sequence that one workgroup counts by itself
constexpr int kCountAlonePeak = 65536;

struct Bins {
  int32_t n[kCountCopies][kBalMaxE + 8];
  __device__ inline void clear(int E) {
    for (int e = threadIdx.x; e < E; e += kCountThreads)
#pragma unroll
      for (int c = 0; c < kCountCopies; ++c) n[c][e] = 0;
  }
  // ids [from, to) of idx
  __device__ inline void add(const int32_t *__restrict__ idx, int from, int to, int E) {
    int32_t *mine = n[threadIdx.x % kCountCopies];
    for (unsigned i = from + 4 * threadIdx.x; i < (unsigned)to; i += 4 * kCountThreads) {
      int id[4];
      if (to - i >= 4)
        __builtin_memcpy(id, idx + i, 16);
      else
        for (int j = 0; j < 4; ++j) id[j] = i + j < (unsigned)to ? idx[i + j] : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((unsigned)id[j] < (unsigned)E) atomicAdd(&mine[id[j]], 1);
    }
  }
  __device__ inline int32_t of(int e) const {
    int32_t v = 0;
#pragma unroll
    for (int c = 0; c < kCountCopies; ++c) v += n[c][e];
    return v;
  }
};

// A workgroup per sequence.
__global__ __launch_bounds__(kCountThreads) void k_count_sequences(const int32_t *__restrict__ idx, Sequences s, int E,
                                                                  int K, int32_t *__restrict__ counts) {
  __shared__ Bins bins;
  const int b = blockIdx.x, lo = first_token(s, b), hi = max(last_token(s, b), lo);
  bins.clear(E);
  __syncthreads();
  bins.add(idx, lo * K, hi * K, E);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kCountThreads) counts[(long long)b * E + e] = bins.of(e);
}

__global__ __launch_bounds__(kCountThreads) void k_count_zero(int32_t *__restrict__ counts, long long n) {
  for (long long i = (long long)blockIdx.x * kCountThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kCountThreads)
    counts[i] = 0;
}

// Adds the ids of `tokens` tokens, sequence by sequence (whole numbers: the order of the additions changes nothing).
__global__ __launch_bounds__(kCountThreads) void k_count_chunks(const int32_t *__restrict__ idx, Sequences s, int E, int K,
                                                               int tokens, int32_t *__restrict__ counts) {
  __shared__ Bins bins;
  int t = (int)min((long long)blockIdx.x * tokens, (long long)s.T);
  const int end = (int)min((long long)t + tokens, (long long)s.T);
  while (t < end) {
    const int b = sequences_of(s, t, t).x;
    if (b >= s.n) break;
    const int stop = !s.cu ? end : min(end, b < 0 ? s.cu[0] : s.cu[b + 1]);  // above t
    if (b >= 0) {
      bins.clear(E);
      __syncthreads();
      bins.add(idx, t * K, stop * K, E);
      __syncthreads();
      for (int e = threadIdx.x; e < E; e += kCountThreads) {
        const int32_t v = bins.of(e);
        if (v) atomicAdd(&counts[(long long)b * E + e], v);
      }
      __syncthreads();
    }
    t = stop;
  }
}

// ---- rows of logits ----------------------------------------------------------------------------

constexpr float kLog2e = 1.44269504f;

// exp(d): the argument is rounded in the product with log2(e), below 2^-126 the result is 0.
__device__ inline float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// Four logits as they lie in memory, -inf behind the last expert.
template <bool BF16>
struct Raw4;

template <>
struct Raw4<true> {
  uint2 t;
  __device__ inline void load(const void *p, long long i, int n) {
    const uint16_t *q = (const uint16_t *)p + i;
    if (n >= 4) {
      __builtin_memcpy(&t, q, 8);
    } else {
      t.x = (n > 0 ? q[0] : 0xFF80u) | (n > 1 ? (uint32_t)q[1] : 0xFF80u) << 16;
      t.y = (n > 2 ? q[2] : 0xFF80u) | 0xFF800000u;
    }
  }
  __device__ inline f32x4 values() const { return (f32x4){bf16_lo(t.x), bf16_hi(t.x), bf16_lo(t.y), bf16_hi(t.y)}; }
};

template <>
struct Raw4<false> {
  f32x4 t;
  __device__ inline void load(const void *p, long long i, int n) {
    const float *q = (const float *)p + i;
    if (n >= 4) {
      __builtin_memcpy(&t, q, 16);
    } else {
      const float ninf = -__builtin_inff();
      t = (f32x4){n > 0 ? q[0] : ninf, n > 1 ? q[1] : ninf, n > 2 ? q[2] : ninf, ninf};
    }
  }
  __device__ inline f32x4 values() const { return t; }
};

// Token t's row in the registers of its L lanes: group i of lane l holds the 4 experts from 4 (l + L i) on.
template <int L, int G, bool BF16>
__device__ inline void read_row(const void *logits, long long t, int E, int l, Raw4<BF16> (&x)[G]) {
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int e = 4 * (l + L * i);
    x[i].load(logits, t * E + e, E - e);
  }
}

// Largest value of a token's lanes; a NaN passes by (it comes back through the sums).  0 where all are -inf, so that
// no difference of infinities arises.
template <int L>
__device__ inline float lanes_max(float m) {
  const uint32_t k = token_max<L>(m == -__builtin_inff() ? 0u : order_key(m));
  return k ? key_value(k) : 0.0f;
}

// A token's logits as numerators of its probabilities: p over sp for the balance loss, z over sz (exp(x - m)) for the
// z loss.  With softmax scores the two are one.  The logistic is 1 / (1 + t) or t / (1 + t) with t = exp(-|x|).  Where all
// logits are below 0, t is exp(x - m) exp(m) and p is left over exp(m): only a logit's distance from the largest one goes
// through an exponential that tells the experts apart.  With exp(-|x|) alone the rounded argument cost P up to 1.3e-6 of itself
// at -40 and 2.6e-6 at -60, and below -87 t is 0; exp(m) is the same for all of them, and its error reaches P only through 1 + t.
template <int L, int G, bool SIGMOID, bool Z>
struct TokenRow {
  f32x4 p[G], z[SIGMOID && Z ? G : 1], rest[SIGMOID ? G : 1];  // rest: 1 - logistic
  float m, sp, sz;
  template <bool BF16>
  __device__ inline void work(const Raw4<BF16> (&raw)[G]) {
    f32x4 x[G];
#pragma unroll
    for (int i = 0; i < G; ++i) x[i] = raw[i].values();
    m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, x[i][j]);
    m = lanes_max<L>(m);
    sp = sz = 0.0f;
    const float low = fminf(m, 0.0f), scale = exp_of(low);
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = x[i][j];
        if constexpr (SIGMOID) {
          const float t = exp_of(-fabsf(v) - low), r = __builtin_amdgcn_rcpf(fmaf(t, scale, 1.0f)), tr = t * r;
          p[i][j] = v >= 0.0f ? r : tr;  // a v above 0 has scale 1
          rest[i][j] = v >= 0.0f ? tr : r;
          if constexpr (Z) sz += z[i][j] = exp_of(v - m);
        } else {
          p[i][j] = exp_of(v - m);
        }
        sp += p[i][j];
      }
    sp = token_sum<L>(sp);
    sz = !SIGMOID ? sp : Z ? token_sum<L>(sz) : 0.0f;
  }
  __device__ inline float znum(int i, int j) const {
    if constexpr (SIGMOID && Z) return z[i][j];
    return p[i][j];
  }
  // log of the sum of exp(logits); 0 where all are -inf
  __device__ inline float lse() const { return sz == 0.0f ? 0.0f : m + logf(sz); }
};

// Counts of sequence b as this lane's experts have them; 0 behind the last expert.
template <int L, int G>
__device__ inline void read_counts(const int32_t *counts, int b, int E, int l, f32x4 (&c)[G]) {
  const int32_t *of = counts + (long long)b * E;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int e = 4 * (l + L * i);
    int v[4] = {0, 0, 0, 0};
    if (e + 4 <= E)
      __builtin_memcpy(v, of + e, 16);
    else
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < E) v[j] = of[e + j];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = (float)v[j];
  }
}

// sum_e c_e P_e of a token (E / sum(c) is left out) and its lse^2, in all its lanes.
template <int L, int G, bool BF16, bool SIGMOID, bool Z>
__device__ inline float2 token_losses(const Raw4<BF16> (&x)[G], const f32x4 (&c)[G]) {
  TokenRow<L, G, SIGMOID, Z> r;
  r.work(x);
  float d = 0.0f;
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) d = fmaf(c[q][j], r.p[q][j], d);
  d = token_sum<L>(d);
  const float lse = Z ? r.lse() : 0.0f;
  return {r.sp == 0.0f ? 0.0f : d * __builtin_amdgcn_rcpf(r.sp), lse * lse};
}

// A workgroup per chunk of `tokens` tokens: parts[chunk + sequence] = sums of what token_losses gives.  Where the chunk
// lies in one sequence, the counts stay in registers and a group adds up its tokens' by itself.
template <int L, int V, bool BF16, bool SIGMOID, bool Z>
__global__ __launch_bounds__(kBalThreads) void k_balance_rows(const void *__restrict__ logits, Sequences s,
                                                             const int32_t *__restrict__ counts, int E, int tokens,
                                                             float2 *__restrict__ parts) {
  constexpr int G = V / 4, GROUPS = kBalThreads / L;
  __shared__ float2 sum_of[kMaxTokens];
  __shared__ int seq_of[kMaxTokens];
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int t0 = blockIdx.x * tokens, tn = min(tokens, s.T - t0);
  Raw4<BF16> x[G];
  if (group < tn) read_row<L, G, BF16>(logits, t0 + group, E, l, x);
  const int2 at = sequences_of(s, t0, t0 + tn - 1);
  f32x4 c[G];
  if (at.x == at.y) {
    const int b = at.x;
    if (b < 0 || b >= s.n) return;
    read_counts<L, G>(counts, b, E, l, c);
    float2 v = {0.0f, 0.0f};
    for (int i = group; i < tn; i += GROUPS) {
      Raw4<BF16> now[G];
#pragma unroll
      for (int q = 0; q < G; ++q) now[q] = x[q];
      if (i + GROUPS < tn) read_row<L, G, BF16>(logits, t0 + i + GROUPS, E, l, x);
      const float2 one = token_losses<L, G, BF16, SIGMOID, Z>(now, c);
      v.x += one.x, v.y += one.y;
    }
    if (l == 0) sum_of[group] = v;
    __syncthreads();
    if (threadIdx.x) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) v.x += sum_of[g].x, v.y += sum_of[g].y;
    parts[(long long)blockIdx.x + b] = v;
    return;
  }
  for (int i = group; i < tn; i += GROUPS) {
    const int b = sequence_between(s, t0 + i, at);
    float2 v = {0.0f, 0.0f};
    if (b >= 0 && b < s.n) {
      read_row<L, G, BF16>(logits, t0 + i, E, l, x);
      read_counts<L, G>(counts, b, E, l, c);
      v = token_losses<L, G, BF16, SIGMOID, Z>(x, c);
    }
    if (l == 0) sum_of[i] = v, seq_of[i] = b;
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i >= tn) return;
  const int b = seq_of[i];
  if (b < 0 || b >= s.n || (i > 0 && seq_of[i - 1] == b)) return;
  double d = 0.0, z = 0.0;
  for (int k = i; k < tn && seq_of[k] == b; ++k) d += sum_of[k].x, z += sum_of[k].y;
  parts[(long long)blockIdx.x + b] = {(float)d, (float)z};
}

// Sum of one value over a wave, the same in every lane, in a fixed order.
__device__ inline double wave_total(double v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// The losses of sequence b of n tokens: d and z summed over its tokens, c over its counts.
__device__ inline void write_losses(int b, int n, int E, double d, double z, double c, float *balance, float *zloss) {
  balance[b] = c > 0.0 ? (float)(d * E / (c * max(n, 1))) : 0.0f;
  if (zloss) zloss[b] = (float)(z / max(n, 1));
}

// A workgroup per sequence: its partial sums added up, in 64 bits (there may be millions of tokens).
__global__ __launch_bounds__(kBalThreads) void k_balance_total(const float2 *__restrict__ parts, Sequences s, int tokens,
                                                              const int32_t *__restrict__ counts, int E,
                                                              float *__restrict__ balance, float *__restrict__ zloss) {
  __shared__ double part[3][kBalThreads / kWave];
  const int b = blockIdx.x, lo = first_token(s, b), hi = last_token(s, b);
  double v[3] = {0.0, 0.0, 0.0};
  if (lo < hi) {
    const int last = (hi - 1) / tokens;
    for (int i0 = lo / tokens + threadIdx.x; i0 <= last; i0 += 8 * kBalThreads) {
      float2 t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = i0 + k * kBalThreads <= last ? parts[(long long)i0 + k * kBalThreads + b] : float2{0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[0] += t[k].x, v[1] += t[k].y;
    }
    for (int e = threadIdx.x; e < E; e += kBalThreads) v[2] += counts[(long long)b * E + e];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = wave_total(v[k]);
    if ((threadIdx.x & 63) == 0) part[k][threadIdx.x >> 6] = v[k];
  }
  __syncthreads();
  if (threadIdx.x) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = 0.0;
    for (int w = 0; w < kBalThreads / kWave; ++w) v[k] += part[k][w];
  }
  write_losses(b, hi - lo, E, v[0], v[1], v[2], balance, zloss);
}

// Few tokens: one workgroup for all of it.
constexpr int kAloneThreads = 1024;
constexpr int kAlonePasses = 3;  // tokens a group of lanes (1.5 us each, where the second launch costs 2 and the host 2.7)
constexpr int kAloneTokens = kAlonePasses * kAloneThreads / 16, kAloneSequences = 64;
template <int L, int V, bool BF16, bool SIGMOID, bool Z>
__global__ __launch_bounds__(kAloneThreads) void k_balance_alone(const void *__restrict__ logits, Sequences s,
                                                                const int32_t *__restrict__ counts, int E,
                                                                float *__restrict__ balance, float *__restrict__ zloss) {
  constexpr int GROUPS = kAloneThreads / L;
  __shared__ float2 sum_of[kAloneTokens];
  const int l = threadIdx.x % L;
  const int2 at = sequences_of(s, 0, max(s.T - 1, 0));
  for (int t = threadIdx.x / L; t < s.T; t += GROUPS) {
    const int b = sequence_between(s, t, at);
    if (b < 0 || b >= s.n) continue;
    Raw4<BF16> x[V / 4];
    f32x4 c[V / 4];
    read_row<L, V / 4, BF16>(logits, t, E, l, x);
    read_counts<L, V / 4>(counts, b, E, l, c);
    const float2 v = token_losses<L, V / 4, BF16, SIGMOID, Z>(x, c);
    if (l == 0) sum_of[t] = v;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  for (int b = threadIdx.x >> 6; b < s.n; b += kAloneThreads / kWave) {
    const int lo = first_token(s, b), hi = last_token(s, b);
    double d = 0.0, z = 0.0, c = 0.0;
    for (int t = lo + lane; t < hi; t += kWave) d += sum_of[t].x, z += sum_of[t].y;
    if (lo < hi)
      for (int e = lane; e < E; e += kWave) c += counts[(long long)b * E + e];
    d = wave_total(d), z = wave_total(z), c = wave_total(c);
    if (lane == 0) write_losses(b, hi - lo, E, d, z, c, balance, zloss);
  }
}

// What a sequence brings to its tokens' gradients: its counts and their sum, dbalance / n E / sum(c), 2 dzloss / n.
template <int L, int G, bool Z>
struct SequenceGrad {
  f32x4 c[G];
  float kb, kz;
  __device__ inline void read(const Sequences &s, const int32_t *counts, int b, int E, int l, const float *dbalance,
                              const float *dzloss) {
    read_counts<L, G>(counts, b, E, l, c);
    const float n = (float)max(last_token(s, b) - first_token(s, b), 1);
    const float db = dbalance ? dbalance[b] : 0.0f;
    kz = Z ? 2.0f * dzloss[b] / n : 0.0f;
    float total = 0.0f;
#pragma unroll
    for (int q = 0; q < G; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) total += c[q][j];
    total = token_sum<L>(total);
    kb = total > 0.0f ? db / n * ((float)E / total) : 0.0f;
  }
};

// dlogits of a token, with f_e = E c_e / sum(c) and D = sum_e f_e P_e:
//   dbalance / n * P_e (f_e - D) [* (1 - logistic(x_e))]  +  2 dzloss / n * lse * softmax_e
template <int L, int G, bool BF16, bool SIGMOID, bool Z>
__device__ inline void token_grad(const Raw4<BF16> (&x)[G], const Raw4<BF16> (&a)[G], bool add,
                                  const SequenceGrad<L, G, Z> &s, void *dlogits, long long t, int E, int l) {
  TokenRow<L, G, SIGMOID, Z> r;
  r.work(x);
  float d = 0.0f;
#pragma unroll
  for (int q = 0; q < G; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) d = fmaf(s.c[q][j], r.p[q][j], d);
  const float rs = r.sp == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(r.sp);
  d = token_sum<L>(d) * rs;
  const float kb = s.kb * rs, kz = Z && r.sz != 0.0f ? s.kz * r.lse() * __builtin_amdgcn_rcpf(r.sz) : 0.0f;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int e = 4 * (l + L * q);
    if (e >= E) continue;
    f32x4 g;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (SIGMOID) {
        g[j] = kb * r.p[q][j] * (s.c[q][j] - d) * r.rest[q][j];
        if (Z) g[j] = fmaf(kz, r.znum(q, j), g[j]);
      } else {
        g[j] = r.p[q][j] * fmaf(kb, s.c[q][j] - d, kz);
      }
    }
    if (add) g += a[q].values();
    const long long o = t * E + e;
    if (e + 4 <= E) {
      if constexpr (BF16) {
        const uint2 w = {pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
        __builtin_memcpy((uint16_t *)dlogits + o, &w, 8);
      } else {
        __builtin_memcpy((float *)dlogits + o, &g, 16);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e + j >= E) continue;
        if constexpr (BF16)
          ((uint16_t *)dlogits)[o + j] = (uint16_t)pack_bf16x2(g[j], 0.0f);
        else
          ((float *)dlogits)[o + j] = g[j];
      }
    }
  }
}

// A workgroup per chunk of tokens, as in k_balance_rows.
template <int L, int V, bool BF16, bool SIGMOID, bool Z>
__global__ __launch_bounds__(kBalThreads) void k_balance_bwd(const void *__restrict__ logits, Sequences s,
                                                            const int32_t *__restrict__ counts, int E, int tokens,
                                                            const float *__restrict__ dbalance,
                                                            const float *__restrict__ dzloss, const void *add,
                                                            void *dlogits) {
  constexpr int G = V / 4, GROUPS = kBalThreads / L;
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int t0 = blockIdx.x * tokens, tn = min(tokens, s.T - t0);
  Raw4<BF16> x[G], a[G];
  auto fetch = [&](int i) {
    read_row<L, G, BF16>(logits, t0 + i, E, l, x);
    if (add) read_row<L, G, BF16>(add, t0 + i, E, l, a);
  };
  if (group < tn) fetch(group);
  const int2 at = sequences_of(s, t0, t0 + tn - 1);
  SequenceGrad<L, G, Z> of;
  if (at.x == at.y) {
    if (at.x < 0 || at.x >= s.n) return;
    of.read(s, counts, at.x, E, l, dbalance, dzloss);
    for (int i = group; i < tn; i += GROUPS) {
      Raw4<BF16> now[G], plus[G];
#pragma unroll
      for (int q = 0; q < G; ++q) now[q] = x[q], plus[q] = a[q];
      if (i + GROUPS < tn) fetch(i + GROUPS);
      token_grad<L, G, BF16, SIGMOID, Z>(now, plus, add != nullptr, of, dlogits, t0 + i, E, l);
    }
    return;
  }
  for (int i = group; i < tn; i += GROUPS) {
    const int b = sequence_between(s, t0 + i, at);
    if (b < 0 || b >= s.n) continue;
    fetch(i);
    of.read(s, counts, b, E, l, dbalance, dzloss);
    token_grad<L, G, BF16, SIGMOID, Z>(x, a, add != nullptr, of, dlogits, t0 + i, E, l);
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

// Calls f with the type, the score and whether there is a z loss.
template <class F>
static void with_kind(moe_dtype dtype, moe_score score, bool z, F f) {
  using std::bool_constant;
  auto third = [&](auto bf16, auto sigmoid) { z ? f(bf16, sigmoid, std::true_type{}) : f(bf16, sigmoid, std::false_type{}); };
  auto second = [&](auto bf16) { score == MOE_SCORE_SIGMOID ? third(bf16, std::true_type{}) : third(bf16, std::false_type{}); };
  dtype == MOE_BF16 ? second(std::true_type{}) : second(std::false_type{});
}

// Tokens per chunk: one for each group of lanes until the chip is full of workgroups.
constexpr int kChunksPerCu = 8;
static int chunk_tokens(int64_t T, int lanes) {
  const int groups = kBalThreads / lanes;
  const int64_t n = T / ((int64_t)groups * kChunksPerCu * device_cu_count()) * groups;
  return (int)(n < groups ? groups : n > kMaxTokens ? kMaxTokens : n);
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
  if (T * K <= (int64_t)kCountAlone * n_seq && T * K <= kCountAlonePeak) {
    hipLaunchKernelGGL(k_count_sequences, dim3(n_seq), dim3(kCountThreads), 0, stream, topk_idx, s, E, K, counts);
    return launch_status();
  }
  const int64_t n = (int64_t)n_seq * E, fill = (n + kCountThreads - 1) / kCountThreads;
  hipLaunchKernelGGL(k_count_zero, dim3((unsigned)(fill < 4096 ? fill : 4096)), dim3(kCountThreads), 0, stream, counts, n);
  const int tokens = kCountIds / K < 1 ? 1 : kCountIds / K;
  hipLaunchKernelGGL(k_count_chunks, dim3(ceil_div(T, tokens)), dim3(kCountThreads), 0, stream, topk_idx, s, E, K, tokens,
                     counts);
  return launch_status();
}

extern "C" size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t n_seq) {
  if (T < 0 || T >= (1LL << 31) || n_seq < 1) return 0;
  return ((size_t)ceil_div(T, kMinTokens) + n_seq) * sizeof(float2);
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
  bool alone = false;
  int tokens = kMinTokens;
  if (T)
    with_kind(dtype, score, zloss != nullptr, [&](auto bf16, auto sigmoid, auto z) {
      with_lanes(E, [&](auto l, auto v) {
        tokens = chunk_tokens(T, l.value);
        alone = T <= kAlonePasses * kAloneThreads / l.value && n_seq <= kAloneSequences;
        if (alone)
          hipLaunchKernelGGL((k_balance_alone<l.value, v.value, bf16.value, sigmoid.value, z.value>), dim3(1),
                             dim3(kAloneThreads), 0, stream, logits, s, counts, E, balance, zloss);
        else
          hipLaunchKernelGGL((k_balance_rows<l.value, v.value, bf16.value, sigmoid.value, z.value>), dim3(ceil_div(T, tokens)),
                             dim3(kBalThreads), 0, stream, logits, s, counts, E, tokens, parts);
      });
    });
  if (!alone)
    hipLaunchKernelGGL(k_balance_total, dim3(n_seq), dim3(kBalThreads), 0, stream, (const float2 *)parts, s, tokens, counts, E,
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
  with_kind(dtype, score, dzloss != nullptr, [&](auto bf16, auto sigmoid, auto z) {
    with_lanes(E, [&](auto l, auto v) {
      const int tokens = chunk_tokens(T, l.value);
      hipLaunchKernelGGL((k_balance_bwd<l.value, v.value, bf16.value, sigmoid.value, z.value>), dim3(ceil_div(T, tokens)),
                         dim3(kBalThreads), 0, stream, logits, s, counts, E, tokens, dbalance, dzloss, add, dlogits);
    });
  });
  return launch_status();
}
