// moe_grad_sumsq, moe_grad_clip: the sum of squares over many gradient tensors, and the
// gradients scaled to a largest norm.  Both only stream the tensors: HBM-bound.  Two fp32
// tensors of 285 M values together (3.4 GB: two reads and a write) take 565 us, 6.1 TB/s, where the best
// copy reaches 5.9: part of the second read meets the memory-side cache (256 MB).  61 short ones (0.13 M
// values) take 8 us in three launches.
//
// The tensors' addresses travel as kernel arguments, kGradBatch tensors a launch; each is cut
// into chunks of kGradChunk elements.  Squares are summed in 64 bits: a square of a large
// fp32 value does not fit 32 bits, and the sum runs over billions of terms.
#include "common.hpp"

namespace moe {

constexpr int kGradBatch = 64;
constexpr int kGradThreads = 256;
constexpr int kGradChunk = 1 << 14;    // elements per chunk
constexpr int kGradParts = 2048;       // partial sums (and the sum kernel's largest grid)
// Chunks that one workgroup sums by itself, in one launch (us, one launch / two: 1 chunk 3.5 / 5.5, 2 5.0 / 5.6,
// 4 full ones 8.0 / 5.7; each launch is 2.7 more on the host)
constexpr int kGradAlone = 2;

struct GradBatch {
  const void *g[kGradBatch];
  void *o[kGradBatch];
  long long n[kGradBatch];
  int first[kGradBatch + 1];  // first chunk of each tensor
  uint8_t bf16[kGradBatch];
  int count;
};

// Tensor of chunk c.
__device__ inline int grad_tensor(const GradBatch &b, int c) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

// 16 bytes of a gradient as fp32 values: 4 of fp32, 8 of bf16.
template <bool BF16>
__device__ inline void widen(u32x4 t, float (&v)[8]) {
  const f32x4 f = __builtin_bit_cast(f32x4, t);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (BF16) {
      v[2 * q] = bf16_lo(t[q]);
      v[2 * q + 1] = bf16_hi(t[q]);
    } else {
      v[q] = f[q];
    }
  }
}

__device__ inline float grad_at(const void *g, bool bf16, long long i) {
  return bf16 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t *)g)[i] << 16) : ((const float *)g)[i];
}

// Sum of one value per thread, the same in every thread, in a fixed order.
template <int THREADS>
__device__ inline double block_sum(double v) {
  __shared__ double part[THREADS / kWave];
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) s += part[w];
  __syncthreads();
  return s;
}

constexpr int kGradFlight = 4;  // 16-byte loads a thread has in flight

// This thread's squares of one chunk whose address is a multiple of 16: whole vectors, then the rest.
template <bool BF16>
__device__ inline double chunk_squares(const char *g, int n, double s) {
  constexpr int V = BF16 ? 8 : 4;
  const u32x4 *p = (const u32x4 *)g;
  const int vecs = n / V;
  for (int i = threadIdx.x; i < vecs; i += kGradThreads * kGradFlight) {
    u32x4 t[kGradFlight];
#pragma unroll
    for (int u = 0; u < kGradFlight; ++u) {
      t[u] = (u32x4){0, 0, 0, 0};
      if (i + u * kGradThreads < vecs) t[u] = p[i + u * kGradThreads];
    }
#pragma unroll
    for (int u = 0; u < kGradFlight; ++u) {
      float v[8];
      widen<BF16>(t[u], v);
#pragma unroll
      for (int e = 0; e < V; ++e) s = fma((double)v[e], (double)v[e], s);
    }
  }
  for (int i = vecs * V + threadIdx.x; i < n; i += kGradThreads) {
    const double v = grad_at(g, BF16, i);
    s = fma(v, v, s);
  }
  return s;
}

// parts[blockIdx] += the squares of every gridDim-th chunk of the batch; the parts from `have`
// on are set instead (no earlier launch of the call wrote them).
__global__ __launch_bounds__(kGradThreads) void k_grad_sumsq(GradBatch b, double *__restrict__ parts,
                                                            int have) {
  double s = 0.0;
  for (int c = blockIdx.x; c < b.first[b.count]; c += gridDim.x) {
    const int t = grad_tensor(b, c);
    const long long i0 = (long long)(c - b.first[t]) * kGradChunk;
    const int n = (int)min((long long)kGradChunk, b.n[t] - i0);
    const bool bf = b.bf16[t];
    const char *g = (const char *)b.g[t] + i0 * (bf ? 2 : 4);
    if ((uintptr_t)g % 16 == 0) {
      s = bf ? chunk_squares<true>(g, n, s) : chunk_squares<false>(g, n, s);
    } else {
      for (int i = threadIdx.x; i < n; i += kGradThreads) {
        const double v = grad_at(g, bf, i);
        s = fma(v, v, s);
      }
    }
  }
  s = block_sum<kGradThreads>(s);
  if (threadIdx.x == 0) parts[blockIdx.x] = (int)blockIdx.x < have ? parts[blockIdx.x] + s : s;
}

constexpr int kGradSumThreads = 1024;
__global__ __launch_bounds__(kGradSumThreads) void k_grad_total(const double *__restrict__ parts, int n,
                                                               double *__restrict__ sumsq) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kGradSumThreads) s += parts[i];
  s = block_sum<kGradSumThreads>(s);
  if (threadIdx.x == 0) *sumsq = s;
}

// min(1, max_norm / (norm + 1e-6)); NaN for a NaN norm
__device__ inline float clip_coef(double sumsq, double max_norm) {
  const double c = max_norm / (sqrt(sumsq) + 1e-6);
  return c >= 1.0 ? 1.0f : (float)c;
}

template <bool BF16>
__device__ inline void chunk_scale(const char *g, char *o, int n, float coef) {
  constexpr int V = BF16 ? 8 : 4;
  const u32x4 *p = (const u32x4 *)g;
  u32x4 *d = (u32x4 *)o;
  const int vecs = n / V;
  for (int i = threadIdx.x; i < vecs; i += kGradThreads * kGradFlight) {
    u32x4 t[kGradFlight];
#pragma unroll
    for (int u = 0; u < kGradFlight; ++u)
      if (i + u * kGradThreads < vecs) t[u] = __builtin_nontemporal_load(p + i + u * kGradThreads);
#pragma unroll
    for (int u = 0; u < kGradFlight; ++u) {
      if (i + u * kGradThreads >= vecs) break;
      float v[8];
      widen<BF16>(t[u], v);
      u32x4 r;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        r[q] = BF16 ? pack_bf16x2(coef * v[2 * q], coef * v[2 * q + 1]) : __builtin_bit_cast(uint32_t, coef * v[q]);
      __builtin_nontemporal_store(r, d + i + u * kGradThreads);
    }
  }
  for (int i = vecs * V + threadIdx.x; i < n; i += kGradThreads) {
    const float v = coef * grad_at(g, BF16, i);
    if (BF16)
      ((uint16_t *)o)[i] = (uint16_t)pack_bf16x2(v, 0.0f);
    else
      ((float *)o)[i] = v;
  }
}

// Chunks from the last to the first: the sum read the last ones last, so they may still be cached.
__global__ __launch_bounds__(kGradThreads) void k_grad_clip(GradBatch b, const double *__restrict__ sumsq,
                                                           double max_norm, float *__restrict__ norm) {
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)sqrt(*sumsq);
  const float coef = clip_coef(*sumsq, max_norm);
  for (int c = b.first[b.count] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int t = grad_tensor(b, c);
    if (coef == 1.0f && b.g[t] == b.o[t]) continue;
    const long long i0 = (long long)(c - b.first[t]) * kGradChunk;
    const int n = (int)min((long long)kGradChunk, b.n[t] - i0);
    const bool bf = b.bf16[t];
    const char *g = (const char *)b.g[t] + i0 * (bf ? 2 : 4);
    char *o = (char *)b.o[t] + i0 * (bf ? 2 : 4);
    if (((uintptr_t)g | (uintptr_t)o) % 16 == 0) {
      bf ? chunk_scale<true>(g, o, n, coef) : chunk_scale<false>(g, o, n, coef);
    } else {
      for (int i = threadIdx.x; i < n; i += kGradThreads) {
        const float v = coef * grad_at(g, bf, i);
        if (bf)
          ((uint16_t *)o)[i] = (uint16_t)pack_bf16x2(v, 0.0f);
        else
          ((float *)o)[i] = v;
      }
    }
  }
}

// Fills the next batch from tensor `from` on (empty tensors are passed over) and returns the
// tensor after it; chunks of one launch stay below 2^31.
static int fill_batch(GradBatch *b, int from, int n, const void *const *g, void *const *o,
                      const int64_t *numel, const moe_dtype *dtype) {
  b->count = 0;
  b->first[0] = 0;
  int i = from;
  for (; i < n && b->count < kGradBatch; ++i) {
    if (numel[i] == 0) continue;
    const int64_t chunks = (numel[i] + kGradChunk - 1) / kGradChunk;
    if (b->first[b->count] + chunks >= (1LL << 31)) break;
    b->g[b->count] = g[i];
    b->o[b->count] = o ? o[i] : nullptr;
    b->n[b->count] = numel[i];
    b->bf16[b->count] = dtype[i] == MOE_BF16;
    b->first[b->count + 1] = (int)(b->first[b->count] + chunks);
    ++b->count;
  }
  return i;
}

static bool grads_ok(int n, const void *const *g, const int64_t *numel, const moe_dtype *dtype) {
  if (n < 0 || (n > 0 && (!g || !numel || !dtype))) return false;
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] >= (1LL << 40)) return false;
    if (dtype[i] != MOE_BF16 && dtype[i] != MOE_F32) return false;
    if (numel[i] > 0 && (!g[i] || (uintptr_t)g[i] % (dtype[i] == MOE_BF16 ? 2 : 4))) return false;
  }
  return true;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_grad_sumsq_workspace_bytes(void) { return kGradParts * sizeof(double); }

extern "C" moe_status_t moe_grad_sumsq(int32_t n, const void *const *grads, const int64_t *numel,
                                       const moe_dtype *dtype, double *sumsq, void *ws,
                                       size_t ws_bytes, hipStream_t stream) {
  if (!grads_ok(n, grads, numel, dtype) || !sumsq || !ws) return MOE_EINVAL;
  if ((uintptr_t)sumsq & 7 || (uintptr_t)ws & 7) return MOE_EINVAL;
  if (ws_bytes < moe_grad_sumsq_workspace_bytes()) return MOE_ENOSPACE;
  int parts = 0;
  GradBatch b;
  for (int at = 0; at < n;) {
    at = fill_batch(&b, at, n, grads, nullptr, numel, dtype);
    if (!b.count) break;
    if (parts == 0 && at == n && b.first[b.count] <= kGradAlone) {
      hipLaunchKernelGGL(k_grad_sumsq, dim3(1), dim3(kGradThreads), 0, stream, b, sumsq, 0);
      return launch_status();
    }
    const int grid = b.first[b.count] < kGradParts ? b.first[b.count] : kGradParts;
    hipLaunchKernelGGL(k_grad_sumsq, dim3(grid), dim3(kGradThreads), 0, stream, b, (double *)ws, parts);
    parts = grid > parts ? grid : parts;
  }
  hipLaunchKernelGGL(k_grad_total, dim3(1), dim3(kGradSumThreads), 0, stream, (const double *)ws, parts, sumsq);
  return launch_status();
}

extern "C" moe_status_t moe_grad_clip(int32_t n, const void *const *grads, const int64_t *numel,
                                      const moe_dtype *dtype, const double *sumsq, double max_norm,
                                      float *norm, void *const *outs, hipStream_t stream) {
  if (!grads_ok(n, grads, numel, dtype) || (n > 0 && !outs) || !sumsq) return MOE_EINVAL;
  if ((uintptr_t)sumsq & 7 || (uintptr_t)norm & 3 || !(max_norm >= 0.0)) return MOE_EINVAL;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0 && (!outs[i] || (uintptr_t)outs[i] % (dtype[i] == MOE_BF16 ? 2 : 4))) return MOE_EINVAL;
  GradBatch b;
  int at = 0;
  do {
    at = fill_batch(&b, at, n, grads, outs, numel, dtype);
    const int chunks = b.first[b.count];
    if (chunks || norm)
      hipLaunchKernelGGL(k_grad_clip, dim3(chunks < 1 ? 1 : chunks < (1 << 22) ? chunks : 1 << 22),
                         dim3(kGradThreads), 0, stream, b, sumsq, max_norm, norm);
    norm = nullptr;  // written by the first launch
  } while (at < n);
  return launch_status();
}
