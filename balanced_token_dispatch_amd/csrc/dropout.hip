// moe_dropout: out = residual + drop(x).  Streams its tensors once.
#include "dropout.hpp"

namespace moe {

constexpr int kDropThreads = 256;

template <bool BF16, bool RES, bool DROP>
__global__ __launch_bounds__(kDropThreads) void k_dropout(const void *x, const void *residual, void *out,
                                                         long long n, Drop d) {
  DropKey key{};
  if (DROP) key = drop_key(d);
  const long long step = (long long)gridDim.x * kDropThreads;
  for (long long b = (long long)blockIdx.x * kDropThreads + threadIdx.x; 8 * b < n; b += step) {
    const int m = (int)min(8LL, n - 8 * b);
    float v[8], r[8];
    load_8<BF16>(x, 8 * b, m, v);
    if (RES) load_8<BF16>(residual, 8 * b, m, r);
    if (DROP && RES) drop_8(philox((unsigned long long)b, key), d, v, r);
    if (DROP && !RES) drop_8(philox((unsigned long long)b, key), d, v);
    if (!DROP && RES)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    store_8<BF16>(out, 8 * b, m, v);
  }
}

template <bool BF16>
static void launch_dropout(dim3 grid, hipStream_t stream, const void *x, const void *residual, void *out,
                           long long n, const Drop &d) {
  auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(kDropThreads), 0, stream, x, residual, out, n, d); };
  if (residual)
    d.below ? go(k_dropout<BF16, true, true>) : go(k_dropout<BF16, true, false>);
  else
    d.below ? go(k_dropout<BF16, false, true>) : go(k_dropout<BF16, false, false>);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_dropout(moe_dtype dtype, int64_t n, const void *x, const void *residual,
                                    double p, const int64_t *rng, int64_t offset, void *out,
                                    hipStream_t stream) {
  if ((dtype != MOE_BF16 && dtype != MOE_F32) || n < 0 || n >= (1LL << 48) || !drop_ok(p, rng)) return MOE_EINVAL;
  if (n == 0) return MOE_OK;
  const size_t size = dtype == MOE_BF16 ? 2 : 4, bytes = (size_t)n * size;
  if (!x || !out || ((uintptr_t)x | (uintptr_t)residual | (uintptr_t)out) % size) return MOE_EINVAL;
  if (shares(out, bytes, x, bytes, true) || shares(out, bytes, residual, bytes, true) ||
      shares(out, bytes, rng, 16, false))
    return MOE_EINVAL;
  const Drop d = make_drop(p, rng, offset);
  const int64_t blocks = (n + 8 * kDropThreads - 1) / (8 * kDropThreads);
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : 1 << 22));
  dtype == MOE_BF16 ? launch_dropout<true>(grid, stream, x, residual, out, n, d)
                    : launch_dropout<false>(grid, stream, x, residual, out, n, d);
  return launch_status();
}
