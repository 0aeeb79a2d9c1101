// moe_dropout: out = residual + drop(x).  Streams its tensors once: HBM-bound.  8192 x 7168 bf16 with residual (352 MB) take
// 54 to 59 us, 6.0 to 6.5 TB/s, where torch's copy moves 5.1; without residual 41 to 43, where the ten rounds for 8 elements
// take about half of the arithmetic's time; 6 x 1408 2.5 us.
#include <type_traits>

#include "dropout.hpp"

namespace moe {

constexpr int kDropThreads = 256;
constexpr int64_t kDropMaxGrid = 1 << 22;

// A run of 8 a thread.  (Walking the runs with the next one's loads under way was slower: 8192 x 7168 bf16 with residual
// 55.4 us, with 2 workgroups per CU that walk 55.8, with 4 57.6, with 8 60.0.)
template <bool BF16, bool RES, bool DROP, bool STREAM>
__global__ __launch_bounds__(kDropThreads) void k_dropout(const void *x, const void *residual, void *out,
                                                         long long n, Drop d) {
  DropKey key{};
  if (DROP) key = drop_key(d);
  const long long step = (long long)gridDim.x * kDropThreads;
  for (long long b = (long long)blockIdx.x * kDropThreads + threadIdx.x; 8 * b < n; b += step) {
    const int m = (int)min(8LL, n - 8 * b);
    const long long bytes = bytes_of<BF16>(8 * b);
    float v[8], r[8] = {};
    if (m == 8) {
      Raw<BF16> xs, rs;
      xs.template load<STREAM>(row_at(x, bytes), 0);
      if (RES) rs.template load<STREAM>(row_at(residual, bytes), 0);
      xs.values(v);
      if (RES) rs.values(r);
    } else {
      load_8<BF16>(x, 8 * b, m, v);
      if (RES) load_8<BF16>(residual, 8 * b, m, r);
    }
    if constexpr (DROP) {
      const u32x4 bits = philox((unsigned long long)b, key);
      if constexpr (RES) drop_8(bits, d, v, r); else drop_8(bits, d, v);
    } else if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    if (m == 8)
      Raw<BF16>(v).template store<STREAM>(row_at(out, bytes), 0);
    else
      store_8<BF16>(out, 8 * b, m, v);
  }
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
  const dim3 grid((unsigned)(blocks < kDropMaxGrid ? blocks : kDropMaxGrid));
  auto go = [&](auto bf16, auto res, auto drop, auto st) {
    hipLaunchKernelGGL((k_dropout<bf16.value, res.value, drop.value, st.value>), grid, dim3(kDropThreads), 0, stream, x,
                       residual, out, n, d);
  };
  const int64_t moved = (int64_t)bytes * (residual ? 3 : 2);
  using std::false_type;
  using std::true_type;
  auto third = [&](auto b, auto r, auto k) { moved >= kStreamBytes ? go(b, r, k, true_type{}) : go(b, r, k, false_type{}); };
  auto second = [&](auto b, auto r) { d.below ? third(b, r, true_type{}) : third(b, r, false_type{}); };
  auto first = [&](auto b) { residual ? second(b, true_type{}) : second(b, false_type{}); };
  dtype == MOE_BF16 ? first(true_type{}) : first(false_type{});
  return launch_status();
}
