// Momentum from a reduction's result, sparse pairs or dense, as the device
// record says: m = mu * m + scale * g, and the update m, or scale * g + mu * m
// with Nesterov.
#include <algorithm>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kTile = 4096;  // positions of one workgroup

// First j in [0, n) with idx[j] >= at, n if there is none.
__device__ __forceinline__ uint64_t lower_bound(const uint32_t* idx, uint64_t n, uint64_t at) {
  uint64_t lo = 0;
  while (lo < n) {
    const uint64_t mid = (lo + n) / 2;
    if (idx[mid] < at) lo = mid + 1;
    else n = mid;
  }
  return lo;
}

template <class U>
__global__ __launch_bounds__(kThreads) void k_momentum(uint64_t N, const ReduceResultDev* result, const uint32_t* idx,
                                                       uint64_t idx_cap, const float* val, float* m, float mu,
                                                       float scale, uint32_t nesterov, U* update) {
  __shared__ float g[kTile];
  const uint64_t begin = (uint64_t)blockIdx.x * kTile, end = min(begin + kTile, N);
  const bool dense = result->is_dense != 0;
  if (!dense) {
    const uint64_t K = min((uint64_t)result->nnz, min(idx_cap, N));
    for (uint32_t i = threadIdx.x; i < kTile; i += kThreads) g[i] = 0.0f;
    const uint64_t j0 = lower_bound(idx, K, begin), j1 = lower_bound(idx, K, end);
    __syncthreads();
    for (uint64_t j = j0 + threadIdx.x; j < j1; j += kThreads) {
      const uint64_t i = idx[j];
      if (i >= begin && i < end) g[i - begin] = val[j];
    }
    __syncthreads();
  }
  for (uint64_t i = begin + threadIdx.x; i < end; i += kThreads) {
    const float s = (dense ? val[i] : g[i - begin]) * scale;
    const float v = fmaf(mu, m[i], s);
    m[i] = v;
    if (update) update[i] = from_f32<U>(nesterov ? fmaf(mu, v, s) : v);
  }
}

}  // namespace

hipError_t momentum_launch(uint64_t N, const ReduceResultDev* result, const uint32_t* idx, uint64_t idx_cap,
                           const float* val, float* momentum, float mu, float scale, bool nesterov,
                           uint32_t update_type, void* update, hipStream_t stream) {
  return for_type(update_type, [&](auto t) {
    using U = decltype(t);
    hipLaunchKernelGGL(k_momentum<U>, dim3((uint32_t)((N + kTile - 1) / kTile)), dim3(kThreads), 0, stream, N, result,
                       idx, idx_cap, val, momentum, mu, scale, nesterov ? 1u : 0u, (U*)update);
    return hipGetLastError();
  });
}

}  // namespace sparcml
