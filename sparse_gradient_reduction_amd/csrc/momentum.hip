// Momentum from a reduction's result, sparse pairs or dense, as the device
// record says: m = mu * m + scale * g, and the update m, or scale * g + mu * m
// with Nesterov.
//
// Bound by memory: 8 bytes of momentum, the update's 2 or 4 and 4 (dense) or
// 8 per pair (sparse) of gradient for each position, all read and written
// once. A workgroup owns a tile of positions. It starts its momentum's loads,
// finds the tile's pairs (the indices ascend) while they are under way, turns
// the pairs into a dense tile in LDS and finishes the tile from there, so the
// sparse form needs no pass that clears or scatters in memory.
#include <algorithm>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

constexpr int kThreads = 256;

// First j in [0, n) with idx[j] >= at, n if there is none; the same in every
// lane of the wave. Each round reads 64 places that cut the range into 65
// parts: 5 rounds of one load for 2^27 pairs where halving takes 27.
__device__ __forceinline__ uint64_t wave_lower_bound(const uint32_t* idx, uint64_t n, uint64_t at) {
  uint64_t lo = 0;  // the answer is in [lo, n]
  while (lo < n) {
    const uint64_t len = n - lo, lane = lane_id();
    const uint64_t probe = lo + len * lane / kWave;  // lane 0: lo; ascending, < n
    // lanes whose probe lies below `at`: the answer is past the last of them, at most the next one's
    const uint32_t below = popc64(ballot(idx[probe] < at));
    if (below == 0) return lo;
    const uint64_t next = below < kWave ? lo + len * below / kWave : n;
    lo = lo + len * (below - 1) / kWave + 1;
    n = max(lo, next);  // of unsorted indices too
  }
  return lo;
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Q: groups of four positions of a thread. A wave's groups lie next to each other.
template <class U, int Q>
__global__ __launch_bounds__(kThreads) void k_momentum(uint64_t N, const ReduceResultDev* result, const uint32_t* idx,
                                                       uint64_t idx_cap, const float* val, float* m, float mu,
                                                       float scale, uint32_t nesterov, U* update) {
  constexpr uint32_t kTile = kThreads * Q * 4;
  typedef U U4 __attribute__((ext_vector_type(4)));
  typedef U4 U4u __attribute__((aligned(sizeof(U))));
  __shared__ f32x4 g[kTile / 4];
  __shared__ uint64_t range[2];
  const uint64_t begin = (uint64_t)blockIdx.x * kTile, end = min(begin + kTile, N);
  const bool whole = end - begin == kTile;
  const bool dense = result->is_dense != 0;
  f32x4 v[Q], s[Q];
  if (whole) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      v[q] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(m + begin) + q * kThreads + threadIdx.x);
  }
  if (dense) {
    if (whole) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        s[q] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(val + begin) + q * kThreads + threadIdx.x);
    }
  } else {
    const uint64_t K = min((uint64_t)result->nnz, min(idx_cap, N));
    const uint32_t wid = threadIdx.x / kWave;
    if (wid < 2) {
      const uint64_t at = wave_lower_bound(idx, K, wid == 0 ? begin : end);
      if (lane_id() == 0) range[wid] = at;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) g[q * kThreads + threadIdx.x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    const uint64_t j1 = range[1];
    for (uint64_t j = range[0] + threadIdx.x; j < j1; j += kThreads) {
      const uint64_t i = idx[j];
      if (i >= begin && i < end) reinterpret_cast<float*>(g)[i - begin] = val[j];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < Q; ++q) s[q] = g[q * kThreads + threadIdx.x];
  }
  if (whole) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      U4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float t = s[q][e] * scale;
        v[q][e] = fmaf(mu, v[q][e], t);
        u[e] = from_f32<U>(nesterov ? fmaf(mu, v[q][e], t) : v[q][e]);
      }
      const uint32_t at = q * kThreads + threadIdx.x;
      __builtin_nontemporal_store(v[q], reinterpret_cast<f32x4u*>(m + begin) + at);
      if (update) *(reinterpret_cast<U4u*>(update + begin) + at) = u;
    }
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t i = begin + (q * kThreads + threadIdx.x) * 4 + e;
        if (i < end) {
          const float t = (dense ? val[i] : s[q][e]) * scale, w = fmaf(mu, m[i], t);
          m[i] = w;
          if (update) update[i] = from_f32<U>(nesterov ? fmaf(mu, w, t) : w);
        }
      }
  }
}

}  // namespace

hipError_t momentum_launch(uint64_t N, const ReduceResultDev* result, const uint32_t* idx, uint64_t idx_cap,
                           const float* val, float* momentum, float mu, float scale, bool nesterov,
                           uint32_t update_type, void* update, hipStream_t stream) {
  return for_type(update_type, [&](auto t) {
    using U = decltype(t);
    // tiles of 4096 positions where they fill the chip several times, else of 1024
    if (N >= (1u << 22))
      hipLaunchKernelGGL((k_momentum<U, 4>), dim3((uint32_t)((N + 4095) / 4096)), dim3(kThreads), 0, stream, N,
                         result, idx, idx_cap, val, momentum, mu, scale, nesterov ? 1u : 0u, (U*)update);
    else
      hipLaunchKernelGGL((k_momentum<U, 1>), dim3((uint32_t)((N + 1023) / 1024)), dim3(kThreads), 0, stream, N,
                         result, idx, idx_cap, val, momentum, mu, scale, nesterov ? 1u : 0u, (U*)update);
    return hipGetLastError();
  });
}

}  // namespace sparcml
