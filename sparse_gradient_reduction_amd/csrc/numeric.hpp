// Element types of the dense operators (fp32, bf16, fp16) and fp32 / fp64
// sums over waves and workgroups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "sparcml.h"

namespace sparcml {

typedef __bf16 bf16;
typedef _Float16 f16;

// Every value of a 16-bit type is an fp32 value; the way back rounds to
// nearest even, once.
template <class T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}
template <class T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}

// N elements of T that move as one load or store.
template <class T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// Sum over the 64 lanes of a wave, the same in every lane and in the same
// order whatever the launch.
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// Sum over a workgroup of NT threads, the same in every thread. `scratch`
// holds NT / 64 values. Contains barriers: all threads call it.
template <int NT>
__device__ __forceinline__ float block_sum_f32(float v, float* scratch) {
  constexpr int NW = NT / kWave;
  v = wave_sum_f32(v);
  if (NW == 1) return v;
  if (lane_id() == 0) scratch[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += scratch[w];
  __syncthreads();
  return s;
}
template <int NT>
__device__ __forceinline__ double block_sum_f64(double v, double* scratch) {
  constexpr int NW = NT / kWave;
  v = wave_sum_f64(v);
  if (NW == 1) return v;
  if (lane_id() == 0) scratch[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += scratch[w];
  __syncthreads();
  return s;
}

// Calls f with a value of the type that `type` names (SPARCML_F32, _BF16 or
// _F16); the caller has checked that it is one of them.
template <class F>
hipError_t for_type(uint32_t type, F&& f) {
  switch (type) {
    case SPARCML_BF16: return f(bf16{});
    case SPARCML_F16: return f(f16{});
    default: return f(float{});
  }
}

}  // namespace sparcml
