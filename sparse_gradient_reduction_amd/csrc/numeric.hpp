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

// 16 bytes of consecutive elements, at any element's border (the memory path
// takes unaligned 16-byte accesses; whole 16-byte borders are the fast case).
template <class T>
struct Pack {
  static constexpr int N = 16 / sizeof(T);
  typedef T V __attribute__((ext_vector_type(N)));
  typedef V U __attribute__((aligned(sizeof(T))));
};

// `n` elements from p on, at most Pack<T>::N; 0 where there are none.
template <class T>
__device__ __forceinline__ typename Pack<T>::V load_pack(const T* p, int64_t n) {
  typename Pack<T>::V v = {};
  if (n >= Pack<T>::N) {
    v = *reinterpret_cast<const typename Pack<T>::U*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < Pack<T>::N - 1; ++e)
      if (e < n) v[e] = p[e];
  }
  return v;
}
template <class T>
__device__ __forceinline__ void store_pack(typename Pack<T>::V v, T* p, int64_t n) {
  if (n >= Pack<T>::N) {
    *reinterpret_cast<typename Pack<T>::U*>(p) = v;
  } else {
#pragma unroll
    for (int e = 0; e < Pack<T>::N - 1; ++e)
      if (e < n) p[e] = v[e];
  }
}

// v plus its value in the lane that a DPP control names.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over aligned groups of L lanes (8, 16, 32 or 64), the same in every lane
// of the group; the lanes of a group are all active.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);  // row_half_mirror: the other quad of 8
  if (L >= 16) v = dpp_add<0x140>(v);  // row_mirror: the other half of 16
  if (L == 32) v += __shfl_xor(v, 16, kWave);
  if (L == 64) {
    v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0)) +
        __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16)) +
        (__int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32)) +
         __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48)));
  }
  return v;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// Sum over a workgroup of NT threads, the same in every thread and in the same
// order whatever the launch. `scratch` holds NT / 64 values. Contains barriers:
// all threads call it.
template <int NT>
__device__ __forceinline__ float block_sum_f32(float v, float* scratch) {
  constexpr int NW = NT / kWave;
  v = lanes_sum<kWave>(v);
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
