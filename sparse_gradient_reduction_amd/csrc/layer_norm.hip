// Layer norm over rows, forward and backward, with the reduction of the
// weight's and the bias's gradients over the rows of each node.
//
//   forward   v = x, or round(x + residual) (returned as `total`)
//             mean = sum v / D, rstd = 1 / sqrt(sum (v - mean)^2 / D + eps)
//             y = (v - mean) * rstd * weight + bias
//   backward  h = (x - mean) * rstd, g = dy * weight
//             dx = rstd * (g - sum g / D - h * sum(g h) / D) [+ dresidual]
//             dweight_p = sum of dy * h, dbias_p = sum of dy over node p's rows
//
// All sums and statistics are fp32; inputs and outputs of 16 bits are rounded
// once, at the store.
#include <algorithm>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ float normed_value(const T* x, const T* r, uint32_t i) {
  const float v = to_f32(x[i]);
  return r ? to_f32(from_f32<T>(v + to_f32(r[i]))) : v;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_layer_norm(uint64_t rows, uint32_t cols, const T* x, uint64_t x_stride,
                                                         const T* residual, uint64_t r_stride, const float* weight,
                                                         const float* bias, float eps, T* y, T* total, float* mean,
                                                         float* rstd) {
  __shared__ float scratch[kThreads / kWave];
  for (uint64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * x_stride;
    const T* rr = residual ? residual + row * r_stride : nullptr;
    float s = 0.0f;
    for (uint32_t i = threadIdx.x; i < cols; i += kThreads) s += normed_value(xr, rr, i);
    const float mu = block_sum_f32<kThreads>(s, scratch) / (float)cols;
    s = 0.0f;
    for (uint32_t i = threadIdx.x; i < cols; i += kThreads) {
      const float d = normed_value(xr, rr, i) - mu;
      s = fmaf(d, d, s);
    }
    const float var = block_sum_f32<kThreads>(s, scratch) / (float)cols;
    const float rs = 1.0f / sqrtf(var + eps);
    for (uint32_t i = threadIdx.x; i < cols; i += kThreads) {
      const float v = normed_value(xr, rr, i);
      if (total) total[row * cols + i] = from_f32<T>(v);
      y[row * cols + i] = from_f32<T>(fmaf((v - mu) * rs, weight ? weight[i] : 1.0f, bias ? bias[i] : 0.0f));
    }
    if (threadIdx.x == 0) {
      mean[row] = mu;
      rstd[row] = rs;
    }
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_layer_norm_dx(uint64_t rows, uint32_t cols, const T* dy,
                                                            uint64_t dy_stride, const T* x, uint64_t x_stride,
                                                            const T* dres, uint64_t dres_stride, const float* weight,
                                                            const float* mean, const float* rstd, T* dx) {
  __shared__ float scratch[kThreads / kWave];
  for (uint64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* gr = dy + row * dy_stride;
    const T* xr = x + row * x_stride;
    const float mu = mean[row], rs = rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (uint32_t i = threadIdx.x; i < cols; i += kThreads) {
      const float g = to_f32(gr[i]) * (weight ? weight[i] : 1.0f);
      s0 += g;
      s1 = fmaf(g, (to_f32(xr[i]) - mu) * rs, s1);
    }
    s0 = block_sum_f32<kThreads>(s0, scratch) / (float)cols;
    s1 = block_sum_f32<kThreads>(s1, scratch) / (float)cols;
    for (uint32_t i = threadIdx.x; i < cols; i += kThreads) {
      const float g = to_f32(gr[i]) * (weight ? weight[i] : 1.0f);
      const float h = (to_f32(xr[i]) - mu) * rs;
      float d = rs * (g - s0 - h * s1);
      if (dres) d += to_f32(dres[row * dres_stride + i]);
      dx[row * cols + i] = from_f32<T>(d);
    }
  }
}

// One thread per column of one node, down that node's rows.
template <class T>
__global__ __launch_bounds__(kThreads) void k_layer_norm_dw(uint64_t rows, uint32_t cols, const T* dy,
                                                            uint64_t dy_stride, const T* x, uint64_t x_stride,
                                                            const float* mean, const float* rstd, float* dweight,
                                                            uint64_t dw_stride, float* dbias, uint64_t db_stride) {
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x, p = blockIdx.y;
  if (c >= cols) return;
  float w = 0.0f, b = 0.0f;
  for (uint64_t row = p * rows; row < (p + 1) * rows; ++row) {
    const float g = to_f32(dy[row * dy_stride + c]);
    b += g;
    w = fmaf(g, (to_f32(x[row * x_stride + c]) - mean[row]) * rstd[row], w);
  }
  if (dweight) dweight[p * dw_stride + c] = w;
  if (dbias) dbias[p * db_stride + c] = b;
}

}  // namespace

hipError_t layer_norm_launch(uint32_t type, uint64_t rows, uint32_t cols, const void* x, uint64_t x_stride,
                             const void* residual, uint64_t r_stride, const float* weight, const float* bias,
                             float eps, void* y, void* total, float* mean, float* rstd, hipStream_t stream) {
  return for_type(type, [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL(k_layer_norm<T>, dim3((uint32_t)std::min<uint64_t>(rows, 1u << 16)), dim3(kThreads), 0, stream,
                       rows, cols, (const T*)x, x_stride, (const T*)residual, r_stride, weight, bias, eps, (T*)y,
                       (T*)total, mean, rstd);
    return hipGetLastError();
  });
}

size_t layer_norm_backward_workspace_bytes(uint32_t, uint64_t, uint32_t) { return 256; }

hipError_t layer_norm_backward_launch(uint32_t type, uint32_t nodes, uint64_t rows, uint32_t cols, const void* dy,
                                      uint64_t dy_stride, const void* x, uint64_t x_stride, const void* dresidual,
                                      uint64_t dres_stride, const float* weight, const float* mean, const float* rstd,
                                      void* dx, float* dweight, uint64_t dw_stride, float* dbias, uint64_t db_stride,
                                      void*, hipStream_t stream) {
  return for_type(type, [&](auto t) {
    using T = decltype(t);
    const uint64_t all = nodes * rows;
    if (all > 0) {
      hipLaunchKernelGGL(k_layer_norm_dx<T>, dim3((uint32_t)std::min<uint64_t>(all, 1u << 16)), dim3(kThreads), 0,
                         stream, all, cols, (const T*)dy, dy_stride, (const T*)x, x_stride, (const T*)dresidual,
                         dres_stride, weight, mean, rstd, (T*)dx);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_layer_norm_dw<T>, dim3((cols + kThreads - 1) / kThreads, nodes), dim3(kThreads), 0, stream,
                       rows, cols, (const T*)dy, dy_stride, (const T*)x, x_stride, mean, rstd, dweight, dw_stride,
                       dbias, db_stride);
    return hipGetLastError();
  });
}

}  // namespace sparcml
