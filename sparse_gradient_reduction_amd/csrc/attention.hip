// Attention forward and backward: plain kernels, one wave a query or a key.
//
//   s = scale q k^T over the keys seen, lse = log sum exp s, out = exp(s - lse) v
//   p = exp(s - lse), ds = p (dout v^T - sum dout out)
//   dv = p^T dout, dq = scale ds k, dk = scale ds^T q
#include <algorithm>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

typedef sparcml_attention_args Args;

// A sequence's own lengths, and the keys [first, last) that its query i sees.
struct Sequence {
  int n, m, before, after;
  __device__ __forceinline__ Sequence(const Args& a, uint32_t b) {
    n = a.queries, m = a.keys;
    if (a.q_lengths) n = (uint32_t)a.q_lengths[b] <= a.queries ? a.q_lengths[b] : a.q_lengths[b] < 0 ? 0 : n;
    if (a.k_lengths) m = (uint32_t)a.k_lengths[b] <= a.keys ? a.k_lengths[b] : a.k_lengths[b] < 0 ? 0 : m;
    before = min(a.before, 1u << 30), after = min(a.after, 1u << 30);
  }
  __device__ __forceinline__ int first(int i) const { return max(0, i + m - n - before); }
  __device__ __forceinline__ int last(int i) const { return min(m, i + m - n + after + 1); }
};

template <class T>
__device__ __forceinline__ T* row_of(const sparcml_heads& x, uint64_t b, uint64_t t, uint64_t h) {
  return static_cast<T*>(x.data) + b * x.batch + t * x.token + h * x.head;
}

template <class T>
__device__ __forceinline__ float dot(const T* a, const T* b, uint32_t dim) {
  float s = 0.0f;
  for (uint32_t e = 0; e < dim; ++e) s = fmaf(to_f32(a[e]), to_f32(b[e]), s);
  return s;
}

template <class T>
__global__ __launch_bounds__(kWave) void k_attention(Args a) {
  __shared__ float p[kWave];
  const uint32_t i = blockIdx.x % a.queries, bh = blockIdx.x / a.queries, h = bh % a.heads, b = bh / a.heads;
  const uint32_t g = h / (a.heads / a.groups), lane = threadIdx.x;
  const Sequence s(a, b);
  const T* q = row_of<T>(a.q, b, i, h);
  float top = -INFINITY, sum = 0.0f, o0 = 0.0f, o1 = 0.0f;
  const int end = (int)i < s.n ? s.last(i) : 0;
  for (int j0 = s.first(i); j0 < end; j0 += kWave) {
    const int j = j0 + lane;
    const float v = j < end ? dot(q, row_of<T>(a.k, b, j, g), a.dim) * a.scale : -INFINITY;
    const float now = fmaxf(top, wave_max(v)), keep = expf(top - now), e = expf(v - now);
    top = now;
    sum = sum * keep + lanes_sum<kWave>(e);
    o0 *= keep, o1 *= keep;
    __syncthreads();
    p[lane] = e;
    __syncthreads();
    for (int k = 0; k < min(kWave, end - j0); ++k) {
      const T* r = row_of<T>(a.v, b, j0 + k, g);
      if (lane < a.dim) o0 = fmaf(p[k], to_f32(r[lane]), o0);
      if (lane + kWave < a.dim) o1 = fmaf(p[k], to_f32(r[lane + kWave]), o1);
    }
  }
  T* out = row_of<T>(a.out, b, i, h);
  const float over = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (lane < a.dim) out[lane] = from_f32<T>(o0 * over);
  if (lane + kWave < a.dim) out[lane + kWave] = from_f32<T>(o1 * over);
  if (lane == 0) a.lse[(uint64_t)bh * a.queries + i] = top + logf(sum);
}

template <class T>
__global__ __launch_bounds__(kWave) void k_attention_dq(Args a) {
  __shared__ float p[kWave];
  const uint32_t i = blockIdx.x % a.queries, bh = blockIdx.x / a.queries, h = bh % a.heads, b = bh / a.heads;
  const uint32_t g = h / (a.heads / a.groups), lane = threadIdx.x;
  const Sequence s(a, b);
  const T *q = row_of<T>(a.q, b, i, h), *dout = row_of<T>(a.dout, b, i, h);
  float o0 = 0.0f, o1 = 0.0f;
  const int begin = s.first(i), end = (int)i < s.n ? s.last(i) : 0;
  if (begin < end) {
    const float lse = a.lse[(uint64_t)bh * a.queries + i], delta = dot(dout, row_of<T>(a.out, b, i, h), a.dim);
    for (int j0 = begin; j0 < end; j0 += kWave) {
      const int j = j0 + lane;
      float ds = 0.0f;
      if (j < end) {
        ds = expf(dot(q, row_of<T>(a.k, b, j, g), a.dim) * a.scale - lse);
        ds *= dot(dout, row_of<T>(a.v, b, j, g), a.dim) - delta;
      }
      __syncthreads();
      p[lane] = ds;
      __syncthreads();
      for (int k = 0; k < min(kWave, end - j0); ++k) {
        const T* r = row_of<T>(a.k, b, j0 + k, g);
        if (lane < a.dim) o0 = fmaf(p[k], to_f32(r[lane]), o0);
        if (lane + kWave < a.dim) o1 = fmaf(p[k], to_f32(r[lane + kWave]), o1);
      }
    }
  }
  T* out = row_of<T>(a.dq, b, i, h);
  if (lane < a.dim) out[lane] = from_f32<T>(o0 * a.scale);
  if (lane + kWave < a.dim) out[lane + kWave] = from_f32<T>(o1 * a.scale);
}

template <class T>
__global__ __launch_bounds__(kWave) void k_attention_dkv(Args a) {
  __shared__ float p[kWave], d[kWave];
  const uint32_t j = blockIdx.x % a.keys, bg = blockIdx.x / a.keys, g = bg % a.groups, b = bg / a.groups;
  const uint32_t each = a.heads / a.groups, lane = threadIdx.x;
  const Sequence s(a, b);
  const T *k = row_of<T>(a.k, b, j, g), *v = row_of<T>(a.v, b, j, g);
  float k0 = 0.0f, k1 = 0.0f, v0 = 0.0f, v1 = 0.0f;
  // the queries that see key j: j - after <= i + m - n <= j + before
  const int begin = max(0, (int)j - s.after - s.m + s.n);
  const int end = (int)j < s.m ? min(s.n, (int)j + s.before - s.m + s.n + 1) : 0;
  for (uint32_t h = g * each; h < (g + 1) * each; ++h) {
    for (int i0 = begin; i0 < end; i0 += kWave) {
      const int i = i0 + lane;
      float e = 0.0f, ds = 0.0f;
      if (i < end) {
        const T* dout = row_of<T>(a.dout, b, i, h);
        e = expf(dot(row_of<T>(a.q, b, i, h), k, a.dim) * a.scale - a.lse[((uint64_t)b * a.heads + h) * a.queries + i]);
        ds = e * (dot(dout, v, a.dim) - dot(dout, row_of<T>(a.out, b, i, h), a.dim));
      }
      __syncthreads();
      p[lane] = e;
      d[lane] = ds;
      __syncthreads();
      for (int r = 0; r < min(kWave, end - i0); ++r) {
        const T *q = row_of<T>(a.q, b, i0 + r, h), *dout = row_of<T>(a.dout, b, i0 + r, h);
        if (lane < a.dim) {
          k0 = fmaf(d[r], to_f32(q[lane]), k0);
          v0 = fmaf(p[r], to_f32(dout[lane]), v0);
        }
        if (lane + kWave < a.dim) {
          k1 = fmaf(d[r], to_f32(q[lane + kWave]), k1);
          v1 = fmaf(p[r], to_f32(dout[lane + kWave]), v1);
        }
      }
    }
  }
  T *dk = row_of<T>(a.dk, b, j, g), *dv = row_of<T>(a.dv, b, j, g);
  if (lane < a.dim) {
    dk[lane] = from_f32<T>(k0 * a.scale);
    dv[lane] = from_f32<T>(v0);
  }
  if (lane + kWave < a.dim) {
    dk[lane + kWave] = from_f32<T>(k1 * a.scale);
    dv[lane + kWave] = from_f32<T>(v1);
  }
}

}  // namespace

size_t attention_workspace_bytes(const Args&) { return 256; }

hipError_t attention_launch(const Args& a, void*, hipStream_t stream) {
  if (a.queries == 0) return hipSuccess;
  return for_type(a.type, [&](auto t) {
    hipLaunchKernelGGL(k_attention<decltype(t)>, dim3(a.batch * a.heads * a.queries), dim3(kWave), 0, stream, a);
    return hipGetLastError();
  });
}

size_t attention_backward_workspace_bytes(const Args&) { return 256; }

hipError_t attention_backward_launch(const Args& a, void*, hipStream_t stream) {
  return for_type(a.type, [&](auto t) {
    if (a.queries > 0)
      hipLaunchKernelGGL(k_attention_dq<decltype(t)>, dim3(a.batch * a.heads * a.queries), dim3(kWave), 0, stream, a);
    if (a.keys > 0)
      hipLaunchKernelGGL(k_attention_dkv<decltype(t)>, dim3(a.batch * a.groups * a.keys), dim3(kWave), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace sparcml
