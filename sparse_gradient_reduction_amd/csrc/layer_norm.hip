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
//
// Both are bound by memory. A row is read once, 16 bytes a lane, and stays in
// registers: L lanes hold it, E elements each, so that rows of up to 16384
// elements take one pass and the variance is that of the differences from the
// mean. Small rows share a wave (L = 8, 16, 32), rows past 1024 take a
// workgroup. A lane keeps the same columns for all the rows it walks, so the
// weight, the bias and the two gradients' sums stay in registers too: read from
// memory for every row, fp32 weight and bias alone would be twice a 16-bit
// row's bytes. Longer rows (past 16384) are read again for each pass.
#include <algorithm>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kBlocks = 2048;   // workgroups that walk the rows: 8 to a CU
constexpr int kBackRows = 8;         // waves of a backward workgroup whose rows take a wave or less
constexpr uint32_t kHeld = 16384;    // elements of the longest row that is held in registers

// A row held by L lanes, E elements each: packs of 16 bytes, neighbouring
// lanes next to each other. NT: threads of the workgroup.
template <class T, int L_, int E_, int NT_>
struct Held {
  static constexpr int L = L_, E = E_, NT = NT_, V = Pack<T>::N, P = E / V, R = NT / L;
  static __device__ __forceinline__ int lane() { return threadIdx.x % L; }
  static __device__ __forceinline__ int at(int p) { return (p * L + lane()) * V; }
};

// Sums of N values each over the L lanes that hold a row. Where that is more
// than a wave, `scratch` (N * NT / 64 words) must not be in use since the
// last barrier but one.
template <class H, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float* scratch) {
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = lanes_sum<(H::L < kWave ? H::L : kWave)>(s[k]);
  if constexpr (H::L > kWave) {
    constexpr int NW = H::NT / kWave;
    if (lane_id() == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) scratch[k * NW + threadIdx.x / kWave] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      s[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s[k] += scratch[k * NW + w];
    }
  }
}

template <class H>
__device__ __forceinline__ void load_vector(float (&v)[H::E], const float* p, uint32_t cols, float none) {
#pragma unroll
  for (int q = 0; q < H::P; ++q)
#pragma unroll
    for (int e = 0; e < H::V; ++e) {
      const uint32_t c = H::at(q) + e;
      v[q * H::V + e] = p && c < cols ? p[c] : none;
    }
}

template <class T, class H>
__global__ __launch_bounds__(H::NT) void k_layer_norm(uint64_t rows, uint32_t cols, const T* x, uint64_t x_stride,
                                                      const T* residual, uint64_t r_stride, const float* weight,
                                                      const float* bias, float eps, T* y, T* total, float* mean,
                                                      float* rstd) {
  __shared__ float scratch[2][H::NT / kWave];
  float w[H::E], b[H::E];
  load_vector<H>(w, weight, cols, 1.0f);
  load_vector<H>(b, bias, cols, 0.0f);
  const float over = 1.0f / (float)cols;
  for (uint64_t row = (uint64_t)blockIdx.x * H::R + threadIdx.x / H::L; row < rows;
       row += (uint64_t)gridDim.x * H::R) {
    float v[H::E];
    typename Pack<T>::V px[H::P], pr[H::P];
#pragma unroll
    for (int q = 0; q < H::P; ++q) px[q] = load_pack(x + row * x_stride + H::at(q), (int64_t)cols - H::at(q));
    if (residual) {
#pragma unroll
      for (int q = 0; q < H::P; ++q) pr[q] = load_pack(residual + row * r_stride + H::at(q), (int64_t)cols - H::at(q));
#pragma unroll
      for (int q = 0; q < H::P; ++q) {
#pragma unroll
        for (int e = 0; e < H::V; ++e) px[q][e] = from_f32<T>(to_f32((T)px[q][e]) + to_f32((T)pr[q][e]));
        store_pack(px[q], total + row * cols + H::at(q), (int64_t)cols - H::at(q));
      }
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int q = 0; q < H::P; ++q)
#pragma unroll
      for (int e = 0; e < H::V; ++e) s[0] += v[q * H::V + e] = to_f32((T)px[q][e]);
    row_sums<H>(s, scratch[0]);
    const float mu = s[0] * over;
    s[0] = 0.0f;
#pragma unroll
    for (int q = 0; q < H::P; ++q)
#pragma unroll
      for (int e = 0; e < H::V; ++e) {
        const float d = v[q * H::V + e] - mu;
        v[q * H::V + e] = d;
        s[0] = H::at(q) + e < cols ? fmaf(d, d, s[0]) : s[0];
      }
    row_sums<H>(s, scratch[1]);
    const float rs = 1.0f / sqrtf(fmaf(s[0], over, eps));
#pragma unroll
    for (int q = 0; q < H::P; ++q) {
      typename Pack<T>::V o;
#pragma unroll
      for (int e = 0; e < H::V; ++e)
        o[e] = from_f32<T>(fmaf(v[q * H::V + e] * rs, w[q * H::V + e], b[q * H::V + e]));
      store_pack(o, y + row * cols + H::at(q), (int64_t)cols - H::at(q));
    }
    if (H::lane() == 0) {
      mean[row] = mu;
      rstd[row] = rs;
    }
  }
}

// One workgroup: rows [c * each, (c + 1) * each) of node p, c and p from the
// workgroup's number. Writes dx and this chunk's sums of dy * h and dy, to the
// node's gradients where it is the only chunk, else to part [p][c][2][cols].
template <class T, class H>
__global__ __launch_bounds__(H::NT) void k_layer_norm_backward(uint64_t rows, uint32_t cols, uint32_t chunks,
                                                               uint64_t each, const T* dy, uint64_t dy_stride,
                                                               const T* x, uint64_t x_stride, const T* dres,
                                                               uint64_t dres_stride, const float* weight,
                                                               const float* mean, const float* rstd, T* dx,
                                                               float* dweight, uint64_t dw_stride, float* dbias,
                                                               uint64_t db_stride, float* part) {
  __shared__ float scratch[2][2 * H::NT / kWave];
  float w[H::E], sw[H::E] = {}, sb[H::E] = {};
  load_vector<H>(w, weight, cols, 1.0f);
  const float over = 1.0f / (float)cols;
  const uint32_t p = blockIdx.x / chunks, c = blockIdx.x % chunks;
  const uint64_t begin = min(c * each, rows), end = min(begin + each, rows);
  uint32_t turn = 0;
  for (uint64_t r = begin + threadIdx.x / H::L; r < end; r += H::R, turn ^= 1) {
    const uint64_t row = p * rows + r;
    typename Pack<T>::V pg[H::P], px[H::P], pr[H::P];
#pragma unroll
    for (int q = 0; q < H::P; ++q) {
      pg[q] = load_pack(dy + row * dy_stride + H::at(q), (int64_t)cols - H::at(q));
      px[q] = load_pack(x + row * x_stride + H::at(q), (int64_t)cols - H::at(q));
    }
    if (dres) {
#pragma unroll
      for (int q = 0; q < H::P; ++q) pr[q] = load_pack(dres + row * dres_stride + H::at(q), (int64_t)cols - H::at(q));
    }
    const float mu = mean[row], rs = rstd[row];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < H::P; ++q)
#pragma unroll
      for (int e = 0; e < H::V; ++e) {
        const int k = q * H::V + e;
        const float g0 = to_f32((T)pg[q][e]);  // 0 past the row's end, so these columns add nothing
        const float h = (to_f32((T)px[q][e]) - mu) * rs, g = g0 * w[k];
        s[0] += g;
        s[1] = fmaf(g, h, s[1]);
        sb[k] += g0;
        sw[k] = fmaf(g0, h, sw[k]);
      }
    row_sums<H>(s, scratch[turn]);
    const float s0 = s[0] * over, s1 = s[1] * over;
#pragma unroll
    for (int q = 0; q < H::P; ++q) {
      typename Pack<T>::V o;
#pragma unroll
      for (int e = 0; e < H::V; ++e) {
        const float h = (to_f32((T)px[q][e]) - mu) * rs, g = to_f32((T)pg[q][e]) * w[q * H::V + e];
        float d = rs * (g - s0 - h * s1);
        if (dres) d += to_f32((T)pr[q][e]);
        o[e] = from_f32<T>(d);
      }
      store_pack(o, dx + row * cols + H::at(q), (int64_t)cols - H::at(q));
    }
  }
  float* ow = chunks == 1 ? (dweight ? dweight + p * dw_stride : nullptr) : part + (uint64_t)blockIdx.x * 2 * cols;
  float* ob = chunks == 1 ? (dbias ? dbias + p * db_stride : nullptr) : part + ((uint64_t)blockIdx.x * 2 + 1) * cols;
  if constexpr (H::L < H::NT) {  // several rows at a time: their lanes' sums come together
#pragma unroll
    for (int d = H::L; d < kWave; d <<= 1)
#pragma unroll
      for (int k = 0; k < H::E; ++k) {
        sw[k] += __shfl_xor(sw[k], d, kWave);
        sb[k] += __shfl_xor(sb[k], d, kWave);
      }
    constexpr int NW = H::NT / kWave;
    __shared__ float all[NW / 2][2][H::E][H::L];
    const bool first = lane_id() < (uint32_t)H::L;
    const int wid = threadIdx.x / kWave;
    for (int half = NW / 2; half > 0; half >>= 1) {  // the upper half's sums to the lower half
      if (wid >= half && wid < 2 * half && first) {
#pragma unroll
        for (int k = 0; k < H::E; ++k) {
          all[wid - half][0][k][H::lane()] = sw[k];
          all[wid - half][1][k][H::lane()] = sb[k];
        }
      }
      __syncthreads();
      if (wid < half && first) {
#pragma unroll
        for (int k = 0; k < H::E; ++k) {
          sw[k] += all[wid][0][k][H::lane()];
          sb[k] += all[wid][1][k][H::lane()];
        }
      }
      __syncthreads();
    }
    if (wid != 0 || !first) return;
  }
#pragma unroll
  for (int q = 0; q < H::P; ++q)
#pragma unroll
    for (int e = 0; e < H::V; ++e) {
      const uint32_t col = H::at(q) + e;
      if (col < cols) {
        if (ow) ow[col] = sw[q * H::V + e];
        if (ob) ob[col] = sb[q * H::V + e];
      }
    }
}

// The chunks' sums, 64 columns of one gradient of one node at a time, in 16
// slices of the chunks (with 4, the 128 chunks of 8 nodes' 4096 columns took
// 20 us for 33 MB).
constexpr int kSlices = 16;
__global__ __launch_bounds__(kSlices * 64) void k_join_chunks(uint32_t nodes, uint32_t cols, uint32_t chunks,
                                                              const float* part, float* dweight, uint64_t dw_stride,
                                                              float* dbias, uint64_t db_stride) {
  __shared__ float s[kSlices][64];
  const uint32_t lane = threadIdx.x % 64, slice = threadIdx.x / 64;
  const uint64_t across = (cols + 63) / 64, items = across * nodes * 2;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint64_t col = it % across * 64 + lane, p = it / across / 2, which = it / across % 2;
    float v = 0.0f;
    if (col < cols) {
#pragma unroll 4
      for (uint32_t c = slice; c < chunks; c += kSlices) v += part[((p * chunks + c) * 2 + which) * cols + col];
    }
    __syncthreads();  // the last item's sums have been read
    s[slice][lane] = v;
    __syncthreads();
    float* out = which ? dbias : dweight;
    if (slice == 0 && col < cols && out) {
#pragma unroll
      for (int k = 1; k < kSlices; ++k) v += s[k][lane];
      out[p * (which ? db_stride : dw_stride) + col] = v;
    }
  }
}

// ---- rows too long to be held ------------------------------------------------
template <class T>
__device__ __forceinline__ float normed_value(const T* x, const T* r, uint32_t i) {
  const float v = to_f32(x[i]);
  return r ? to_f32(from_f32<T>(v + to_f32(r[i]))) : v;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_layer_norm_long(uint64_t rows, uint32_t cols, const T* x,
                                                              uint64_t x_stride, const T* residual, uint64_t r_stride,
                                                              const float* weight, const float* bias, float eps, T* y,
                                                              T* total, float* mean, float* rstd) {
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
__global__ __launch_bounds__(kThreads) void k_layer_norm_dx_long(uint64_t rows, uint32_t cols, const T* dy,
                                                                 uint64_t dy_stride, const T* x, uint64_t x_stride,
                                                                 const T* dres, uint64_t dres_stride,
                                                                 const float* weight, const float* mean,
                                                                 const float* rstd, T* dx) {
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

// One thread per column of one chunk of one node's rows.
template <class T>
__global__ __launch_bounds__(kThreads) void k_layer_norm_dw_long(uint32_t nodes, uint64_t rows, uint32_t cols,
                                                                 uint32_t chunks, uint64_t each, const T* dy,
                                                                 uint64_t dy_stride, const T* x, uint64_t x_stride,
                                                                 const float* mean, const float* rstd, float* part) {
  const uint64_t across = (cols + kThreads - 1) / kThreads, items = across * nodes * chunks;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint64_t col = it % across * kThreads + threadIdx.x, pc = it / across, p = pc / chunks;
    if (col >= cols) continue;
    const uint64_t begin = min(pc % chunks * each, rows), end = min(begin + each, rows);
    float w = 0.0f, b = 0.0f;
    for (uint64_t row = p * rows + begin; row < p * rows + end; ++row) {
      const float g = to_f32(dy[row * dy_stride + col]);
      b += g;
      w = fmaf(g, (to_f32(x[row * x_stride + col]) - mean[row]) * rstd[row], w);
    }
    part[pc * 2 * cols + col] = w;
    part[(pc * 2 + 1) * cols + col] = b;
  }
}

// Calls f with the Held of the fewest lanes and elements that hold a row;
// returns false where none does. NL: threads where a row takes a wave or less.
template <class T, int NL, class F>
bool held_by(uint32_t cols, F&& f) {
  if (cols <= 64) f(Held<T, 8, 8, NL>{});
  else if (cols <= 128) f(Held<T, 16, 8, NL>{});
  else if (cols <= 256) f(Held<T, 32, 8, NL>{});
  else if (cols <= 512) f(Held<T, 64, 8, NL>{});
  else if (cols <= 1024) f(Held<T, 64, 16, NL>{});
  else if (cols <= 2048) f(Held<T, 256, 8, 256>{});
  else if (cols <= 4096) f(Held<T, 256, 16, 256>{});
  else if (cols <= 8192) f(Held<T, 1024, 8, 1024>{});
  else if (cols <= kHeld) f(Held<T, 1024, 16, 1024>{});
  else return false;
  return true;
}

// The rows of a node are cut into chunks, one workgroup each: enough of them
// to fill the chip, and no more, since each writes and the last kernel reads
// 8 bytes a column. A chunk takes at least two turns of the rows that its
// workgroup holds at a time (one chunk needs no last kernel: 4 nodes of 16
// rows of 1024 fp32 are one launch). Past 1024 columns that is two rows, whose
// sums are more bytes than the rows: 2048 rows of 4096 bf16 take 40 us where
// their bytes alone take 10, 8192 rows of 16384 319 us where they take 163.
uint32_t chunks_of(uint32_t nodes, uint64_t rows, uint32_t cols) {
  const uint64_t at_once = cols <= 1024 ? kBackRows * kWave / std::max(8u, std::min(64u, cols / 8)) : 1;
  const uint64_t most = (1024 + nodes - 1) / nodes, wanted = (rows + 2 * at_once - 1) / (2 * at_once);
  return (uint32_t)std::max<uint64_t>(1, std::min(most, wanted));
}

}  // namespace

hipError_t layer_norm_launch(uint32_t type, uint64_t rows, uint32_t cols, const void* x, uint64_t x_stride,
                             const void* residual, uint64_t r_stride, const float* weight, const float* bias,
                             float eps, void* y, void* total, float* mean, float* rstd, hipStream_t stream) {
  return for_type(type, [&](auto t) {
    using T = decltype(t);
    const bool held = held_by<T, kThreads>(cols, [&](auto h) {
      using H = decltype(h);
      const uint64_t blocks = std::min<uint64_t>((rows + H::R - 1) / H::R, kBlocks * kThreads / H::NT);
      hipLaunchKernelGGL((k_layer_norm<T, H>), dim3((uint32_t)blocks), dim3(H::NT), 0, stream, rows, cols,
                         (const T*)x, x_stride, (const T*)residual, r_stride, weight, bias, eps, (T*)y, (T*)total,
                         mean, rstd);
    });
    if (!held)
      hipLaunchKernelGGL(k_layer_norm_long<T>, dim3((uint32_t)std::min<uint64_t>(rows, kBlocks)), dim3(kThreads), 0,
                         stream, rows, cols, (const T*)x, x_stride, (const T*)residual, r_stride, weight, bias, eps,
                         (T*)y, (T*)total, mean, rstd);
    return hipGetLastError();
  });
}

size_t layer_norm_backward_workspace_bytes(uint32_t nodes, uint64_t rows, uint32_t cols) {
  return (size_t)nodes * chunks_of(nodes, rows, cols) * 2 * cols * sizeof(float) + 256;
}

hipError_t layer_norm_backward_launch(uint32_t type, uint32_t nodes, uint64_t rows, uint32_t cols, const void* dy,
                                      uint64_t dy_stride, const void* x, uint64_t x_stride, const void* dresidual,
                                      uint64_t dres_stride, const float* weight, const float* mean, const float* rstd,
                                      void* dx, float* dweight, uint64_t dw_stride, float* dbias, uint64_t db_stride,
                                      void* ws, hipStream_t stream) {
  return for_type(type, [&](auto t) {
    using T = decltype(t);
    float* part = static_cast<float*>(ws);
    const uint32_t chunks = chunks_of(nodes, rows, cols);
    const uint64_t each = (rows + chunks - 1) / chunks;
    const bool held = held_by<T, kBackRows * kWave>(cols, [&](auto h) {
      using H = decltype(h);
      hipLaunchKernelGGL((k_layer_norm_backward<T, H>), dim3(nodes * chunks), dim3(H::NT), 0, stream, rows, cols,
                         chunks, each, (const T*)dy, dy_stride, (const T*)x, x_stride, (const T*)dresidual,
                         dres_stride, weight, mean, rstd, (T*)dx, dweight, dw_stride, dbias, db_stride, part);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (held && chunks == 1)) return e;
    if (!held) {
      const uint64_t all = nodes * rows, items = (uint64_t)((cols + kThreads - 1) / kThreads) * nodes * chunks;
      if (all > 0)
        hipLaunchKernelGGL(k_layer_norm_dx_long<T>, dim3((uint32_t)std::min<uint64_t>(all, kBlocks)), dim3(kThreads),
                           0, stream, all, cols, (const T*)dy, dy_stride, (const T*)x, x_stride, (const T*)dresidual,
                           dres_stride, weight, mean, rstd, (T*)dx);
      hipLaunchKernelGGL(k_layer_norm_dw_long<T>, dim3((uint32_t)std::min<uint64_t>(items, 4 * kBlocks)),
                         dim3(kThreads), 0, stream, nodes, rows, cols, chunks, each, (const T*)dy, dy_stride,
                         (const T*)x, x_stride, mean, rstd, part);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return join_chunks_launch(nodes, cols, chunks, part, dweight, dw_stride, dbias, db_stride, stream);
  });
}

hipError_t join_chunks_launch(uint32_t nodes, uint32_t cols, uint32_t chunks, const float* part, float* first,
                              uint64_t first_stride, float* second, uint64_t second_stride, hipStream_t stream) {
  const uint64_t items = (uint64_t)((cols + 63) / 64) * nodes * 2;
  hipLaunchKernelGGL(k_join_chunks, dim3((uint32_t)std::min<uint64_t>(items, 4 * kBlocks)), dim3(kSlices * 64), 0,
                     stream, nodes, cols, chunks, part, first, first_stride, second, second_stride);
  return hipGetLastError();
}

}  // namespace sparcml
