// Orthogonalised updates: every matrix of a flat update by Newton-Schulz
// steps, written out or applied to the weights.
//
//   X0 = G / (|G|_F + eps), the wide way round (m = the shorter side <= n)
//   A = X X^T,  X <- a X + (b A + c A A) X          `steps` times
//   out = X, or w = (1 - lr * decay) * w - lr * sqrt(max(1, rows / cols)) * X
//
// Each step is three products, all of the form D = alpha * A B^T + beta * C:
//   A = X X^T (symmetric), M = c A A + b A (symmetric), X' = M X + a X,
// so one kernel multiplies tiles whose operands both run along the summed
// index. Symmetric results are computed for the tiles on and below the
// diagonal and stored twice; X is kept in both orders (X and X^T), since the
// first product sums along its rows and the third along its columns.
//
// Numbers: the matrix cores multiply fp16 and add in fp32. A value v is held
// as hi = fp16(v * scale), lo = fp16(v * scale - hi), 22 bits in all, and a
// product of two values is hi hi + hi lo + lo hi: the dropped lo lo is below
// 2^-22 of it, the same order as fp32's own rounding of a long sum. The scale
// is a power of two (2^12 for X and A, 2^8 for M) that keeps lo out of fp16's
// underflow for the small entries of large matrices; entries of X reach 1.3
// with the usual coefficients and may reach 15 before hi overflows.
#include <algorithm>
#include <cmath>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kTile = 128;      // rows and columns of one workgroup's tile of a product
constexpr uint32_t kDepth = 32;      // summed index per pass through LDS
constexpr uint32_t kPad = 64;        // sides are padded with zeros to this
constexpr uint32_t kGroups = 24;     // groups of equal matrices in one set of launches
constexpr uint32_t kParts = 256;     // partial sums of squares of one matrix, at most
constexpr float kScaleX = 4096.0f;   // of X, X^T, A
constexpr float kScaleM = 256.0f;    // of M

typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__host__ __device__ __forceinline__ uint32_t up(uint32_t v, uint32_t to) { return (v + to - 1) / to * to; }

// Equal matrices that follow each other in the flat update.
struct Group {
  uint64_t at;     // position of the first one in the flat update
  uint64_t ws;     // byte of the workspace where its buffers start
  uint64_t ws_of;  // bytes of each one's buffers
  uint32_t count, rows, cols, tiles;

  __host__ __device__ bool tall() const { return rows > cols; }
  __host__ __device__ uint32_t m() const { return up(rows < cols ? rows : cols, kPad); }
  __host__ __device__ uint32_t n() const { return up(rows < cols ? cols : rows, kPad); }
};
struct Groups {
  Group g[kGroups];
  uint32_t count;
};

// A matrix's buffers: partial sums, then X, X^T, the next X and X^T, A and M.
// Each buffer is a plane of hi and a plane of lo.
enum Buffer : uint32_t { kX0, kXT0, kX1, kXT1, kA, kM, kBuffers };

struct Planes {
  f16* hi;
  f16* lo;
  uint32_t ld;
};
__host__ __device__ __forceinline__ uint64_t buffers_bytes(uint32_t m, uint32_t n) {
  return kParts * sizeof(double) + 4ull * (4ull * m * n + (uint64_t)(kBuffers - kA) * m * m);
}
__device__ __forceinline__ Planes planes(unsigned char* base, uint32_t m, uint32_t n, uint32_t b) {
  f16* p = reinterpret_cast<f16*>(base + kParts * sizeof(double));
  const uint64_t x = (uint64_t)m * n, s = (uint64_t)m * m;
  if (b < kA) return Planes{p + 2 * x * b, p + 2 * x * b + x, (b & 1) ? m : n};
  p += 2 * x * kA + 2 * s * (b - kA);
  return Planes{p, p + s, m};
}

// This workgroup's item among the groups' `tiles` per matrix: the group, the
// matrix in it and the tile in the matrix.
struct Item {
  uint32_t g, k, tile;
};
__device__ __forceinline__ Item item_of(const Groups& gs, uint32_t b) {
  uint32_t g = 0;
  while (g + 1 < gs.count && b >= gs.g[g].count * gs.g[g].tiles) {
    b -= gs.g[g].count * gs.g[g].tiles;
    ++g;
  }
  return Item{g, b / gs.g[g].tiles, b % gs.g[g].tiles};
}

__device__ __forceinline__ uint32_t parts_of(uint64_t size) {
  const uint64_t p = (size + 8191) / 8192;
  return p < kParts ? (uint32_t)p : kParts;
}

// Sums of squares, fp64, in parts of a fixed order.
template <class T>
__global__ __launch_bounds__(kThreads) void k_squares(Groups gs, const T* update, unsigned char* ws) {
  __shared__ double scratch[kThreads / kWave];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  const uint64_t size = (uint64_t)g.rows * g.cols, each = (size + g.tiles - 1) / g.tiles;
  const T* x = update + g.at + it.k * size;
  const uint64_t begin = it.tile * each, end = min(begin + each, size);
  double s = 0.0;
  for (uint64_t i = begin + threadIdx.x; i < end; i += kThreads) {
    const double v = to_f32(x[i]);
    s += v * v;
  }
  s = block_sum_f64<kThreads>(s, scratch);
  if (threadIdx.x == 0) reinterpret_cast<double*>(ws + g.ws + it.k * g.ws_of)[it.tile] = s;
}

// X0 and its transpose, one 64 x 64 tile of the padded matrix.
template <class T>
__global__ __launch_bounds__(kThreads) void k_split(Groups gs, const T* update, float eps, unsigned char* ws) {
  __shared__ float t[64][65];
  __shared__ double scratch[kThreads / kWave];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  unsigned char* base = ws + g.ws + it.k * g.ws_of;
  const uint64_t size = (uint64_t)g.rows * g.cols;
  const uint32_t parts = parts_of(size);
  const double* part = reinterpret_cast<const double*>(base);
  const double sum = block_sum_f64<kThreads>(threadIdx.x < parts ? part[threadIdx.x] : 0.0, scratch);
  const double by = (double)kScaleX / (sqrt(sum) + (double)eps);
  const uint32_t pr = up(g.rows, kPad), pc = up(g.cols, kPad);
  const uint32_t r0 = it.tile / (pc / 64) * 64, c0 = it.tile % (pc / 64) * 64;
  const T* x = update + g.at + it.k * size;
  const uint32_t tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  // as stored: the wide X if rows <= cols, else X^T
  const Planes same = planes(base, g.m(), g.n(), g.tall() ? kXT0 : kX0);
  const Planes turned = planes(base, g.m(), g.n(), g.tall() ? kX0 : kXT0);
  for (uint32_t y = ty; y < 64; y += 4) {
    const uint32_t r = r0 + y, c = c0 + tx;
    const float v = r < g.rows && c < g.cols ? (float)((double)to_f32(x[(uint64_t)r * g.cols + c]) * by) : 0.0f;
    t[y][tx] = v;
    const f16 hi = (f16)v;
    same.hi[(uint64_t)r * pc + c] = hi;
    same.lo[(uint64_t)r * pc + c] = (f16)(v - (float)hi);
  }
  __syncthreads();
  for (uint32_t y = ty; y < 64; y += 4) {
    const float v = t[tx][y];
    const f16 hi = (f16)v;
    const uint64_t at = (uint64_t)(c0 + y) * pr + r0 + tx;
    turned.hi[at] = hi;
    turned.lo[at] = (f16)(v - (float)hi);
  }
}

// One product of every matrix: D = alpha * A B^T + beta * C in stored units.
// i runs over A's rows (m of them), j over B's.
struct Product {
  uint32_t a, b;        // operands, rows along the summed index
  uint32_t c_ji;        // C, stored [j][i]
  uint32_t d_ij, d_ji;  // D in both orders (planes only)
  uint32_t sym;         // D symmetric: a == b's rows, tiles j <= i
  float alpha, beta;
};
enum Out { kPlanes, kResult, kWeight };

// (i, j), j <= i, of the t-th tile on and below the diagonal
__device__ __forceinline__ void lower_tile(uint32_t t, uint32_t& i, uint32_t& j) {
  i = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((uint64_t)i * (i + 1) / 2 > t) --i;
  while ((uint64_t)(i + 1) * (i + 2) / 2 <= t) ++i;
  j = t - (uint32_t)((uint64_t)i * (i + 1) / 2);
}

// Scale of the result for the weights: w = keep * w - move * s * X.
struct Move {
  float keep, move;
};

template <int OUT, class T>
__global__ __launch_bounds__(kThreads) void k_product(Groups gs, Product p, unsigned char* ws, T* out, Move mv) {
  __shared__ f16x8 lds[4][kTile * kDepth / 8];  // A hi, A lo, B hi, B lo
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  const uint32_t m = g.m(), n = g.n();
  unsigned char* base = ws + g.ws + it.k * g.ws_of;
  const Planes a = planes(base, m, n, p.a), b = planes(base, m, n, p.b);
  const uint32_t J = p.sym ? m : n, K = a.ld;
  uint32_t ti, tj;
  if (p.sym) {
    lower_tile(it.tile, ti, tj);
  } else {
    const uint32_t across = up(J, kTile) / kTile;
    ti = it.tile / across;
    tj = it.tile % across;
  }
  const uint32_t lane = lane_id(), wid = threadIdx.x / kWave;
  const uint32_t wi = wid / 2 * 64, wj = wid % 2 * 64;
  const bool on = ti * kTile + wi < m && tj * kTile + wj < J;  // this wave's 64 x 64 is inside

  f32x16 acc[2][2] = {};
  for (uint32_t k0 = 0; k0 < K; k0 += kDepth) {
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t chunk = threadIdx.x + h * kThreads, row = chunk / 4, c = chunk % 4;
      const uint32_t slot = row * 4 + (c ^ (row >> 1 & 3));  // 8 rows of one chunk fall into 8 bank groups
      const uint64_t ra = (uint64_t)min(ti * kTile + row, m - 1) * K + k0 + c * 8;
      const uint64_t rb = (uint64_t)min(tj * kTile + row, J - 1) * K + k0 + c * 8;
      lds[0][slot] = *reinterpret_cast<const f16x8*>(a.hi + ra);
      lds[1][slot] = *reinterpret_cast<const f16x8*>(a.lo + ra);
      lds[2][slot] = *reinterpret_cast<const f16x8*>(b.hi + rb);
      lds[3][slot] = *reinterpret_cast<const f16x8*>(b.lo + rb);
    }
    __syncthreads();
    if (on) {
#pragma unroll
      for (uint32_t ks = 0; ks < kDepth / 16; ++ks) {
        f16x8 f[4][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t ra = wi + q * 32 + lane % 32, rb = wj + q * 32 + lane % 32, c = ks * 2 + lane / 32;
          f[0][q] = lds[0][ra * 4 + (c ^ (ra >> 1 & 3))];
          f[1][q] = lds[1][ra * 4 + (c ^ (ra >> 1 & 3))];
          f[2][q] = lds[2][rb * 4 + (c ^ (rb >> 1 & 3))];
          f[3][q] = lds[3][rb * 4 + (c ^ (rb >> 1 & 3))];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[0][x], f[2][y], acc[x][y], 0, 0, 0);
            acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[0][x], f[3][y], acc[x][y], 0, 0, 0);
            acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[1][x], f[2][y], acc[x][y], 0, 0, 0);
          }
      }
    }
  }
  if (!on) return;
  const Planes c = planes(base, m, n, p.c_ji), dij = planes(base, m, n, p.d_ij), dji = planes(base, m, n, p.d_ji);
  const float move = mv.move * sqrtf(fmaxf(1.0f, (float)g.rows / (float)g.cols));
  T* o = out + g.at + it.k * (uint64_t)g.rows * g.cols;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint32_t j = tj * kTile + wj + y * 32 + lane % 32;
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // 4 consecutive i
        const uint32_t i = ti * kTile + wi + x * 32 + q * 8 + lane / 32 * 4;
        f16x4 ch = {}, cl = {};
        if (p.beta != 0.0f) {
          ch = *reinterpret_cast<const f16x4*>(c.hi + (uint64_t)j * c.ld + i);
          cl = *reinterpret_cast<const f16x4*>(c.lo + (uint64_t)j * c.ld + i);
        }
        f16x4 dh, dl;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = fmaf(p.alpha, acc[x][y][q * 4 + e], p.beta * ((float)ch[e] + (float)cl[e]));
          if (OUT == kPlanes) {
            dh[e] = (f16)v;
            dl[e] = (f16)(v - (float)dh[e]);
            if (!(p.sym && ti == tj)) {
              dij.hi[(uint64_t)(i + e) * dij.ld + j] = dh[e];
              dij.lo[(uint64_t)(i + e) * dij.ld + j] = dl[e];
            }
          } else {
            const uint32_t r = g.tall() ? j : i + e, col = g.tall() ? i + e : j;
            if (r < g.rows && col < g.cols) {
              const uint64_t at = (uint64_t)r * g.cols + col;
              o[at] = from_f32<T>(OUT == kWeight ? fmaf(mv.keep, to_f32(o[at]), -move * v) : v);
            }
          }
        }
        if (OUT == kPlanes) {
          *reinterpret_cast<f16x4*>(dji.hi + (uint64_t)j * dji.ld + i) = dh;
          *reinterpret_cast<f16x4*>(dji.lo + (uint64_t)j * dji.ld + i) = dl;
        }
      }
    }
}

// No steps: the normalised update itself.
template <int OUT, class S, class T>
__global__ __launch_bounds__(kThreads) void k_normalised(Groups gs, const S* update, float eps, unsigned char* ws,
                                                         T* out, Move mv) {
  __shared__ double scratch[kThreads / kWave];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  const uint64_t size = (uint64_t)g.rows * g.cols, each = (size + g.tiles - 1) / g.tiles;
  const double* part = reinterpret_cast<const double*>(ws + g.ws + it.k * g.ws_of);
  const double sum = block_sum_f64<kThreads>(threadIdx.x < g.tiles ? part[threadIdx.x] : 0.0, scratch);
  const double by = 1.0 / (sqrt(sum) + (double)eps);
  const float move = mv.move * sqrtf(fmaxf(1.0f, (float)g.rows / (float)g.cols));
  const uint64_t begin = it.tile * each, end = min(begin + each, size), at = g.at + it.k * size;
  for (uint64_t i = at + begin + threadIdx.x; i < at + end; i += kThreads) {
    const float v = (float)((double)to_f32(update[i]) * by);
    out[i] = from_f32<T>(OUT == kWeight ? fmaf(mv.keep, to_f32(out[i]), -move * v) : v);
  }
}

// Cuts the matrices into groups of equal ones that follow each other, and
// lays their buffers out in the workspace. Calls f(groups) for every kGroups
// of them; returns the bytes used.
template <class F>
uint64_t for_groups(const OrthoMatrices& ms, F&& f) {
  Groups gs = {};
  uint64_t used = 0;
  for (uint32_t k = 0; k < ms.count; ++k) {
    const uint32_t rows = ms.rows[k], cols = ms.cols[k];
    if (rows == 0 || cols == 0) continue;
    Group* last = gs.count ? &gs.g[gs.count - 1] : nullptr;
    if (last && last->rows == rows && last->cols == cols &&
        last->at + (uint64_t)last->count * rows * cols == ms.offsets[k]) {
      ++last->count;
      used += last->ws_of;
      continue;
    }
    if (gs.count == kGroups) {
      f(gs);
      gs.count = 0;
    }
    Group& g = gs.g[gs.count++];
    g = Group{ms.offsets[k], used, 0, 1, rows, cols, 0};
    g.ws_of = buffers_bytes(g.m(), g.n());
    used += g.ws_of;
  }
  if (gs.count) f(gs);
  return used;
}

// Sets the groups' tiles by `of` and returns the launch's workgroups.
template <class F>
uint32_t tiled(Groups& gs, F&& of) {
  uint64_t all = 0;
  for (uint32_t k = 0; k < gs.count; ++k) {
    gs.g[k].tiles = of(gs.g[k]);
    all += (uint64_t)gs.g[k].tiles * gs.g[k].count;
  }
  return (uint32_t)all;
}
uint32_t parts_of_host(const Group& g) {
  return (uint32_t)std::min<uint64_t>(((uint64_t)g.rows * g.cols + 8191) / 8192, kParts);
}

template <int OUT, class T>
hipError_t launch_product(Groups& gs, const Product& p, unsigned char* ws, T* out, Move mv, hipStream_t stream) {
  const uint32_t blocks = tiled(gs, [&](const Group& g) {
    const uint32_t i = up(g.m(), kTile) / kTile, j = up(g.n(), kTile) / kTile;
    return p.sym ? i * (i + 1) / 2 : i * j;
  });
  hipLaunchKernelGGL((k_product<OUT, T>), dim3(blocks), dim3(kThreads), 0, stream, gs, p, ws, out, mv);
  return hipGetLastError();
}

template <int OUT, class S, class T>
hipError_t run(Groups& gs, const OrthoSteps& s, const S* update, T* out, Move mv, unsigned char* ws,
               hipStream_t stream) {
  uint32_t blocks = tiled(gs, parts_of_host);
  hipLaunchKernelGGL(k_squares<S>, dim3(blocks), dim3(kThreads), 0, stream, gs, update, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (s.steps == 0) {
    hipLaunchKernelGGL((k_normalised<OUT, S, T>), dim3(blocks), dim3(kThreads), 0, stream, gs, update, s.eps, ws, out,
                       mv);
    return hipGetLastError();
  }
  blocks = tiled(gs, [](const Group& g) { return g.m() / 64 * (g.n() / 64); });
  hipLaunchKernelGGL(k_split<S>, dim3(blocks), dim3(kThreads), 0, stream, gs, update, s.eps, ws);
  e = hipGetLastError();
  for (uint32_t k = 0; k < s.steps && e == hipSuccess; ++k) {
    const uint32_t x = k % 2 ? kX1 : kX0, y = k % 2 ? kX0 : kX1;  // the step's X and the next
    e = launch_product<kPlanes, T>(gs, Product{x, x, x, kA, kA, 1, 1.0f / kScaleX, 0.0f}, ws, nullptr, mv, stream);
    if (e != hipSuccess) break;
    e = launch_product<kPlanes, T>(gs,
                                   Product{kA, kA, kA, kM, kM, 1, s.c * kScaleM / (kScaleX * kScaleX),
                                           s.b * kScaleM / kScaleX},
                                   ws, nullptr, mv, stream);
    if (e != hipSuccess) break;
    const bool last = k + 1 == s.steps;
    const float unit = last ? 1.0f / kScaleX : 1.0f;
    const Product px{kM, x + 1, x + 1, y, y + 1, 0, unit / kScaleM, unit * s.a};
    e = last ? launch_product<OUT, T>(gs, px, ws, out, mv, stream)
             : launch_product<kPlanes, T>(gs, px, ws, nullptr, mv, stream);
  }
  return e;
}

}  // namespace

uint64_t ortho_tiles(uint64_t rows, uint64_t cols) {
  const uint64_t m = std::min(rows, cols), n = std::max(rows, cols);
  if (m > (1u << 16) || n > (1u << 24) || m * n > (1ull << 32)) return 0;
  return (m + 63) / 64 * ((n + 63) / 64);
}

size_t ortho_workspace_bytes(const OrthoMatrices& ms) {
  return (size_t)for_groups(ms, [](Groups&) {}) + 256;
}

hipError_t ortho_launch(const OrthoMatrices& ms, const OrthoSteps& steps, uint32_t update_type, const void* update,
                        uint32_t out_type, void* out, bool is_weight, float keep, float move, void* ws,
                        hipStream_t stream) {
  hipError_t e = hipSuccess;
  const Move mv{keep, move};
  for_groups(ms, [&](Groups& gs) {
    if (e != hipSuccess) return;
    e = for_type(update_type, [&](auto s) {
      return for_type(out_type, [&](auto t) {
        using S = decltype(s);
        using T = decltype(t);
        unsigned char* w = static_cast<unsigned char*>(ws);
        return is_weight ? run<kWeight, S, T>(gs, steps, (const S*)update, (T*)out, mv, w, stream)
                         : run<kResult, S, T>(gs, steps, (const S*)update, (T*)out, mv, w, stream);
      });
    });
  });
  return e;
}

}  // namespace sparcml
