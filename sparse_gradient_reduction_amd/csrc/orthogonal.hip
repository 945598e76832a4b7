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
// diagonal and stored twice: exactly symmetric, because a rounding that makes
// A B^T differ from A B grows from step to step (20 times in three steps taken
// as one, below); X is kept in both orders (X and X^T), since the
// first product sums along its rows and the third along its columns.
//
// Numbers: the matrix cores multiply fp16 and add in fp32. A value v is held
// as hi = fp16(v * scale), lo = fp16(v * scale - hi), 22 bits in all, and a
// product of two values is hi hi + hi lo + lo hi: the dropped lo lo is below
// 2^-22 of it, the same order as fp32's own rounding of a long sum. The scale
// is a power of two (2^12 for X and A, 2^8 for M) that keeps lo out of fp16's
// underflow for the small entries of large matrices. hi overflows at 65504: A's
// entries may reach 16 and so X's rows a norm of 4 (1.3 with the usual
// coefficients), those of Q = a I + M and of the product of two steps' Q 255 (13).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kernels.hpp"
#include "numeric.hpp"
#include "orthogonal_tiles.hpp"

namespace sparcml {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kGroups = 24;     // groups of equal matrices in one set of launches
constexpr uint32_t kParts = 1024;    // partial sums of squares of one matrix, at most
constexpr float kScaleX = 4096.0f;   // of X, X^T, A
constexpr float kScaleM = 256.0f;    // of M

typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

// A matrix's buffers: partial sums, then X, X^T, the next X and X^T, and the
// square ones: A, the step's M, Q A, and the product of the steps' Q (two).
// A row of `ld` values holds 2 * ld fp16: 32 hi, 32 lo and so on, so that 128
// bytes of a row are a pass's operands (64 bytes at a time, memory gives a
// workgroup 59 GB/s instead of 100).
enum Buffer : uint32_t { kX0, kXT0, kX1, kXT1, kA, kM, kT, kP, kP2, kBuffers };

struct Plane {
  f16* p;
  uint32_t ld;
  __device__ __forceinline__ f16* row(uint64_t r) const { return p + r * 2 * ld; }
  // element e's hi part; its lo part is kToLo further on
  __device__ __forceinline__ f16* hi(uint64_t r, uint32_t e) const { return row(r) + e + e / 32 * 32; }
};
constexpr uint32_t kToLo = 32;
__host__ __device__ __forceinline__ uint64_t buffers_bytes(uint32_t m, uint32_t n) {
  return kParts * sizeof(double) + 4ull * (4ull * m * n + (uint64_t)(kBuffers - kA) * m * m);
}
__device__ __forceinline__ Plane plane(unsigned char* base, uint32_t m, uint32_t n, uint32_t b) {
  f16* p = reinterpret_cast<f16*>(base + kParts * sizeof(double));
  const uint64_t x = 2ull * m * n, s = 2ull * m * m;
  return b < kA ? Plane{p + x * b, (b & 1) ? m : n} : Plane{p + x * kA + s * (b - kA), m};
}

// Workgroups of a launch come in groups of `count * tiles`, rounded up to 8 so
// that the workgroups of one group spread over the XCDs alike and each XCD
// walks neighbouring tiles. k may be past the last matrix: nothing to do.
struct Item {
  uint32_t g, k, tile;
};
__host__ __device__ __forceinline__ uint32_t items_of(const Group& g) { return up(g.count * g.tiles, kXcds); }
__device__ __forceinline__ Item item_of(const Groups& gs, uint32_t b) {
  uint32_t g = 0;
  while (g + 1 < gs.count && b >= items_of(gs.g[g])) {
    b -= items_of(gs.g[g]);
    ++g;
  }
  b = xcd_contiguous(b, items_of(gs.g[g]));
  return Item{g, b / gs.g[g].tiles, b % gs.g[g].tiles};
}

__device__ __forceinline__ uint32_t parts_of(uint64_t size) {
  const uint64_t p = (size + 8191) / 8192;
  return p < kParts ? (uint32_t)p : kParts;
}

// Sums of squares, fp64, in parts of a fixed order.
__device__ __forceinline__ double sum_of_parts(const double* part, uint32_t parts, double* scratch) {
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return block_sum_f64<kThreads>(s, scratch);
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_squares(Groups gs, const T* update, unsigned char* ws) {
  __shared__ double scratch[kThreads / kWave];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  if (it.k >= g.count) return;
  const uint64_t size = (uint64_t)g.rows * g.cols, each = (size + 8ull * g.tiles - 1) / (8ull * g.tiles) * 8;
  const T* x = update + g.at + it.k * size;
  const uint64_t begin = it.tile * each, end = min(begin + each, size);
  constexpr int V = Pack<T>::N;
  double s = 0.0;
#pragma unroll 4
  for (uint64_t i = begin + threadIdx.x * V; i < end; i += kThreads * V) {
    const typename Pack<T>::V v = load_pack(x + i, (int64_t)(end - i));
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const double w = to_f32((T)v[e]);
      s = fma(w, w, s);
    }
  }
  s = block_sum_f64<kThreads>(s, scratch);
  if (threadIdx.x == 0) reinterpret_cast<double*>(ws + g.ws + it.k * g.ws_of)[it.tile] = s;
}

// 16 values to a row's elements e .. e + 15 as hi and lo parts.
__device__ __forceinline__ void store_parts(const float (&v)[16], f16* hi) {
  f16x8 h[2], l[2];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    h[e / 8][e % 8] = (f16)v[e];
    l[e / 8][e % 8] = (f16)fmaf((float)h[e / 8][e % 8], -1.0f, v[e]);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    reinterpret_cast<f16x8*>(hi)[q] = h[q];
    reinterpret_cast<f16x8*>(hi + kToLo)[q] = l[q];
  }
}

// X0 and its transpose, one 64 x 64 tile of the padded matrix; a thread takes
// 16 elements of a row, then 16 of a row of the transpose.
template <class T>
__global__ __launch_bounds__(kThreads) void k_split(Groups gs, const T* update, float eps, unsigned char* ws) {
  __shared__ float t[64][65];
  __shared__ double scratch[kThreads / kWave];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  if (it.k >= g.count) return;
  unsigned char* base = ws + g.ws + it.k * g.ws_of;
  const uint64_t size = (uint64_t)g.rows * g.cols;
  const uint32_t across = up(g.cols, kPad) / 64;
  const uint32_t r0 = it.tile / across * 64, c0 = it.tile % across * 64;
  const T* x = update + g.at + it.k * size;
  const uint32_t row = threadIdx.x / 4, seg = threadIdx.x % 4 * 16;
  const uint32_t r = r0 + row, c = c0 + seg;
  constexpr int V = Pack<T>::N;
  typename Pack<T>::V w[16 / V];
#pragma unroll
  for (int q = 0; q < 16 / V; ++q) {
    const int64_t room = r < g.rows ? (int64_t)g.cols - c - q * V : 0;
    w[q] = load_pack(x + (uint64_t)r * g.cols + c + q * V, room);
  }
  const double sum = sum_of_parts(reinterpret_cast<const double*>(base), parts_of(size), scratch);
  const double by = (double)kScaleX / (sqrt(sum) + (double)eps);
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    v[e] = r < g.rows && c + e < g.cols ? (float)((double)to_f32((T)w[e / V][e % V]) * by) : 0.0f;
    t[row][seg + e] = v[e];
  }
  // as stored: the wide X if rows <= cols, else X^T
  const bool tall = g.tall();
  const Plane same = plane(base, g.m(), g.n(), tall ? kXT0 : kX0), turned = plane(base, g.m(), g.n(), tall ? kX0 : kXT0);
  store_parts(v, same.hi(r, c));
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = t[seg + e][row];
  store_parts(v, turned.hi(c0 + row, r0 + seg));
}

// One product of every matrix: D = alpha * A B^T + beta * C + gamma * C2 in stored units.
// i runs over A's rows (m of them), j over B's.
struct Product {
  uint32_t a, b;        // operands, rows along the summed index
  uint32_t c_ji, c2;    // C, stored [j][i]; C2, symmetric
  uint32_t d_ij, d_ji;  // D in both orders (planes only)
  uint32_t sym;         // D symmetric: what lies above the diagonal is the mirror of what lies below
  float alpha, beta, gamma;
};
enum Out { kPlanes, kResult, kWeight };

// Scale of the result for the weights: w = keep * w - move * s * X.
struct Move {
  float keep, move;
};

// Tiles of a product, I x J of them, or those on and below the diagonal. They
// are taken in bands of 4 rows, column by column, so that neighbouring ones,
// which share an XCD's L2, read few rows of A and B. Every number is a tile: a
// workgroup without one would take a CU's LDS from another's first turn (72
// such among 288 made a product of six matrices of width 1024 take 34 us, not
// 21).
constexpr uint32_t kBand = 4;
// (i, j), j <= i, of the t-th pair in the order (0, 0), (1, 0), (1, 1), (2, 0) ...
__host__ __device__ __forceinline__ void pair_at(uint32_t t, uint32_t& i, uint32_t& j) {
  i = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((uint64_t)i * (i + 1) / 2 > t) --i;
  while ((uint64_t)(i + 1) * (i + 2) / 2 <= t) ++i;
  j = t - (uint32_t)((uint64_t)i * (i + 1) / 2);
}
__host__ __device__ __forceinline__ void tile_at(uint32_t t, uint32_t I, uint32_t J, bool sym, uint32_t& ti,
                                                 uint32_t& tj) {
  uint32_t r0, u;
  if (sym) {
    pair_at(t, ti, tj);
    r0 = ti / kBand * kBand;
    u = t - r0 * (r0 + 1) / 2;
  } else {
    r0 = t / (kBand * J) * kBand;
    u = t - r0 * J;
  }
  const uint32_t h = min(kBand, I - r0);  // rows of the band
  if (!sym || u < r0 * h) {
    ti = r0 + u % h;
    tj = u / h;
  } else {  // the band's own triangle
    pair_at(u - r0 * h, ti, tj);
    ti += r0;
    tj += r0;
  }
}

// 16 bytes a lane from memory straight into LDS, at `to` + 16 * lane.
__device__ __forceinline__ void load_to_lds(const char* from, f16x8* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Orders the wave's LDS accesses, whose lanes read what other lanes wrote; the
// hardware runs them in order.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Waits until at most N of this wave's memory operations are under way and its
// LDS reads have arrived, then for the workgroup's other waves to be there too.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | N / 16 << 14);  // vmcnt N, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The shape of a workgroup's tile: WI x WJ waves, each TI x TJ blocks of
// 32 x 32, and the LDS buffers.
template <int WI_, int WJ_, int TI_, int TJ_, int BUFFERS_>
struct Shape {
  static constexpr int WI = WI_, WJ = WJ_, TI = TI_, TJ = TJ_, BUFFERS = BUFFERS_;
  static constexpr int W = WI * WJ, NT = W * kWave, I = WI * TI * 32, J = WJ * TJ * 32;
  static constexpr int DEPTH = 32;  // summed index of a pass: rows of 128 bytes, hi and lo
  static constexpr int SIZE = (I + J) * 8;
  static constexpr int PITCH = 36;  // of a block of 32 x 32 that a wave turns
  static constexpr int FIRST = SIZE > W * 32 * PITCH / 4 ? SIZE : W * 32 * PITCH / 4;  // the first buffer: the turned blocks too
  static_assert(W % 2 == 0, "a lane's chunk is the same in every load");
};

// Tells the scheduler to spread NV memory loads and ND LDS reads over NM
// multiplications.
template <int I, int NM, int NV, int ND>
struct Spread {
  static __device__ __forceinline__ void over() {
    constexpr int v = (I + 1) * NV / NM - I * NV / NM, d = (I + 1) * ND / NM - I * ND / NM;
    if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x20, v, 0);
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if constexpr (I + 1 < NM) Spread<I + 1, NM, NV, ND>::over();
  }
};

// A workgroup multiplies I x J tiles. LDS buffers of (I + J) rows of 128 bytes:
// while the waves multiply from one, the rows of the next passes go from memory
// straight into the others. A row's eight 16-byte chunks are stored in an order
// that differs by pairs of rows (chunk c at c ^ (row / 2 % 8)): sixteen lanes
// that read the same chunk of sixteen rows then read all 64 banks once.
template <class S, int OUT, class T>
__global__ __launch_bounds__(S::NT, S::NT == 512 ? 2 : 1) void k_product(Groups gs, Product p, unsigned char* ws,
                                                                        T* out, Move mv) {
  __shared__ f16x8 lds0[S::FIRST], lds1[S::SIZE], lds2[S::BUFFERS > 2 ? S::SIZE : 1], lds3[S::BUFFERS > 2 ? S::SIZE : 1];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  if (it.k >= g.count) return;
  const uint32_t m = g.m(), n = g.n();
  const uint32_t J = p.sym ? m : n;
  uint32_t ti, tj;
  tile_at(it.tile, (m + S::I - 1) / S::I, (J + S::J - 1) / S::J, p.sym, ti, tj);
  const uint32_t i0 = ti * S::I, j0 = tj * S::J;
  unsigned char* base = ws + g.ws + it.k * g.ws_of;
  const Plane a = plane(base, m, n, p.a), b = plane(base, m, n, p.b);
  const uint32_t K = a.ld;
  const uint32_t lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t wi = wid / S::WJ * (S::TI * 32), wj = wid % S::WJ * (S::TJ * 32);

  // this lane's part of the 8 rows that its wave loads at once: row lane / 8, stored chunk lane % 8
  const uint32_t from = (lane % 8 ^ (wid % 2 * 4 + lane / 16)) * 8;
  constexpr int LA = S::I / 8 / S::W, LN = LA + S::J / 8 / S::W;
  const char *pa = (const char*)a.row(i0), *pb = (const char*)b.row(j0);
  uint32_t src[LN];  // bytes from there; at most 256 rows of 2 * 2^21 fp16
#pragma unroll
  for (int t = 0; t < LN; ++t) {
    const uint32_t r = ((t < LA ? t : t - LA) * S::W + wid) * 8 + lane / 8;
    src[t] = (min(r, (t < LA ? m - i0 : J - j0) - 1) * 2 * K + from) * sizeof(f16);
  }
  const auto load = [&](f16x8* lds) {  // of a pass
#pragma unroll
    for (int t = 0; t < LN; ++t) load_to_lds((t < LA ? pa : pb) + src[t], lds + (t * S::W + wid) * kWave);
    pa += 128;
    pb += 128;
    asm("" : "+s"(pa), "+s"(pb));  // stays a scalar base and 32-bit offsets
  };

  // C and C2, 32 columns at a time. A tile of few registers loads them ahead of
  // the products. They are added before anything is stored: a load behind
  // stores would wait for them, block after block.
  constexpr bool AHEAD = S::TI * S::TJ <= 4;
  const auto outside = [&](int x, int y) {  // blocks of 32 lie inside or outside
    return i0 + wi + x * 32 >= m || j0 + wj + y * 32 >= J;
  };
  // A lane loads 16 bytes of a column, the halves of the wave different eights
  // of its 32 rows, and they swap fours when these are used: half the loads of
  // 8 bytes each.
  struct Columns {
    f16x8 hi[S::TI][2], lo[S::TI][2];
  };
  const auto load_c = [&](const Plane& c, int y, Columns& to) {
    to = Columns{};
    const uint32_t j = j0 + wj + y * 32 + lane % 32, i = i0 + wi + lane / 32 * 16;
#pragma unroll
    for (int x = 0; x < S::TI; ++x)
      if (!outside(x, y)) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f16* at = c.hi(j, i + x * 32 + q * 8);
          to.hi[x][q] = *reinterpret_cast<const f16x8*>(at);
          to.lo[x][q] = *reinterpret_cast<const f16x8*>(at + kToLo);
        }
      }
  };
  // rows 8 q + 4 (lane / 32) + e of eights q and q + 2
  const auto fours = [&](f16x8 eight, f16x4 (&to)[4], int q) {
    const u32x4 w = __builtin_bit_cast(u32x4, eight);
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    to[q] = __builtin_bit_cast(f16x4, u32x2{a[0], b[0]});
    to[q + 2] = __builtin_bit_cast(f16x4, u32x2{a[1], b[1]});
  };
  Columns ahead[2][AHEAD ? S::TJ : 1];
  if constexpr (AHEAD) {
#pragma unroll
    for (int y = 0; y < S::TJ; ++y) {
      if (p.beta != 0.0f) load_c(plane(base, m, n, p.c_ji), y, ahead[0][y]);
      if (p.gamma != 0.0f) load_c(plane(base, m, n, p.c2), y, ahead[1][y]);
    }
  }

  // The sums add up 8 passes (256 of the summed index, 48 additions) at a time:
  // in one chain of thousands of roundings an fp32 result of 196 x 8000
  // is off by 7e-6 of its norm, not 2e-6. Tiles of 256 x 256 have no registers
  // left for it: 25 matrices of 1024 x 8192, which take them, are off by 3.2e-6
  // each and 4 of them, which do not, by 2.2e-6 (fp32 products: 3.9e-6).
  constexpr bool STAGES = S::BUFFERS > 2;
  f32x16 acc[S::TI][S::TJ] = {}, total[STAGES ? S::TI : 1][STAGES ? S::TJ : 1] = {};
  const auto stage = [&] {
#pragma unroll
    for (int x = 0; x < S::TI; ++x)
#pragma unroll
      for (int y = 0; y < S::TJ; ++y)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          total[x][y][e] += acc[x][y][e];
          acc[x][y][e] = 0.0f;
        }
  };
  struct Parts {
    f16x8 a[2][S::TI], b[2][S::TJ];  // hi and lo of 16 of a pass's 32: its first half in f[0], its second in f[1]
  } f[2];
  const auto read = [&](const f16x8* lds, int ks, Parts& to) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = (ks * 2 + h * 4 + lane / 32) ^ lane / 2 % 8;
#pragma unroll
      for (int q = 0; q < S::TI; ++q) to.a[h][q] = lds[(wi + q * 32 + lane % 32) * 8 + c];
#pragma unroll
      for (int q = 0; q < S::TJ; ++q) to.b[h][q] = lds[(S::I + wj + q * 32 + lane % 32) * 8 + c];
    }
  };
  const auto multiply = [&](const Parts& by) {
#pragma unroll
    for (int x = 0; x < S::TI; ++x)
#pragma unroll
      for (int y = 0; y < S::TJ; ++y) {
        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(by.a[0][x], by.b[0][y], acc[x][y], 0, 0, 0);
        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(by.a[0][x], by.b[1][y], acc[x][y], 0, 0, 0);
        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(by.a[1][x], by.b[0][y], acc[x][y], 0, 0, 0);
      }
  };

  // The operands of half a pass are read while the half before it is
  // multiplied. So at a pass's barrier all of its operands are in registers:
  // its buffer is free for the pass BUFFERS later, and the second half is
  // multiplied behind the barrier, while the next pass's first operands arrive.
  // The barrier waits for the next pass's loads only. The loads are spread
  // between the multiplications: issued at once, a pass's 64 hold the waves up
  // for a thousand cycles. Passes past the last load what follows in the
  // workspace, and nothing reads it.
  constexpr int NM = S::TI * S::TJ * 3, ND = 2 * (S::TI + S::TJ);
  const uint32_t passes = K / S::DEPTH;  // even, as K is padded to 64
  const auto pass = [&](f16x8* now, const f16x8* next) {
    read(now, 1, f[1]);
    multiply(f[0]);
    Spread<0, NM, 0, ND>::over();
    __builtin_amdgcn_sched_barrier(0);
    wait_and_meet<(S::BUFFERS - 2) * LN>();
    load(now);
    read(next, 0, f[0]);
    multiply(f[1]);
    Spread<0, NM, LN, ND>::over();
    __builtin_amdgcn_sched_barrier(0);
  };
  load(lds0);
  if constexpr (S::BUFFERS == 2) {
    load(lds1);
    wait_and_meet<LN>();
    read(lds0, 0, f[0]);
    for (uint32_t k = 0; k < passes; k += 2) {
      pass(lds0, lds1);
      pass(lds1, lds0);
    }
  } else {
    load(lds1);
    load(lds2);
    load(lds3);
    wait_and_meet<3 * LN>();
    read(lds0, 0, f[0]);
    uint32_t k = 0;
    for (; k + 4 <= passes; k += 4) {
      pass(lds0, lds1);
      pass(lds1, lds2);
      pass(lds2, lds3);
      pass(lds3, lds0);
      if constexpr (STAGES) {
        if (k % 8 == 4) stage();
      }
    }
    if (k < passes) {
      pass(lds0, lds1);
      pass(lds1, lds2);
    }
    if constexpr (STAGES) {
#pragma unroll
      for (int x = 0; x < S::TI; ++x)
#pragma unroll
        for (int y = 0; y < S::TJ; ++y)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[x][y][e] += total[x][y][e];
    }
  }

#pragma unroll
  for (int x = 0; x < S::TI; ++x)
#pragma unroll
    for (int y = 0; y < S::TJ; ++y)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[x][y][e] *= p.alpha;
  const auto add = [&](uint32_t buffer, int which, float by) {
#pragma unroll
    for (int y = 0; y < S::TJ; ++y) {
      Columns c;
      if constexpr (AHEAD) c = ahead[which][y];
      else load_c(plane(base, m, n, buffer), y, c);
#pragma unroll
      for (int x = 0; x < S::TI; ++x) {
        f16x4 hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          fours(c.hi[x][q], hi, q);
          fours(c.lo[x][q], lo, q);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          acc[x][y][e] = fmaf(by, (float)hi[e / 4][e % 4] + (float)lo[e / 4][e % 4], acc[x][y][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (p.beta != 0.0f) add(p.c_ji, 0, p.beta);
  if (p.gamma != 0.0f) add(p.c2, 1, p.gamma);

  // A wave turns its blocks of 32 x 32 through LDS: lane l stores row l / 2,
  // half l % 2, of the block's 32 rows of 32, 32 bytes at a time. The loads past
  // the last pass also end in LDS: every wave waits for its own before the
  // waves meet, so that none of them lands on another's turned blocks.
  wait_and_meet<0>();
  constexpr int PITCH = S::PITCH;
  uint32_t* turn = reinterpret_cast<uint32_t*>(lds0) + wid * 32 * PITCH;
  const uint32_t row = lane / 2, half = lane % 2 * 16;
  u32x4* put = reinterpret_cast<u32x4*>(turn + lane % 32 * PITCH + lane / 32 * 4);
  const u32x4* along = reinterpret_cast<const u32x4*>(turn + row * PITCH + half);
  const uint32_t* across = turn + half * PITCH + row;
  if constexpr (OUT == kPlanes) {
    const Plane dij = plane(base, m, n, p.d_ij), dji = plane(base, m, n, p.d_ji);
    const auto store = [&](const uint32_t (&w)[16], f16* hi) {
      f16x8 h[2], l[2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        h[e / 8][e % 8] = __builtin_bit_cast(f16, (uint16_t)w[e]);
        l[e / 8][e % 8] = __builtin_bit_cast(f16, (uint16_t)(w[e] >> 16));
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        reinterpret_cast<f16x8*>(hi)[q] = h[q];
        reinterpret_cast<f16x8*>(hi + kToLo)[q] = l[q];
      }
    };
#pragma unroll
    for (int x = 0; x < S::TI; ++x)
#pragma unroll
      for (int y = 0; y < S::TJ; ++y) {
        asm volatile("" : "+v"(acc[x][y]));  // not converted before its turn
        if (outside(x, y)) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = acc[x][y][q * 4 + e];
            const f16 h = (f16)v, l = (f16)fmaf((float)h, -1.0f, v);
            w[e] = (uint32_t)__builtin_bit_cast(uint16_t, h) | (uint32_t)__builtin_bit_cast(uint16_t, l) << 16;
          }
          put[q * 2] = w;
        }
        wave_fence();
        const uint32_t ix = i0 + wi + x * 32, jx = j0 + wj + y * 32;
        if (p.sym && ix < jx) continue;  // the mirror of another block
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) w[q * 4 + e] = along[q][e];
        if (p.sym && ix == jx) {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = half + e >= row ? w[e] : across[e * PITCH];
        }
        store(w, dji.hi(jx + row, ix + half));
        if (!(p.sym && ix == jx)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = across[e * PITCH];
          store(w, dij.hi(ix + row, jx + half));
        }
        wave_fence();  // before the next block's values
        __builtin_amdgcn_sched_barrier(0);
      }
  } else {
    constexpr int N = Pack<T>::N;
    const float move = mv.move * sqrtf(fmaxf(1.0f, (float)g.rows / (float)g.cols));
    T* o = out + g.at + it.k * (uint64_t)g.rows * g.cols;
#pragma unroll
    for (int x = 0; x < S::TI; ++x) {
      typename Pack<T>::V w[S::TJ][16 / N];
      T* at[S::TJ];
      int64_t room[S::TJ];
#pragma unroll
      for (int y = 0; y < S::TJ; ++y) {  // the result's rows are j where it is tall, else i
        const uint32_t ix = i0 + wi + x * 32, jx = j0 + wj + y * 32;
        const uint32_t r = (g.tall() ? jx : ix) + row, col = (g.tall() ? ix : jx) + half;
        at[y] = o + (uint64_t)r * g.cols + col;
        room[y] = r < g.rows && !outside(x, y) ? (int64_t)g.cols - col : 0;
#pragma unroll
        for (int q = 0; q < 16 / N; ++q)
          if (OUT == kWeight) w[y][q] = load_pack(at[y] + q * N, room[y] - q * N);
      }
#pragma unroll
      for (int y = 0; y < S::TJ; ++y) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(acc[x][y][q * 4 + e]);
          put[q * 2] = v;
        }
        wave_fence();
        float v[16];
        if (g.tall()) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(along[e / 4][e % 4]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(across[e * PITCH]);
        }
#pragma unroll
        for (int q = 0; q < 16 / N; ++q) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            w[y][q][e] = from_f32<T>(OUT == kWeight ? fmaf(mv.keep, to_f32((T)w[y][q][e]), -move * v[q * N + e])
                                                    : v[q * N + e]);
          store_pack(w[y][q], at[y] + q * N, room[y] - q * N);
        }
        wave_fence();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

// ---- matrices of a shorter side of at most 64 ---------------------------------
//
// One workgroup takes a matrix through all of its steps, two taken as one, so
// the chain of some twenty dependent products costs no launches. The square
// matrices stay in LDS (64 x 64, hi and lo). X passes by in blocks of 32
// columns, a block to a wave at a time, and never through LDS: the index that a
// product sums over may run in any order that both operands share, and in the
// order below the registers that hold a product's result are, once split into
// parts, the operand of the next one. That needs X the way P X leaves it (a
// lane holds rows of one column) for the next P X, and the way X^T P leaves it
// (columns of one row) for X X^T. Both are computed from the same operands,
// and a pass over X has no barrier but those of the last sum over the waves.
// Between passes only the first is kept (a workgroup has 100 GB/s to memory,
// which both would exhaust), in registers where a wave has one block only.
//
// Q = a I + M and P, the product of two steps' Q, are held whole: as P - a a I
// next to a a X they would cancel to a tenth of their size. The products of the
// lo parts are added up before those of the hi parts, whose sums round more.
//
// Bound by the chain: at 64 x 2048 (116 us) the matrix cores work a third of the
// time and the vector units two fifths, one after the other, since the waves
// keep step. 16 x 27 takes 14 us, 64 x 576 48 us, and 20 matrices of 16 x 16 ..
// 64 x 576 take 55 us, little more than the largest one.
constexpr int kSmallThreads = 512, kSmallWaves = kSmallThreads / kWave;
constexpr uint32_t kSmallSide = 64, kSmallLong = 2048, kSmallLong32 = 16384;
constexpr int kRow = 72;  // fp16 of a row in LDS: sixteen rows' 16-byte chunks fall into different banks

typedef float f32x4v __attribute__((ext_vector_type(4)));

// Blocks of 32 columns, each of 64 rows, fp32.
__host__ __device__ __forceinline__ uint64_t small_bytes(uint32_t n) { return (uint64_t)up(n, 32) * 64 * sizeof(float); }

// Where a row's k-th value lies: lane group g of 16 finds k = 4 g .. 4 g + 3 and
// 16 more, as two blocks of a result hold them, in 16 bytes.
__device__ __forceinline__ uint32_t pos_of(uint32_t k) {
  return (k & ~31u) | (k >> 2 & 3) << 3 | (k >> 4 & 1) << 2 | (k & 3);
}

// lo = v - hi in one instruction of mixed types, which the compiler takes for a
// product and a sum but not for a difference: it does not get to know the -1.
__device__ __forceinline__ void split4(f32x4v v, f16x4& hi, f16x4& lo) {
  float minus = -1.0f;
  asm("" : "+s"(minus));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = (f16)v[e];
    lo[e] = (f16)fmaf((float)hi[e], minus, v[e]);
  }
}
// Two of a result's blocks as an operand.
__device__ __forceinline__ void split8(f32x4v u, f32x4v v, f16x8& hi, f16x8& lo) {
  f16x4 h[2], l[2];
  split4(u, h[0], l[0]);
  split4(v, h[1], l[1]);
  hi = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
  lo = __builtin_shufflevector(l[0], l[1], 0, 1, 2, 3, 4, 5, 6, 7);
}
// Blocks of 16 x 16 of a row-major matrix from its first row r0 and column c0
// on: `along` holds 4 columns of a row, `down` 4 rows of a column. Inside the
// matrix the places are a base that the wave shares and a lane's offset; at its
// edges every load is made all the same, at a place inside.
template <class S>
struct Blocks16 {
  const S* x;
  uint32_t rows, cols, in, four;

  __device__ __forceinline__ f32x4v along(uint32_t r0, uint32_t c0, bool inside) const {
    f32x4v v;
    if (inside) {
      typedef S S4 __attribute__((ext_vector_type(4)));
      typedef S4 S4u __attribute__((aligned(sizeof(S))));
      const S4 w = *reinterpret_cast<const S4u*>(reinterpret_cast<const char*>(x + ((uint64_t)r0 * cols + c0)) +
                                                 (in * cols + four) * (uint32_t)sizeof(S));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = to_f32((S)w[e]);
      return v;
    }
    const uint32_t r = r0 + in, c = c0 + four;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = to_f32(x[(uint64_t)min(r, rows - 1) * cols + min(c + e, cols - 1)]);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r < rows && c + e < cols ? v[e] : 0.0f;
    return v;
  }
  __device__ __forceinline__ f32x4v down(uint32_t r0, uint32_t c0, bool inside) const {
    f32x4v v;
    if (inside) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = to_f32(*reinterpret_cast<const S*>(reinterpret_cast<const char*>(x + ((uint64_t)(r0 + e) * cols + c0)) +
                                                  (four * cols + in) * (uint32_t)sizeof(S)));
      return v;
    }
    const uint32_t r = r0 + four, c = c0 + in;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = to_f32(x[(uint64_t)min(r + e, rows - 1) * cols + min(c, cols - 1)]);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r + e < rows && c < cols ? v[e] : 0.0f;
    return v;
  }
};

typedef f16 Part[64 * kRow];
enum { kSqA, kSqM, kSqQ, kSqP, kSqP2, kSquares };
// Behind A, the waves' sums of X X^T take the place of the other squares.
struct SmallLds {
  static constexpr int kSums = kSmallWaves * 10 * kWave * (int)sizeof(f32x4v);
  static constexpr int kOthers = (kSquares - 1) * 2 * (int)sizeof(Part);
  __align__(16) unsigned char bytes[2 * sizeof(Part) + (kSums > kOthers ? kSums : kOthers)];
  double scratch[kSmallWaves];
};

// RB: blocks of 16 rows, 2 (a short side of up to 32) or 4.
template <int RB, int OUT, class S, class T>
__device__ __forceinline__ void small_steps(SmallLds& lds, const Group& g, uint32_t steps, float a, float b, float c,
                                            float eps, const S* x, f32x4v* kept, T* o, Move mv) {
  constexpr int kPairs = RB * (RB + 1) / 2;  // blocks of 16 x 16 on and below the diagonal
  constexpr int SL = RB / 2;                 // slabs of 32 of the index of rows
  Part(*const sq)[2] = reinterpret_cast<Part(*)[2]>(lds.bytes);
  f32x4v* const sums = reinterpret_cast<f32x4v*>(lds.bytes + 2 * sizeof(Part));
  const bool tall = g.tall();
  const uint32_t m = tall ? g.cols : g.rows, n = tall ? g.rows : g.cols, blocks = (n + 31) / 32;
  const uint32_t lane = lane_id(), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t in = lane % 16, four = lane / 16 * 4;  // a result's block: this lane's column, and its rows from there
  const bool held = blocks <= (uint32_t)kSmallWaves;  // a wave has one block at most: it stays in registers

  // A block of X: xu[c][b][e] at row 16 b + four + e, column 16 c + in.
  f32x4v xu[2][RB];
  const auto place = [&](uint32_t blk, int q) {  // a base that the wave shares, and a lane's offset
    return reinterpret_cast<f32x4v*>(reinterpret_cast<char*>(kept) + ((uint64_t)blk * 8 + q) * 1024 + lane * 16);
  };
  const auto keep = [&](uint32_t blk) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < RB; ++b) *place(blk, c * 4 + b) = xu[c][b];
  };
  const auto fetch = [&](uint32_t blk, f32x4v (&to)[2][RB]) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < RB; ++b) to[c][b] = *place(blk, c * 4 + b);
  };

  double sum = 0.0;
  const Blocks16<S> from{x, g.rows, g.cols, in, four};
  const auto load = [&](uint32_t blk, auto inside) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const uint32_t i0 = b * 16, j0 = blk * 32 + c * 16;
        xu[c][b] = tall ? from.along(j0, i0, inside()) : from.down(i0, j0, inside());
      }
  };
  for (uint32_t blk = wid; blk < blocks; blk += kSmallWaves) {
    if (m == RB * 16 && blk * 32 + 32 <= n) load(blk, std::true_type{});
    else load(blk, std::false_type{});
    if (!held) keep(blk);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double v = xu[c][b][e];
          sum = fma(v, v, sum);
        }
  }
  // v * by as v * 2^power * (hi + lo), whatever the update's magnitude
  const double by = (double)kScaleX / (sqrt(block_sum_f64<kSmallThreads>(sum, lds.scratch)) + (double)eps);
  int power;
  const double rest = frexp(by, &power);
  const float by_hi = (float)rest, by_lo = by_hi - by_hi == 0.0f ? (float)(rest - (double)by_hi) : 0.0f;
  const auto normalise = [&](f32x4v& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = ldexpf(v[e], power);
      v[e] = fmaf(w, by_hi, w * by_lo);
    }
  };
  // A block's parts, h and l, are the operand of P X and X^T P. Against the unit
  // matrix they give the block turned, exactly: columns 16 c + four + e of row
  // 16 b + in.
  f16x8 h[2][SL], l[2][SL], unit[2];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int t = 0; t < 8; ++t) unit[b][t] = t / 4 == b && four + t % 4 == in ? (f16)1.0f : (f16)0.0f;
  const auto split = [&] {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int s = 0; s < SL; ++s) split8(xu[c][2 * s], xu[c][2 * s + 1], h[c][s], l[c][s]);
  };
  const auto turned = [&](int b, int c) {
    f32x4v v = {};
    v = __builtin_amdgcn_mfma_f32_16x16x32_f16(h[c][b / 2], unit[b % 2], v, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(l[c][b / 2], unit[b % 2], v, 0, 0, 0);
  };

  // X X^T: block (b, q), q <= b, of this wave's columns, from their turned parts
  f32x4v gram[kPairs];
  f16x8 th[RB], tl[RB];
  const auto clear_gram = [&] {
#pragma unroll
    for (int t = 0; t < kPairs; ++t) gram[t] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
  };
  const auto add_to_gram = [&] {
    // a part at a time: a product waits for the one before it in the same block;
    // hi lo and lo hi first, whose sums' roundings are small
    f32x4v t[kPairs];
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int q = 0; q <= b; ++q) {
          f32x4v& to = t[b * (b + 1) / 2 + q];
          if (part == 0) to = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
          to = __builtin_amdgcn_mfma_f32_16x16x32_f16(part == 1 ? tl[b] : th[b], part == 0 ? tl[q] : th[q], to, 0, 0, 0);
        }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) gram[k] += t[k];
  };

  // Rows i .. i + 3 of column j of a symmetric matrix, those on and below the
  // diagonal, and their mirror.
  const auto put_symmetric = [&](Part (&to)[2], uint32_t i, uint32_t j, f32x4v v) {
    f16x4 hi, lo;
    split4(v, hi, lo);
    if (i >= j) {
      *reinterpret_cast<f16x4*>(&to[0][j * kRow + pos_of(i)]) = hi;
      *reinterpret_cast<f16x4*>(&to[1][j * kRow + pos_of(i)]) = lo;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e < j) continue;
      to[0][(i + e) * kRow + pos_of(j)] = hi[e];
      to[1][(i + e) * kRow + pos_of(j)] = lo[e];
      if (i < j) {
        to[0][j * kRow + pos_of(i + e)] = hi[e];
        to[1][j * kRow + pos_of(i + e)] = lo[e];
      }
    }
  };
  // A = X X^T of the waves' parts of it, in the order of the waves
  const auto join_gram = [&] {
    __syncthreads();  // the squares have been read
    const uint32_t waves = min(blocks, (uint32_t)kSmallWaves);
    if (wid < waves) {
#pragma unroll
      for (int t = 0; t < kPairs; ++t) sums[(wid * kPairs + t) * kWave + lane] = gram[t];
    }
    __syncthreads();
    for (uint32_t t = wid; t < (uint32_t)kPairs; t += kSmallWaves) {
      f32x4v v = sums[t * kWave + lane];
      for (uint32_t w = 1; w < waves; ++w) v += sums[(w * kPairs + t) * kWave + lane];
      uint32_t b, q;
      pair_at(t, b, q);
      put_symmetric(sq[kSqA], b * 16 + four, q * 16 + in, v * (1.0f / kScaleX));
    }
    __syncthreads();
  };

  // d = alpha l r + beta r + diagonal I, all symmetric: a wave takes the blocks on
  // and below the diagonal of (row bi, columns bj and bj + 1). Each is computed
  // both ways round, from the same operands and with the same roundings, so that
  // a lane writes four values of a row at once: the mirror written from one of
  // them, two bytes at a time, would take twice as long as all the rest.
  const uint32_t bi = wid / SL, bj = wid % SL * 2;
  const auto square = [&](int l, int r, int d, float alpha, float beta, float diagonal) {
    const uint32_t at = in * kRow + lane / 16 * 8;
    const auto operand = [&](int of, uint32_t blk, f16x8 (&h)[SL], f16x8 (&o)[SL]) {
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        h[s] = *reinterpret_cast<const f16x8*>(&sq[of][0][blk * 16 * kRow + at + s * 32]);
        o[s] = *reinterpret_cast<const f16x8*>(&sq[of][1][blk * 16 * kRow + at + s * 32]);
      }
    };
    if (bi < (uint32_t)RB && bj <= bi) {
      f16x8 lh[SL], ll[SL];
      operand(l, bi, lh, ll);
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // the second one may lie above the diagonal: computed, not stored
        const uint32_t i = bi * 16, j = (bj + q) * 16;
        const uint32_t down_at = (j + in) * kRow + pos_of(i + four), along_at = (i + in) * kRow + pos_of(j + four);
        const auto add = [&](int m, uint32_t of, float by, f32x4v to) {
          const f16x4 h = *reinterpret_cast<const f16x4*>(&sq[m][0][of]);
          const f16x4 o4 = *reinterpret_cast<const f16x4*>(&sq[m][1][of]);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = fmaf((float)h[e], by, fmaf((float)o4[e], by, to[e]));
          return to;
        };
        f16x8 rh[SL], rl[SL];
        operand(r, bj + q, rh, rl);
        f32x4v below = {}, above = {};  // rows i + four + e of column j + in, and row i + in's columns j + four + e
#pragma unroll
        for (int part = 0; part < 3; ++part)  // hi hi last, as above
#pragma unroll
          for (int s = 0; s < SL; ++s) {
            const f16x8 of_l = part == 1 ? ll[s] : lh[s], of_r = part == 0 ? rl[s] : rh[s];
            below = __builtin_amdgcn_mfma_f32_16x16x32_f16(of_l, of_r, below, 0, 0, 0);
            above = __builtin_amdgcn_mfma_f32_16x16x32_f16(of_r, of_l, above, 0, 0, 0);
          }
        f32x4v v = below * alpha, w = above * alpha;
        if (beta != 0.0f) {
          v = add(r, down_at, beta, v);
          w = add(r, along_at, beta, w);
        }
        if (i == j) {  // what lies above the diagonal from below it
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = in == four + e ? w[e] + diagonal : in > four + e ? w[e] : v[e];
        }
        f16x4 vh, vl, wh, wl;
        split4(v, vh, vl);
        split4(w, wh, wl);
        if (j < i) {
          *reinterpret_cast<f16x4*>(&sq[d][0][down_at]) = vh;
          *reinterpret_cast<f16x4*>(&sq[d][1][down_at]) = vl;
        }
        if (j <= i) {
          *reinterpret_cast<f16x4*>(&sq[d][0][along_at]) = wh;
          *reinterpret_cast<f16x4*>(&sq[d][1][along_at]) = wl;
        }
      }
    }
    __syncthreads();
  };

  clear_gram();
  f32x4v next[2][RB];
  if (!held && wid < blocks) fetch(wid, next);
  for (uint32_t blk = wid; blk < blocks; blk += kSmallWaves) {
    if (!held) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int b = 0; b < RB; ++b) xu[c][b] = next[c][b];
      if (blk + kSmallWaves < blocks) fetch(blk + kSmallWaves, next);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < RB; ++b) normalise(xu[c][b]);
    split();
#pragma unroll
    for (int b = 0; b < RB; ++b) split8(turned(b, 0), turned(b, 1), th[b], tl[b]);
    add_to_gram();
  }
  join_gram();
  const float to_m = kScaleM / kScaleX;
  // The smallest matrices take as long one step at a time, and come out nearer.
  const uint32_t together = RB == 2 && held ? 1 : 2;
  for (uint32_t done = 0; done < steps; done += together) {
    const bool pair = together == 2 && done + 1 < steps, last = done + together >= steps;
    // P, the product of the one or two steps' Q = a I + b A + c A A
    square(kSqA, kSqA, kSqP, c * to_m / kScaleX, b * to_m, a * kScaleM);
    if (pair) {
      square(kSqP, kSqA, kSqQ, 1.0f / kScaleM, 0.0f, 0.0f);
      square(kSqP, kSqQ, kSqA, 1.0f / kScaleM, 0.0f, 0.0f);
      square(kSqA, kSqA, kSqM, c * to_m / kScaleX, b * to_m, a * kScaleM);
      square(kSqM, kSqP, kSqP2, 1.0f / kScaleM, 0.0f, 0.0f);
    }
    const Part(&p)[2] = sq[pair ? kSqP2 : kSqP];
    // P X in xu and X^T P, its columns 16 c + four + e of row 16 b + in, in xt
    f32x4v xt[2][RB];
    const auto move_block = [&](auto want_u, auto want_t) {
      split();
      uint32_t at = in * kRow + lane / 16 * 8;
      asm volatile("" : "+v"(at));  // P is read for every block: its 64 registers are not there to hold it
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        f16x8 ph[SL], pl[SL];
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          ph[s] = *reinterpret_cast<const f16x8*>(&p[0][at + b * 16 * kRow + s * 32]);
          pl[s] = *reinterpret_cast<const f16x8*>(&p[1][at + b * 16 * kRow + s * 32]);
        }
        f32x4v u[2] = {}, t[2] = {};
        // up to four chains of products side by side
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int s = 0; s < SL; ++s)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const f16x8 of_p = part == 1 ? pl[s] : ph[s], of_x = part == 0 ? l[c][s] : h[c][s];
              if (want_u()) u[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(of_p, of_x, u[c], 0, 0, 0);
              if (want_t()) t[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(of_x, of_p, t[c], 0, 0, 0);
            }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (want_u()) xu[c][b] = u[c] * (1.0f / kScaleM);
          if (want_t()) xt[c][b] = t[c] * (1.0f / kScaleM);
        }
        if (want_u() && want_t()) split8(xt[0][b], xt[1][b], th[b], tl[b]);
      }
    };
    constexpr std::true_type yes;
    constexpr std::false_type no;
    clear_gram();
    if (!held && wid < blocks) fetch(wid, next);
    for (uint32_t blk = wid; blk < blocks; blk += kSmallWaves) {
      if (!held) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int b = 0; b < RB; ++b) xu[c][b] = next[c][b];
        if (blk + kSmallWaves < blocks) fetch(blk + kSmallWaves, next);
        if (done == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int b = 0; b < RB; ++b) normalise(xu[c][b]);
        }
      }
      if (!last) {
        move_block(yes, yes);
        if (!held) keep(blk);
        add_to_gram();
        continue;
      }
      if (tall) move_block(yes, no);
      else move_block(no, yes);
      const float move = mv.move * sqrtf(fmaxf(1.0f, (float)g.rows / (float)g.cols));
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const uint32_t i0 = b * 16, j0 = blk * 32 + c * 16;
          const uint32_t r = (tall ? j0 : i0) + in, col = (tall ? i0 : j0) + four;
          if (r >= g.rows) continue;
          T* at = o + (uint64_t)r * g.cols + col;
          const f32x4v v = (tall ? xu[c][b] : xt[c][b]) * (1.0f / kScaleX);
          typedef T T4 __attribute__((ext_vector_type(4)));
          typedef T4 T4u __attribute__((aligned(sizeof(T))));
          if (col + 4 <= g.cols) {
            T4 w = {};
            if (OUT == kWeight) w = *reinterpret_cast<const T4u*>(at);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = from_f32<T>(OUT == kWeight ? fmaf(mv.keep, to_f32((T)w[e]), -move * v[e]) : v[e]);
            *reinterpret_cast<T4u*>(at) = w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (col + e < g.cols)
                at[e] = from_f32<T>(OUT == kWeight ? fmaf(mv.keep, to_f32(at[e]), -move * v[e]) : v[e]);
          }
        }
    }
    if (!last) join_gram();
  }
}

template <int OUT, class S, class T>
__global__ __launch_bounds__(kSmallThreads) void k_small(Groups gs, uint32_t steps, float a, float b, float c, float eps,
                                                         const S* update, unsigned char* ws, T* out, Move mv) {
  __shared__ SmallLds lds;
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  if (it.k >= g.count) return;
  const uint64_t at = g.at + it.k * (uint64_t)g.rows * g.cols;
  f32x4v* kept = reinterpret_cast<f32x4v*>(ws + g.ws + it.k * g.ws_of);
  if (min(g.rows, g.cols) <= 32) small_steps<2, OUT>(lds, g, steps, a, b, c, eps, update + at, kept, out + at, mv);
  else small_steps<4, OUT>(lds, g, steps, a, b, c, eps, update + at, kept, out + at, mv);
}

// No steps: the normalised update itself.
template <int OUT, class S, class T>
__global__ __launch_bounds__(kThreads) void k_normalised(Groups gs, const S* update, float eps, unsigned char* ws,
                                                         T* out, Move mv) {
  __shared__ double scratch[kThreads / kWave];
  const Item it = item_of(gs, blockIdx.x);
  const Group& g = gs.g[it.g];
  if (it.k >= g.count) return;
  const uint64_t size = (uint64_t)g.rows * g.cols, each = (size + g.tiles - 1) / g.tiles;
  const double* part = reinterpret_cast<const double*>(ws + g.ws + it.k * g.ws_of);
  const double sum = sum_of_parts(part, g.tiles, scratch);
  // an infinite norm would leave zeros beside the infinities: no direction is left, so all are NaN
  const double by = isinf(sum) ? (double)NAN : 1.0 / (sqrt(sum) + (double)eps);
  const float move = mv.move * sqrtf(fmaxf(1.0f, (float)g.rows / (float)g.cols));
  const uint64_t begin = it.tile * each, end = min(begin + each, size), at = g.at + it.k * size;
  for (uint64_t i = at + begin + threadIdx.x; i < at + end; i += kThreads) {
    const float v = (float)((double)to_f32(update[i]) * by);
    out[i] = from_f32<T>(OUT == kWeight ? fmaf(mv.keep, to_f32(out[i]), -move * v) : v);
  }
}

// The kinds of matrices: those that one workgroup takes through its steps, up
// to where the chip's other CUs are nearly as fast (64 x 2048: 116 us, against
// 128 by products over all CUs; 32 x 16384: 361 against 492), and by the shorter side
// the narrow and the wide ones, whose steps are paired or not on their own.
enum Kind { kSmall, kNarrow, kWide, kKinds };
Kind kind_of(uint32_t rows, uint32_t cols) {
  const uint32_t m = std::min(rows, cols), n = std::max(rows, cols);
  return m <= kSmallSide && n <= (m <= 32 ? kSmallLong32 : kSmallLong) ? kSmall : m <= 128 ? kNarrow : kWide;
}

// Cuts the matrices of one kind into groups of equal ones that follow each
// other, and lays their buffers out in the workspace from `used` on. Calls
// f(groups) for every kGroups of them; returns the workspace's new end.
template <class F>
uint64_t for_groups(const OrthoMatrices& ms, Kind kind, uint64_t used, F&& f) {
  Groups gs = {};
  for (uint32_t k = 0; k < ms.count; ++k) {
    const uint32_t rows = ms.rows[k], cols = ms.cols[k];
    if (rows == 0 || cols == 0 || kind_of(rows, cols) != kind) continue;
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
    g.ws_of = kind == kSmall ? small_bytes(g.n()) : buffers_bytes(g.m(), g.n());
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
    all += items_of(gs.g[k]);
  }
  return (uint32_t)all;
}
uint32_t parts_of_host(const Group& g) {
  return (uint32_t)std::min<uint64_t>(((uint64_t)g.rows * g.cols + 8191) / 8192, kParts);
}

template <int OUT, class T>
hipError_t launch_product(Groups& gs, const Product& p, unsigned char* ws, T* out, Move mv, hipStream_t stream) {
  using Large = Shape<2, 4, 4, 2, 2>;  // 256 x 256, 8 waves
  using Small = Shape<2, 2, 2, 2, 4>;  // 128 x 128, 4 waves
  using Tiny = Shape<2, 2, 1, 1, 4>;   // 64 x 64, 4 waves
  const auto tiles = [&](uint32_t side) {
    uint64_t all = 0;
    for (uint32_t k = 0; k < gs.count; ++k)
      all += (uint64_t)gs.g[k].count * tiles_by(gs.g[k].m(), gs.g[k].n(), p.sym, side);
    return all;
  };
  const auto launch = [&](auto shape) {
    using S = decltype(shape);
    static_assert(S::I == S::J, "square tiles");
    const uint32_t blocks = tiled(gs, [&](const Group& g) { return tiles_by(g.m(), g.n(), p.sym, S::I); });
    hipLaunchKernelGGL((k_product<S, OUT, T>), dim3(blocks), dim3(S::NT), 0, stream, gs, p, ws, out, mv);
    return hipGetLastError();
  };
  switch (tile_side(tiles(64), tiles(128), tiles(256))) {
    case 64: return launch(Tiny{});
    case 128: return launch(Small{});
    default: return launch(Large{});
  }
}

// One step, or two taken as one: with A = X X^T, Q = a I + M, M = b A + c A A,
// the next step's A is Q A Q = Q (Q A) (they commute, so both products are
// symmetric) and X moves once, by the product of the two Q. That trades two of
// X's products (3 m m n) for three halves more of m x m ones and keeps the
// accuracy; at three (2e-6 .. 6e-6 of the norm where one and two leave 4e-7 ..
// 1.2e-6) A's small singular values begin to be lost beside its large ones.
//
// Every product takes both parts of its operands, whatever the result's type.
// The error that single fp16 products (a third of the multiplications) leave in
// a step is a matter of the spectrum: with two of five steps in both parts it
// was 8e-4 of the norm for noise, 1.5e-3 for noise thinned to 0.5%, 4e-5 for
// noise with a few strong directions, where fp16's rounding is 2.1e-4; four of
// five still left 1.5e-4 where rows differ in size.
//
// Operations of `steps` steps with or without pairs, and what their launches
// cost in operations: about 5 us each at 5e14 a second.
double steps_cost(uint32_t steps, bool paired, const Groups& gs) {
  double all = 0.0;
  for (uint32_t done = 0; done < steps; done += paired ? 2 : 1) {
    const double squares = paired && done + 1 < steps ? 5 : 1;
    for (uint32_t j = 0; j < gs.count; ++j) {
      const double m = gs.g[j].m(), n = gs.g[j].n();
      all += gs.g[j].count * 3 * m * m * (3 * n + squares * m);
    }
    all += 2.5e9 * (2 + squares);
  }
  return all;
}

template <int OUT, class S, class T>
hipError_t run(Groups& gs, Kind kind, const OrthoSteps& s, const S* update, T* out, Move mv,
               unsigned char* ws, hipStream_t stream) {
  if (kind == kSmall && s.steps > 0) {
    const uint32_t blocks = tiled(gs, [](const Group&) { return 1u; });
    hipLaunchKernelGGL((k_small<OUT, S, T>), dim3(blocks), dim3(kSmallThreads), 0, stream, gs, s.steps, s.a, s.b, s.c,
                       s.eps, update, ws, out, mv);
    return hipGetLastError();
  }
  // the longest sums first, so that they do not start when the others end
  std::sort(gs.g, gs.g + gs.count, [](const Group& x, const Group& y) { return x.n() > y.n(); });
  uint32_t blocks = tiled(gs, parts_of_host);
  hipLaunchKernelGGL(k_squares<S>, dim3(blocks), dim3(kThreads), 0, stream, gs, update, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (s.steps == 0) {
    hipLaunchKernelGGL((k_normalised<OUT, S, T>), dim3(blocks), dim3(kThreads), 0, stream, gs, update, s.eps, ws, out,
                       mv);
    return hipGetLastError();
  }
  const bool paired = steps_cost(s.steps, true, gs) < steps_cost(s.steps, false, gs);
  blocks = tiled(gs, [](const Group& g) { return g.m() / 64 * (g.n() / 64); });
  hipLaunchKernelGGL(k_split<S>, dim3(blocks), dim3(kThreads), 0, stream, gs, update, s.eps, ws);
  e = hipGetLastError();

  // symmetric: D = alpha * A B + beta * B + gamma * C2
  const auto square = [&](uint32_t a, uint32_t b, uint32_t c2, uint32_t d, float alpha, float beta, float gamma) {
    if (e == hipSuccess)
      e = launch_product<kPlanes, float>(gs, Product{a, b, b, c2, d, d, 1, alpha, beta, gamma}, ws, nullptr, mv, stream);
  };
  const float to_m = kScaleM / kScaleX;
  uint32_t x = kX0, y = kX1;  // X and the next
  for (uint32_t done = 0; done < s.steps;) {
    square(x, x, x, kA, 1.0f / kScaleX, 0.0f, 0.0f);
    square(kA, kA, kA, kP, s.c * to_m / kScaleX, s.b * to_m, 0.0f);
    uint32_t pp = kP;  // P - p0 I
    float p0 = s.a;
    ++done;
    if (paired && done < s.steps) {
      square(kP, kA, kA, kT, 1.0f / kScaleM, s.a, 0.0f);
      square(kP, kT, kT, kA, 1.0f / kScaleM, s.a, 0.0f);  // the next step's A
      square(kA, kA, kA, kM, s.c * to_m / kScaleX, s.b * to_m, 0.0f);
      square(kM, kP, kM, kP2, 1.0f / kScaleM, s.a, p0);  // (a I + M) (p0 I + P)
      pp = kP2;
      p0 *= s.a;
      ++done;
    }
    const bool last = done == s.steps;
    const float unit = last ? 1.0f / kScaleX : 1.0f;
    const Product px{pp, x + 1, x + 1, x, y, y + 1, 0, unit / kScaleM, unit * p0, 0.0f};
    if (e == hipSuccess)
      e = last ? launch_product<OUT, T>(gs, px, ws, out, mv, stream)
               : launch_product<kPlanes, float>(gs, px, ws, nullptr, mv, stream);
    std::swap(x, y);
  }
  return e;
}

}  // namespace

uint64_t ortho_tiles(uint64_t rows, uint64_t cols) {
  const uint64_t m = std::min(rows, cols), n = std::max(rows, cols);
  if (m > (1u << 16) || n > (1u << 21) || m * n > (1ull << 32)) return 0;
  return (m + 63) / 64 * ((n + 63) / 64);
}

size_t ortho_workspace_bytes(const OrthoMatrices& ms) {
  uint64_t used = 0;
  for (int kind = 0; kind < kKinds; ++kind) used = for_groups(ms, (Kind)kind, used, [](Groups&) {});
  return (size_t)used + 1024;  // passes past the last load up to 512 bytes past a buffer
}

hipError_t ortho_launch(const OrthoMatrices& ms, const OrthoSteps& steps, uint32_t update_type, const void* update,
                        uint32_t out_type, void* out, bool is_weight, float keep, float move, void* ws,
                        hipStream_t stream) {
  hipError_t e = hipSuccess;
  const Move mv{keep, move};
  uint64_t used = 0;
  for (int kind = 0; kind < kKinds; ++kind)
    used = for_groups(ms, (Kind)kind, used, [&](Groups& gs) {
      if (e != hipSuccess) return;
      e = for_type(update_type, [&](auto s) {
        return for_type(out_type, [&](auto t) {
          using S = decltype(s);
          using T = decltype(t);
          unsigned char* w = static_cast<unsigned char*>(ws);
          return is_weight
                     ? run<kWeight, S, T>(gs, (Kind)kind, steps, (const S*)update, (T*)out, mv, w, stream)
                     : run<kResult, S, T>(gs, (Kind)kind, steps, (const S*)update, (T*)out, mv, w, stream);
        });
      });
    });
  return e;
}

}  // namespace sparcml
