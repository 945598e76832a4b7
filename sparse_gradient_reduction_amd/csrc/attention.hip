// Attention forward and backward, on the matrix cores.
//
//   forward   s = scale q k^T over the keys seen, lse = log sum exp s,
//             out = exp(s - lse) v
//   backward  p = exp(s - lse), ds = p (dout v^T - sum dout out)
//             dv = p^T dout, dq = scale ds k, dk = scale ds^T q
//
// One pass over the keys (forward, dq) or the queries (dk and dv), with tiles
// of probabilities that stay in registers. A product's 32 x 32 result leaves a
// lane one column and 16 rows, which is what the next product wants of its
// right operand (the summed index runs in the same order on both sides), so
// scores are computed turned: keys are rows and queries columns where the next
// sum is over keys, the other way round where it is over queries. A row's
// maximum, sum and rescaling are then one lane's, but for one exchange between
// the two halves of a wave.
//
// The tiles that are walked over go from memory to LDS without passing through
// registers, one tile ahead, in an order in which neither the rows (the first
// product) nor the columns (the second, read turned) meet in a bank.
//
// The query heads that share a key and value head are rows of one tile, so that
// its keys and values are loaded once for all of them, and dk and dv are summed
// over them on the way.
#include <algorithm>
#include <type_traits>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

typedef sparcml_attention_args Args;
typedef float Acc __attribute__((ext_vector_type(16)));
typedef int I4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A sequence's own lengths; query i's place among the keys is i + m - n.
struct Sequence {
  int n, m, before, after;
  __device__ __forceinline__ Sequence(const Args& a, uint32_t b) {
    n = a.queries, m = a.keys;
    if (a.q_lengths) n = min(max(a.q_lengths[b], 0), n);
    if (a.k_lengths) m = min(max(a.k_lengths[b], 0), m);
    before = min(a.before, 1u << 30), after = min(a.after, 1u << 30);
  }
  __device__ __forceinline__ int first(int i) const { return max(0, i + m - n - before); }
  __device__ __forceinline__ int last(int i) const { return min(m - 1, i + m - n + after); }
};

template <class T>
__device__ __forceinline__ T* at(const sparcml_heads& x, uint64_t b, uint64_t t, uint64_t h) {
  return static_cast<T*>(x.data) + b * x.batch + t * x.token + h * x.head;
}

// ---- the matrix instructions --------------------------------------------------
// A Frag is a lane's 16 bytes of an operand. Of a left operand's row or a right
// operand's column (lane % 32), half h = lane / 32 of the wave holds, of step s
// of STEP summed indices,
//   16-bit   16 s + 8 h + 0..7, where rows are read along the head, or
//            16 s + 4 h + 0..3 and 16 s + 8 + 4 h + 0..3, as results leave them
//   fp32     8 s + 4 h + 0..3 in both cases, taken one by one.
// A result's lane has column lane % 32 and rows 8 (r / 4) + 4 h + r % 4.
template <class T>
struct Mma {
  static constexpr int STEP = 16;
  typedef T Frag __attribute__((ext_vector_type(8)));
  typedef T Four __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ Acc mul(Frag a, Frag b, Acc c);
  // rows s * STEP .. of a result, as a right operand
  static __device__ __forceinline__ Frag frag(const Acc& p, int s) {
    Frag f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = from_f32<T>(p[8 * s + j]);
    return f;
  }
};
template <>
__device__ __forceinline__ Acc Mma<bf16>::mul(Frag a, Frag b, Acc c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ Acc Mma<f16>::mul(Frag a, Frag b, Acc c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
template <>
struct Mma<float> {
  static constexpr int STEP = 8;
  typedef float Frag __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ Acc mul(Frag a, Frag b, Acc c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag frag(const Acc& p, int s) {
    return Frag{p[4 * s], p[4 * s + 1], p[4 * s + 2], p[4 * s + 3]};
  }
};

// ---- tiles in LDS ---------------------------------------------------------------
// ROWS heads of DP elements, 16-byte chunks, W elements a row; the chunks of a
// row are exchanged in an order that differs between the rows that are read at
// once: 8 rows' chunk c (a 16-byte read of 8 lanes) and 4 rows' 32 bytes (a
// turned read of 16 lanes) are in different banks.
template <class T, int DP, int ROWS_>
struct Tile {
  typedef Mma<T> M;
  typedef typename M::Frag Frag;
  static constexpr int ROWS = ROWS_, W = DP <= 64 ? 64 : 128, CH = W * (int)sizeof(T) / 16, SIZE = ROWS * CH;
  static constexpr int STEPS = DP / M::STEP, PACK = 16 / (int)sizeof(T);

  static __device__ __forceinline__ int order(int row) { return CH == 8 ? (row >> 1 & 3) << 1 : (row & 7) << 1; }

  // step s of row `base` + lane % 32 (base a multiple of 32)
  static __device__ __forceinline__ Frag row(const I4* lds, int base, int s) {
    const int r = lane_id() % 32, h = lane_id() / 32;
    return __builtin_bit_cast(Frag, lds[(base + r) * CH + ((2 * s + h) ^ order(r))]);
  }
  // column 32 t + lane % 32 of rows base + s * STEP .. (base a multiple of 32)
  static __device__ __forceinline__ Frag column(const I4* lds, int base, int s, int t) {
    const int lane = lane_id(), h = lane / 32;
    if constexpr (sizeof(T) == 2) {
      typedef short S4 __attribute__((ext_vector_type(4)));
      const int i = lane % 16, r = 4 * h + i / 4, c = 4 * t + lane / 16 % 2 * 2 + i % 4 / 2;
      typedef __attribute__((address_space(3))) S4 L;
      const char* p = reinterpret_cast<const char*>(lds + (base + 16 * s + r) * CH + (c ^ order(r))) + i % 2 * 8;
      const S4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p);
      const S4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p + 8 * CH * 16));
      return __builtin_bit_cast(Frag, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      Frag f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * h + j, d = 32 * t + lane % 32;
        f[j] = reinterpret_cast<const float*>(lds + (base + 8 * s + r) * CH + (d / 4 ^ order(r)))[d % 4];
      }
      return f;
    }
  }
};

// The rows of a tile: `ip` queries with `hp` of the heads that share a key and
// value head, row r being query r / hp and head r % hp. `nh` tiles take all of
// a query's heads: hp divides them.
struct Packing {
  uint32_t hp, ip, nh;
};


// Waits for this wave's loads and LDS accesses, then for the workgroup's other
// waves to be there too.
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt 0, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Loads of a tile's rows by NT threads, 16 bytes a thread at a time. What is
// not there (past a head's end, past the last query or key) becomes 0 and is
// not read. DIRECT: memory to LDS, for heads on 16-byte borders whose rows are
// within 2^31 bytes of the tile's first; otherwise through registers.
template <class T, class TL, int NT, bool DIRECT>
struct Loader {
  static constexpr int N = TL::SIZE / NT;
  static_assert(TL::SIZE % NT == 0, "whole chunks to a thread");
  static constexpr int kNothing = 0x7FFFFFF0;  // past the records
  int offset[N], query[N];  // bytes from the tile's first row; its query, past all of them where it is never there
  uint64_t token, head;
  uint32_t hp, dim;

  __device__ __forceinline__ Loader(const sparcml_heads& x, const Packing& pk, uint32_t dim_)
      : token(x.token), head(x.head), hp(pk.hp), dim(dim_) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t c = k * NT + threadIdx.x, row = c / TL::CH, i = row / pk.hp, h = row % pk.hp;
      const uint32_t e = (c % TL::CH ^ TL::order(row)) * TL::PACK;
      query[k] = i < pk.ip && e < dim ? (int)i : 1 << 30;
      offset[k] = DIRECT ? (int)((i * token + h * head + e) * sizeof(T)) : (int)(h << 8 | e);
    }
  }
  // the queries or keys from .. to - 1, counted from the tile's first one
  __device__ __forceinline__ void load(const T* base, int from, int to, I4* lds) const {
    if constexpr (DIRECT) {
#if __HIP_DEVICE_COMPILE__  // the host's pass has no such type, and would leave the kernel out
      const auto memory = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, kNothing, 0x00027000);
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
#pragma unroll
      for (int k = 0; k < N; ++k)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            memory, (__attribute__((address_space(3))) void*)(lds + k * NT + wave * kWave), 16,
            query[k] >= from && query[k] < to ? offset[k] : kNothing, 0, 0, 0);
#endif
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        typename Pack<T>::V v = {};
        const int e = offset[k] & 255;
        if (query[k] >= from && query[k] < to) v = load_pack(base + query[k] * token + (offset[k] >> 8) * head + e, (int64_t)dim - e);
        lds[k * NT + threadIdx.x] = __builtin_bit_cast(I4, v);
      }
    }
  }
};

__device__ __forceinline__ float both_halves_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_halves_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A lane's row (lane % 32 of its wave's 32) of a tile of queries, and what the
// wave and the workgroup see.
template <int NW>
struct Rows {
  int i, head;            // the query and its head
  bool there, live;       // in the batch; within the sequence, and sees a key
  int lo;                 // keys seen: lo .. lo + span
  uint32_t span;
  int wave_first, wave_last;  // some row of the wave sees these
  int wave_all_first, wave_all_last;  // all live rows see what lies between
  int first, last;        // some row of the workgroup sees these; last < first: none does
  __device__ __forceinline__ Rows(const Args& a, const Sequence& s, const Packing& pk, uint32_t tile, uint32_t g) {
    const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t r = wid * 32 + lane_id() % 32, q = r / pk.hp;
    const int i0 = tile / pk.nh * pk.ip;
    i = i0 + q, head = g * (a.heads / a.groups) + tile % pk.nh * pk.hp + r % pk.hp;
    there = q < pk.ip && i < (int)a.queries;
    lo = s.first(i), span = s.last(i) - lo;
    live = there && i < s.n && (int)span >= 0;
    if (!live) lo = 1 << 30, span = 0;
    const int w0 = i0 + wid * 32 / pk.hp, w1 = min(i0 + (int)min(pk.ip - 1, (wid * 32 + 31) / pk.hp), s.n - 1);
    const int i1 = min(i0 + (int)pk.ip, s.n) - 1;
    wave_first = s.first(w0), wave_last = w0 <= w1 ? s.last(w1) : -1;
    wave_all_first = s.first(w1), wave_all_last = s.last(w0);
    first = s.first(i0), last = i0 <= i1 ? s.last(i1) : -1;
  }
};

// a row of a head, 16 bytes of it to a Frag; 0 past its end
template <class T, class TL>
__device__ __forceinline__ void load_row(typename TL::Frag (&f)[TL::STEPS], const T* p, bool there, uint32_t dim) {
#pragma unroll
  for (int s = 0; s < TL::STEPS; ++s) {
    const int e = (2 * s + lane_id() / 32) * TL::PACK;
    f[s] = __builtin_bit_cast(typename TL::Frag, load_pack(p + e, there ? (int64_t)dim - e : 0));
  }
}

// A turned result's column to a row in memory.
template <class T, int DP>
__device__ __forceinline__ void store_row(const Acc (&acc)[DP / 32], float by, T* p, uint32_t dim) {
  typedef T Four __attribute__((ext_vector_type(4)));
  typedef Four Any __attribute__((aligned(sizeof(T))));
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t e = 32 * t + 8 * q + 4 * (lane_id() / 32);
      Four v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = from_f32<T>(acc[t][4 * q + j] * by);
      if (e + 4 <= dim) {
        *reinterpret_cast<Any*>(p + e) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (e + j < dim) p[e + j] = v[j];
      }
    }
}

constexpr int kKeys = 64;  // keys of a tile, 16-bit; 32 with fp32
template <class T>
constexpr int keys_of() { return sizeof(T) == 2 ? kKeys : kKeys / 2; }

// ---- forward --------------------------------------------------------------------
template <class T, int DP, int NW, bool DIRECT>
__global__ __launch_bounds__(NW * kWave, (sizeof(T) == 4 && DP > 64 ? 1 : 2)) void k_attention(Args a, Packing pk, uint32_t tiles) {
  constexpr int BN = keys_of<T>(), NT = NW * kWave;
  typedef Tile<T, DP, BN> TL;
  typedef Mma<T> M;
  __shared__ I4 k0[TL::SIZE], v0[TL::SIZE], k1[TL::SIZE], v1[TL::SIZE];
  const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), bg = id / tiles, tile = tiles - 1 - id % tiles;
  const uint32_t b = bg / a.groups, g = bg % a.groups;
  const Sequence s(a, b);
  const Rows<NW> rows(a, s, pk, tile, g);
  const float c = a.scale * kLog2e;

  typename TL::Frag q[TL::STEPS];
  load_row<T, TL>(q, at<T>(a.q, b, rows.i, rows.head), rows.live, a.dim);
  Acc o[DP / 32] = {};
  float top = -INFINITY, sum = 0.0f;

  const Packing one{1, BN, 1};
  const Loader<T, TL, NT, DIRECT> lk(a.k, one, a.dim), lv(a.v, one, a.dim);
  const T *ks = at<T>(a.k, b, 0, g), *vs = at<T>(a.v, b, 0, g);
  const auto load = [&](int j, I4* kt, I4* vt) {
    lk.load(ks + j * a.k.token, 0, rows.last + 1 - j, kt);
    lv.load(vs + j * a.v.token, 0, rows.last + 1 - j, vt);
  };
  const auto pass = [&](int j, const I4* kt, const I4* vt, I4* kn, I4* vn) {
    wait_and_meet();
    if (j + BN <= rows.last) load(j + BN, kn, vn);
    if (j > rows.wave_last || j + BN - 1 < rows.wave_first) return;
    Acc p[BN / 32] = {};
#pragma unroll
    for (int t = 0; t < BN / 32; ++t)
#pragma unroll
      for (int x = 0; x < TL::STEPS; ++x) p[t] = M::mul(TL::row(kt, 32 * t, x), q[x], p[t]);
    if (j < rows.wave_all_first || j + BN - 1 > rows.wave_all_last) {
      const uint32_t from = j + 4 * (lane_id() / 32) - rows.lo;
#pragma unroll
      for (int t = 0; t < BN / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) p[t][r] = from + (32 * t + 8 * (r / 4) + r % 4) > rows.span ? -INFINITY : p[t][r];
    }
    float now = p[0][0];
#pragma unroll
    for (int t = 0; t < BN / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) now = fmaxf(now, p[t][r]);
    now = both_halves_max(now) * c;
    if (ballot(now > top + 8.0f)) {
      const float higher = fmaxf(now, top), keep = higher == top ? 1.0f : __builtin_amdgcn_exp2f(top - higher);
      top = higher;
      sum *= keep;
#pragma unroll
      for (int t = 0; t < DP / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] *= keep;
    }
    const float off = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int t = 0; t < BN / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        p[t][r] = __builtin_amdgcn_exp2f(fmaf(p[t][r], c, -off));
        sum += p[t][r];
      }
#pragma unroll
    for (int t = 0; t < BN / 32; ++t)
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const typename TL::Frag f = M::frag(p[t], x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) o[y] = M::mul(TL::column(vt, 32 * t, x, y), f, o[y]);
      }
  };
  if (rows.first <= rows.last) load(rows.first, k0, v0);
  for (int j = rows.first; j <= rows.last; j += 2 * BN) {
    pass(j, k0, v0, k1, v1);
    if (j + BN <= rows.last) pass(j + BN, k1, v1, k0, v0);
  }
  sum = rows.live ? both_halves_sum(sum) : 0.0f;
  if (!rows.there) return;
  store_row<T, DP>(o, sum == 0.0f ? 0.0f : 1.0f / sum, at<T>(a.out, b, rows.i, rows.head), a.dim);
  if (lane_id() < 32) a.lse[((uint64_t)b * a.heads + rows.head) * a.queries + rows.i] = sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
}

// ---- backward -------------------------------------------------------------------
// fp16 has 40 binary digits from its smallest to its largest value, fewer than
// probabilities of long rows and ds of small gradients take. So p is held 2^14
// times as large, and ds, which is at most 2 p |dout| |v|, 2^14 f times, f the
// power of two that brings the largest |dout| |v| of a key and value head of a
// sequence to 1/2 .. 1: at most 2^15, and no other digits are lost than those of
// values 2^-25 times as large. bf16 has fp32's range, f and both factors are 1.
template <class T>
constexpr float kBoost = sizeof(T) == 2 && std::is_same<T, f16>::value ? 14.0f : 0.0f;  // as an exponent

// The largest sum of squares of a row of dout and of v, of one of kNormParts
// parts of the rows of each sequence's key and value head.
constexpr int kNormParts = 64;
template <class T>
__global__ __launch_bounds__(4 * kWave) void k_attention_norms(Args a, float* norms) {
  __shared__ float most[2][4];
  const uint32_t bg = blockIdx.x / kNormParts, part = blockIdx.x % kNormParts;
  const uint32_t b = bg / a.groups, g = bg % a.groups, each = a.heads / a.groups;
  const Sequence s(a, b);
  const uint32_t seeing = max(0, s.n - s.m - s.after), in = threadIdx.x % 16 * Pack<T>::N;
  const uint64_t rows[2] = {(uint64_t)max(0, s.n - (int)seeing) * each, (uint64_t)s.m};
  float top[2] = {0.0f, 0.0f};
#pragma unroll
  for (int which = 0; which < 2; ++which)
    for (uint64_t r = part * 16 + threadIdx.x / 16; r < rows[which]; r += 16 * kNormParts) {
      const T* p = which ? at<T>(a.v, b, r, g) : at<T>(a.dout, b, seeing + r / each, g * each + r % each);
      const typename Pack<T>::V v = load_pack(p + in, (int64_t)a.dim - in);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < Pack<T>::N; ++e) sum = fmaf(to_f32((T)v[e]), to_f32((T)v[e]), sum);
      top[which] = fmaxf(top[which], lanes_sum<16>(sum));
    }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const float v = wave_max(top[which]);
    if (lane_id() == 0) most[which][threadIdx.x / kWave] = v;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const float* v = most[threadIdx.x];
    norms[(bg * 2 + threadIdx.x) * kNormParts + part] = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
  }
}
// f of a sequence's key and value head
template <class T>
__device__ __forceinline__ float factor_of(const float* norms, uint32_t bg) {
  if constexpr (kBoost<T> == 0.0f) {
    return 1.0f;
  } else {
    const float* v = norms + bg * 2 * kNormParts + lane_id();
    const float most = sqrtf(wave_max(v[0])) * sqrtf(wave_max(v[kNormParts]));
    if (!(most > 0.0f) || most == INFINITY) return 1.0f;
    int e;
    frexpf(most, &e);
    return ldexpf(1.0f, -e);
  }
}

// ---- backward: dq ---------------------------------------------------------------
// Each row's lse in base 2 less the probabilities' exponent (or +inf, where they
// are 0) and sum of dout * out go to `stats` ([batch][heads][queries] each) for
// dk and dv.
template <class T, int DP, int NW, bool DIRECT>
__global__ __launch_bounds__(NW * kWave, ((sizeof(T) == 4 ? DP > 64 : DP > 96) ? 1 : 2)) void k_attention_dq(Args a, Packing pk, uint32_t tiles, float* stats, const float* norms) {
  constexpr int BN = keys_of<T>(), NT = NW * kWave;
  typedef Tile<T, DP, BN> TL;
  typedef Mma<T> M;
  __shared__ I4 k0[TL::SIZE], v0[TL::SIZE], k1[TL::SIZE], v1[TL::SIZE];
  const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), bg = id / tiles, tile = tiles - 1 - id % tiles;
  const uint32_t b = bg / a.groups, g = bg % a.groups;
  const Sequence s(a, b);
  const Rows<NW> rows(a, s, pk, tile, g);
  const float c = a.scale * kLog2e;

  typename TL::Frag q[TL::STEPS], d[TL::STEPS];
  load_row<T, TL>(q, at<T>(a.q, b, rows.i, rows.head), rows.live, a.dim);
  load_row<T, TL>(d, at<T>(a.dout, b, rows.i, rows.head), rows.live, a.dim);
  float lse = INFINITY, delta = 0.0f;
  {
    typename TL::Frag f[TL::STEPS];
    load_row<T, TL>(f, at<T>(a.out, b, rows.i, rows.head), rows.live, a.dim);
#pragma unroll
    for (int x = 0; x < TL::STEPS; ++x)
#pragma unroll
      for (int e = 0; e < TL::PACK; ++e) delta = fmaf(to_f32((T)f[x][e]), to_f32((T)d[x][e]), delta);
    delta = both_halves_sum(delta);
    const uint64_t where = ((uint64_t)b * a.heads + rows.head) * a.queries + rows.i;
    if (rows.live) lse = a.lse[where] * kLog2e - kBoost<T>;
    if (rows.there && lane_id() < 32) {
      stats[where] = lse;
      stats[where + (uint64_t)a.batch * a.heads * a.queries] = delta;
    }
  }
  const float f = factor_of<T>(norms, bg);
  delta *= f;
  Acc o[DP / 32] = {};

  const Packing one{1, BN, 1};
  const Loader<T, TL, NT, DIRECT> lk(a.k, one, a.dim), lv(a.v, one, a.dim);
  const T *ks = at<T>(a.k, b, 0, g), *vs = at<T>(a.v, b, 0, g);
  const auto load = [&](int j, I4* kt, I4* vt) {
    lk.load(ks + j * a.k.token, 0, rows.last + 1 - j, kt);
    lv.load(vs + j * a.v.token, 0, rows.last + 1 - j, vt);
  };
  const auto pass = [&](int j, const I4* kt, const I4* vt, I4* kn, I4* vn) {
    wait_and_meet();
    if (j + BN <= rows.last) load(j + BN, kn, vn);
    if (j > rows.wave_last || j + BN - 1 < rows.wave_first) return;
    const bool masked = j < rows.wave_all_first || j + BN - 1 > rows.wave_all_last;
#pragma unroll
    for (int t = 0; t < BN / 32; ++t) {
      Acc p = {}, e = {};
#pragma unroll
      for (int x = 0; x < TL::STEPS; ++x) {
        p = M::mul(TL::row(kt, 32 * t, x), q[x], p);
        e = M::mul(TL::row(vt, 32 * t, x), d[x], e);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) p[r] = __builtin_amdgcn_exp2f(fmaf(p[r], c, -lse));
      if (masked) {
        const uint32_t from = j + 4 * (lane_id() / 32) - rows.lo;
#pragma unroll
        for (int r = 0; r < 16; ++r) p[r] = from + (32 * t + 8 * (r / 4) + r % 4) > rows.span ? 0.0f : p[r];
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) p[r] *= kBoost<T> == 0.0f ? e[r] - delta : fmaf(e[r], f, -delta);
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const typename TL::Frag f = M::frag(p, x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) o[y] = M::mul(TL::column(kt, 32 * t, x, y), f, o[y]);
      }
    }
  };
  if (rows.first <= rows.last) load(rows.first, k0, v0);
  for (int j = rows.first; j <= rows.last; j += 2 * BN) {
    pass(j, k0, v0, k1, v1);
    if (j + BN <= rows.last) pass(j + BN, k1, v1, k0, v0);
  }
  if (rows.there) store_row<T, DP>(o, a.scale / f * exp2f(-kBoost<T>), at<T>(a.dq, b, rows.i, rows.head), a.dim);
}

// ---- backward: dk and dv --------------------------------------------------------
// A wave has 32 keys and walks over the tiles of queries that see one of the
// workgroup's.
template <class T, int DP, int NW, bool DIRECT>
__global__ __launch_bounds__(NW * kWave, (DP > 64 ? 1 : 2)) void k_attention_dkv(Args a, Packing pk, uint32_t tiles,
                                                                 const float* stats, const float* norms) {
  constexpr int BM = keys_of<T>(), NT = NW * kWave;
  typedef Tile<T, DP, BM> TL;
  typedef Mma<T> M;
  __shared__ I4 q0[TL::SIZE], d0[TL::SIZE], q1[TL::SIZE], d1[TL::SIZE];
  __shared__ float stat[2][2][BM];
  __shared__ int query[BM];
  const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), bg = id / tiles, tile = id % tiles;
  const uint32_t b = bg / a.groups, g = bg % a.groups, each = a.heads / a.groups;
  const Sequence s(a, b);
  const float c = a.scale * kLog2e;
  const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int j0 = tile * NW * 32, w0 = j0 + wid * 32, j = w0 + lane % 32, end = min(j0 + NW * 32, s.m);
  const bool there = j < (int)a.keys;

  typename TL::Frag k[TL::STEPS], v[TL::STEPS];
  load_row<T, TL>(k, at<T>(a.k, b, j, g), j < s.m, a.dim);
  load_row<T, TL>(v, at<T>(a.v, b, j, g), j < s.m, a.dim);
  const float f = factor_of<T>(norms, bg);
  Acc dk[DP / 32] = {}, dv[DP / 32] = {};

  // queries first .. last see one of the workgroup's keys
  const int first = max(0, j0 - s.after - s.m + s.n), last = j0 < end ? min(s.n - 1, end - 1 + s.before - s.m + s.n) : -1;
  const int t0 = first / (int)pk.ip * (int)pk.nh, t1 = last < first ? t0 : (last / (int)pk.ip + 1) * (int)pk.nh;

  const Loader<T, TL, NT, DIRECT> lq(a.q, pk, a.dim), ld(a.dout, pk, a.dim);
  const int seeing = max(0, s.n - s.m - s.after);  // the first query that sees a key
  const uint32_t my_i = threadIdx.x / pk.hp, my_h = threadIdx.x % pk.hp;
  if (threadIdx.x < BM) query[threadIdx.x] = my_i;
  const auto load = [&](int t, I4* qt, I4* dt, int turn) {
    const uint32_t h = g * each + t % pk.nh * pk.hp;
    const int i0 = t / pk.nh * pk.ip;
    lq.load(at<T>(a.q, b, i0, h), seeing - i0, s.n - i0, qt);
    ld.load(at<T>(a.dout, b, i0, h), seeing - i0, s.n - i0, dt);
    if (threadIdx.x < BM) {
      const uint32_t r = threadIdx.x;
      const int i = i0 + my_i;
      float lse = INFINITY, delta = 0.0f;
      if (my_i < pk.ip && i >= seeing && i < s.n) {
        const uint64_t where = ((uint64_t)b * a.heads + h + my_h) * a.queries + i;
        lse = stats[where];
        delta = stats[where + (uint64_t)a.batch * a.heads * a.queries];
      }
      stat[turn][0][r] = lse;
      stat[turn][1][r] = delta * f;
    }
  };
  const auto pass = [&](int t, const I4* qt, const I4* dt, I4* qn, I4* dn, int turn) {
    wait_and_meet();
    if (t + 1 < t1) load(t + 1, qn, dn, turn ^ 1);
    const int i0 = t / pk.nh * pk.ip, i1 = min(i0 + (int)pk.ip, s.n) - 1;
    // keys that the tile's first and last queries see
    if (w0 > s.last(i1) || min(w0 + 31, end - 1) < s.first(i0) || w0 >= end) return;
    const bool masked = w0 < s.first(i1) || w0 + 31 > s.last(i0);
#pragma unroll
    for (int u = 0; u < BM / 32; ++u) {
      Acc p = {}, e = {};
#pragma unroll
      for (int x = 0; x < TL::STEPS; ++x) {
        p = M::mul(TL::row(qt, 32 * u, x), k[x], p);
        e = M::mul(TL::row(dt, 32 * u, x), v[x], e);
      }
      const int h4 = 32 * u + 4 * (lane / 32);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        p[r] = __builtin_amdgcn_exp2f(fmaf(p[r], c, -stat[turn][0][h4 + 8 * (r / 4) + r % 4]));
      if (masked) {
        const int far = j - i0 - s.m + s.n;  // from the place of the tile's first query
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int ahead = far - query[h4 + 8 * (r / 4) + r % 4];
          p[r] = ahead > s.after || ahead < -s.before || j >= s.m ? 0.0f : p[r];
        }
      }
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const typename TL::Frag f = M::frag(p, x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) dv[y] = M::mul(TL::column(dt, 32 * u, x, y), f, dv[y]);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float delta = stat[turn][1][h4 + 8 * (r / 4) + r % 4];
        p[r] *= kBoost<T> == 0.0f ? e[r] - delta : fmaf(e[r], f, -delta);
      }
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const typename TL::Frag f = M::frag(p, x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) dk[y] = M::mul(TL::column(qt, 32 * u, x, y), f, dk[y]);
      }
    }
  };
  if (t0 < t1) load(t0, q0, d0, 0);
  for (int t = t0; t < t1; t += 2) {
    pass(t, q0, d0, q1, d1, 0);
    if (t + 1 < t1) pass(t + 1, q1, d1, q0, d0, 1);
  }
  if (!there) return;
  store_row<T, DP>(dk, a.scale / f * exp2f(-kBoost<T>), at<T>(a.dk, b, j, g), a.dim);
  store_row<T, DP>(dv, exp2f(-kBoost<T>), at<T>(a.dv, b, j, g), a.dim);
}

// ---- launches -------------------------------------------------------------------
// The tiles of `rows` rows that take the fewest for all queries and heads; of
// those that take as few the one with the most heads, which share loads.
Packing packing_of(const Args& a, uint32_t rows, uint64_t& tiles) {
  const uint32_t each = a.heads / a.groups;
  Packing best{};
  tiles = ~0ull;
  for (uint32_t hp = 1; hp <= std::min(each, rows); ++hp) {
    if (each % hp != 0) continue;
    const uint32_t ip = rows / hp, nh = each / hp;
    const uint64_t n = (uint64_t)((a.queries + ip - 1) / ip) * nh;
    if (n <= tiles) tiles = n, best = Packing{hp, ip, nh};
  }
  return best;
}

// Whether a tile of these heads can go to LDS without passing through registers.
bool direct_ok(const Args& a, const sparcml_heads& x, uint32_t rows, uint32_t heads) {
  const uint64_t size = a.type == SPARCML_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x.data) & 15u) || a.dim * size % 16 != 0) return false;
  if (x.batch * size % 16 != 0 || x.token * size % 16 != 0 || x.head * size % 16 != 0) return false;
  return (x.token * rows + x.head * heads + a.dim) * size < (1ull << 31) - 64;
}

template <class F>
hipError_t with_dim(const Args& a, bool direct, F&& f) {
  return for_type(a.type, [&](auto t) {
    const auto go = [&](auto dp) {
      if (direct) f(t, dp, std::true_type{});
      else f(t, dp, std::false_type{});
    };
    if (a.dim <= 32) go(std::integral_constant<int, 32>{});
    else if (a.dim <= 64) go(std::integral_constant<int, 64>{});
    else if (a.dim <= 96) go(std::integral_constant<int, 96>{});
    else go(std::integral_constant<int, 128>{});
    return hipGetLastError();
  });
}

constexpr int kWaves = 4;

}  // namespace

size_t attention_workspace_bytes(const Args&) { return 256; }

hipError_t attention_launch(const Args& a, void*, hipStream_t stream) {
  uint64_t tiles;
  const Packing pk = packing_of(a, kWaves * 32, tiles);
  const bool direct = a.keys == 0 || (direct_ok(a, a.k, kKeys, 1) && direct_ok(a, a.v, kKeys, 1));
  return with_dim(a, direct, [&](auto t, auto dp, auto d) {
    hipLaunchKernelGGL((k_attention<decltype(t), dp, kWaves, d>), dim3((uint32_t)(tiles * a.batch * a.groups)),
                       dim3(kWaves * kWave), 0, stream, a, pk, (uint32_t)tiles);
  });
}

size_t attention_backward_workspace_bytes(const Args& a) {
  const size_t norms = a.type == SPARCML_F16 ? (size_t)a.batch * a.groups * 2 * kNormParts : 0;
  return ((size_t)a.batch * a.heads * a.queries * 2 + norms) * sizeof(float) + 256;
}

hipError_t attention_backward_launch(const Args& a, void* ws, hipStream_t stream) {
  float* stats = static_cast<float*>(ws);
  float* norms = stats + (size_t)a.batch * a.heads * a.queries * 2;
  if (a.type == SPARCML_F16) {
    hipLaunchKernelGGL(k_attention_norms<f16>, dim3(a.batch * a.groups * kNormParts), dim3(4 * kWave), 0, stream, a, norms);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.queries > 0) {
    uint64_t tiles;
    const Packing pk = packing_of(a, kWaves * 32, tiles);
    const bool direct = a.keys == 0 || (direct_ok(a, a.k, kKeys, 1) && direct_ok(a, a.v, kKeys, 1));
    const hipError_t e = with_dim(a, direct, [&](auto t, auto dp, auto d) {
      hipLaunchKernelGGL((k_attention_dq<decltype(t), dp, kWaves, d>), dim3((uint32_t)(tiles * a.batch * a.groups)),
                         dim3(kWaves * kWave), 0, stream, a, pk, (uint32_t)tiles, stats, norms);
    });
    if (e != hipSuccess) return e;
  }
  if (a.keys == 0) return hipSuccess;
  uint64_t none;
  const uint32_t tiles = (a.keys + kWaves * 32 - 1) / (kWaves * 32);
  const Packing pk = packing_of(a, a.type == SPARCML_F32 ? kKeys / 2 : kKeys, none);
  const bool direct = a.queries == 0 || (direct_ok(a, a.q, pk.ip, pk.hp) && direct_ok(a, a.dout, pk.ip, pk.hp));
  return with_dim(a, direct, [&](auto t, auto dp, auto d) {
    hipLaunchKernelGGL((k_attention_dkv<decltype(t), dp, kWaves, d>), dim3(tiles * a.batch * a.groups),
                       dim3(kWaves * kWave), 0, stream, a, pk, tiles, stats, norms);
  });
}

}  // namespace sparcml
