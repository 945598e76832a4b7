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
  // Keys from here on, up to m, are seen by some query, those before it by none:
  // they may hold anything, and a probability of 0 times what is not finite is
  // no 0.
  __device__ __forceinline__ int first_seen() const { return n > 0 ? first(0) : m; }
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
// ROWS heads of DP elements, W elements a row, in 16-byte chunks; row r's chunk
// c is at c ^ order(r). LDS serves 256 bytes at a time, from 64 banks: a chunk
// of 16 rows (a 16-byte read's quarter), and 64 bytes of 4 rows (half of a read
// that turns 16-bit values), have to be in different banks. With 16-bit values
// order takes a row's lowest bits to the chunk's highest for the latter and the
// next ones below for the former; with rows of 2 to the 256 bytes, the lowest
// bit is in the place already. fp32's columns are 32 neighbours of 2 rows,
// rows 4 apart; its rows are two to a bank, as its matrix instructions take 16
// times as long for as many products.
template <class T, int DP, int ROWS_>
struct Tile {
  typedef Mma<T> M;
  typedef typename M::Frag Frag;
  static constexpr int ROWS = ROWS_, W = DP <= 64 ? 64 : 128, CH = W * (int)sizeof(T) / 16, SIZE = ROWS * CH;
  static constexpr int STEPS = DP / M::STEP, PACK = 16 / (int)sizeof(T);

  static __device__ __forceinline__ int order(int row) {
    if (sizeof(T) == 4) return (row & 7) << 1;
    return CH == 8 ? (row >> 1 & 1) << 2 | (row >> 2 & 3) : (row & 3) << 2 | (row >> 2 & 3);
  }

  // A lane's byte offsets into a tile: of step 0 of its row, of its column 0.
  // The others differ from them in single bits, which exclusive ors set. They
  // are made new to the compiler where a tile's products begin, so that it does
  // not keep a register for each place it can compute ahead.
  struct Places {
    int row, column;
    __device__ __forceinline__ Places() {
      const int lane = lane_id(), h = lane / 32, r = lane % 32;
      row = (r * CH + (h ^ order(r))) * 16;
      if constexpr (sizeof(T) == 2) {  // 4 rows of 16 columns turn to 16 lanes of 4 rows
        const int i = lane % 16, v = 4 * h + i / 4;
        column = (v * CH + ((lane / 16 % 2 * 2 + i % 4 / 2) ^ order(v))) * 16 + i % 2 * 8;
      } else {
        column = (4 * h * CH + (r / 4 ^ order(4 * h))) * 16 + r % 4 * 4;
      }
    }
    __device__ __forceinline__ void make_new() { asm volatile("" : "+v"(row), "+v"(column)); }
  };
  // step s of row `base` + lane % 32 (base a multiple of 32)
  static __device__ __forceinline__ Frag row(const I4* lds, const Places& at, int base, int s) {
    return *reinterpret_cast<const Frag*>(reinterpret_cast<const char*>(lds) + (at.row ^ s << 5) + base * CH * 16);
  }
  // column 32 t + lane % 32 of rows base + s * STEP .. (base a multiple of 32)
  static __device__ __forceinline__ Frag column(const I4* lds, const Places& at, int base, int s, int t) {
    const char* p = reinterpret_cast<const char*>(lds) + (base + M::STEP * s) * CH * 16;
    if constexpr (sizeof(T) == 2) {
      typedef short S4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) S4 L;
      const S4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p + (at.column ^ t << 6)));
      const S4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p + (at.column ^ t << 6 ^ 32) + 8 * CH * 16));
      return __builtin_bit_cast(Frag, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      Frag f;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const float*>(p + (at.column ^ t << 7 ^ j << 5) + j * CH * 16);
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
// within 2^31 bytes of the tile's first; otherwise through registers. PACKED:
// rows as `pk` has them, else one a key.
template <class T, class TL, int NT, bool DIRECT, bool PACKED>
struct Loader {
  static constexpr int N = TL::SIZE / NT, STEP = NT / TL::CH, KEPT = PACKED ? N : 1;
  static_assert(TL::SIZE % NT == 0 && NT % TL::CH == 0, "whole chunks to a thread, whole rows to a turn");
  static constexpr int kNothing = 0x7FFFFFF0;  // past the records
  // of each turn (not PACKED: of the first, the others being STEP rows further
  // each, at the same chunk): bytes from the tile's first row, and its query or
  // key, past all of them where it is never there
  int offset[KEPT], query[KEPT];
  uint64_t token, head;
  uint32_t dim;
  int all;  // queries or keys of a tile

  __device__ __forceinline__ Loader(const sparcml_heads& x, const Packing& pk, uint32_t dim_)
      : token(x.token), head(x.head), dim(dim_), all(PACKED ? pk.ip : TL::ROWS) {
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
      const uint32_t c = k * NT + threadIdx.x, row = c / TL::CH;
      const uint32_t i = PACKED ? row / pk.hp : row, h = PACKED ? row % pk.hp : 0;
      const uint32_t e = (c % TL::CH ^ TL::order(row)) * TL::PACK;
      const bool never = i >= (uint32_t)all || e >= dim;
      query[k] = never ? 1 << 30 : (int)i;
      offset[k] = !DIRECT ? (int)(h << 8 | e) : never ? kNothing : (int)((i * token + h * head + e) * sizeof(T));
    }
  }
  // the queries or keys from .. to - 1, counted from the tile's first one
  __device__ __forceinline__ void load(const T* base, int from, int to, I4* lds) const {
    if constexpr (DIRECT) {
      if (from <= 0 && to >= all) turns<true>(base, from, to, lds);
      else turns<false>(base, from, to, lds);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        typename Pack<T>::V v = {};
        const int q = PACKED ? query[k] : query[0] + k * STEP, x = offset[PACKED ? k : 0], e = x & 255;
        if (q >= from && q < to) v = load_pack(base + q * token + (x >> 8) * head + e, (int64_t)dim - e);
        lds[k * NT + threadIdx.x] = __builtin_bit_cast(I4, v);
      }
    }
  }
  template <bool WHOLE>
  __device__ __forceinline__ void turns(const T* base, int from, int to, I4* lds) const {
#if __HIP_DEVICE_COMPILE__  // the host's pass has no such type, and would leave the kernel out
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const T* first = PACKED ? base : base + k * STEP * token;
      const int q = PACKED ? query[k] : query[0] + k * STEP, x = offset[PACKED ? k : 0];
      const auto memory = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(first), 0, kNothing, 0x00027000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          memory, (__attribute__((address_space(3))) void*)(lds + k * NT + wave * kWave), 16,
          WHOLE || (q >= from && q < to) ? x : kNothing, 0, 0, 0);
    }
#endif
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
    place(a, pk, tile, g, wid * 32 + lane_id() % 32);
    const int i0 = tile / pk.nh * pk.ip;
    lo = s.first(i), span = s.last(i) - lo;
    live = there && i < s.n && (int)span >= 0;
    if (!live) lo = 1 << 30, span = 0;
    const int w0 = i0 + wid * 32 / pk.hp, w1 = min(i0 + (int)min(pk.ip - 1, (wid * 32 + 31) / pk.hp), s.n - 1);
    const int i1 = min(i0 + (int)pk.ip, s.n) - 1;
    wave_first = s.first(w0), wave_last = w0 <= w1 ? s.last(w1) : -1;
    wave_all_first = s.first(w1), wave_all_last = s.last(w0);
    first = s.first(i0), last = i0 <= i1 ? s.last(i1) : -1;
  }
  // part `part` of `parts` of the keys, in whole tiles of BN
  template <int BN>
  __device__ __forceinline__ void take(uint32_t part, uint32_t parts) {
    if (parts == 1 || last < first) return;
    const int tiles = (last - first) / BN + 1, each = (tiles + parts - 1) / parts * BN;
    const int64_t from = first + (int64_t)part * each;
    last = min((int64_t)last, from + each - 1);
    wave_last = min(wave_last, last);
    first = min(from, (int64_t)last + 1);
  }
  __device__ __forceinline__ Rows() {}
  // row r of the tile
  __device__ __forceinline__ void place(const Args& a, const Packing& pk, uint32_t tile, uint32_t g, uint32_t r) {
    i = tile / pk.nh * pk.ip + r / pk.hp;
    head = g * (a.heads / a.groups) + tile % pk.nh * pk.hp + r % pk.hp;
    there = r / pk.hp < pk.ip && i < (int)a.queries;
  }
};

// A row of a head, 16 bytes of it to a Frag; 0 past its end, and where it is
// not `there`. WHOLE: 16 bytes divide it; what is not there is then read from
// the tensor's first head instead, which keeps the loads free of branches.
template <class T, class TL, bool WHOLE>
__device__ __forceinline__ void load_row(typename TL::Frag (&f)[TL::STEPS], const sparcml_heads& x, uint64_t b,
                                         int i, uint32_t h, bool there, uint32_t dim) {
  if constexpr (WHOLE) {
    const T* p = there ? at<T>(x, b, i, h) : static_cast<const T*>(x.data);
#pragma unroll
    for (int s = 0; s < TL::STEPS; ++s) {
      const uint32_t e = (2 * s + lane_id() / 32) * TL::PACK;
      f[s] = __builtin_bit_cast(typename TL::Frag, *reinterpret_cast<const typename Pack<T>::U*>(p + (e < dim ? e : 0)));
    }
#pragma unroll
    for (int s = 0; s < TL::STEPS; ++s)
      if (!there || (2 * s + lane_id() / 32) * TL::PACK >= dim) f[s] = typename TL::Frag{};
  } else {
    const T* p = at<T>(x, b, i, h);
#pragma unroll
    for (int s = 0; s < TL::STEPS; ++s) {
      const int e = (2 * s + lane_id() / 32) * TL::PACK;
      f[s] = __builtin_bit_cast(typename TL::Frag, load_pack(p + e, there ? (int64_t)dim - e : 0));
    }
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

// The same in fp32, DP elements a row, for a later kernel to join.
template <int DP>
__device__ __forceinline__ void store_part(const Acc (&acc)[DP / 32], float by, float* p) {
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<f32x4*>(p + 32 * t + 8 * q + 4 * (lane_id() / 32)) =
          f32x4{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]} * by;
}

constexpr int kKeys = 64;  // keys of a tile, 16-bit; 32 with fp32
template <class T>
constexpr int keys_of() { return sizeof(T) == 2 ? kKeys : kKeys / 2; }

constexpr int kJoinThreads = 256;

// ---- forward --------------------------------------------------------------------
// The probabilities go to the second product in the type, since 4-byte operands
// would take 16 times as long: each is rounded by half a step at most, their sum
// is taken before that. With bf16 the result is then off by 2.1e-3 of its norm
// at 4 x 4096 tokens, where its own rounding leaves 1.6e-3.
//
// They are held 2^kHeld times as large below the running maximum, which is moved
// on where a score passes it by a factor of 2^kPast. fp16 has 40 binary digits
// from its smallest to its largest value: at 2^13 and 2^2 past that, at most
// 2^15, those of 2^-27 of the maximum have all their digits and those of 2^-38
// are lost (at 1, 2^-14 and 2^-25: a row whose result is made of many such keys
// beside a large one of value 0 lost its result). The larger kPast, the fewer
// rescalings: at 2^7 and 2^8 past that, 4 x 4096 tokens of 32 heads of 128 take
// 597 us for 600, 65 queries of 16384 keys 20.6 for 21.2. bf16 has fp32's range.
template <class T>
constexpr float kHeld = std::is_same<T, f16>::value ? 13.0f : 0.0f;  // both as exponents
template <class T>
constexpr float kBack = kHeld<T> == 0.0f ? 1.0f : 0x1p-13f;  // 2^-kHeld: takes it off sums exactly
template <class T>
constexpr float kPast = std::is_same<T, f16>::value ? 2.0f : 8.0f;

// Two tiles to a turn, since each is at another place in LDS; the second of the
// last turn may be past the end, where a wave passes it over like any tile it
// does not see. (Leaving the loop between the two cost 36 register moves a tile,
// a fifteenth of the time.) 4 x 4096 tokens of 32 heads of 128, bf16: 567 us, 970
// TFLOP/s. The matrix cores are busy half the time; the rest is the softmax's, 6
// vector instructions to each matrix one, which two waves to a SIMD hide in part.
template <class T, int DP, int NW, bool DIRECT>
__global__ __launch_bounds__(NW * kWave, (sizeof(T) == 4 && DP > 64 ? 1 : 2)) void k_attention(Args a, Packing pk, uint32_t tiles,
                                                                         uint32_t parts, float* part) {
  constexpr int BN = keys_of<T>(), NT = NW * kWave;
  typedef Tile<T, DP, BN> TL;
  typedef Mma<T> M;
  __shared__ I4 k0[TL::SIZE], v0[TL::SIZE], k1[TL::SIZE], v1[TL::SIZE];
  const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), bg = id / parts / tiles, tile = tiles - 1 - id / parts % tiles;
  const uint32_t b = bg / a.groups, g = bg % a.groups;
  const Sequence s(a, b);
  Rows<NW> rows(a, s, pk, tile, g);
  rows.template take<BN>(id % parts, parts);
  const float c = a.scale * kLog2e;

  typename TL::Frag q[TL::STEPS];
  load_row<T, TL, DIRECT>(q, a.q, b, rows.i, rows.head, rows.live, a.dim);
  Acc o[DP / 32] = {};
  float top = -INFINITY, sum = 0.0f;

  const Packing one{1, BN, 1};
  const Loader<T, TL, NT, DIRECT, false> lk(a.k, one, a.dim), lv(a.v, one, a.dim);
  const T *ks = at<T>(a.k, b, rows.first, g), *vs = at<T>(a.v, b, rows.first, g);  // of the next tile
  const uint64_t k_step = BN * a.k.token, v_step = BN * a.v.token;
  const auto load = [&](int j, I4* kt, I4* vt) {
    lk.load(ks, 0, rows.last + 1 - j, kt);
    lv.load(vs, 0, rows.last + 1 - j, vt);
    ks += k_step, vs += v_step;
  };
  typename TL::Places places;
  const auto products = [&](auto masked, int j, const I4* kt, const I4* vt) {
    places.make_new();
    Acc p[BN / 32] = {};
#pragma unroll
    for (int t = 0; t < BN / 32; ++t)
#pragma unroll
      for (int x = 0; x < TL::STEPS; ++x) p[t] = M::mul(TL::row(kt, places, 32 * t, x), q[x], p[t]);
    if constexpr (masked) {
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
    if (ballot(now > top + kPast<T>)) {
      const float higher = fmaxf(now, top), keep = higher == top ? 1.0f : __builtin_amdgcn_exp2f(top - higher);
      top = higher;
      sum *= keep;
#pragma unroll
      for (int t = 0; t < DP / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] *= keep;
    }
    const float off = top == -INFINITY ? 0.0f : top - kHeld<T>;
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
        for (int y = 0; y < DP / 32; ++y) o[y] = M::mul(TL::column(vt, places, 32 * t, x, y), f, o[y]);
      }
  };
  const auto pass = [&](int j, const I4* kt, const I4* vt, I4* kn, I4* vn) {
    wait_and_meet();
    if (j + BN <= rows.last) load(j + BN, kn, vn);
    if (j > rows.wave_last || j + BN - 1 < rows.wave_first) return;
    if (j < rows.wave_all_first || j + BN - 1 > rows.wave_all_last) products(std::true_type{}, j, kt, vt);
    else products(std::false_type{}, j, kt, vt);
  };
  if (rows.first <= rows.last) load(rows.first, k0, v0);
  for (int j = rows.first; j <= rows.last; j += 2 * BN) {
    pass(j, k0, v0, k1, v1);
    pass(j + BN, k1, v1, k0, v0);
  }
  sum = rows.live ? both_halves_sum(sum) * kBack<T> : 0.0f;
  if (!rows.there) return;
  if (parts > 1) {
    const uint64_t row = (uint64_t)id * (NW * 32) + threadIdx.x / kWave * 32 + lane_id() % 32;
    if (lane_id() < 32) reinterpret_cast<float2*>(part)[row] = make_float2(top, sum);
    store_part<DP>(o, kBack<T>, part + (uint64_t)gridDim.x * (NW * 32) * 2 + row * DP);
    return;
  }
  store_row<T, DP>(o, sum == 0.0f ? 0.0f : kBack<T> / sum, at<T>(a.out, b, rows.i, rows.head), a.dim);
  if (lane_id() < 32) a.lse[((uint64_t)b * a.heads + rows.head) * a.queries + rows.i] = sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
}

// Where a thread of a joining kernel is: L lanes join row r of the ROWS of a
// tile, 4 elements each from e on. MANY parts: a wave joins a row, its L lanes
// each taking every SLICES-th part, since a few rows' parts one after the other
// would take as long as they are many.
constexpr uint32_t kManyParts = 8;
template <int DP, int ROWS, bool MANY>
struct Joined {
  static constexpr int L = DP <= 32 ? 8 : DP <= 64 ? 16 : 32, SLICES = MANY ? kWave / L : 1, LANES = L * SLICES;
  uint64_t row;
  uint32_t id, r, e, slice;
  __device__ __forceinline__ Joined() {
    row = (uint64_t)blockIdx.x * (kJoinThreads / LANES) + threadIdx.x / LANES;
    id = row / ROWS, r = row % ROWS, e = lane_id() % L * 4, slice = lane_id() % LANES / L;
  }
  static uint32_t blocks(uint64_t rows) { return (uint32_t)(rows / (kJoinThreads / LANES)); }  // ROWS is a multiple of it
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int d = L; d < LANES; d <<= 1) v += __shfl_xor(v, d, kWave);
    return v;
  }
  static __device__ __forceinline__ f32x4 sum(f32x4 v) { return f32x4{sum(v[0]), sum(v[1]), sum(v[2]), sum(v[3])}; }
  // the largest of f(k), k < parts, for the row
  template <class F>
  __device__ __forceinline__ float most(uint32_t parts, F&& f) const {
    float v = -INFINITY;
    for (uint32_t k = lane_id() % LANES; k < parts; k += LANES) v = fmaxf(v, f(k));
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
  }
  template <class T>
  __device__ __forceinline__ void store(f32x4 o, T* p, uint32_t dim) const {
    typedef T Four __attribute__((ext_vector_type(4)));
    typedef Four Any __attribute__((aligned(sizeof(T))));
    if (e + 4 <= dim) {
      Four v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = from_f32<T>(o[j]);
      *reinterpret_cast<Any*>(p + e) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (e + j < dim) p[e + j] = from_f32<T>(o[j]);
    }
  }
};

// Joins the parts of a row: out = sum of 2^(top - most) o, over the sum of 2^(top
// - most) sum.
template <class T, int DP, int NW, bool MANY>
__global__ __launch_bounds__(kJoinThreads) void k_attention_join(Args a, Packing pk, uint32_t tiles, uint32_t parts,
                                                                 const float* part) {
  constexpr int ROWS = NW * 32;
  const Joined<DP, ROWS, MANY> in;
  const uint64_t all = (uint64_t)tiles * a.batch * a.groups * ROWS;
  const uint32_t bg = in.id / tiles, b = bg / a.groups;
  Rows<NW> rows;
  rows.place(a, pk, tiles - 1 - in.id % tiles, bg % a.groups, in.r);
  if (!rows.there) return;
  const float2* tops = reinterpret_cast<const float2*>(part) + (uint64_t)in.id * parts * ROWS + in.r;
  const float* os = part + all * parts * 2 + ((uint64_t)in.id * parts * ROWS + in.r) * DP + in.e;
  const float most = in.most(parts, [&](uint32_t k) { return tops[k * ROWS].x; });
  float sum = 0.0f;
  f32x4 o = {};
#pragma unroll 4
  for (uint32_t k = in.slice; k < parts; k += in.SLICES) {
    const float2 t = tops[k * ROWS];
    const float by = t.x == most ? 1.0f : __builtin_amdgcn_exp2f(t.x - most);
    sum = fmaf(t.y, by, sum);
    if (in.e < DP) o += *reinterpret_cast<const f32x4*>(os + (uint64_t)k * ROWS * DP) * by;
  }
  sum = in.sum(sum), o = in.sum(o);
  if (in.slice != 0) return;
  in.store(o * (sum == 0.0f ? 0.0f : 1.0f / sum), at<T>(a.out, b, rows.i, rows.head), a.dim);
  if (in.e == 0) a.lse[((uint64_t)b * a.heads + rows.head) * a.queries + rows.i] = sum == 0.0f ? -INFINITY : most * kLn2 + logf(sum);
}

// ---- backward -------------------------------------------------------------------
// fp16 has 40 binary digits from its smallest to its largest value, fewer than
// probabilities of long rows and ds of small gradients take. So p is held 2^14
// times as large, and ds, which is at most 2 p |dout| |v|, 2^14 f times, f a
// power of two that brings |dout| |v| to 1/2 .. 1: at most 2^15, and digits of a
// ds are lost below 2^-28 |dout| |v| and all of it below 2^-39. |v| is the largest
// of the key and value head's in a sequence; |dout| is the row's own for dq, so
// that rows of any size keep their digits, and for dk, whose sums run over the
// rows, the largest, too: keys that only rows of far smaller dout see lose
// digits of their dk. bf16 has fp32's range, f and both factors are 1.
template <class T>
constexpr float kBoost = sizeof(T) == 2 && std::is_same<T, f16>::value ? 14.0f : 0.0f;  // as an exponent

// The largest sum of squares of a row of dout and of v, of one of kNormParts
// parts of the rows of each sequence's key and value head that take part: the
// queries that see something and the keys that are seen. The others may hold
// anything.
constexpr int kNormParts = 64;
template <class T>
__global__ __launch_bounds__(4 * kWave) void k_attention_norms(Args a, float* norms) {
  __shared__ float most[2][4];
  const uint32_t items = a.batch * a.groups * kNormParts;
  for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint32_t bg = it / kNormParts, part = it % kNormParts;
    const uint32_t b = bg / a.groups, g = bg % a.groups, each = a.heads / a.groups;
    const Sequence s(a, b);
    const uint32_t seeing = max(0, s.n - s.m - s.after), seen = s.first_seen(), in = threadIdx.x % 16 * Pack<T>::N;
    const uint64_t rows[2] = {(uint64_t)max(0, s.n - (int)seeing) * each, (uint64_t)max(0, s.m - (int)seen)};
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int which = 0; which < 2; ++which)
      for (uint64_t r = part * 16 + threadIdx.x / 16; r < rows[which]; r += 16 * kNormParts) {
        const T* p = which ? at<T>(a.v, b, seen + r, g) : at<T>(a.dout, b, seeing + r / each, g * each + r % each);
        const typename Pack<T>::V v = load_pack(p + in, (int64_t)a.dim - in);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < Pack<T>::N; ++e) sum = fmaf(to_f32((T)v[e]), to_f32((T)v[e]), sum);
        top[which] = fmaxf(top[which], lanes_sum<16>(sum));
      }
    __syncthreads();  // the last item's have been read
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
}
// The largest norm of a row of dout (which = 0) or v (1) of a sequence's key and value head.
__device__ __forceinline__ float largest_norm(const float* norms, uint32_t bg, int which) {
  return sqrtf(wave_max(norms[(bg * 2 + which) * kNormParts + lane_id()]));
}
// the power of two that brings `most` to 1/2 .. 1
__device__ __forceinline__ float factor_of(float most) {
  if (!(most > 0.0f) || most == INFINITY) return 1.0f;
  int e;
  frexpf(most, &e);
  return ldexpf(1.0f, -e);
}

// ---- backward: dq ---------------------------------------------------------------
// For dk and dv, what their products take off goes to `stats` ([batch][heads]
// [queries] each): each row's lse in base 2 less the probabilities' exponent, or
// +inf where they are 0, with 16-bit types as a score, before its scaling; and
// its sum of dout * out. ds is rounded to the type for its product with k, like
// the forward pass's probabilities and for the same reason. 4 x 4096 tokens of
// 32 heads of 128: 765 us, 1080 TFLOP/s, matrix cores busy 59 of 100 of it.
template <class T, int DP, int NW, bool DIRECT>
__global__ __launch_bounds__(NW * kWave, (sizeof(T) == 4 && DP > 64 ? 1 : 2)) void k_attention_dq(Args a, Packing pk, uint32_t tiles, float* stats,
                                                                            const float* norms, uint32_t parts, float* part) {
  constexpr int BN = keys_of<T>(), NT = NW * kWave;
  typedef Tile<T, DP, BN> TL;
  typedef Mma<T> M;
  __shared__ I4 k0[TL::SIZE], v0[TL::SIZE], k1[TL::SIZE], v1[TL::SIZE];
  const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), bg = id / parts / tiles, tile = tiles - 1 - id / parts % tiles;
  const uint32_t b = bg / a.groups, g = bg % a.groups;
  const Sequence s(a, b);
  Rows<NW> rows(a, s, pk, tile, g);
  rows.template take<BN>(id % parts, parts);
  const float c = a.scale * kLog2e;

  typename TL::Frag q[TL::STEPS], d[TL::STEPS];
  load_row<T, TL, DIRECT>(q, a.q, b, rows.i, rows.head, rows.live, a.dim);
  load_row<T, TL, DIRECT>(d, a.dout, b, rows.i, rows.head, rows.live, a.dim);
  float lse = INFINITY, delta = 0.0f;
  {
    typename TL::Frag f[TL::STEPS];
    load_row<T, TL, DIRECT>(f, a.out, b, rows.i, rows.head, rows.live, a.dim);
#pragma unroll
    for (int x = 0; x < TL::STEPS; ++x)
#pragma unroll
      for (int e = 0; e < TL::PACK; ++e) delta = fmaf(to_f32((T)f[x][e]), to_f32((T)d[x][e]), delta);
    delta = both_halves_sum(delta);
    const uint64_t where = ((uint64_t)b * a.heads + rows.head) * a.queries + rows.i;
    if (rows.live) lse = a.lse[where] * kLog2e - kBoost<T>;
    if (rows.there && lane_id() < 32 && id % parts == 0) {
      stats[where] = sizeof(T) == 2 ? -lse / c : -lse;
      stats[where + (uint64_t)a.batch * a.heads * a.queries] = -delta;
    }
  }
  float f = 1.0f;
  if constexpr (kBoost<T> != 0.0f) {
    float size = 0.0f;
#pragma unroll
    for (int x = 0; x < TL::STEPS; ++x)
#pragma unroll
      for (int e = 0; e < TL::PACK; ++e) size = fmaf(to_f32((T)d[x][e]), to_f32((T)d[x][e]), size);
    f = factor_of(sqrtf(both_halves_sum(size)) * largest_norm(norms, bg, 1));
    delta *= f;
  }
  Acc o[DP / 32] = {};

  const Packing one{1, BN, 1};
  const Loader<T, TL, NT, DIRECT, false> lk(a.k, one, a.dim), lv(a.v, one, a.dim);
  const T *ks = at<T>(a.k, b, rows.first, g), *vs = at<T>(a.v, b, rows.first, g);  // of the next tile
  const uint64_t k_step = BN * a.k.token, v_step = BN * a.v.token;
  const auto load = [&](int j, I4* kt, I4* vt) {
    lk.load(ks, 0, rows.last + 1 - j, kt);
    lv.load(vs, 0, rows.last + 1 - j, vt);
    ks += k_step, vs += v_step;
  };
  typename TL::Places places;
  const auto products = [&](auto masked, int j, const I4* kt, const I4* vt) {
    places.make_new();
    const uint32_t from = j + 4 * (lane_id() / 32) - rows.lo;
#pragma unroll
    for (int t = 0; t < BN / 32; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      Acc p = {}, e = {};
#pragma unroll
      for (int x = 0; x < TL::STEPS; ++x) {
        p = M::mul(TL::row(kt, places, 32 * t, x), q[x], p);
        e = M::mul(TL::row(vt, places, 32 * t, x), d[x], e);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        p[r] = __builtin_amdgcn_exp2f(fmaf(p[r], c, -lse));
        if constexpr (masked) p[r] = from + (32 * t + 8 * (r / 4) + r % 4) > rows.span ? 0.0f : p[r];
        p[r] *= kBoost<T> == 0.0f ? e[r] - delta : fmaf(e[r], f, -delta);
      }
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const typename TL::Frag b = M::frag(p, x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) o[y] = M::mul(TL::column(kt, places, 32 * t, x, y), b, o[y]);
      }
    }
  };
  const auto pass = [&](int j, const I4* kt, const I4* vt, I4* kn, I4* vn) {
    wait_and_meet();
    if (j + BN <= rows.last) load(j + BN, kn, vn);
    if (j > rows.wave_last || j + BN - 1 < rows.wave_first) return;
    if (j < rows.wave_all_first || j + BN - 1 > rows.wave_all_last) products(std::true_type{}, j, kt, vt);
    else products(std::false_type{}, j, kt, vt);
  };
  if (rows.first <= rows.last) load(rows.first, k0, v0);
  for (int j = rows.first; j <= rows.last; j += 2 * BN) {
    pass(j, k0, v0, k1, v1);
    pass(j + BN, k1, v1, k0, v0);
  }
  if (!rows.there) return;
  const float by = a.scale * (exp2f(-kBoost<T>) / f);
  if (parts == 1) store_row<T, DP>(o, by, at<T>(a.dq, b, rows.i, rows.head), a.dim);
  else store_part<DP>(o, by, part + ((uint64_t)id * (NW * 32) + threadIdx.x / kWave * 32 + lane_id() % 32) * DP);
}

// The sum of the parts of a row of dq.
template <class T, int DP, int NW, bool MANY>
__global__ __launch_bounds__(kJoinThreads) void k_attention_join_dq(Args a, Packing pk, uint32_t tiles, uint32_t parts,
                                                                    const float* part) {
  constexpr int ROWS = NW * 32;
  const Joined<DP, ROWS, MANY> in;
  const uint32_t bg = in.id / tiles;
  Rows<NW> rows;
  rows.place(a, pk, tiles - 1 - in.id % tiles, bg % a.groups, in.r);
  if (!rows.there) return;
  f32x4 o = {};
  if (in.e < DP) {
#pragma unroll 4
    for (uint32_t k = in.slice; k < parts; k += in.SLICES)
      o += *reinterpret_cast<const f32x4*>(part + (((uint64_t)in.id * parts + k) * ROWS + in.r) * DP + in.e);
  }
  o = in.sum(o);
  if (in.slice == 0) in.store(o, at<T>(a.dq, bg / a.groups, rows.i, rows.head), a.dim);
}

// ---- backward: dk and dv --------------------------------------------------------
// A wave has 32 keys and walks over the tiles of queries that see one of the
// workgroup's. It holds k, v, dk and dv, with 128-element heads 192 registers, so
// that there is one wave to a SIMD (the second one's spills took 2800 us instead
// of 1960 for the gradients of 4 x 4096 tokens of 32 heads of 128) and nothing
// hides the vector instructions between the products, nor the reads from LDS:
// matrix cores busy 42 of 100 of the time, 870 TFLOP/s of its own four products.
// s and dout v^T are computed here and for dq: sharing them would take sums in
// memory that several workgroups add to, in an order that changes results.
// p is rounded to the type for its product with dout, ds for that with q.
// The mask is applied in the middle of the one way through a tile's products:
// a way of its own for masked tiles had the results moved to other registers at
// its end, 2150 us instead of 1960.
template <class T, int DP, int NW, bool DIRECT>
__global__ __launch_bounds__(NW * kWave, (DP > 64 ? 1 : 2)) void k_attention_dkv(
    Args a, Packing pk, uint32_t tiles, const float* stats, const float* norms, uint32_t parts, float* part) {
  constexpr int BM = keys_of<T>(), NT = NW * kWave, KEYS = NW * 32;
  typedef Tile<T, DP, BM> TL;
  typedef Mma<T> M;
  typedef typename TL::Frag Frag;
  __shared__ I4 q0[TL::SIZE], d0[TL::SIZE], q1[TL::SIZE], d1[TL::SIZE];
  __shared__ __align__(16) float stat[2][2][BM];
  __shared__ uint32_t query[BM];
  const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), bg = id / parts / tiles, tile = id / parts % tiles;
  const uint32_t b = bg / a.groups, g = bg % a.groups, each = a.heads / a.groups;
  const Sequence s(a, b);
  const float c = a.scale * kLog2e;
  const uint32_t wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int j0 = tile * KEYS, w0 = j0 + wid * 32, j = w0 + lane % 32, end = min(j0 + KEYS, s.m);
  const bool there = j < (int)a.keys;

  Frag k[TL::STEPS], v[TL::STEPS];
  const bool seen = j >= s.first_seen() && j < s.m;
  load_row<T, TL, DIRECT>(k, a.k, b, j, g, seen, a.dim);
  load_row<T, TL, DIRECT>(v, a.v, b, j, g, seen, a.dim);
  float f = 1.0f;
  if constexpr (kBoost<T> != 0.0f) f = factor_of(largest_norm(norms, bg, 0) * largest_norm(norms, bg, 1));
  Acc dk[DP / 32] = {}, dv[DP / 32] = {};

  // queries first .. last see one of the workgroup's keys
  const int first = max(0, j0 - s.after - s.m + s.n), last = j0 < end ? min(s.n - 1, end - 1 + s.before - s.m + s.n) : -1;
  int t0 = first / (int)pk.ip * (int)pk.nh, t1 = last < first ? t0 : (last / (int)pk.ip + 1) * (int)pk.nh;
  if (parts > 1) {
    const int64_t each = (t1 - t0 + parts - 1) / parts, from = t0 + id % parts * each;
    t1 = min((int64_t)t1, from + each);
    t0 = min(from, (int64_t)t1);
  }

  const int count = t1 - t0;

  const Loader<T, TL, NT, DIRECT, true> lq(a.q, pk, a.dim), ld(a.dout, pk, a.dim);
  const int seeing = max(0, s.n - s.m - s.after);  // the first query that sees a key
  const uint32_t my_i = threadIdx.x / pk.hp, my_h = threadIdx.x % pk.hp;
  if (threadIdx.x < BM) query[threadIdx.x] = my_i;
  // Where the next tile is: its first query, its heads, and what follows from
  // them. Moved on instead of computed again, since divisions and products of
  // 64 bits between two tiles would take longer than the tile.
  struct {
    int i0;
    uint32_t chunk;
    const T *q, *d;
    const float* stat;
  } at_tile;
  const uint64_t all_stats = (uint64_t)a.batch * a.heads * a.queries;
  const auto go_to = [&](int i0, uint32_t chunk) {
    const uint32_t h = g * each + chunk * pk.hp;
    at_tile = {i0, chunk, at<T>(a.q, b, i0, h), at<T>(a.dout, b, i0, h), stats + ((uint64_t)b * a.heads + h) * a.queries + i0};
  };
  const uint64_t q_step = pk.ip * a.q.token, d_step = pk.ip * a.dout.token;
  const auto step_back = [&]() {
    if (pk.nh > 1) {
      const bool wrap = at_tile.chunk == 0;
      go_to(at_tile.i0 - (wrap ? (int)pk.ip : 0), wrap ? pk.nh - 1 : at_tile.chunk - 1);
    } else {
      at_tile.i0 -= pk.ip, at_tile.q -= q_step, at_tile.d -= d_step, at_tile.stat -= pk.ip;
    }
  };
  // the rows' lse and delta pass through registers: they are stored when the
  // tiles' loads, which were asked for after them, have had time
  const uint64_t my_stat = (uint64_t)my_h * a.queries + my_i;
  const bool mine = threadIdx.x < BM && my_i < pk.ip;
  const auto stats_of = [&]() {
    float2 v = make_float2(-INFINITY, 0.0f);
    const int i = at_tile.i0 + my_i;
    if (mine && i >= seeing && i < s.n) v = make_float2(at_tile.stat[my_stat], at_tile.stat[my_stat + all_stats]);
    return v;
  };
  const auto keep = [&](float2 v, int turn) {
    if (threadIdx.x < BM) {
      stat[turn][0][threadIdx.x] = v.x;
      stat[turn][1][threadIdx.x] = v.y;
    }
  };
  const auto load = [&](I4* qt, I4* dt) {
    lq.load(at_tile.q, seeing - at_tile.i0, s.n - at_tile.i0, qt);
    ld.load(at_tile.d, seeing - at_tile.i0, s.n - at_tile.i0, dt);
  };
  typename TL::Places places;
  const auto products = [&](bool masked, int i0, const I4* qt, const I4* dt, const float (&row)[2][BM]) {
    places.make_new();
    // the key's way from the first one that the tile's first query may see; past all of them where there is no key
    const uint32_t far = j < s.m ? (uint32_t)(j - i0 - s.m + s.n + s.before) : 0xFFFFFF00u;
    const uint32_t span = (uint32_t)s.before + (uint32_t)s.after;
#pragma unroll
    for (int u = 0; u < BM / 32; ++u) {
      const int h4 = 32 * u + 4 * (lane / 32);
      // 16-bit: the products start from -lse and -delta
      const auto start = [&](int which) {
        Acc a = {};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(row[which] + h4 + 8 * r);
#pragma unroll
            for (int x = 0; x < 4; ++x) a[4 * r + x] = v[x];
          }
        }
        return a;
      };
      Acc p = start(0), e = start(1);
#pragma unroll
      for (int x = 0; x < TL::STEPS; ++x) {
        p = M::mul(TL::row(qt, places, 32 * u, x), k[x], p);
        e = M::mul(TL::row(dt, places, 32 * u, x), v[x], e);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        p[r] = __builtin_amdgcn_exp2f(sizeof(T) == 2 ? p[r] * c : fmaf(p[r], c, row[0][h4 + 8 * (r / 4) + r % 4]));
      }
      if (masked) {
#pragma unroll
        for (int r = 0; r < 16; ++r) p[r] = far - query[h4 + 8 * (r / 4) + r % 4] > span ? 0.0f : p[r];
      }
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const Frag b = M::frag(p, x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) dv[y] = M::mul(TL::column(dt, places, 32 * u, x, y), b, dv[y]);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if constexpr (kBoost<T> != 0.0f) p[r] *= f;
        p[r] *= sizeof(T) == 2 ? e[r] : e[r] + row[1][h4 + 8 * (r / 4) + r % 4];
      }
#pragma unroll
      for (int x = 0; x < 32 / M::STEP; ++x) {
        const Frag b = M::frag(p, x);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) dk[y] = M::mul(TL::column(qt, places, 32 * u, x, y), b, dk[y]);
      }
    }
  };
  const auto pass = [&](int n, const I4* qt, const I4* dt, I4* qn, I4* dn, int turn) {
    wait_and_meet();
    const int i0 = at_tile.i0, i1 = min(i0 + (int)pk.ip, s.n) - 1;
    float2 next = {};
    if (n + 1 < count) {
      step_back();
      next = stats_of();
      load(qn, dn);
    }
    // some query of the tile sees some key of the wave, or all see all
    if (n < count && w0 < end && w0 <= s.last(i1) && min(w0 + 31, end - 1) >= s.first(i0)) {
      products(w0 < s.first(i1) || w0 + 31 > s.last(i0), i0, qt, dt, stat[turn]);
    }
    keep(next, turn ^ 1);
  };
  // From the last queries to the first: under a causal mask all workgroups of a
  // head see the last ones, so that those that run together find what they read
  // in L2, where from the first on each is at another place (16384 tokens'
  // gradients are a twentieth slower that way).
  if (count > 0) {
    go_to((t1 - 1) / (int)pk.nh * (int)pk.ip, (t1 - 1) % pk.nh);
    keep(stats_of(), 0);
    load(q0, d0);
    for (int n = 0; n < count; n += 2) {
      pass(n, q0, d0, q1, d1, 0);
      pass(n + 1, q1, d1, q0, d0, 1);
    }
  }
  if (!there) return;
  const float byk = a.scale * (exp2f(-kBoost<T>) / f), byv = exp2f(-kBoost<T>);
  if (parts == 1) {
    store_row<T, DP>(dk, byk, at<T>(a.dk, b, j, g), a.dim);
    store_row<T, DP>(dv, byv, at<T>(a.dv, b, j, g), a.dim);
  } else {
    float* to = part + ((uint64_t)id * 2 * KEYS + wid * 32 + lane % 32) * DP;
    store_part<DP>(dk, byk, to);
    store_part<DP>(dv, byv, to + KEYS * DP);
  }
}

// The sums of the parts of a row of dk and of dv.
template <class T, int DP, int ROWS, bool MANY>
__global__ __launch_bounds__(kJoinThreads) void k_attention_join_dkv(Args a, uint32_t tiles, uint32_t parts,
                                                                     const float* part) {
  const Joined<DP, ROWS, MANY> in;
  const uint32_t bg = in.id / tiles, j = in.id % tiles * ROWS + in.r;
  if (j >= a.keys) return;
  f32x4 k = {}, v = {};
  if (in.e < DP) {
#pragma unroll 4
    for (uint32_t n = in.slice; n < parts; n += in.SLICES) {
      const float* from = part + (((uint64_t)in.id * parts + n) * 2 * ROWS + in.r) * DP + in.e;
      k += *reinterpret_cast<const f32x4*>(from);
      v += *reinterpret_cast<const f32x4*>(from + ROWS * DP);
    }
  }
  k = in.sum(k), v = in.sum(v);
  if (in.slice != 0) return;
  in.store(k, at<T>(a.dk, bg / a.groups, j, bg % a.groups), a.dim);
  in.store(v, at<T>(a.dv, bg / a.groups, j, bg % a.groups), a.dim);
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

// f(whether there are many), where there are parts to join
template <class F>
void join(uint32_t parts, F&& f) {
  if (parts >= kManyParts) f(std::true_type{});
  else if (parts > 1) f(std::false_type{});
}

constexpr int kWaves = 4, kRows = kWaves * 32;  // of a workgroup; its queries and heads, or keys

// How a call is cut up: the tiles of queries of a sequence's key and value
// head (forward, dq) and of its keys (dk, dv), and the parts that the keys or
// queries that a tile walks over are split into.
struct Plan {
  Packing rows, walked;  // of the tiles of queries that stay, and of those that are walked over for dk and dv
  uint64_t tiles, key_tiles;
  uint32_t parts, key_parts;
  bool direct, key_direct;
  size_t dp;

  // Few workgroups with long ways are split so that all compute units are
  // full: two workgroups each, one of those that hold 128-element heads' dk and
  // dv (5 sequences of 1001, 80-element heads, in 3 parts: gradients 80 us, in
  // one 74). Parts have `shortest` tiles at least, and a way that has fewer than
  // `least` is not worth the kernel that joins it: 512 tokens of 16 heads of 64
  // take 12 us, in parts of 4 tiles 17; an fp32 tile takes about 6 times as long,
  // and 128 queries of 512 keys 17 us in parts of 2, in one 44. The rule knows the
  // sizes alone: workgroups past a sequence's length count, too.
  static uint32_t parts_of(const Args& a, uint64_t workgroups, uint64_t way, uint64_t full) {
    const uint64_t shortest = a.type == SPARCML_F32 ? 2 : 4, least = a.type == SPARCML_F32 ? 4 : 16;
    if (workgroups == 0 || workgroups * 2 > full || way < least) return 1;
    return (uint32_t)std::min(full / workgroups, way / shortest);
  }

  explicit Plan(const Args& a) {
    const uint32_t bn = a.type == SPARCML_F32 ? kKeys / 2 : kKeys;
    const uint64_t bg = (uint64_t)a.batch * a.groups, reach = (uint64_t)a.before + a.after;
    uint64_t walked_tiles;
    rows = packing_of(a, kRows, tiles);
    walked = packing_of(a, bn, walked_tiles);
    key_tiles = (a.keys + kRows - 1) / kRows;
    parts = parts_of(a, tiles * bg, std::min<uint64_t>(a.keys, reach + rows.ip) / bn, 512);
    key_parts = parts_of(a, key_tiles * bg, std::min<uint64_t>(a.queries, reach + kRows) / walked.ip * walked.nh, a.dim > 64 ? 256 : 512);
    direct = a.dim * (a.type == SPARCML_F32 ? 4 : 2) % 16 == 0 && (a.keys == 0 || (direct_ok(a, a.k, bn, 1) && direct_ok(a, a.v, bn, 1)));
    key_direct = a.dim * (a.type == SPARCML_F32 ? 4 : 2) % 16 == 0 && (a.queries == 0 || (direct_ok(a, a.q, walked.ip, walked.hp) && direct_ok(a, a.dout, walked.ip, walked.hp)));
    dp = (a.dim + 31) / 32 * 32;
  }
  size_t part_floats(const Args& a) const {
    return parts > 1 ? tiles * a.batch * a.groups * parts * kRows * (dp + 2) : 0;
  }
  size_t key_part_floats(const Args& a) const {
    return key_parts > 1 ? key_tiles * a.batch * a.groups * key_parts * kRows * 2 * dp : 0;
  }
};

}  // namespace

size_t attention_workspace_bytes(const Args& a) { return Plan(a).part_floats(a) * sizeof(float); }

hipError_t attention_launch(const Args& a, void* ws, hipStream_t stream) {
  const Plan plan(a);
  float* part = static_cast<float*>(ws);
  const uint32_t tiles = (uint32_t)plan.tiles, all = tiles * a.batch * a.groups;
  return with_dim(a, plan.direct, [&](auto t, auto dp, auto d) {
    typedef decltype(t) T;
    hipLaunchKernelGGL((k_attention<T, dp, kWaves, d>), dim3(all * plan.parts), dim3(kWaves * kWave), 0, stream, a,
                       plan.rows, tiles, plan.parts, part);
    join(plan.parts, [&](auto many) {
      hipLaunchKernelGGL((k_attention_join<T, dp, kWaves, many>), dim3(Joined<dp, kRows, many>::blocks((uint64_t)all * kRows)),
                         dim3(kJoinThreads), 0, stream, a, plan.rows, tiles, plan.parts, part);
    });
  });
}

// the rows' sums, fp16's norms, the parts: dq's are done with when dk's and dv's come
static size_t stats_floats(const Args& a) {
  const size_t norms = a.type == SPARCML_F16 ? (size_t)a.batch * a.groups * 2 * kNormParts : 0;
  return ((size_t)a.batch * a.heads * a.queries * 2 + norms + 63) / 64 * 64;
}

size_t attention_backward_workspace_bytes(const Args& a) {
  const Plan plan(a);
  return (stats_floats(a) + std::max(plan.part_floats(a), plan.key_part_floats(a))) * sizeof(float);
}

hipError_t attention_backward_launch(const Args& a, void* ws, hipStream_t stream) {
  const Plan plan(a);
  float *stats = static_cast<float*>(ws), *norms = stats + (size_t)a.batch * a.heads * a.queries * 2;
  float* part = stats + stats_floats(a);
  if (a.type == SPARCML_F16)
    hipLaunchKernelGGL(k_attention_norms<f16>, dim3(std::min(a.batch * a.groups * kNormParts, 1u << 16)), dim3(4 * kWave), 0,
                       stream, a, norms);
  if (a.queries > 0) {
    const uint32_t tiles = (uint32_t)plan.tiles, all = tiles * a.batch * a.groups;
    const hipError_t e = with_dim(a, plan.direct, [&](auto t, auto dp, auto d) {
      typedef decltype(t) T;
      hipLaunchKernelGGL((k_attention_dq<T, dp, kWaves, d>), dim3(all * plan.parts), dim3(kWaves * kWave), 0, stream, a,
                         plan.rows, tiles, stats, norms, plan.parts, part);
      join(plan.parts, [&](auto many) {
        hipLaunchKernelGGL((k_attention_join_dq<T, dp, kWaves, many>),
                           dim3(Joined<dp, kRows, many>::blocks((uint64_t)all * kRows)), dim3(kJoinThreads), 0, stream, a,
                           plan.rows, tiles, plan.parts, part);
      });
    });
    if (e != hipSuccess) return e;
  }
  if (a.keys == 0) return hipGetLastError();
  const uint32_t tiles = (uint32_t)plan.key_tiles, all = tiles * a.batch * a.groups;
  return with_dim(a, plan.key_direct, [&](auto t, auto dp, auto d) {
    typedef decltype(t) T;
    hipLaunchKernelGGL((k_attention_dkv<T, dp, kWaves, d>), dim3(all * plan.key_parts), dim3(kWaves * kWave), 0, stream,
                       a, plan.walked, tiles, stats, norms, plan.key_parts, part);
    join(plan.key_parts, [&](auto many) {
      hipLaunchKernelGGL((k_attention_join_dkv<T, dp, kRows, many>), dim3(Joined<dp, kRows, many>::blocks((uint64_t)all * kRows)),
                         dim3(kJoinThreads), 0, stream, a, tiles, plan.key_parts, part);
    });
  });
}

}  // namespace sparcml
