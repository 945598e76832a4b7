// Norms of the queries and keys of every head with the rotation by position in
// the same pass, forward and backward, with the reduction of the two weights'
// gradients over the tokens and heads of each node.
//
//   forward   r = 1 / sqrt(sum x^2 / D + eps), y = R(x * r * weight), where R
//             turns the pairs of the first `rotated` elements by position *
//             frequency: (a, b) -> (a cos - b sin, b cos + a sin)
//   backward  u = R^T dy, h = x * r, g = u * weight
//             dx = r * (g - h * sum(g h) / D), dweight_p = sum of u * h over
//             the tokens and heads of node p
//
// Sums are fp32; an angle is 64 bits up to its place in the turn; 16-bit
// results are rounded once, at the store.
//
// Both are bound by memory, large calls by its rate (65536 tokens of 32 + 8 heads
// of 128, bf16: forward 247 us, 5.4 TB/s, backward 383 us, 5.3 TB/s; a large copy
// reaches 4.95), small ones by the launch (8 tokens: 4.6 us of a call's 12.6).
// With one or two heads a token the angles, in 64 bits, count too (3 nodes of
// 275557 tokens, 1 + 1 heads of 80: gradients 342 us, without turning 238, 161 by
// the bytes). What is read and written is touched once and goes past the caches,
// which takes 4 of 100 off. A head's D elements are held by L lanes, two packs
// of V elements each, chosen so that a pair is in one lane (halves: the packs
// are as far apart as the pair's elements; interleaved: the packs are next to
// each other). A wave takes a token with all its heads, or several tokens where
// they have few: its lanes compute each cosine and sine once, exchange them
// through LDS and keep their own for all heads of the token, so that no table is
// read.
#include <algorithm>

#include "kernels.hpp"
#include "numeric.hpp"

namespace sparcml {
namespace {

constexpr int kWaves = 4;  // of a workgroup; forward they share nothing, backward the last sums
constexpr int kThreads = kWaves * kWave;

// V elements at any element's border.
template <class T, int V>
struct Part {
  typedef T W __attribute__((ext_vector_type(V)));
  typedef W U __attribute__((aligned(sizeof(T))));
};

// What a lane holds of a head: K times two packs of V elements. Slot s, of
// lane s % L, is the pairs s * V .. s * V + V - 1; past the rotated pairs its
// packs are the next 2 V elements.
template <class T, int V_, int L_, int K_, bool HALVES>
struct Slots {
  typedef T Type;
  static constexpr int V = V_, L = L_, K = K_, E = 2 * V * K, H = kWave / L;
  static constexpr bool kApart = HALVES || V == 1;  // a pair's elements are e and V + e, else 2 e and 2 e + 1
  uint32_t dim, pairs;

  static __device__ __forceinline__ uint32_t slot(int k) { return lane_id() % L + L * k; }
  __device__ __forceinline__ bool turns(int k) const { return slot(k) * V < pairs; }
  __device__ __forceinline__ uint32_t a(int k) const { return slot(k) * V * (HALVES && turns(k) ? 1 : 2); }
  __device__ __forceinline__ uint32_t b(int k) const { return a(k) + (HALVES && turns(k) ? pairs : V); }
  // a pack is there as a whole or not at all: V_of below
  __device__ __forceinline__ bool there(int k, int pack) const { return (pack ? b(k) : a(k)) < dim; }

  __device__ __forceinline__ void load(float (&x)[E], const T* p) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      typename Part<T, V>::W wa = {}, wb = {};
      if (there(k, 0)) wa = __builtin_nontemporal_load(reinterpret_cast<const typename Part<T, V>::U*>(p + a(k)));
      if (there(k, 1)) wb = __builtin_nontemporal_load(reinterpret_cast<const typename Part<T, V>::U*>(p + b(k)));
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[2 * V * k + e] = to_f32((T)wa[e]);
        x[2 * V * k + V + e] = to_f32((T)wb[e]);
      }
    }
  }
  __device__ __forceinline__ void store(const float (&x)[E], T* p) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      typename Part<T, V>::W wa, wb;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        wa[e] = from_f32<T>(x[2 * V * k + e]);
        wb[e] = from_f32<T>(x[2 * V * k + V + e]);
      }
      if (there(k, 0)) __builtin_nontemporal_store(wa, reinterpret_cast<typename Part<T, V>::U*>(p + a(k)));
      if (there(k, 1)) __builtin_nontemporal_store(wb, reinterpret_cast<typename Part<T, V>::U*>(p + b(k)));
    }
  }
  __device__ __forceinline__ void weight(float (&w)[E], const float* p) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        const uint32_t c = e < V ? a(k) + e : b(k) + e - V;
        w[2 * V * k + e] = c < dim ? (p ? p[c] : 1.0f) : 0.0f;
      }
  }
};

// The cosines and sines of the lane's pairs.
template <class S>
struct Turn {
  float c[S::V * S::K], s[S::V * S::K];

  // The lanes compute those of the pairs of the wave's tokens t .. t + count - 1
  // into `shared`, which is the wave's own, and read those of their pairs of
  // token t + mine.
  __device__ __forceinline__ void at(const S& slots, const int32_t* positions, uint64_t t, uint32_t count, uint32_t mine,
                                     const double* frequency, float2* shared) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");  // the last tokens' have been read
    __builtin_amdgcn_wave_barrier();
    uint32_t i = lane_id(), n = 0;  // pair i of token t + n
    while (i >= slots.pairs && n < count) i -= slots.pairs, ++n;
    while (n < count) {
      const double turns = (double)positions[t + n] * frequency[i] * 0.15915494309189533577;  // 1 / (2 pi)
      float sine, cosine;
      sincospif((float)(2.0 * (turns - rint(turns))), &sine, &cosine);
      shared[n * slots.pairs + i] = make_float2(cosine, sine);
      i += kWave;
      while (i >= slots.pairs && n < count) i -= slots.pairs, ++n;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int k = 0; k < S::K; ++k)
#pragma unroll
      for (int e = 0; e < S::V; ++e) {
        const float2 v = slots.turns(k) ? shared[mine * slots.pairs + S::slot(k) * S::V + e] : make_float2(1.0f, 0.0f);
        c[S::V * k + e] = v.x;
        s[S::V * k + e] = v.y;
      }
  }
  template <bool BACK>
  __device__ __forceinline__ void apply(const S& slots, float (&x)[S::E]) const {
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
      if (!slots.turns(k)) continue;  // an infinity next to it stays where it is
#pragma unroll
      for (int e = 0; e < S::V; ++e) {
        float& a = x[2 * S::V * k + (S::kApart ? e : 2 * e)];
        float& b = x[2 * S::V * k + (S::kApart ? S::V + e : 2 * e + 1)];
        const float co = c[S::V * k + e], si = BACK ? -s[S::V * k + e] : s[S::V * k + e];
        const float a0 = a, b0 = b;
        a = fmaf(a0, co, -(b0 * si));
        b = fmaf(b0, co, a0 * si);
      }
    }
  }
};

// How a wave's S::H groups of lanes are dealt: to `tokens` tokens, `heads` groups
// each, a power of two that takes a token's heads at once where there are as
// many (a call of 58454 tokens of 2 query and 2 key heads of 64 takes 23 us so,
// with all groups to one token's heads 53).
template <class S>
struct Dealt {
  uint32_t heads, tokens, token, head;  // token, head: the lane's first
  __device__ __forceinline__ explicit Dealt(const sparcml_head_norm_args& g) {
    const uint32_t most = max(g.heads, g.groups);
    heads = 1;
    while (heads < (uint32_t)S::H && heads < most) heads <<= 1;
    tokens = S::H / heads;
    token = lane_id() / S::L / heads, head = lane_id() / S::L % heads;
  }
  // float2 of LDS for a wave: tokens * pairs, each of the S::H groups' lanes having V * K pairs
  static constexpr int SHARED = kWave * S::V * S::K;
};

template <int L>
__device__ __forceinline__ float head_sum(float v) {
  if (L == 4) return dpp_add<0x4E>(dpp_add<0xB1>(v));  // quad_perm [1,0,3,2], [2,3,0,1]
  return lanes_sum<(L < 8 ? 8 : L)>(v);
}

// A wave's tokens: their query heads, then their key heads.
template <class S>
__global__ __launch_bounds__(kThreads) void k_head_norm_rotate(sparcml_head_norm_args g) {
  typedef typename S::Type T;
  __shared__ float2 shared[kWaves][Dealt<S>::SHARED];
  const S slots{g.dim, g.rotated / 2};
  float wq[S::E], wk[S::E];
  slots.weight(wq, g.q_weight);
  slots.weight(wk, g.k_weight);
  const float over = 1.0f / (float)g.dim;
  const uint32_t wid = threadIdx.x / kWave;
  const Dealt<S> dealt(g);
  for (uint64_t t0 = ((uint64_t)blockIdx.x * kWaves + wid) * dealt.tokens; t0 < g.tokens;
       t0 += (uint64_t)gridDim.x * kWaves * dealt.tokens) {
    const uint64_t t = t0 + dealt.token;
    Turn<S> turn;
    turn.at(slots, g.positions, t0, g.rotated ? min((uint64_t)dealt.tokens, g.tokens - t0) : 0, dealt.token, g.frequencies,
            shared[wid]);
    if (t >= g.tokens) continue;
    const auto heads = [&](uint32_t count, const sparcml_heads& in, const sparcml_heads& out, const float (&w)[S::E]) {
      const T* src = static_cast<const T*>(in.data) + t * in.token;
      T* dst = static_cast<T*>(out.data) + t * out.token;
      for (uint32_t i = dealt.head; i < count; i += dealt.heads) {
        float x[S::E], s = 0.0f;
        slots.load(x, src + i * in.head);
#pragma unroll
        for (int e = 0; e < S::E; ++e) s = fmaf(x[e], x[e], s);
        const float r = 1.0f / sqrtf(fmaf(head_sum<S::L>(s), over, g.eps));
#pragma unroll
        for (int e = 0; e < S::E; ++e) x[e] = x[e] * r * w[e];
        turn.template apply<false>(slots, x);
        slots.store(x, dst + i * out.head);
      }
    };
    heads(g.heads, g.q, g.q_out, wq);
    heads(g.groups, g.k, g.k_out, wk);
  }
}

// One workgroup: tokens [c * each, (c + 1) * each) of node p, c and p from the
// workgroup's number. Writes dx and this chunk's sums of u * h of both
// weights, to the node's gradients where it is the only chunk, else to part
// [p][c][2][dim].
template <class S>
__global__ __launch_bounds__(kThreads) void k_head_norm_rotate_backward(sparcml_head_norm_args g, uint32_t chunks,
                                                                        uint64_t each, float* part) {
  typedef typename S::Type T;
  __shared__ float2 shared[kWaves][Dealt<S>::SHARED];
  const S slots{g.dim, g.rotated / 2};
  float wq[S::E], wk[S::E], sq[S::E] = {}, sk[S::E] = {};
  slots.weight(wq, g.q_weight);
  slots.weight(wk, g.k_weight);
  const float over = 1.0f / (float)g.dim;
  const uint32_t wid = threadIdx.x / kWave;
  const Dealt<S> dealt(g);
  const uint32_t p = blockIdx.x / chunks, c = blockIdx.x % chunks;
  const uint64_t begin = min(c * each, g.tokens), end = min(begin + each, g.tokens);
  for (uint64_t n = begin + wid * dealt.tokens; n < end; n += kWaves * dealt.tokens) {
    const uint64_t t = p * g.tokens + n + dealt.token;
    Turn<S> turn;
    turn.at(slots, g.positions, p * g.tokens + n, g.rotated ? min((uint64_t)dealt.tokens, end - n) : 0, dealt.token,
            g.frequencies, shared[wid]);
    if (n + dealt.token >= end) continue;
    const auto heads = [&](uint32_t count, const sparcml_heads& in, const sparcml_heads& grad, const sparcml_heads& out,
                           const float (&w)[S::E], float (&sw)[S::E]) {
      const T* src = static_cast<const T*>(in.data) + t * in.token;
      const T* dy = static_cast<const T*>(grad.data) + t * grad.token;
      T* dst = static_cast<T*>(out.data) + t * out.token;
      for (uint32_t i = dealt.head; i < count; i += dealt.heads) {
        float x[S::E], u[S::E], s = 0.0f, gh = 0.0f;
        slots.load(x, src + i * in.head);
        slots.load(u, dy + i * grad.head);
#pragma unroll
        for (int e = 0; e < S::E; ++e) s = fmaf(x[e], x[e], s);
        const float r = 1.0f / sqrtf(fmaf(head_sum<S::L>(s), over, g.eps));
        turn.template apply<true>(slots, u);
#pragma unroll
        for (int e = 0; e < S::E; ++e) {
          x[e] *= r;
          sw[e] = fmaf(u[e], x[e], sw[e]);
          u[e] *= w[e];
          gh = fmaf(u[e], x[e], gh);
        }
        const float m = head_sum<S::L>(gh) * over;
#pragma unroll
        for (int e = 0; e < S::E; ++e) u[e] = r * fmaf(-x[e], m, u[e]);
        slots.store(u, dst + i * out.head);
      }
    };
    heads(g.heads, g.q, g.dq, g.q_out, wq, sq);
    heads(g.groups, g.k, g.dk, g.k_out, wk, sk);
  }
  // the lanes that hold the same columns, then the waves, always in one order
#pragma unroll
  for (int d = S::L; d < kWave; d <<= 1)
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
      sq[e] += __shfl_xor(sq[e], d, kWave);
      sk[e] += __shfl_xor(sk[e], d, kWave);
    }
  __shared__ float all[kWaves][2][S::E][S::L];
  if (lane_id() < S::L) {
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
      all[wid][0][e][lane_id()] = sq[e];
      all[wid][1][e][lane_id()] = sk[e];
    }
  }
  __syncthreads();
  if (wid >= 2 || lane_id() >= S::L) return;
  float* out = chunks == 1 ? (wid ? g.dk_weight : g.dq_weight) : part;
  if (!out) return;
  out += chunks == 1 ? p * (wid ? g.dk_stride : g.dq_stride) : ((uint64_t)blockIdx.x * 2 + wid) * g.dim;
#pragma unroll
  for (int k = 0; k < S::K; ++k)
#pragma unroll
    for (int e = 0; e < 2 * S::V; ++e) {
      const uint32_t col = e < S::V ? slots.a(k) + e : slots.b(k) + e - S::V;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += all[w][wid][2 * S::V * k + e][lane_id()];
      if (col < g.dim) out[col] = v;
    }
}

// Calls f with the Slots of the widest packs that hold a head: V divides the
// rotated pairs, and 2 V what is left of the head.
template <class T, int V, bool HALVES, class F>
void with_lanes(uint32_t dim, F&& f) {
  if (dim <= 64) f(Slots<T, V, 32 / V, 1, HALVES>{});
  else if (dim <= 128) f(Slots<T, V, 64 / V, 1, HALVES>{});
  else f(Slots<T, V, V == 1 ? 64 : 128 / V, V == 1 ? 2 : 1, HALVES>{});
}
template <class T, bool HALVES, class F>
void with_packs(uint32_t dim, uint32_t rotated, F&& f) {
  const auto fits = [&](uint32_t v) { return rotated / 2 % v == 0 && (dim - rotated) % (2 * v) == 0; };
  if (sizeof(T) == 2 && fits(8)) with_lanes<T, sizeof(T) == 2 ? 8 : 4, HALVES>(dim, f);
  else if (fits(4)) with_lanes<T, 4, HALVES>(dim, f);
  else if (fits(2)) with_lanes<T, 2, HALVES>(dim, f);
  else with_lanes<T, 1, HALVES>(dim, f);
}
template <class F>
hipError_t with_slots(const sparcml_head_norm_args& g, F&& f) {
  return for_type(g.type, [&](auto t) {
    using T = decltype(t);
    if (g.interleaved) with_packs<T, false>(g.dim, g.rotated, f);
    else with_packs<T, true>(g.dim, g.rotated, f);
    return hipGetLastError();
  });
}

// Workgroups of a node, 8 to a CU in all, each of whose waves has `least` tokens
// at least: backward 4, since a workgroup's sums of its weights' gradients take
// as long as a token's heads do (a call of 64 nodes of 98 tokens, 32 + 4 heads of
// 32, takes 30 us so, with 1 token 42, with 2 35, with 8 40; where the chip is not
// full anyway, 3 nodes of 1001 tokens, 6 + 2 fp32 heads of 80, kernels 21 us, with
// 1 token 17, which the call hides: 24.6 and 24.4).
constexpr uint32_t kLeastTokens = 4;
uint32_t chunks_of(uint32_t nodes, uint64_t tokens, uint32_t least) {
  const uint64_t most = (2048 + nodes - 1) / nodes, wanted = (tokens + kWaves * least - 1) / (kWaves * least);
  return (uint32_t)std::max<uint64_t>(1, std::min(most, wanted));
}
// tokens of a chunk, as many for each wave
uint64_t each_of(uint64_t tokens, uint32_t chunks) {
  return ((tokens + chunks - 1) / chunks + kWaves - 1) / kWaves * kWaves;
}

}  // namespace

hipError_t head_norm_rotate_launch(const sparcml_head_norm_args& g, hipStream_t stream) {
  return with_slots(g, [&](auto s) {
    using S = decltype(s);
    hipLaunchKernelGGL(k_head_norm_rotate<S>, dim3(chunks_of(1, g.tokens, 1)), dim3(kThreads), 0, stream, g);
  });
}

size_t head_norm_rotate_backward_workspace_bytes(uint32_t nodes, uint64_t tokens, uint32_t dim) {
  return (size_t)nodes * chunks_of(nodes, tokens, kLeastTokens) * 2 * dim * sizeof(float) + 256;
}

hipError_t head_norm_rotate_backward_launch(const sparcml_head_norm_args& g, void* ws, hipStream_t stream) {
  float* part = static_cast<float*>(ws);
  const uint32_t chunks = chunks_of(g.nodes, g.tokens, kLeastTokens);
  const hipError_t e = with_slots(g, [&](auto s) {
    using S = decltype(s);
    hipLaunchKernelGGL(k_head_norm_rotate_backward<S>, dim3(g.nodes * chunks), dim3(kThreads), 0, stream, g, chunks,
                       each_of(g.tokens, chunks), part);
  });
  if (e != hipSuccess || chunks == 1) return e;
  return join_chunks_launch(g.nodes, g.dim, chunks, part, g.dq_weight, g.dq_stride, g.dk_weight, g.dk_stride, stream);
}

}  // namespace sparcml
