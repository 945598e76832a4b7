// C ABI of the SparCML hot path: argument checks, workspace sizing, launch.
// The declarations and their contracts are in include/sparcml.h and, for the
// measurement variants, include/sparcml_bench.h.
#include "sparcml.h"
#include "sparcml_bench.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "kernels.hpp"

// Scratch of the allocation-free reduce: one copy per GPU, held until the
// process ends. Host code never passes this name to a kernel; it uses the
// device address that hipGetSymbolAddress gives on each device.
static __device__ __align__(256) unsigned char scratch[SPARCML_REDUCE_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 256;
std::atomic<void*> g_scratch[kMaxDevices];  // device address of `scratch`, per device ordinal
std::mutex g_scratch_mu;

// Device address of the current device's `scratch`, looked up once per device.
hipError_t scratch_of_current_device(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  void* p = g_scratch[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
      e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
      if (e != hipSuccess) return e;
      if (p == nullptr) return hipErrorInvalidSymbol;
      g_scratch[dev].store(p, std::memory_order_release);
    }
  }
  *out = p;
  return hipSuccess;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

sparcml_status from_hip(hipError_t e) { return e == hipSuccess ? SPARCML_OK : SPARCML_ERR_HIP; }

constexpr uint64_t kMaxN = 0xFFFFFFFFull;       // indices are uint32
constexpr uint64_t kMaxTopkN = 0xFFF80000ull;   // 2^32 - 2^19: candidate slot offsets stay below 2^32 - 2^18

// T = ceil(delta * N) in double, clamped to [0, N + 1]
uint64_t dense_threshold(double delta, uint64_t N) {
  const double t = std::ceil(delta * (double)N);
  if (!(t > 0.0)) return 0;
  if (t > (double)N) return N + 1;
  return (uint64_t)t;
}

}  // namespace

extern "C" {

const char* sparcml_status_string(sparcml_status status) {
  switch (status) {
    case SPARCML_OK: return "SPARCML_OK";
    case SPARCML_ERR_INVALID_ARG: return "SPARCML_ERR_INVALID_ARG: invalid argument";
    case SPARCML_ERR_WORKSPACE: return "SPARCML_ERR_WORKSPACE: workspace missing or too small";
    case SPARCML_ERR_HIP: return "SPARCML_ERR_HIP: HIP runtime or launch error";
    case SPARCML_ERR_SCRATCH_LIMIT:
      return "SPARCML_ERR_SCRATCH_LIMIT: the call needs more than SPARCML_REDUCE_SCRATCH_BYTES of scratch";
  }
  return "SPARCML: unknown status";
}

// --------------------------------------------------------------------------
size_t sparcml_topk_ef_workspace(uint32_t P, uint64_t N, uint64_t k) {
  if (P == 0 || N > kMaxTopkN || k > N || P > 65535u) return 0;
  return sparcml::topk_workspace_bytes(P, N, k);
}

// runs: null, or the run table of the output to write (sparcml_topk_ef_runs)
static sparcml_status topk_common(uint32_t P, uint64_t N, uint64_t k, const float* grad, float* residual,
                                  uint32_t* out_idx, float* out_val, uint32_t* runs, void* ws, size_t ws_bytes,
                                  hipStream_t stream, const sparcml::OpEvents* ev) {
  if (P == 0 || P > 65535u || N > kMaxTopkN || k > N) return SPARCML_ERR_INVALID_ARG;
  if (runs && (uint64_t)P * k > kMaxN - 15) return SPARCML_ERR_INVALID_ARG;  // table positions are uint32
  if ((uint64_t)P * N >= (1ull << 40)) return SPARCML_ERR_INVALID_ARG;
  // one 256-thread workgroup per 1024-element tile slot (a node's tiles start at
  // the 128-byte line of its first element), in one grid dimension of < 2^32 work-items
  if ((uint64_t)P * ((N + 31 + 1023) / 1024) >= (1ull << 24)) return SPARCML_ERR_INVALID_ARG;
  if (N == 0) return SPARCML_OK;
  if (!grad || !residual || !aligned16(grad) || !aligned16(residual)) return SPARCML_ERR_INVALID_ARG;
  if (k > 0 && (!out_idx || !out_val)) return SPARCML_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || ws_bytes < sparcml::topk_workspace_bytes(P, N, k)) return SPARCML_ERR_WORKSPACE;
  // short rows in a small call: one workgroup per node beats the candidate pipeline's kernel chain
  if (N <= SPARCML_TOPK_ROW_MAX && (uint64_t)P * N <= SPARCML_TOPK_ROW_TOTAL_MAX) {
    hipError_t e =
        sparcml::topk_row_launch(P, N, k, grad, residual, out_idx, out_val, static_cast<uint32_t*>(ws), stream, ev);
    // the row kernel has no emit pass: the table comes from its output
    if (e == hipSuccess && runs) e = sparcml::topk_runs_of_output_launch(P, N, k, out_idx, runs, stream);
    return from_hip(e);
  }
  return from_hip(sparcml::topk_ef_launch(P, N, k, grad, residual, out_idx, out_val, runs, ws, stream, ev));
}

sparcml_status sparcml_topk_ef(uint32_t P, uint64_t N, uint64_t k, const float* grad, float* residual,
                               uint32_t* out_idx, float* out_val, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  return topk_common(P, N, k, grad, residual, out_idx, out_val, nullptr, ws, ws_bytes, stream, nullptr);
}

sparcml_status sparcml_topk_ef_runs(uint32_t P, uint64_t N, uint64_t k, const float* grad, float* residual,
                                    uint32_t* out_idx, float* out_val, uint32_t* runs, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  if (!runs) return SPARCML_ERR_INVALID_ARG;
  return topk_common(P, N, k, grad, residual, out_idx, out_val, runs, ws, ws_bytes, stream, nullptr);
}

// --------------------------------------------------------------------------
// layers: off[0] = 0 < ... nondecreasing ... off[nl] = N, k[l] <= off[l+1] - off[l]
static bool layers_ok(uint32_t P, uint64_t N, uint32_t nl, const uint64_t* off, const uint64_t* k) {
  if (P == 0 || P > 65535u || nl == 0 || (uint64_t)P * nl > 65535u || N > kMaxTopkN) return false;
  if (!off || !k || off[0] != 0 || off[nl] != N) return false;
  for (uint32_t l = 0; l < nl; ++l)
    if (off[l + 1] < off[l] || k[l] > off[l + 1] - off[l]) return false;
  if ((uint64_t)P * N >= (1ull << 40)) return false;
  // one 256-thread workgroup per tile of every layer, in one grid dimension
  return sparcml::topk_layers_stream_blocks(P, N, nl, off, k) < (1ull << 24);
}

size_t sparcml_topk_ef_layers_workspace(uint32_t P, uint64_t N, uint32_t nlayers, const uint64_t* h_layer_offsets,
                                        const uint64_t* h_k) {
  if (!layers_ok(P, N, nlayers, h_layer_offsets, h_k)) return 0;
  return sparcml::topk_layers_workspace_bytes(P, N, nlayers, h_layer_offsets, h_k);
}

sparcml_status sparcml_topk_ef_layers(uint32_t P, uint64_t N, uint32_t nlayers, const uint64_t* h_layer_offsets,
                                      const uint64_t* h_k, const float* grad, float* residual, uint32_t* out_idx,
                                      float* out_val, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!layers_ok(P, N, nlayers, h_layer_offsets, h_k)) return SPARCML_ERR_INVALID_ARG;
  if (N == 0) return SPARCML_OK;
  if (!grad || !residual || !aligned16(grad) || !aligned16(residual)) return SPARCML_ERR_INVALID_ARG;
  uint64_t K = 0;
  for (uint32_t l = 0; l < nlayers; ++l) K += h_k[l];
  if (K > 0 && (!out_idx || !out_val)) return SPARCML_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) ||
      ws_bytes < sparcml::topk_layers_workspace_bytes(P, N, nlayers, h_layer_offsets, h_k))
    return SPARCML_ERR_WORKSPACE;
  uint64_t longest = 0;
  for (uint32_t l = 0; l < nlayers; ++l) longest = std::max(longest, h_layer_offsets[l + 1] - h_layer_offsets[l]);
  if (longest <= SPARCML_TOPK_ROW_MAX && (uint64_t)P * N <= SPARCML_TOPK_ROW_TOTAL_MAX &&
      ws_bytes >= sparcml::topk_layer_rows_workspace_bytes(P, nlayers))
    return from_hip(sparcml::topk_layer_rows_launch(P, N, nlayers, h_layer_offsets, h_k, grad, residual, out_idx,
                                                    out_val, ws, stream));  // only short layers: one workgroup each
  return from_hip(sparcml::topk_layers_launch(P, N, nlayers, h_layer_offsets, h_k, grad, residual, out_idx, out_val,
                                              ws, stream));
}

// --------------------------------------------------------------------------
static bool bucket_ok(uint32_t bucket) {
  return bucket == 64 || bucket == 128 || bucket == 256 || bucket == 512 || bucket == 1024;
}

uint64_t sparcml_topk_bucketed_count(uint64_t N, uint32_t bucket, uint32_t k_per_bucket) {
  if (!bucket_ok(bucket) || N > kMaxN) return 0;
  return sparcml::topk_bucketed_count(N, bucket, k_per_bucket);
}

sparcml_status sparcml_topk_ef_bucketed(uint32_t P, uint64_t N, uint32_t bucket, uint32_t k_per_bucket,
                                        const float* grad, float* residual, uint32_t* out_idx, float* out_val,
                                        hipStream_t stream) {
  if (P == 0 || P > 65535u || N > kMaxN || !bucket_ok(bucket)) return SPARCML_ERR_INVALID_ARG;
  if ((uint64_t)P * N >= (1ull << 40)) return SPARCML_ERR_INVALID_ARG;
  if (N == 0) return SPARCML_OK;
  if (!grad || !residual) return SPARCML_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(grad) | reinterpret_cast<uintptr_t>(residual)) & 3u) return SPARCML_ERR_INVALID_ARG;
  if (sparcml::topk_bucketed_count(N, bucket, k_per_bucket) > 0 && (!out_idx || !out_val))
    return SPARCML_ERR_INVALID_ARG;
  return from_hip(sparcml::topk_bucketed_launch(P, N, bucket, k_per_bucket, grad, residual, out_idx, out_val,
                                                stream));
}

// --------------------------------------------------------------------------
static bool qsgd_args_ok(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket) {
  if (bits != 2 && bits != 4 && bits != 8) return false;
  if (P == 0 || P > 65535u) return false;
  if (bucket < 8 || bucket > (1u << 20) || (bucket % 8) != 0) return false;
  if (n >= (1ull << 34)) return false;
  return true;  // any number of buckets: the kernels loop over them
}

static sparcml_status qsgd_common(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket, uint64_t seed,
                                  uint32_t step, uint32_t node0, const float* val, uint8_t* codes, float* scales,
                                  hipStream_t stream, const sparcml::OpEvents* ev) {
  if (!qsgd_args_ok(bits, P, n, bucket)) return SPARCML_ERR_INVALID_ARG;
  if ((uint64_t)node0 + P - 1 > 0xFFFFFFFFull) return SPARCML_ERR_INVALID_ARG;
  if (n == 0) return SPARCML_OK;
  if (!val || !codes || !scales || !aligned16(val)) return SPARCML_ERR_INVALID_ARG;
  return from_hip(
      sparcml::qsgd_launch(bits, P, n, bucket, seed, step, node0, nullptr, val, codes, scales, stream, ev));
}

static sparcml_status dqsgd_common(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket, const uint8_t* codes,
                                   const float* scales, float* val, hipStream_t stream, const sparcml::OpEvents* ev) {
  if (!qsgd_args_ok(bits, P, n, bucket)) return SPARCML_ERR_INVALID_ARG;
  if (n == 0) return SPARCML_OK;
  if (!val || !codes || !scales || !aligned16(val)) return SPARCML_ERR_INVALID_ARG;
  return from_hip(sparcml::dqsgd_launch(bits, P, n, bucket, codes, scales, val, stream, ev));
}

sparcml_status sparcml_qsgd(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket, uint64_t seed, uint32_t step,
                            uint32_t node0, const float* val, uint8_t* codes, float* scales, hipStream_t stream) {
  return qsgd_common(bits, P, n, bucket, seed, step, node0, val, codes, scales, stream, nullptr);
}

sparcml_status sparcml_dqsgd(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket, const uint8_t* codes,
                             const float* scales, float* val, hipStream_t stream) {
  return dqsgd_common(bits, P, n, bucket, codes, scales, val, stream, nullptr);
}

sparcml_status sparcml_q4(uint32_t P, uint64_t n, uint32_t bucket, uint64_t seed, uint32_t step,
                          const float* val, uint8_t* codes, float* scales, hipStream_t stream) {
  return sparcml_qsgd(4, P, n, bucket, seed, step, 0u, val, codes, scales, stream);
}

sparcml_status sparcml_dq4(uint32_t P, uint64_t n, uint32_t bucket, const uint8_t* codes, const float* scales,
                           float* val, hipStream_t stream) {
  return sparcml_dqsgd(4, P, n, bucket, codes, scales, val, stream);
}

sparcml_status sparcml_qsgd_dense_result(uint32_t bits, uint64_t N, uint32_t bucket, uint64_t seed, uint32_t step,
                                         uint32_t node, const sparcml_reduce_result* d_result, const float* val,
                                         uint8_t* codes, float* scales, hipStream_t stream) {
  if (!qsgd_args_ok(bits, 1, N, bucket) || N > kMaxN || !d_result) return SPARCML_ERR_INVALID_ARG;
  if (N == 0) return SPARCML_OK;
  if (!val || !codes || !scales || !aligned16(val)) return SPARCML_ERR_INVALID_ARG;
  return from_hip(sparcml::qsgd_launch(bits, 1, N, bucket, seed, step, node, &d_result->is_dense, val, codes,
                                       scales, stream));
}

// --------------------------------------------------------------------------
double sparcml_estimate_nnz(uint32_t P, uint64_t N, const uint64_t* h_offsets) {
  if (!h_offsets || N == 0) return 0.0;
  double miss = 1.0, sum = 0.0;
  for (uint32_t p = 0; p < P; ++p) {
    const double c = (double)(h_offsets[p + 1] - h_offsets[p]);
    sum += c;
    const double q = c / (double)N;
    miss *= (q >= 1.0 ? 0.0 : 1.0 - q);
  }
  const double e = (double)N * (1.0 - miss);
  return e < sum ? e : sum;
}

size_t sparcml_sparse_reduce_workspace(uint32_t P, uint64_t N, uint64_t total_nnz) {
  if (P == 0 || P > 1024u || N == 0 || N > kMaxN || total_nnz > kMaxN) return 0;
  return sparcml::reduce_workspace_bytes(P, N, total_nnz);
}

// runs: null, or the caller's run table; phase: both phases, or one of them
// (the union phase needs neither values nor outputs)
static sparcml_status reduce_common(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                    const uint32_t* idx, const float* val, const sparcml::ReduceQuantized* quant,
                                    const uint32_t* runs, uint64_t expected_nnz_hint, uint32_t* out_idx,
                                    float* out_val, sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                    hipStream_t stream, const sparcml::OpEvents* ev = nullptr,
                                    int phase = sparcml::kReduceBoth) {
  const bool sums = (phase & sparcml::kReduceSums) != 0;
  if (P == 0 || P > 1024u || N == 0 || N > kMaxN || !std::isfinite(delta)) return SPARCML_ERR_INVALID_ARG;
  if (!h_offsets || !d_result || (sums && (!out_val || !aligned16(out_val)))) return SPARCML_ERR_INVALID_ARG;
  if (h_offsets[0] != 0) return SPARCML_ERR_INVALID_ARG;
  for (uint32_t p = 0; p < P; ++p)
    if (h_offsets[p + 1] < h_offsets[p]) return SPARCML_ERR_INVALID_ARG;
  const uint64_t total = h_offsets[P];
  if (total > kMaxN - 15) return SPARCML_ERR_INVALID_ARG;  // positions and quad ends fit in 32 bits
  if (total > 0 && (!idx || (sums && (quant ? (!quant->codes || !quant->scales) : !val))))
    return SPARCML_ERR_INVALID_ARG;
  const uint64_t T = dense_threshold(delta, N);
  const uint64_t cap = T == 0 ? 0 : (T - 1 < N ? T - 1 : N);
  if (sums && cap > 0 && !out_idx) return SPARCML_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || ws_bytes < sparcml::reduce_workspace_bytes(P, N, total)) return SPARCML_ERR_WORKSPACE;
  // the model's union estimate sizes the writer groups; a hint, where given,
  // picks the writer in its place
  const double model = sparcml_estimate_nnz(P, N, h_offsets);
  const double est = expected_nnz_hint ? (double)expected_nnz_hint : model;
  const bool dense_first = est >= (double)T;
  return from_hip(sparcml::sparse_reduce_launch(P, N, T, h_offsets, idx, val, quant, runs, dense_first, model,
                                                out_idx, cap, out_val,
                                                reinterpret_cast<sparcml::ReduceResultDev*>(d_result), ws, stream,
                                                ev, phase));
}

sparcml_status sparcml_sparse_reduce(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                     const uint32_t* idx, const float* val, uint64_t expected_nnz_hint,
                                     uint32_t* out_idx, float* out_val, sparcml_reduce_result* d_result,
                                     void* ws, size_t ws_bytes, hipStream_t stream) {
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, nullptr, expected_nnz_hint, out_idx, out_val, d_result, ws,
                       ws_bytes, stream);
}

sparcml_status sparcml_sparse_reduce_runs(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                          const uint32_t* idx, const float* val, const uint32_t* runs,
                                          uint64_t expected_nnz_hint, uint32_t* out_idx, float* out_val,
                                          sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                          hipStream_t stream) {
  if (!runs) return SPARCML_ERR_INVALID_ARG;
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, runs, expected_nnz_hint, out_idx, out_val,
                       d_result, ws, ws_bytes, stream);
}

sparcml_status sparcml_sparse_reduce_union(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                           const uint32_t* idx, const uint32_t* runs, uint64_t expected_nnz_hint,
                                           sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                           hipStream_t stream) {
  return reduce_common(P, N, delta, h_offsets, idx, nullptr, nullptr, runs, expected_nnz_hint, nullptr, nullptr,
                       d_result, ws, ws_bytes, stream, nullptr, sparcml::kReduceUnion);
}

sparcml_status sparcml_sparse_reduce_sums(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                          const uint32_t* idx, const float* val, const uint32_t* runs,
                                          uint64_t expected_nnz_hint, uint32_t* out_idx, float* out_val,
                                          sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                          hipStream_t stream) {
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, runs, expected_nnz_hint, out_idx, out_val,
                       d_result, ws, ws_bytes, stream, nullptr, sparcml::kReduceSums);
}

sparcml_status sparcml_sparse_reduce_noalloc(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                             const uint32_t* idx, const float* val, uint64_t expected_nnz_hint,
                                             uint32_t* out_idx, float* out_val, sparcml_reduce_result* d_result,
                                             hipStream_t stream) {
  if (P == 0 || P > 1024u || N == 0 || N > kMaxN || !h_offsets) return SPARCML_ERR_INVALID_ARG;
  if (h_offsets[P] > kMaxN) return SPARCML_ERR_INVALID_ARG;
  if (sparcml::reduce_workspace_bytes(P, N, h_offsets[P]) > SPARCML_REDUCE_SCRATCH_BYTES)
    return SPARCML_ERR_SCRATCH_LIMIT;
  void* ws = nullptr;
  if (scratch_of_current_device(&ws) != hipSuccess) return SPARCML_ERR_HIP;
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, nullptr, expected_nnz_hint, out_idx, out_val, d_result, ws,
                       SPARCML_REDUCE_SCRATCH_BYTES, stream);
}

static sparcml_status reduce_qsgd_common(uint32_t bits, uint32_t bucket, uint32_t P, uint64_t N, double delta,
                                         const uint64_t* h_offsets, const uint32_t* idx, const uint8_t* codes,
                                         const float* scales, const uint32_t* runs, uint64_t expected_nnz_hint,
                                         uint32_t* out_idx, float* out_val, sparcml_reduce_result* d_result,
                                         void* ws, size_t ws_bytes, hipStream_t stream,
                                         const sparcml::OpEvents* ev = nullptr) {
  if (!qsgd_args_ok(bits, 1, 0, bucket)) return SPARCML_ERR_INVALID_ARG;
  const sparcml::ReduceQuantized q{bits, bucket, codes, scales};
  return reduce_common(P, N, delta, h_offsets, idx, nullptr, &q, runs, expected_nnz_hint, out_idx, out_val,
                       d_result, ws, ws_bytes, stream, ev);
}

sparcml_status sparcml_sparse_reduce_qsgd(uint32_t bits, uint32_t bucket, uint32_t P, uint64_t N, double delta,
                                          const uint64_t* h_offsets, const uint32_t* idx, const uint8_t* codes,
                                          const float* scales, uint64_t expected_nnz_hint, uint32_t* out_idx,
                                          float* out_val, sparcml_reduce_result* d_result, void* ws,
                                          size_t ws_bytes, hipStream_t stream) {
  return reduce_qsgd_common(bits, bucket, P, N, delta, h_offsets, idx, codes, scales, nullptr, expected_nnz_hint,
                            out_idx, out_val, d_result, ws, ws_bytes, stream);
}

sparcml_status sparcml_sparse_reduce_qsgd_runs(uint32_t bits, uint32_t bucket, uint32_t P, uint64_t N,
                                               double delta, const uint64_t* h_offsets, const uint32_t* idx,
                                               const uint8_t* codes, const float* scales, const uint32_t* runs,
                                               uint64_t expected_nnz_hint, uint32_t* out_idx, float* out_val,
                                               sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                               hipStream_t stream) {
  if (!runs) return SPARCML_ERR_INVALID_ARG;
  return reduce_qsgd_common(bits, bucket, P, N, delta, h_offsets, idx, codes, scales, runs, expected_nnz_hint,
                            out_idx, out_val, d_result, ws, ws_bytes, stream);
}

// --------------------------------------------------------------------------
// The dense operators around the reduction: arguments are checked here, before
// anything is launched.
// --------------------------------------------------------------------------
static bool type_ok(uint32_t type) { return type <= SPARCML_F16; }
static bool typed_ok(const void* p, uint32_t type) {
  return p && (reinterpret_cast<uintptr_t>(p) & (type == SPARCML_F32 ? 3u : 1u)) == 0;
}
static bool f32_ok(const float* p) { return typed_ok(p, SPARCML_F32); }

sparcml_status sparcml_layer_norm(uint32_t type, uint64_t rows, uint32_t cols, const void* x, uint64_t x_stride,
                                  const void* residual, uint64_t r_stride, const float* weight, const float* bias,
                                  float eps, void* y, void* total, float* mean, float* rstd, hipStream_t stream) {
  if (!type_ok(type) || cols == 0 || cols > 0x7FFFFFFFu || !std::isfinite(eps) || eps < 0.0f)
    return SPARCML_ERR_INVALID_ARG;
  if (rows >= (1ull << 40) / cols || (residual == nullptr) != (total == nullptr)) return SPARCML_ERR_INVALID_ARG;
  if (rows == 0) return SPARCML_OK;
  if (!typed_ok(x, type) || !typed_ok(y, type) || !f32_ok(mean) || !f32_ok(rstd)) return SPARCML_ERR_INVALID_ARG;
  if (residual && (!typed_ok(residual, type) || !typed_ok(total, type))) return SPARCML_ERR_INVALID_ARG;
  if ((weight && !f32_ok(weight)) || (bias && !f32_ok(bias))) return SPARCML_ERR_INVALID_ARG;
  return from_hip(sparcml::layer_norm_launch(type, rows, cols, x, x_stride, residual, r_stride, weight, bias, eps, y,
                                             total, mean, rstd, stream));
}

static bool layer_norm_backward_sizes_ok(uint32_t nodes, uint64_t rows, uint32_t cols) {
  if (nodes == 0 || nodes > 65535u || cols == 0 || cols > 0x7FFFFFFFu) return false;
  return rows < (1ull << 40) / cols / nodes;
}

size_t sparcml_layer_norm_backward_workspace(uint32_t nodes, uint64_t rows, uint32_t cols) {
  if (!layer_norm_backward_sizes_ok(nodes, rows, cols)) return 0;
  return sparcml::layer_norm_backward_workspace_bytes(nodes, rows, cols);
}

sparcml_status sparcml_layer_norm_backward(uint32_t type, uint32_t nodes, uint64_t rows, uint32_t cols,
                                           const void* dy, uint64_t dy_stride, const void* x, uint64_t x_stride,
                                           const void* dresidual, uint64_t dres_stride, const float* weight,
                                           const float* mean, const float* rstd, void* dx, float* dweight,
                                           uint64_t dw_stride, float* dbias, uint64_t db_stride, void* ws,
                                           size_t ws_bytes, hipStream_t stream) {
  if (!type_ok(type) || !layer_norm_backward_sizes_ok(nodes, rows, cols)) return SPARCML_ERR_INVALID_ARG;
  if (rows > 0 && (!typed_ok(dy, type) || !typed_ok(x, type) || !typed_ok(dx, type) || !f32_ok(mean) || !f32_ok(rstd)))
    return SPARCML_ERR_INVALID_ARG;
  if ((dresidual && !typed_ok(dresidual, type)) || (weight && !f32_ok(weight))) return SPARCML_ERR_INVALID_ARG;
  if ((dweight && (!f32_ok(dweight) || dw_stride < cols)) || (dbias && (!f32_ok(dbias) || db_stride < cols)))
    return SPARCML_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || ws_bytes < sparcml::layer_norm_backward_workspace_bytes(nodes, rows, cols))
    return SPARCML_ERR_WORKSPACE;
  return from_hip(sparcml::layer_norm_backward_launch(type, nodes, rows, cols, dy, dy_stride, x, x_stride, dresidual,
                                                      dres_stride, weight, mean, rstd, dx, dweight, dw_stride, dbias,
                                                      db_stride, ws, stream));
}

// --------------------------------------------------------------------------
static bool heads_ok(const sparcml_heads& x, uint32_t type) {
  return typed_ok(x.data, type) && x.batch < (1ull << 40) && x.token < (1ull << 40) && x.head < (1ull << 40);
}

static bool head_norm_sizes_ok(uint32_t nodes, uint64_t tokens, uint32_t dim) {
  return nodes > 0 && nodes <= 65535u && dim > 0 && dim <= sparcml::kHeadNormDim && tokens < (1ull << 31) / nodes;
}

static bool head_norm_args_ok(const sparcml_head_norm_args& a) {
  if (!type_ok(a.type) || !head_norm_sizes_ok(a.nodes, a.tokens, a.dim)) return false;
  if (a.heads == 0 || a.heads > 65535u || a.groups == 0 || a.groups > 65535u) return false;
  if (a.rotated > a.dim || a.rotated % 2 != 0 || !std::isfinite(a.eps) || a.eps < 0.0f) return false;
  if ((a.q_weight && !f32_ok(a.q_weight)) || (a.k_weight && !f32_ok(a.k_weight))) return false;
  if (a.tokens == 0) return true;
  if (a.rotated > 0 && (!a.positions || (reinterpret_cast<uintptr_t>(a.positions) & 3u) || !a.frequencies ||
                        (reinterpret_cast<uintptr_t>(a.frequencies) & 7u)))
    return false;
  return heads_ok(a.q, a.type) && heads_ok(a.k, a.type) && heads_ok(a.q_out, a.type) && heads_ok(a.k_out, a.type);
}

sparcml_status sparcml_head_norm_rotate(const sparcml_head_norm_args* args, hipStream_t stream) {
  if (!args || !head_norm_args_ok(*args) || args->nodes != 1) return SPARCML_ERR_INVALID_ARG;
  if (args->tokens == 0) return SPARCML_OK;
  return from_hip(sparcml::head_norm_rotate_launch(*args, stream));
}

size_t sparcml_head_norm_rotate_backward_workspace(uint32_t nodes, uint64_t tokens, uint32_t dim) {
  if (!head_norm_sizes_ok(nodes, tokens, dim)) return 0;
  return sparcml::head_norm_rotate_backward_workspace_bytes(nodes, tokens, dim);
}

sparcml_status sparcml_head_norm_rotate_backward(const sparcml_head_norm_args* args, void* ws, size_t ws_bytes,
                                                 hipStream_t stream) {
  if (!args || !head_norm_args_ok(*args)) return SPARCML_ERR_INVALID_ARG;
  const sparcml_head_norm_args& a = *args;
  if (a.tokens > 0 && (!heads_ok(a.dq, a.type) || !heads_ok(a.dk, a.type))) return SPARCML_ERR_INVALID_ARG;
  if ((a.dq_weight && (!f32_ok(a.dq_weight) || a.dq_stride < a.dim)) ||
      (a.dk_weight && (!f32_ok(a.dk_weight) || a.dk_stride < a.dim)))
    return SPARCML_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || ws_bytes < sparcml::head_norm_rotate_backward_workspace_bytes(a.nodes, a.tokens, a.dim))
    return SPARCML_ERR_WORKSPACE;
  return from_hip(sparcml::head_norm_rotate_backward_launch(a, ws, stream));
}

// --------------------------------------------------------------------------
// what the workspaces are sized by; a launch has fewer than 2^24 workgroups of
// 256 threads, which take 128 queries of a head, or keys
static bool attention_sizes_ok(const sparcml_attention_args& a) {
  if (!type_ok(a.type) || a.batch > 65535u || a.queries >= (1u << 29) || a.keys >= (1u << 29)) return false;
  if (a.heads == 0 || a.heads > 65535u || a.groups == 0 || a.heads % a.groups != 0) return false;
  const uint64_t bh = (uint64_t)a.batch * a.heads, most = std::max(a.queries, a.keys) / 128 + 1;
  return a.dim > 0 && a.dim <= sparcml::kAttentionDim && (bh == 0 || most < (1ull << 24) / bh);
}

// The kernels multiply the scale by log2 e and, for fp16, by up to 2^26, and
// divide by it: all of that stays finite.
static bool attention_scale_ok(float scale) { return scale >= 1e-30f && scale <= 1e30f; }

static bool attention_args_ok(const sparcml_attention_args& a, bool backward) {
  if (!attention_sizes_ok(a) || !attention_scale_ok(a.scale)) return false;
  if ((a.q_lengths && (reinterpret_cast<uintptr_t>(a.q_lengths) & 3u)) ||
      (a.k_lengths && (reinterpret_cast<uintptr_t>(a.k_lengths) & 3u)))
    return false;
  if (a.batch == 0) return true;
  if (a.queries > 0 && (!heads_ok(a.q, a.type) || !heads_ok(a.out, a.type) || !f32_ok(a.lse))) return false;
  if (a.keys > 0 && (!heads_ok(a.k, a.type) || !heads_ok(a.v, a.type))) return false;
  if (!backward) return true;
  if (a.queries > 0 && (!heads_ok(a.dout, a.type) || !heads_ok(a.dq, a.type))) return false;
  return a.keys == 0 || (heads_ok(a.dk, a.type) && heads_ok(a.dv, a.type));
}

size_t sparcml_attention_workspace(const sparcml_attention_args* args) {
  return args && attention_sizes_ok(*args) ? sparcml::attention_workspace_bytes(*args) : 0;
}

sparcml_status sparcml_attention(const sparcml_attention_args* args, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!args || !attention_args_ok(*args, false)) return SPARCML_ERR_INVALID_ARG;
  const size_t need = sparcml::attention_workspace_bytes(*args);
  if (need > 0 && (!ws || !aligned256(ws) || ws_bytes < need)) return SPARCML_ERR_WORKSPACE;
  if (args->batch == 0 || args->queries == 0) return SPARCML_OK;
  return from_hip(sparcml::attention_launch(*args, ws, stream));
}

size_t sparcml_attention_backward_workspace(const sparcml_attention_args* args) {
  return args && attention_sizes_ok(*args) ? sparcml::attention_backward_workspace_bytes(*args) : 0;
}

sparcml_status sparcml_attention_backward(const sparcml_attention_args* args, void* ws, size_t ws_bytes,
                                          hipStream_t stream) {
  if (!args || !attention_args_ok(*args, true)) return SPARCML_ERR_INVALID_ARG;
  const size_t need = sparcml::attention_backward_workspace_bytes(*args);
  if (need > 0 && (!ws || !aligned256(ws) || ws_bytes < need)) return SPARCML_ERR_WORKSPACE;
  if (args->batch == 0) return SPARCML_OK;
  return from_hip(sparcml::attention_backward_launch(*args, ws, stream));
}

// --------------------------------------------------------------------------
sparcml_status sparcml_momentum_step(uint64_t N, const sparcml_reduce_result* d_result, const uint32_t* idx,
                                     uint64_t idx_cap, const float* val, float* momentum, float mu, float scale,
                                     uint32_t nesterov, uint32_t update_type, void* update, hipStream_t stream) {
  if (N == 0 || N > kMaxN || !type_ok(update_type)) return SPARCML_ERR_INVALID_ARG;
  if (!d_result || (reinterpret_cast<uintptr_t>(d_result) & 7u) || !f32_ok(val) || !f32_ok(momentum))
    return SPARCML_ERR_INVALID_ARG;
  if (idx_cap > 0 && (!idx || (reinterpret_cast<uintptr_t>(idx) & 3u))) return SPARCML_ERR_INVALID_ARG;
  if (update && !typed_ok(update, update_type)) return SPARCML_ERR_INVALID_ARG;
  return from_hip(sparcml::momentum_launch(N, reinterpret_cast<const sparcml::ReduceResultDev*>(d_result), idx,
                                           idx_cap, val, momentum, mu, scale, nesterov != 0, update_type, update,
                                           stream));
}

// --------------------------------------------------------------------------
// the matrices follow each other inside the N elements, and their tiles fit one launch
static bool matrices_ok(uint64_t N, const sparcml::OrthoMatrices& ms) {
  if (N >= (1ull << 40) || (ms.count > 0 && (!ms.offsets || !ms.rows || !ms.cols))) return false;
  uint64_t end = 0, tiles = 0;
  for (uint32_t k = 0; k < ms.count; ++k) {
    const uint64_t rows = ms.rows[k], cols = ms.cols[k];
    if (ms.offsets[k] < end || ms.offsets[k] > N || rows * cols > N - ms.offsets[k]) return false;
    end = ms.offsets[k] + rows * cols;
    if (rows == 0 || cols == 0) continue;
    const uint64_t t = sparcml::ortho_tiles(rows, cols);
    tiles += t;
    if (t == 0 || tiles >= (1ull << 24)) return false;
  }
  return true;
}

size_t sparcml_orthogonalize_workspace(uint64_t N, uint32_t count, const uint64_t* h_offsets, const uint32_t* h_rows,
                                       const uint32_t* h_cols) {
  const sparcml::OrthoMatrices ms{count, h_offsets, h_rows, h_cols};
  return matrices_ok(N, ms) ? sparcml::ortho_workspace_bytes(ms) : 0;
}

static sparcml_status ortho_common(uint64_t N, const sparcml::OrthoMatrices& ms, const sparcml::OrthoSteps& s,
                                   uint32_t update_type, const void* update, uint32_t out_type, void* out,
                                   bool is_weight, float keep, float move, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  if (!type_ok(update_type) || !type_ok(out_type) || !matrices_ok(N, ms)) return SPARCML_ERR_INVALID_ARG;
  if (s.steps > 64 || !std::isfinite(s.a) || !std::isfinite(s.b) || !std::isfinite(s.c) || !std::isfinite(s.eps) ||
      s.eps < 0.0f)
    return SPARCML_ERR_INVALID_ARG;
  if (!std::isfinite(keep) || !std::isfinite(move)) return SPARCML_ERR_INVALID_ARG;
  if (ms.count == 0 || N == 0) return SPARCML_OK;
  if (!typed_ok(update, update_type) || !typed_ok(out, out_type)) return SPARCML_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || ws_bytes < sparcml::ortho_workspace_bytes(ms)) return SPARCML_ERR_WORKSPACE;
  return from_hip(sparcml::ortho_launch(ms, s, update_type, update, out_type, out, is_weight, keep, move, ws, stream));
}

sparcml_status sparcml_orthogonalize(uint64_t N, uint32_t count, const uint64_t* h_offsets, const uint32_t* h_rows,
                                     const uint32_t* h_cols, uint32_t steps, float a, float b, float c, float eps,
                                     uint32_t update_type, const void* update, uint32_t out_type, void* out,
                                     void* ws, size_t ws_bytes, hipStream_t stream) {
  return ortho_common(N, {count, h_offsets, h_rows, h_cols}, {steps, a, b, c, eps}, update_type, update, out_type,
                      out, false, 0.0f, 0.0f, ws, ws_bytes, stream);
}

sparcml_status sparcml_orthogonal_step(uint64_t N, uint32_t count, const uint64_t* h_offsets, const uint32_t* h_rows,
                                       const uint32_t* h_cols, uint32_t steps, float a, float b, float c, float eps,
                                       uint32_t update_type, const void* update, uint32_t weight_type, void* weight,
                                       double lr, double decay, void* ws, size_t ws_bytes, hipStream_t stream) {
  return ortho_common(N, {count, h_offsets, h_rows, h_cols}, {steps, a, b, c, eps}, update_type, update, weight_type,
                      weight, true, (float)(1.0 - lr * decay), (float)lr, ws, ws_bytes, stream);
}

// --------------------------------------------------------------------------
// Measurement entry points: the calls above with caller-owned events
// attached to their kernel dispatches.
// --------------------------------------------------------------------------
static sparcml::OpEvents op_events(const sparcml_bench_events* ev) {
  sparcml::OpEvents e;
  if (ev) {
    e.op_start = ev->op_start;
    e.op_stop = ev->op_stop;
    e.k_start = ev->kernel_start;
    e.k_stop = ev->kernel_stop;
  }
  return e;
}

sparcml_status sparcml_bench_topk_ef(uint32_t P, uint64_t N, uint64_t k, const float* grad, float* residual,
                                     uint32_t* out_idx, float* out_val, void* ws, size_t ws_bytes,
                                     const sparcml_bench_events* ev, hipStream_t stream) {
  const sparcml::OpEvents e = op_events(ev);
  return topk_common(P, N, k, grad, residual, out_idx, out_val, nullptr, ws, ws_bytes, stream, &e);
}

sparcml_status sparcml_bench_topk_ef_runs(uint32_t P, uint64_t N, uint64_t k, const float* grad, float* residual,
                                          uint32_t* out_idx, float* out_val, uint32_t* runs, void* ws,
                                          size_t ws_bytes, const sparcml_bench_events* ev, hipStream_t stream) {
  if (!runs) return SPARCML_ERR_INVALID_ARG;
  const sparcml::OpEvents e = op_events(ev);
  return topk_common(P, N, k, grad, residual, out_idx, out_val, runs, ws, ws_bytes, stream, &e);
}

sparcml_status sparcml_bench_qsgd(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket, uint64_t seed,
                                  uint32_t step, uint32_t node0, const float* val, uint8_t* codes, float* scales,
                                  const sparcml_bench_events* ev, hipStream_t stream) {
  const sparcml::OpEvents e = op_events(ev);
  return qsgd_common(bits, P, n, bucket, seed, step, node0, val, codes, scales, stream, &e);
}

sparcml_status sparcml_bench_dqsgd(uint32_t bits, uint32_t P, uint64_t n, uint32_t bucket, const uint8_t* codes,
                                   const float* scales, float* val, const sparcml_bench_events* ev,
                                   hipStream_t stream) {
  const sparcml::OpEvents e = op_events(ev);
  return dqsgd_common(bits, P, n, bucket, codes, scales, val, stream, &e);
}

sparcml_status sparcml_bench_sparse_reduce(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                           const uint32_t* idx, const float* val, uint64_t expected_nnz_hint,
                                           uint32_t* out_idx, float* out_val, sparcml_reduce_result* d_result,
                                           void* ws, size_t ws_bytes, const sparcml_bench_events* ev,
                                           hipStream_t stream) {
  const sparcml::OpEvents e = op_events(ev);
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, nullptr, expected_nnz_hint, out_idx, out_val,
                       d_result, ws, ws_bytes, stream, &e);
}

sparcml_status sparcml_bench_sparse_reduce_runs(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                                const uint32_t* idx, const float* val, const uint32_t* runs,
                                                uint64_t expected_nnz_hint, uint32_t* out_idx, float* out_val,
                                                sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                                const sparcml_bench_events* ev, hipStream_t stream) {
  if (!runs) return SPARCML_ERR_INVALID_ARG;
  const sparcml::OpEvents e = op_events(ev);
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, runs, expected_nnz_hint, out_idx, out_val,
                       d_result, ws, ws_bytes, stream, &e);
}

sparcml_status sparcml_bench_sparse_reduce_qsgd_runs(uint32_t bits, uint32_t bucket, uint32_t P, uint64_t N,
                                                     double delta, const uint64_t* h_offsets, const uint32_t* idx,
                                                     const uint8_t* codes, const float* scales,
                                                     const uint32_t* runs, uint64_t expected_nnz_hint,
                                                     uint32_t* out_idx, float* out_val,
                                                     sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                                     const sparcml_bench_events* ev, hipStream_t stream) {
  if (!runs) return SPARCML_ERR_INVALID_ARG;
  const sparcml::OpEvents e = op_events(ev);
  return reduce_qsgd_common(bits, bucket, P, N, delta, h_offsets, idx, codes, scales, runs, expected_nnz_hint,
                            out_idx, out_val, d_result, ws, ws_bytes, stream, &e);
}

sparcml_status sparcml_bench_sparse_reduce_union(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                                 const uint32_t* idx, const uint32_t* runs, uint64_t expected_nnz_hint,
                                                 sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                                 const sparcml_bench_events* ev, hipStream_t stream) {
  const sparcml::OpEvents e = op_events(ev);
  return reduce_common(P, N, delta, h_offsets, idx, nullptr, nullptr, runs, expected_nnz_hint, nullptr, nullptr,
                       d_result, ws, ws_bytes, stream, &e, sparcml::kReduceUnion);
}

sparcml_status sparcml_bench_sparse_reduce_sums(uint32_t P, uint64_t N, double delta, const uint64_t* h_offsets,
                                                const uint32_t* idx, const float* val, const uint32_t* runs,
                                                uint64_t expected_nnz_hint, uint32_t* out_idx, float* out_val,
                                                sparcml_reduce_result* d_result, void* ws, size_t ws_bytes,
                                                const sparcml_bench_events* ev, hipStream_t stream) {
  const sparcml::OpEvents e = op_events(ev);
  return reduce_common(P, N, delta, h_offsets, idx, val, nullptr, runs, expected_nnz_hint, out_idx, out_val,
                       d_result, ws, ws_bytes, stream, &e, sparcml::kReduceSums);
}

}  // extern "C"
