"""MI355X (gfx950) SparCML hot path: error-feedback Top-k, 2/4/8-bit stochastic
quantization and sparse reduction with the dense switch; and around it, layer
norm and the norms of queries and keys with per-node gradients, attention and
its gradients, momentum from a reduction's result and orthogonalised updates.

Thin ctypes binding over the C ABI in include/sparcml.h: it checks tensor
dtype/device/contiguity, allocates outputs and workspaces with torch, and
passes raw pointers and the current HIP stream. Every step of the path runs
in the HIP kernels of libsparcml.so; there is no CPU fallback. If the library
is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsparcml.so")
BENCH_LIB_PATH = os.path.join(_PKG, "libsparcml_bench.so")

OK, ERR_INVALID_ARG, ERR_WORKSPACE, ERR_HIP, ERR_SCRATCH_LIMIT = 0, 1, 2, 3, 4
REDUCE_SCRATCH_BYTES = 32 << 20  # SPARCML_REDUCE_SCRATCH_BYTES: static scratch of sparse_reduce_noalloc
FLAG_INDEX_RANGE, FLAG_NOT_ASCENDING = 1, 2

_lib = None


class SparcmlError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = _load().sparcml_status_string(status).decode()
        super().__init__(f"{what}: {msg}")
        self.status = status


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m sparse_gradient_reduction_amd.build` "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(LIB_PATH)
    u32, u64, sz, vp, f64 = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_double
    st = ctypes.c_int
    L.sparcml_status_string.argtypes = [st]
    L.sparcml_status_string.restype = ctypes.c_char_p
    L.sparcml_topk_ef_workspace.argtypes = [u32, u64, u64]
    L.sparcml_topk_ef_workspace.restype = sz
    L.sparcml_topk_ef.argtypes = [u32, u64, u64, vp, vp, vp, vp, vp, sz, vp]
    L.sparcml_topk_ef.restype = st
    L.sparcml_topk_ef_runs.argtypes = [u32, u64, u64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.sparcml_topk_ef_runs.restype = st
    L.sparcml_topk_ef_layers_workspace.argtypes = [u32, u64, u32, vp, vp]
    L.sparcml_topk_ef_layers_workspace.restype = sz
    L.sparcml_topk_ef_layers.argtypes = [u32, u64, u32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.sparcml_topk_ef_layers.restype = st
    L.sparcml_topk_bucketed_count.argtypes = [u64, u32, u32]
    L.sparcml_topk_bucketed_count.restype = u64
    L.sparcml_topk_ef_bucketed.argtypes = [u32, u64, u32, u32, vp, vp, vp, vp, vp]
    L.sparcml_topk_ef_bucketed.restype = st
    L.sparcml_q4.argtypes = [u32, u64, u32, u64, u32, vp, vp, vp, vp]
    L.sparcml_q4.restype = st
    L.sparcml_dq4.argtypes = [u32, u64, u32, vp, vp, vp, vp]
    L.sparcml_dq4.restype = st
    L.sparcml_qsgd.argtypes = [u32, u32, u64, u32, u64, u32, u32, vp, vp, vp, vp]
    L.sparcml_qsgd.restype = st
    L.sparcml_dqsgd.argtypes = [u32, u32, u64, u32, vp, vp, vp, vp]
    L.sparcml_dqsgd.restype = st
    L.sparcml_qsgd_dense_result.argtypes = [u32, u64, u32, u64, u32, u32, vp, vp, vp, vp, vp]
    L.sparcml_qsgd_dense_result.restype = st
    L.sparcml_sparse_reduce_qsgd.argtypes = [u32, u32, u32, u64, f64, vp, vp, vp, vp, u64, vp, vp, vp, vp, sz, vp]
    L.sparcml_sparse_reduce_qsgd.restype = st
    L.sparcml_sparse_reduce_qsgd_runs.argtypes = [u32, u32, u32, u64, f64, vp, vp, vp, vp, vp, u64, vp, vp, vp, vp,
                                                  sz, vp]
    L.sparcml_sparse_reduce_qsgd_runs.restype = st
    L.sparcml_sparse_reduce_workspace.argtypes = [u32, u64, u64]
    L.sparcml_sparse_reduce_workspace.restype = sz
    L.sparcml_sparse_reduce.argtypes = [u32, u64, f64, vp, vp, vp, u64, vp, vp, vp, vp, sz, vp]
    L.sparcml_sparse_reduce.restype = st
    L.sparcml_sparse_reduce_runs.argtypes = [u32, u64, f64, vp, vp, vp, vp, u64, vp, vp, vp, vp, sz, vp]
    L.sparcml_sparse_reduce_runs.restype = st
    L.sparcml_sparse_reduce_union.argtypes = [u32, u64, f64, vp, vp, vp, u64, vp, vp, sz, vp]
    L.sparcml_sparse_reduce_union.restype = st
    L.sparcml_sparse_reduce_sums.argtypes = [u32, u64, f64, vp, vp, vp, vp, u64, vp, vp, vp, vp, sz, vp]
    L.sparcml_sparse_reduce_sums.restype = st
    L.sparcml_sparse_reduce_noalloc.argtypes = [u32, u64, f64, vp, vp, vp, u64, vp, vp, vp, vp]
    L.sparcml_sparse_reduce_noalloc.restype = st
    f32 = ctypes.c_float
    L.sparcml_layer_norm.argtypes = [u32, u64, u32, vp, u64, vp, u64, vp, vp, f32, vp, vp, vp, vp, vp]
    L.sparcml_layer_norm.restype = st
    L.sparcml_layer_norm_backward_workspace.argtypes = [u32, u64, u32]
    L.sparcml_layer_norm_backward_workspace.restype = sz
    L.sparcml_layer_norm_backward.argtypes = [u32, u32, u64, u32, vp, u64, vp, u64, vp, u64, vp, vp, vp, vp, vp, u64,
                                              vp, u64, vp, sz, vp]
    L.sparcml_layer_norm_backward.restype = st
    L.sparcml_head_norm_rotate.argtypes = [vp, vp]
    L.sparcml_head_norm_rotate.restype = st
    L.sparcml_head_norm_rotate_backward_workspace.argtypes = [u32, u64, u32]
    L.sparcml_head_norm_rotate_backward_workspace.restype = sz
    L.sparcml_head_norm_rotate_backward.argtypes = [vp, vp, sz, vp]
    L.sparcml_head_norm_rotate_backward.restype = st
    L.sparcml_attention_workspace.argtypes = [vp]
    L.sparcml_attention_workspace.restype = sz
    L.sparcml_attention.argtypes = [vp, vp, sz, vp]
    L.sparcml_attention.restype = st
    L.sparcml_attention_backward_workspace.argtypes = [vp]
    L.sparcml_attention_backward_workspace.restype = sz
    L.sparcml_attention_backward.argtypes = [vp, vp, sz, vp]
    L.sparcml_attention_backward.restype = st
    L.sparcml_momentum_step.argtypes = [u64, vp, vp, u64, vp, vp, f32, f32, u32, u32, vp, vp]
    L.sparcml_momentum_step.restype = st
    L.sparcml_orthogonalize_workspace.argtypes = [u64, u32, vp, vp, vp]
    L.sparcml_orthogonalize_workspace.restype = sz
    L.sparcml_orthogonalize.argtypes = [u64, u32, vp, vp, vp, u32, f32, f32, f32, f32, u32, vp, u32, vp, vp, sz, vp]
    L.sparcml_orthogonalize.restype = st
    L.sparcml_orthogonal_step.argtypes = [u64, u32, vp, vp, vp, u32, f32, f32, f32, f32, u32, vp, u32, vp, f64, f64,
                                          vp, sz, vp]
    L.sparcml_orthogonal_step.restype = st
    L.sparcml_estimate_nnz.argtypes = [u32, u64, vp]
    L.sparcml_estimate_nnz.restype = f64
    ev = ctypes.POINTER(BenchEvents)
    L.sparcml_bench_topk_ef.argtypes = [u32, u64, u64, vp, vp, vp, vp, vp, sz, ev, vp]
    L.sparcml_bench_topk_ef.restype = st
    L.sparcml_bench_topk_ef_runs.argtypes = [u32, u64, u64, vp, vp, vp, vp, vp, vp, sz, ev, vp]
    L.sparcml_bench_topk_ef_runs.restype = st
    L.sparcml_bench_qsgd.argtypes = [u32, u32, u64, u32, u64, u32, u32, vp, vp, vp, ev, vp]
    L.sparcml_bench_qsgd.restype = st
    L.sparcml_bench_dqsgd.argtypes = [u32, u32, u64, u32, vp, vp, vp, ev, vp]
    L.sparcml_bench_dqsgd.restype = st
    L.sparcml_bench_sparse_reduce.argtypes = [u32, u64, f64, vp, vp, vp, u64, vp, vp, vp, vp, sz, ev, vp]
    L.sparcml_bench_sparse_reduce.restype = st
    L.sparcml_bench_sparse_reduce_runs.argtypes = [u32, u64, f64, vp, vp, vp, vp, u64, vp, vp, vp, vp, sz, ev, vp]
    L.sparcml_bench_sparse_reduce_runs.restype = st
    L.sparcml_bench_sparse_reduce_union.argtypes = [u32, u64, f64, vp, vp, vp, u64, vp, vp, sz, ev, vp]
    L.sparcml_bench_sparse_reduce_union.restype = st
    L.sparcml_bench_sparse_reduce_sums.argtypes = [u32, u64, f64, vp, vp, vp, vp, u64, vp, vp, vp, vp, sz, ev, vp]
    L.sparcml_bench_sparse_reduce_sums.restype = st
    L.sparcml_bench_sparse_reduce_qsgd_runs.argtypes = [u32, u32, u32, u64, f64, vp, vp, vp, vp, vp, u64, vp, vp, vp,
                                                        vp, sz, ev, vp]
    L.sparcml_bench_sparse_reduce_qsgd_runs.restype = st
    _lib = L
    return L


def lib():
    """The loaded ctypes handle of libsparcml.so."""
    return _load()


class BenchEvents(ctypes.Structure):
    """sparcml_bench_events: HIP events (raw handles, or None) that the
    measurement entry points attach to kernel dispatches."""
    _fields_ = [("op_start", ctypes.c_void_p), ("op_stop", ctypes.c_void_p),
                ("kernel_start", ctypes.c_void_p), ("kernel_stop", ctypes.c_void_p)]


_bench_lib = None


def bench_lib():
    """The loaded ctypes handle of libsparcml_bench.so (measurement only: the
    bandwidth reference kernel)."""
    global _bench_lib
    if _bench_lib is None:
        if not os.path.exists(BENCH_LIB_PATH):
            raise RuntimeError(f"{BENCH_LIB_PATH} is not built; run `python -m sparse_gradient_reduction_amd.build`")
        L = ctypes.CDLL(BENCH_LIB_PATH)
        L.sparcml_bench_reference_stream.argtypes = [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.POINTER(BenchEvents), ctypes.c_void_p]
        L.sparcml_bench_reference_stream.restype = ctypes.c_int
        _bench_lib = L
    return _bench_lib


# the current stream's handle without a Stream object, which takes 3 us; not every torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device.index)


def _check_dev(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor on a GPU")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()  # 0 where there are no elements


def _raise(status: int, what: str):
    if status != OK:
        raise SparcmlError(status, what)


# ---------------------------------------------------------------------------
def topk_ef_workspace_bytes(P: int, N: int, k: int) -> int:
    return int(_load().sparcml_topk_ef_workspace(P, N, k))


SEGMENT = 4096  # indices per segment of a run table (SPARCML_SEGMENT)


def run_table_shape(P: int, N: int):
    """Shape of the run table of P sorted contributions over N indices."""
    return (P, (N + SEGMENT - 1) // SEGMENT + 1)


def topk_ef(grad: torch.Tensor, residual: torch.Tensor, k: int, out_idx: Optional[torch.Tensor] = None,
            out_val: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            events: Optional[BenchEvents] = None, runs: Optional[torch.Tensor] = None):
    """Error-feedback Top-k on [P, N] fp32 `grad`; `residual` is updated in place.
    Returns (idx [P, k] int32 holding uint32 indices, val [P, k] float32).
    `runs` (int32 tensor of run_table_shape(P, N)) routes the call through
    sparcml_topk_ef_runs, which also writes the run table of the output.
    `events` (measurement only) routes the call through sparcml_bench_topk_ef(_runs)."""
    _check_dev(grad, torch.float32, "grad")
    _check_dev(residual, torch.float32, "residual")
    if grad.dim() != 2 or grad.shape != residual.shape:
        raise ValueError("grad and residual must both be [P, N]")
    P, N = grad.shape
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty((P, k), dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty((P, k), dtype=torch.float32, device=dev)
    need = topk_ef_workspace_bytes(P, N, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    L = _load()
    s = ctypes.c_void_p(_stream(dev))
    if runs is not None:
        _check_dev(runs, torch.int32, "runs")
        if tuple(runs.shape) != run_table_shape(P, N) or not runs.is_contiguous():
            raise ValueError(f"runs must be a contiguous {run_table_shape(P, N)} tensor")
        if events is None:
            st = L.sparcml_topk_ef_runs(P, N, k, _ptr(grad), _ptr(residual), _ptr(out_idx), _ptr(out_val),
                                        _ptr(runs), _ptr(workspace), workspace.numel(), s)
        else:
            st = L.sparcml_bench_topk_ef_runs(P, N, k, _ptr(grad), _ptr(residual), _ptr(out_idx), _ptr(out_val),
                                              _ptr(runs), _ptr(workspace), workspace.numel(), ctypes.byref(events),
                                              s)
        _raise(st, "sparcml_topk_ef_runs")
        return out_idx, out_val
    if events is None:
        st = L.sparcml_topk_ef(P, N, k, _ptr(grad), _ptr(residual), _ptr(out_idx), _ptr(out_val),
                               _ptr(workspace), workspace.numel(), s)
    else:
        st = L.sparcml_bench_topk_ef(P, N, k, _ptr(grad), _ptr(residual), _ptr(out_idx), _ptr(out_val),
                                     _ptr(workspace), workspace.numel(), ctypes.byref(events), s)
    _raise(st, "sparcml_topk_ef")
    return out_idx, out_val


def _u64s(xs):
    xs = [int(x) for x in xs]
    return (ctypes.c_uint64 * len(xs))(*xs)


def topk_ef_layers_workspace_bytes(P: int, N: int, layer_offsets: Sequence[int], ks: Sequence[int]) -> int:
    return int(_load().sparcml_topk_ef_layers_workspace(P, N, len(ks), _u64s(layer_offsets), _u64s(ks)))


def topk_ef_layers(grad: torch.Tensor, residual: torch.Tensor, layer_offsets: Sequence[int], ks: Sequence[int],
                   out_idx: Optional[torch.Tensor] = None, out_val: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Error-feedback Top-k of every layer [off[l], off[l+1]) of every node,
    keeping ks[l] of layer l; `residual` is updated in place. Returns (idx
    [P, sum ks] int32 holding node-relative uint32 indices, val [P, sum ks])."""
    _check_dev(grad, torch.float32, "grad")
    _check_dev(residual, torch.float32, "residual")
    if grad.dim() != 2 or grad.shape != residual.shape:
        raise ValueError("grad and residual must both be [P, N]")
    P, N = grad.shape
    K = sum(int(x) for x in ks)
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty((P, K), dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty((P, K), dtype=torch.float32, device=dev)
    need = topk_ef_layers_workspace_bytes(P, N, layer_offsets, ks)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    st = _load().sparcml_topk_ef_layers(P, N, len(ks), _u64s(layer_offsets), _u64s(ks), _ptr(grad), _ptr(residual),
                                        _ptr(out_idx), _ptr(out_val), _ptr(workspace), workspace.numel(),
                                        ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_topk_ef_layers")
    return out_idx, out_val


def topk_bucketed_count(N: int, bucket: int, k_per_bucket: int) -> int:
    return int(_load().sparcml_topk_bucketed_count(N, bucket, k_per_bucket))


def topk_ef_bucketed(grad: torch.Tensor, residual: torch.Tensor, bucket: int, k_per_bucket: int,
                     out_idx: Optional[torch.Tensor] = None, out_val: Optional[torch.Tensor] = None):
    """Error-feedback Top-k within every bucket of `bucket` positions (64 ..
    1024, a power of two); `residual` is updated in place. Returns (idx [P, K]
    int32 holding uint32 indices, val [P, K] float32), K = topk_bucketed_count."""
    _check_dev(grad, torch.float32, "grad")
    _check_dev(residual, torch.float32, "residual")
    if grad.dim() != 2 or grad.shape != residual.shape:
        raise ValueError("grad and residual must both be [P, N]")
    P, N = grad.shape
    K = topk_bucketed_count(N, bucket, k_per_bucket)
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty((P, K), dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty((P, K), dtype=torch.float32, device=dev)
    st = _load().sparcml_topk_ef_bucketed(P, N, bucket, k_per_bucket, _ptr(grad), _ptr(residual), _ptr(out_idx),
                                          _ptr(out_val), ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_topk_ef_bucketed")
    return out_idx, out_val


TOPK_ROW_MAX = 1 << 17  # SPARCML_TOPK_ROW_MAX: rows this short are selected by one workgroup per node ...
TOPK_ROW_TOTAL_MAX = 1 << 24  # SPARCML_TOPK_ROW_TOTAL_MAX: ... in calls of at most this many elements


def topk_ef_paths(workspace: torch.Tensor, P: int) -> torch.Tensor:
    """Per node, which path the last sparcml_topk_ef in `workspace` took
    (0 candidates, 1 exact rescan, 2 one workgroup over a short row), and its
    consistency flag: [2, P] int32."""
    return workspace[: 8 * P].view(torch.int32).view(2, P)


# ---------------------------------------------------------------------------
def q4(val: torch.Tensor, bucket: int, seed: int, step: int, codes: Optional[torch.Tensor] = None,
       scales: Optional[torch.Tensor] = None, events: Optional[BenchEvents] = None):
    """[P, n] fp32 -> (codes [P, ceil(n/2)] uint8, scales [P, ceil(n/bucket)] fp32)."""
    _check_dev(val, torch.float32, "val")
    P, n = val.shape
    dev = val.device
    if codes is None:
        codes = torch.empty((P, (n + 1) // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((P, (n + bucket - 1) // bucket), dtype=torch.float32, device=dev)
    if events is None:
        st = _load().sparcml_q4(P, n, bucket, seed & ((1 << 64) - 1), step, _ptr(val), _ptr(codes), _ptr(scales),
                                ctypes.c_void_p(_stream(dev)))
    else:  # measurement: the same call with events on its kernel
        st = _load().sparcml_bench_qsgd(4, P, n, bucket, seed & ((1 << 64) - 1), step, 0, _ptr(val), _ptr(codes),
                                        _ptr(scales), ctypes.byref(events), ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_q4")
    return codes, scales


def dq4(codes: torch.Tensor, scales: torch.Tensor, n: int, bucket: int, out: Optional[torch.Tensor] = None,
        events: Optional[BenchEvents] = None):
    _check_dev(codes, torch.uint8, "codes")
    _check_dev(scales, torch.float32, "scales")
    P = codes.shape[0]
    if out is None:
        out = torch.empty((P, n), dtype=torch.float32, device=codes.device)
    if events is None:
        st = _load().sparcml_dq4(P, n, bucket, _ptr(codes), _ptr(scales), _ptr(out),
                                 ctypes.c_void_p(_stream(codes.device)))
    else:  # measurement: the same call with events on its kernel
        st = _load().sparcml_bench_dqsgd(4, P, n, bucket, _ptr(codes), _ptr(scales), _ptr(out), ctypes.byref(events),
                                         ctypes.c_void_p(_stream(codes.device)))
    _raise(st, "sparcml_dq4")
    return out


def qsgd_row_bytes(bits: int, n: int) -> int:
    return (n * bits + 7) // 8


def qsgd(val: torch.Tensor, bits: int, bucket: int, seed: int, step: int, node0: int = 0,
         codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """b-bit (2, 4, 8) stochastic quantization of [P, n] fp32; row p is node
    node0 + p. Returns (codes [P, ceil(n*bits/8)] uint8, scales [P, ceil(n/bucket)] fp32)."""
    _check_dev(val, torch.float32, "val")
    P, n = val.shape
    dev = val.device
    if codes is None:
        codes = torch.empty((P, qsgd_row_bytes(bits, n)), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((P, (n + bucket - 1) // bucket), dtype=torch.float32, device=dev)
    st = _load().sparcml_qsgd(bits, P, n, bucket, seed & ((1 << 64) - 1), step, node0, _ptr(val), _ptr(codes),
                              _ptr(scales), ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_qsgd")
    return codes, scales


def dqsgd(codes: torch.Tensor, scales: torch.Tensor, n: int, bits: int, bucket: int,
          out: Optional[torch.Tensor] = None):
    _check_dev(codes, torch.uint8, "codes")
    _check_dev(scales, torch.float32, "scales")
    P = codes.shape[0]
    if out is None:
        out = torch.empty((P, n), dtype=torch.float32, device=codes.device)
    st = _load().sparcml_dqsgd(bits, P, n, bucket, _ptr(codes), _ptr(scales), _ptr(out),
                               ctypes.c_void_p(_stream(codes.device)))
    _raise(st, "sparcml_dqsgd")
    return out


# ---------------------------------------------------------------------------
def dense_threshold(delta: float, N: int) -> int:
    t = math.ceil(delta * float(N))
    return max(0, min(t, N + 1))


def sparse_reduce_workspace_bytes(P: int, N: int, total_nnz: int) -> int:
    return int(_load().sparcml_sparse_reduce_workspace(P, N, total_nnz))


def estimate_nnz(offsets: Sequence[int], N: int) -> float:
    off = (ctypes.c_uint64 * len(offsets))(*[int(x) for x in offsets])
    return float(_load().sparcml_estimate_nnz(len(offsets) - 1, N, off))


class ReduceOutput:
    """Device-resident result of sparse_reduce. `result` is a 16-byte tensor
    holding sparcml_reduce_result; `read()` copies it to the host."""

    def __init__(self, result, out_idx, out_val, N):
        self.result, self.out_idx, self.out_val, self.N = result, out_idx, out_val, N

    def read(self):
        r = self.result.cpu()
        nnz = int(r[:8].view(torch.int64).item())
        is_dense = bool(r[8:12].view(torch.int32).item())
        flags = int(r[12:16].view(torch.int32).item())
        return nnz, is_dense, flags

    def host(self):
        """(K, is_dense, flags, idx, val) as host tensors: dense -> idx empty, val [N];
        sparse -> idx [K] int64, val [K]."""
        K, dense, flags = self.read()
        if dense:
            return K, True, flags, torch.zeros(0, dtype=torch.int64), self.out_val[: self.N].cpu()
        idx = self.out_idx[:K].cpu().to(torch.int64) & 0xFFFFFFFF
        return K, False, flags, idx, self.out_val[:K].cpu()


def _reduce_outputs(offsets, N, delta, dev, out_idx, out_val, result, workspace):
    P = len(offsets) - 1
    T = dense_threshold(delta, N)
    cap = 0 if T == 0 else min(N, T - 1)
    if out_idx is None:
        out_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(N, dtype=torch.float32, device=dev)
    if result is None:
        result = torch.zeros(16, dtype=torch.uint8, device=dev)
    need = sparse_reduce_workspace_bytes(P, N, int(offsets[-1]))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    return out_idx, out_val, result, workspace


def sparse_reduce_qsgd(offsets: Sequence[int], idx: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                       bits: int, bucket: int, N: int, delta: float, expected_nnz_hint: int = 0,
                       out_idx: Optional[torch.Tensor] = None, out_val: Optional[torch.Tensor] = None,
                       result: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, runs: Optional[torch.Tensor] = None,
                       events: Optional[BenchEvents] = None) -> "ReduceOutput":
    """sparse_reduce with node p's values given as b-bit codes: node p's code
    row starts at byte sum_{q<p} ceil(nnz_q*bits/8), its scales at
    sum_{q<p} ceil(nnz_q/bucket) (the layout qsgd writes when every node has
    the same count). `runs` (the run table, as for sparse_reduce) routes the
    call through sparcml_sparse_reduce_qsgd_runs, and with `events`
    (measurement only) through sparcml_bench_sparse_reduce_qsgd_runs."""
    _check_dev(idx, torch.int32, "idx")
    _check_dev(codes, torch.uint8, "codes")
    _check_dev(scales, torch.float32, "scales")
    P = len(offsets) - 1
    off = (ctypes.c_uint64 * (P + 1))(*[int(x) for x in offsets])
    dev = idx.device
    out_idx, out_val, result, workspace = _reduce_outputs(offsets, N, delta, dev, out_idx, out_val, result,
                                                          workspace)
    if runs is not None:
        _check_dev(runs, torch.int32, "runs")
        if tuple(runs.shape) != run_table_shape(P, N):
            raise ValueError(f"runs must be a contiguous {run_table_shape(P, N)} tensor")
        s = ctypes.c_void_p(_stream(dev))
        if events is None:
            st = _load().sparcml_sparse_reduce_qsgd_runs(bits, bucket, P, N, float(delta), off, _ptr(idx), _ptr(codes),
                                                         _ptr(scales), _ptr(runs), int(expected_nnz_hint),
                                                         _ptr(out_idx), _ptr(out_val), _ptr(result), _ptr(workspace),
                                                         workspace.numel(), s)
        else:
            st = _load().sparcml_bench_sparse_reduce_qsgd_runs(bits, bucket, P, N, float(delta), off, _ptr(idx),
                                                               _ptr(codes), _ptr(scales), _ptr(runs),
                                                               int(expected_nnz_hint), _ptr(out_idx), _ptr(out_val),
                                                               _ptr(result), _ptr(workspace), workspace.numel(),
                                                               ctypes.byref(events), s)
        _raise(st, "sparcml_sparse_reduce_qsgd_runs")
        return ReduceOutput(result, out_idx, out_val, N)
    if events is not None:
        raise ValueError("events need the run table (sparcml_bench_sparse_reduce_qsgd_runs)")
    st = _load().sparcml_sparse_reduce_qsgd(bits, bucket, P, N, float(delta), off, _ptr(idx), _ptr(codes),
                                            _ptr(scales), int(expected_nnz_hint), _ptr(out_idx), _ptr(out_val),
                                            _ptr(result), _ptr(workspace), workspace.numel(),
                                            ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_sparse_reduce_qsgd")
    return ReduceOutput(result, out_idx, out_val, N)


def qsgd_dense_result(out: "ReduceOutput", bits: int, bucket: int, seed: int, step: int, node: int = 0,
                      codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """Quantize the reduction's dense result on the device if (and only if)
    it turned out dense; codes/scales are left untouched otherwise. Returns
    (codes [ceil(N*bits/8)] uint8, scales [ceil(N/bucket)] fp32)."""
    N = out.N
    dev = out.out_val.device
    if codes is None:
        codes = torch.zeros(qsgd_row_bytes(bits, N), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.zeros((N + bucket - 1) // bucket, dtype=torch.float32, device=dev)
    _check_dev(codes, torch.uint8, "codes")
    _check_dev(scales, torch.float32, "scales")
    st = _load().sparcml_qsgd_dense_result(bits, N, bucket, seed & ((1 << 64) - 1), step, node, _ptr(out.result),
                                           _ptr(out.out_val), _ptr(codes), _ptr(scales),
                                           ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_qsgd_dense_result")
    return codes, scales


def sparse_reduce(offsets: Sequence[int], idx: torch.Tensor, val: torch.Tensor, N: int, delta: float,
                  expected_nnz_hint: int = 0, out_idx: Optional[torch.Tensor] = None,
                  out_val: Optional[torch.Tensor] = None, result: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, events: Optional[BenchEvents] = None,
                  runs: Optional[torch.Tensor] = None) -> ReduceOutput:
    """Sum of P sparse contributions (node p owns pairs [offsets[p], offsets[p+1])).
    idx: int32 tensor holding uint32 indices, val: float32 tensor. `runs`, the
    run table of these pairs (int32, run_table_shape(P, N), as topk_ef(runs=...)
    writes it), routes the call through sparcml_sparse_reduce_runs. `events`
    (measurement only) routes the call through sparcml_bench_sparse_reduce(_runs)."""
    _check_dev(idx, torch.int32, "idx")
    _check_dev(val, torch.float32, "val")
    P = len(offsets) - 1
    off = (ctypes.c_uint64 * (P + 1))(*[int(x) for x in offsets])
    dev = idx.device
    out_idx, out_val, result, workspace = _reduce_outputs(offsets, N, delta, dev, out_idx, out_val, result,
                                                          workspace)
    if runs is not None:
        _check_dev(runs, torch.int32, "runs")
        if tuple(runs.shape) != run_table_shape(P, N) or not runs.is_contiguous():
            raise ValueError(f"runs must be a contiguous {run_table_shape(P, N)} tensor")
        s = ctypes.c_void_p(_stream(dev))
        if events is None:
            st = _load().sparcml_sparse_reduce_runs(P, N, float(delta), off, _ptr(idx), _ptr(val), _ptr(runs),
                                                    int(expected_nnz_hint), _ptr(out_idx), _ptr(out_val),
                                                    _ptr(result), _ptr(workspace), workspace.numel(), s)
        else:
            st = _load().sparcml_bench_sparse_reduce_runs(P, N, float(delta), off, _ptr(idx), _ptr(val), _ptr(runs),
                                                          int(expected_nnz_hint), _ptr(out_idx), _ptr(out_val),
                                                          _ptr(result), _ptr(workspace), workspace.numel(),
                                                          ctypes.byref(events), s)
        _raise(st, "sparcml_sparse_reduce_runs")
        return ReduceOutput(result, out_idx, out_val, N)
    if events is None:
        st = _load().sparcml_sparse_reduce(P, N, float(delta), off, _ptr(idx), _ptr(val), int(expected_nnz_hint),
                                           _ptr(out_idx), _ptr(out_val), _ptr(result), _ptr(workspace),
                                           workspace.numel(), ctypes.c_void_p(_stream(dev)))
    else:
        st = _load().sparcml_bench_sparse_reduce(P, N, float(delta), off, _ptr(idx), _ptr(val),
                                                 int(expected_nnz_hint), _ptr(out_idx), _ptr(out_val), _ptr(result),
                                                 _ptr(workspace), workspace.numel(), ctypes.byref(events),
                                                 ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_sparse_reduce")
    return ReduceOutput(result, out_idx, out_val, N)


class ReduceUnion:
    """What sparse_reduce_union prepared for sparse_reduce_sums: the call's
    arguments and the device buffers (workspace, result record) it filled."""

    def __init__(self, offsets, off, idx, N, delta, runs, hint, result, workspace):
        self.offsets, self.off, self.idx, self.N, self.delta = offsets, off, idx, N, delta
        self.runs, self.hint, self.result, self.workspace = runs, hint, result, workspace


def _check_runs(runs, P, N):
    _check_dev(runs, torch.int32, "runs")
    if tuple(runs.shape) != run_table_shape(P, N):
        raise ValueError(f"runs must be a contiguous {run_table_shape(P, N)} tensor")


def sparse_reduce_union(offsets: Sequence[int], idx: torch.Tensor, N: int, delta: float,
                        runs: Optional[torch.Tensor] = None, expected_nnz_hint: int = 0,
                        result: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        events: Optional[BenchEvents] = None) -> ReduceUnion:
    """The union phase of the sparse reduce (indices only): run starts, union
    bitmaps and counts, K and the dense decision. sparse_reduce_sums then
    adds the values; together they give sparse_reduce's result."""
    _check_dev(idx, torch.int32, "idx")
    P = len(offsets) - 1
    off = (ctypes.c_uint64 * (P + 1))(*[int(x) for x in offsets])
    dev = idx.device
    if runs is not None:
        _check_runs(runs, P, N)
    if result is None:
        result = torch.zeros(16, dtype=torch.uint8, device=dev)
    if workspace is None:
        need = sparse_reduce_workspace_bytes(P, N, int(offsets[-1]))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    s = ctypes.c_void_p(_stream(dev))
    args = (P, N, float(delta), off, _ptr(idx), _ptr(runs), int(expected_nnz_hint), _ptr(result), _ptr(workspace),
            workspace.numel())
    if events is None:
        st = _load().sparcml_sparse_reduce_union(*args, s)
    else:
        st = _load().sparcml_bench_sparse_reduce_union(*args, ctypes.byref(events), s)
    _raise(st, "sparcml_sparse_reduce_union")
    return ReduceUnion(offsets, off, idx, N, delta, runs, int(expected_nnz_hint), result, workspace)


def sparse_reduce_sums(u: ReduceUnion, val: torch.Tensor, out_idx: Optional[torch.Tensor] = None,
                       out_val: Optional[torch.Tensor] = None,
                       events: Optional[BenchEvents] = None) -> ReduceOutput:
    """The sums phase after sparse_reduce_union (same stream, the indices,
    table and workspace unchanged in between)."""
    _check_dev(val, torch.float32, "val")
    P = len(u.offsets) - 1
    dev = val.device
    out_idx, out_val, result, workspace = _reduce_outputs(u.offsets, u.N, u.delta, dev, out_idx, out_val, u.result,
                                                          u.workspace)
    s = ctypes.c_void_p(_stream(dev))
    args = (P, u.N, float(u.delta), u.off, _ptr(u.idx), _ptr(val), _ptr(u.runs), u.hint, _ptr(out_idx),
            _ptr(out_val), _ptr(result), _ptr(workspace), workspace.numel())
    if events is None:
        st = _load().sparcml_sparse_reduce_sums(*args, s)
    else:
        st = _load().sparcml_bench_sparse_reduce_sums(*args, ctypes.byref(events), s)
    _raise(st, "sparcml_sparse_reduce_sums")
    return ReduceOutput(result, out_idx, out_val, u.N)


def sparse_reduce_noalloc(offsets, idx: torch.Tensor, val: torch.Tensor, N: int, delta: float,
                          out_idx: torch.Tensor, out_val: torch.Tensor, result: torch.Tensor,
                          expected_nnz_hint: int = 0) -> ReduceOutput:
    """sparse_reduce through the allocation-free entry point: the library's
    static per-GPU scratch replaces the workspace, and the caller passes every
    output (out_idx with capacity min(N, T-1), out_val [N], result 16 bytes),
    so nothing is allocated on the device. `offsets` may be a sequence or a
    prepared (ctypes.c_uint64 * (P+1)) array. Calls that overlap in time on
    one GPU share the scratch and race."""
    _check_dev(idx, torch.int32, "idx")
    _check_dev(val, torch.float32, "val")
    _check_dev(out_idx, torch.int32, "out_idx")
    _check_dev(out_val, torch.float32, "out_val")
    _check_dev(result, torch.uint8, "result")
    if isinstance(offsets, ctypes.Array):
        off, P = offsets, len(offsets) - 1
    else:
        P = len(offsets) - 1
        off = (ctypes.c_uint64 * (P + 1))(*[int(x) for x in offsets])
    dev = idx.device
    st = _load().sparcml_sparse_reduce_noalloc(P, N, float(delta), off, _ptr(idx), _ptr(val),
                                               int(expected_nnz_hint), _ptr(out_idx), _ptr(out_val),
                                               _ptr(result), ctypes.c_void_p(_stream(dev)))
    _raise(st, "sparcml_sparse_reduce_noalloc")
    return ReduceOutput(result, out_idx, out_val, N)


# ---------------------------------------------------------------------------
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # SPARCML_F32, SPARCML_BF16, SPARCML_F16


def _type(dtype, name: str) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {dtype}")
    return t


def _row_length(x: torch.Tensor) -> int:
    if not isinstance(x, torch.Tensor) or x.dim() == 0:
        raise TypeError("x must be a tensor of rows")
    cols = x.shape[-1]
    if cols >= 1 << 31:  # more than 2^32 would wrap in the call
        raise ValueError("x's rows must be shorter than 2^31")
    return cols


def _row_stride(t: torch.Tensor, like: torch.Tensor, name: str) -> int:
    """Elements from one row to the next of `t`, a GPU tensor of `like`'s shape
    and type whose rows (the last dimension) are contiguous and evenly spaced."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (t is not like and (t.dtype != like.dtype or
                                                                               t.shape != like.shape)):
        raise TypeError(f"{name} must be a {like.dtype} tensor of shape {tuple(like.shape)} on a GPU")
    if t.is_contiguous():
        return t.shape[-1]
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    step, size = None, 1  # of the dimensions from the inside out
    for d in range(t.dim() - 2, -1, -1):
        n = t.shape[d]
        if n == 1:
            continue
        if step is None:
            step = t.stride(d)
        elif t.stride(d) != step * size:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        size *= n
    return t.shape[-1] if step is None else step


def _vector(t: Optional[torch.Tensor], n: int, name: str):
    if t is not None:
        _check_dev(t, torch.float32, name)
        if t.numel() != n:
            raise ValueError(f"{name} must have {n} elements")


def _workspace(t: Optional[torch.Tensor], need: int, like: torch.Tensor) -> torch.Tensor:
    """The caller's workspace, or a new one on `like`'s device."""
    if t is None:
        return like.new_empty(need, dtype=torch.uint8)
    _check_dev(t, torch.uint8, "workspace")
    if t.device != like.device:
        raise ValueError(f"workspace must be on {like.device}")
    return t


def _given(t: Optional[torch.Tensor], like: torch.Tensor, name: str, shape=None, dtype=None) -> torch.Tensor:
    """The caller's output, or a new one, contiguous, on `like`'s device; of
    its shape and type where none are given."""
    if shape is None:
        if t is None:
            return torch.empty_like(like, memory_format=torch.contiguous_format)
        shape, dtype = like.shape, like.dtype
    elif t is None:
        return like.new_empty(shape, dtype=dtype)
    _check_dev(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
               total: Optional[torch.Tensor] = None):
    """Layer norm over the last dimension of `x` (fp32, bf16 or fp16; rows may
    be slices of a wider buffer), with fp32 `weight` and `bias`. Returns (y,
    mean, rstd), mean and rstd fp32 of x.shape[:-1]; with `residual`, x +
    residual is what is normed, and (y, mean, rstd, total) come back with that sum."""
    cols = _row_length(x)
    t = _type(x.dtype, "x")
    xs = _row_stride(x, x, "x")
    rows = x.numel() // cols if cols else 0
    rs = 0 if residual is None else _row_stride(residual, x, "residual")
    _vector(weight, cols, "weight")
    _vector(bias, cols, "bias")
    dev = x.device
    y = _given(y, x, "y")
    if mean is None and rstd is None:  # one allocation
        mean, rstd = x.new_empty((2,) + x.shape[:-1], dtype=torch.float32).unbind()
    else:
        mean = _given(mean, x, "mean", x.shape[:-1], torch.float32)
        rstd = _given(rstd, x, "rstd", x.shape[:-1], torch.float32)
    if residual is not None:
        total = _given(total, x, "total")
    elif total is not None:
        raise ValueError("total needs a residual")
    st = _load().sparcml_layer_norm(t, rows, cols, _ptr(x), xs, _ptr(residual), rs, _ptr(weight), _ptr(bias), eps,
                                    _ptr(y), _ptr(total), _ptr(mean), _ptr(rstd), _stream(dev))
    _raise(st, "sparcml_layer_norm")
    return (y, mean, rstd) if residual is None else (y, mean, rstd, total)


def layer_norm_backward_workspace_bytes(nodes: int, rows: int, cols: int) -> int:
    if not 0 <= nodes < 1 << 32 or not 0 <= rows < 1 << 64 or not 0 <= cols < 1 << 32:
        raise ValueError("nodes and cols must lie in [0, 2^32), rows in [0, 2^64)")
    return int(_load().sparcml_layer_norm_backward_workspace(nodes, rows, cols))


def _node_rows(t: Optional[torch.Tensor], nodes: int, cols: int, like: torch.Tensor, name: str):
    """A per-node gradient's tensor and the elements from one node to the next."""
    if t is None:
        return like.new_empty((nodes, cols), dtype=torch.float32), cols
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a float32 tensor on a GPU")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if tuple(t.shape) != (nodes, cols) or (cols > 1 and t.stride(1) != 1) or (nodes > 1 and t.stride(0) < cols):
        raise ValueError(f"{name} must be [{nodes}, {cols}] with contiguous rows that do not overlap")
    return t, max(t.stride(0), cols)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, nodes: int = 1, dresidual: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of layer_norm: (dx like x, dweight [nodes, D], dbias [nodes, D],
    both fp32). `x` is what was normed (`total` where there was a residual); its
    rows belong to `nodes` nodes in equal parts, one after the other.
    `dresidual`, the gradient that reaches the residual stream from elsewhere,
    is added to dx. dweight and dbias may be columns of the [P, N] gradients."""
    cols = _row_length(x)
    t = _type(x.dtype, "x")
    xs = _row_stride(x, x, "x")
    ds = _row_stride(dy, x, "dy")
    rs = 0 if dresidual is None else _row_stride(dresidual, x, "dresidual")
    if cols == 0:
        raise ValueError("x's rows are empty")
    rows = x.numel() // cols
    if not 1 <= nodes <= 65535 or rows % nodes:
        raise ValueError(f"{rows} rows do not belong to {nodes} nodes (up to 65535) in equal parts")
    _vector(weight, cols, "weight")
    _check_dev(mean, torch.float32, "mean")
    _check_dev(rstd, torch.float32, "rstd")
    if mean.numel() != rows or rstd.numel() != rows:
        raise ValueError(f"mean and rstd must have {rows} elements")
    dev = x.device
    dx = _given(dx, x, "dx")
    if dweight is None and dbias is None:  # one allocation
        dweight, dbias = x.new_empty((2, nodes, cols), dtype=torch.float32).unbind()
        ws = bs = cols
    else:
        dweight, ws = _node_rows(dweight, nodes, cols, x, "dweight")
        dbias, bs = _node_rows(dbias, nodes, cols, x, "dbias")
    L = _load()
    workspace = _workspace(workspace, L.sparcml_layer_norm_backward_workspace(nodes, rows // nodes, cols), x)
    st = L.sparcml_layer_norm_backward(t, nodes, rows // nodes, cols, _ptr(dy), ds, _ptr(x), xs, _ptr(dresidual), rs,
                                       _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dweight), ws,
                                       _ptr(dbias), bs, _ptr(workspace), workspace.numel(), _stream(dev))
    _raise(st, "sparcml_layer_norm_backward")
    return dx, dweight, dbias


# ---------------------------------------------------------------------------
# sparcml_head_norm_args and sparcml_attention_args; a sparcml_heads is four words
_HEAD_NORM_ARGS = struct.Struct("@7If33Q")
_ATTENTION_ARGS = struct.Struct("@9If35Q")
_NO_HEADS = (0, 0, 0, 0)


def _head_tensor(t: torch.Tensor, dtype, shape, device, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or t.device != device:
        raise TypeError(f"{name} must be a {dtype} tensor on {device if device.type == 'cuda' else 'a GPU'}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _apart(t: torch.Tensor, name: str):
    """Raises unless every element of `t` has a place of its own."""
    end = 1
    for step, n in sorted(zip(t.stride(), t.shape)):
        if n > 1:
            if step < end:
                raise ValueError(f"{name}'s elements must not share a place")
            end = step * (n - 1) + end
    return t


def _output_heads(t: Optional[torch.Tensor], like: torch.Tensor, name: str) -> torch.Tensor:
    """The caller's output, of any strides, or a new contiguous one, of `like`'s shape and type."""
    if t is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _head_tensor(t, like.dtype, like.shape, like.device, name)
    return t if t.numel() == 0 else _apart(t, name)


def _alike(like: torch.Tensor, strides, *tensors) -> bool:
    """Whether `tensors` and `like`, of these strides, are of one type, shape and
    GPU, with contiguous heads: the quick look, before the one that says what is wrong."""
    dtype, shape, dev = like.dtype, like.shape, like.device
    if not like.is_cuda or strides[-1] != 1:
        return False
    for t in tensors:
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.device != dev or t.stride(-1) != 1:
            return False
    return True


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device, call, *args) -> int:
    """call(*args, the current stream of `device`) with that device the current one."""
    if _current_device() == device.index:
        return call(*args, _stream(device))
    with torch.cuda.device(device):
        return call(*args, _stream(device))


def _token_heads(t: torch.Tensor, name: str):
    """sparcml_heads of [..., heads, D] whose tokens are evenly spaced (where there are none, any)."""
    if t.dim() == 3 or t.numel() == 0:
        return t.data_ptr(), 0, t.stride(-3), t.stride(-2)
    step, size = 0, 1  # of the tokens' dimensions from the inside out
    for d in range(t.dim() - 3, -1, -1):
        n = t.shape[d]
        if n == 1:
            continue
        if size == 1:
            step = t.stride(d)
        elif t.stride(d) != step * size:
            raise ValueError(f"{name}'s tokens must be evenly spaced")
        size *= n
    return t.data_ptr(), 0, step, t.stride(-2)


def _head_norm_checks(q, k, q_weight, k_weight, positions, frequencies):
    """(type, tokens, heads, groups, D, rotated) of head_norm_rotate's arguments."""
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() < 2 or k.dim() < 2:
        raise TypeError("q and k must be tensors of [..., heads, D]")
    shape, dev = q.shape, q.device
    heads, cols, groups = shape[-2], shape[-1], k.shape[-2]
    if not (_alike(q, q.stride()) and _alike(k, k.stride()) and k.dtype == q.dtype and k.device == dev
            and k.shape[:-2] == shape[:-2] and k.shape[-1] == cols):
        _head_tensor(q, q.dtype, shape, dev, "q")
        _head_tensor(k, q.dtype, shape[:-2] + (groups, cols), dev, "k")
    tokens = shape[:-2].numel()
    if tokens >= 1 << 31 or max(heads, groups) >= 1 << 16 or min(heads, groups, cols) < 1 or cols > 256:
        raise ValueError("q and k must have 1 to 65535 heads of 1 to 256 elements and fewer than 2^31 tokens")
    if q_weight is not None:
        _dim_vector(q_weight, cols, dev, "q_weight")
    if k_weight is not None:
        _dim_vector(k_weight, cols, dev, "k_weight")
    rotated = 0
    if frequencies is not None:
        rotated = 2 * frequencies.numel()
        _check_dev(frequencies, torch.float64, "frequencies")
        _check_dev(positions, torch.int32, "positions")
        if rotated > cols or positions.numel() != tokens:
            raise ValueError(f"frequencies must have at most {cols // 2} elements, positions {tokens}")
        if frequencies.device != dev or positions.device != dev:
            raise ValueError(f"positions and frequencies must be on {dev}")
    return _type(q.dtype, "q"), tokens, heads, groups, cols, rotated


def _dim_vector(t, cols, device, name):
    _check_dev(t, torch.float32, name)
    if t.device != device or t.numel() != cols:
        raise ValueError(f"{name} must have {cols} elements on {device}")


def rotation_frequencies(rotated: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """base^(-2 i / rotated), i < rotated / 2: the usual frequencies of head_norm_rotate, fp64."""
    if rotated % 2:
        raise ValueError("rotated must be even")
    return base ** (-2.0 * torch.arange(rotated // 2, dtype=torch.float64, device=device) / max(rotated, 1))


def head_norm_rotate(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                     frequencies: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Norms every head of `q` [..., heads, D] and `k` [..., groups, D] (fp32, bf16
    or fp16; views of one projection, say): x / sqrt(mean(x^2) + eps) * weight,
    with fp32 weights of D elements, then turns pair i of its first
    2 * len(frequencies) elements by position * frequencies[i] (int32 positions of
    q.shape[:-2], fp64 frequencies; none: nothing turns, whatever the positions).
    Pair i is elements i and i + len(frequencies), or 2 i and 2 i + 1 where
    `interleaved`. Tokens of several dimensions have to be evenly spaced in memory,
    as those of a contiguous tensor's heads are. Returns (q_out, k_out), which may
    be q and k themselves and overlap nothing else."""
    t, tokens, heads, groups, cols, rotated = _head_norm_checks(q, k, q_weight, k_weight, positions, frequencies)
    q_out, k_out = _output_heads(q_out, q, "q_out"), _output_heads(k_out, k, "k_out")
    args = _HEAD_NORM_ARGS.pack(t, 1, heads, groups, cols, rotated, interleaved, eps, tokens, *_token_heads(q, "q"),
                                *_token_heads(k, "k"), *_token_heads(q_out, "q_out"), *_token_heads(k_out, "k_out"),
                                _ptr(q_weight) or 0, _ptr(k_weight) or 0, _ptr(positions) or 0, _ptr(frequencies) or 0,
                                *_NO_HEADS, *_NO_HEADS, 0, 0, 0, 0)
    st = _on(q.device, _load().sparcml_head_norm_rotate, args)
    if st:
        _raise(st, "sparcml_head_norm_rotate")
    return q_out, k_out


def head_norm_rotate_backward_workspace_bytes(nodes: int, tokens: int, cols: int) -> int:
    """Bytes of the workspace for `tokens` tokens a node."""
    if not 0 <= nodes < 1 << 32 or not 0 <= tokens < 1 << 64 or not 0 <= cols < 1 << 32:
        raise ValueError("nodes and cols must lie in [0, 2^32), tokens in [0, 2^64)")
    return int(_load().sparcml_head_norm_rotate_backward_workspace(nodes, tokens, cols))


def head_norm_rotate_backward(dq: torch.Tensor, dk: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                              positions: Optional[torch.Tensor] = None, frequencies: Optional[torch.Tensor] = None,
                              eps: float = 1e-6, interleaved: bool = False, nodes: int = 1,
                              q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                              dq_weight: Optional[torch.Tensor] = None, dk_weight: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None):
    """Gradients of head_norm_rotate, with `dq` and `dk` those of its results and
    `q` and `k` its inputs: (like q, like k, dq_weight [nodes, D], dk_weight
    [nodes, D], both fp32). The tokens belong to `nodes` nodes in equal parts, one
    after the other. q_out and k_out may be dq and dk (or q and k); dq_weight and
    dk_weight may be columns of the [P, N] gradients. Apart from that nothing that
    is written may overlap anything else."""
    t, tokens, heads, groups, cols, rotated = _head_norm_checks(q, k, q_weight, k_weight, positions, frequencies)
    if not (_alike(q, q.stride(), dq) and _alike(k, k.stride(), dk)):
        _head_tensor(dq, q.dtype, q.shape, q.device, "dq")
        _head_tensor(dk, k.dtype, k.shape, q.device, "dk")
    if not 1 <= nodes <= 65535 or tokens % nodes:
        raise ValueError(f"{tokens} tokens do not belong to {nodes} nodes (up to 65535) in equal parts")
    q_out, k_out = _output_heads(q_out, q, "q_out"), _output_heads(k_out, k, "k_out")
    if dq_weight is None and dk_weight is None:  # one allocation
        dq_weight, dk_weight = q.new_empty((2, nodes, cols), dtype=torch.float32).unbind()
        qs = ks = cols
    else:
        dq_weight, qs = _node_rows(dq_weight, nodes, cols, q, "dq_weight")
        dk_weight, ks = _node_rows(dk_weight, nodes, cols, q, "dk_weight")
    L = _load()
    ws, n, workspace = _call_workspace(
        workspace, L.sparcml_head_norm_rotate_backward_workspace(nodes, tokens // nodes, cols), q)
    args = _HEAD_NORM_ARGS.pack(t, nodes, heads, groups, cols, rotated, interleaved, eps, tokens // nodes,
                                *_token_heads(q, "q"), *_token_heads(k, "k"), *_token_heads(q_out, "q_out"),
                                *_token_heads(k_out, "k_out"), _ptr(q_weight) or 0, _ptr(k_weight) or 0,
                                _ptr(positions) or 0, _ptr(frequencies) or 0, *_token_heads(dq, "dq"),
                                *_token_heads(dk, "dk"), dq_weight.data_ptr(), dk_weight.data_ptr(), qs, ks)
    st = _on(q.device, L.sparcml_head_norm_rotate_backward, args, ws, n)
    _raise(st, "sparcml_head_norm_rotate_backward")
    return q_out, k_out, dq_weight, dk_weight


# ---------------------------------------------------------------------------
def _attention_checks(q, k, v, causal, window, scale, q_lengths, k_lengths):
    """The first words of sparcml_attention_args: sizes, mask, scale, lengths, q, k and v."""
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 4 or k.dim() != 4:
        raise TypeError("q, k and v must be tensors of [batch, tokens, heads, D]")
    shape, dtype, dev = q.shape, q.dtype, q.device
    batch, queries, heads, cols = shape
    k_batch, keys, groups, k_cols = k.shape
    qs, ks = q.stride(), k.stride()
    if not (_alike(q, qs) and _alike(k, ks, v) and k.dtype == dtype and k.device == dev and k_batch == batch and k_cols == cols):
        _head_tensor(q, dtype, shape, dev, "q")
        shape = (batch, keys, groups, cols)
        _head_tensor(k, dtype, shape, dev, "k")
        _head_tensor(v, dtype, shape, dev, "v")
    if batch > 65535 or queries >= 1 << 29 or keys >= 1 << 29 or heads > 65535 or not 1 <= cols <= 128:
        raise ValueError("up to 65535 sequences and heads of 1 to 128 elements, fewer than 2^29 queries and keys")
    if groups < 1 or heads < 1 or heads % groups:
        raise ValueError(f"{heads} heads do not share {groups} groups of keys and values in equal parts")
    if scale is None:
        scale = cols ** -0.5
    elif not 1e-30 <= scale <= 1e30:
        raise ValueError("scale must lie between 1e-30 and 1e30")
    n = m = 0
    if q_lengths is not None:
        n = _lengths(q_lengths, batch, dev, "q_lengths")
    if k_lengths is not None:
        m = _lengths(k_lengths, batch, dev, "k_lengths")
    before = 0xFFFFFFFF
    if window is not None:
        if window < 1:
            raise ValueError("window must be at least 1")
        before = min(window - 1, before)
    t = _TYPES.get(dtype)
    vs = v.stride()
    return (_type(dtype, "q") if t is None else t, batch, queries, keys, heads, groups, cols, before,
            0 if causal else before, scale, n, m, q.data_ptr(), qs[0], qs[1], qs[2], k.data_ptr(), ks[0], ks[1], ks[2],
            v.data_ptr(), vs[0], vs[1], vs[2])


def _lengths(t, batch, device, name):
    _check_dev(t, torch.int32, name)
    if t.device != device or t.numel() != batch:
        raise ValueError(f"{name} must have {batch} elements on {device}")
    return t.data_ptr()


def _batch_heads(t: torch.Tensor):
    b, n, h, _ = t.stride()
    return t.data_ptr(), b, n, h


def _call_workspace(t: Optional[torch.Tensor], need: int, like: torch.Tensor):
    """(address, bytes) of the caller's workspace or a new one, and the tensor that keeps it."""
    if t is None and need == 0:
        return 0, 0, None
    t = _workspace(t, need, like)
    return t.data_ptr(), t.numel(), t


def attention_workspace_bytes(q: torch.Tensor, k: torch.Tensor, backward: bool = False) -> int:
    """Bytes of the workspace that is enough for attention or, `backward`,
    attention_backward of queries and keys like these, whatever the mask."""
    args = _ATTENTION_ARGS.pack(*_attention_checks(q, k, k, False, None, None, None, None), *([0] * 21))
    return int((_load().sparcml_attention_backward_workspace if backward else _load().sparcml_attention_workspace)(args))


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False, window: Optional[int] = None,
              scale: Optional[float] = None, q_lengths: Optional[torch.Tensor] = None,
              k_lengths: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """softmax(scale * q k^T) v for `q` [batch, queries, heads, D] and `k`, `v`
    [batch, keys, groups, D] (fp32, bf16 or fp16, D up to 128, any strides); heads /
    groups query heads share a key and value head. Returns (out like q, lse
    [batch, heads, queries] fp32), lse the logarithm of each row's sum.

    Query i of n sees the keys j of m with j <= i + m - n where `causal`, and less
    than `window` away from i + m - n where that is given. `q_lengths`, `k_lengths`
    [batch] int32 are each sequence's own n and m: what lies behind is not read,
    rows of out there are 0 and lse -inf, as where a query sees nothing. scale:
    1 / sqrt(D) if none is given, else 1e-30 to 1e30. With 16-bit types the
    probabilities are rounded to the type for their product with v, sums are fp32.
    out and lse overlap nothing else."""
    head = _attention_checks(q, k, v, causal, window, scale, q_lengths, k_lengths)
    out = _output_heads(out, q, "out")
    if lse is None:
        lse = q.new_empty((head[1], head[4], head[2]), dtype=torch.float32)
    else:
        _check_lse(lse, head, q)
    args = _ATTENTION_ARGS.pack(*head, *_batch_heads(out), lse.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    L = _load()
    st = ERR_WORKSPACE
    if workspace is None:  # most calls need none; those that do say so
        st = _on(q.device, L.sparcml_attention, args, 0, 0)
    if st == ERR_WORKSPACE:
        ws, n, workspace = _call_workspace(workspace, L.sparcml_attention_workspace(args), q)
        st = _on(q.device, L.sparcml_attention, args, ws, n)
    if st:
        _raise(st, "sparcml_attention")
    return out, lse


def _check_lse(lse, head, q):
    _check_dev(lse, torch.float32, "lse")
    if lse.shape != (head[1], head[4], head[2]) or lse.device != q.device:
        raise ValueError(f"lse must have shape {(head[1], head[4], head[2])} on {q.device}")


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, causal: bool = False, window: Optional[int] = None,
                       scale: Optional[float] = None, q_lengths: Optional[torch.Tensor] = None,
                       k_lengths: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
                       dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients of attention, of whose results `out` and `lse` are needed: (dq, dk,
    dv) like q, k and v; dk and dv are summed over the query heads that share a
    head. They may be given, of any strides (the parts of a projection's gradient,
    say). Behind a sequence's lengths, and for queries that see nothing, they are
    0. Nothing of queries times keys is stored: the probabilities are computed
    again, tile by tile, and with 16-bit types rounded to the type like their
    gradients. With fp16 a dk has fewer digits where only queries see its key whose
    dout is far below the others' (2^-16 and less). The gradients overlap nothing
    else, nor one another."""
    head = _attention_checks(q, k, v, causal, window, scale, q_lengths, k_lengths)
    if not _alike(q, q.stride(), dout, out):
        _head_tensor(dout, q.dtype, q.shape, q.device, "dout")
        _head_tensor(out, q.dtype, q.shape, q.device, "out")
    _check_lse(lse, head, q)
    dq, dk, dv = _output_heads(dq, q, "dq"), _output_heads(dk, k, "dk"), _output_heads(dv, v, "dv")
    args = _ATTENTION_ARGS.pack(*head, *_batch_heads(out), lse.data_ptr(), *_batch_heads(dout), *_batch_heads(dq),
                                *_batch_heads(dk), *_batch_heads(dv))
    L = _load()
    ws, n, workspace = _call_workspace(workspace, L.sparcml_attention_backward_workspace(args), q)
    st = _on(q.device, L.sparcml_attention_backward, args, ws, n)
    _raise(st, "sparcml_attention_backward")
    return dq, dk, dv


# ---------------------------------------------------------------------------
def momentum_step(reduced: "ReduceOutput", momentum: torch.Tensor, mu: float, scale: float = 1.0,
                  nesterov: bool = False, dtype: torch.dtype = torch.float32,
                  update: Optional[torch.Tensor] = None) -> torch.Tensor:
    """momentum = mu * momentum + scale * g in place, g the reduction's result
    (sparse or dense, as the device knows). Returns the update in `dtype` (a
    given `update`: in its own): the momentum, or scale * g + mu * momentum
    with `nesterov`."""
    _check_dev(momentum, torch.float32, "momentum")
    _check_dev(reduced.result, torch.uint8, "result")
    _check_dev(reduced.out_idx, torch.int32, "out_idx")
    _check_dev(reduced.out_val, torch.float32, "out_val")
    N = reduced.N
    if momentum.numel() != N or reduced.out_val.numel() < N or reduced.result.numel() < 16:
        raise ValueError(f"momentum and the reduction's result must hold {N} positions")
    dev = momentum.device
    if update is None:
        update = momentum.new_empty(N, dtype=dtype)
    else:
        _check_dev(update, update.dtype, "update")
        if update.numel() != N:
            raise ValueError(f"update must hold {N} positions")
    st = _load().sparcml_momentum_step(N, _ptr(reduced.result), _ptr(reduced.out_idx), reduced.out_idx.numel(),
                                       _ptr(reduced.out_val), _ptr(momentum), mu, scale, int(nesterov),
                                       _type(update.dtype, "update"), _ptr(update), _stream(dev))
    _raise(st, "sparcml_momentum_step")
    return update


# ---------------------------------------------------------------------------
# quintic whose iterates take (0, 1] to about 0.7 .. 1.2, as published with the Muon optimizer (Jordan et al., 2024)
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def _matrices(matrices):
    """Host arrays of [(position, rows, cols)], in ascending order."""
    n = len(matrices)
    at, rows, cols = zip(*matrices) if n else ((), (), ())
    if n and (min(at) < 0 or max(at) >= 1 << 64 or min(min(rows), min(cols)) < 0 or max(max(rows), max(cols)) >= 1 << 32):
        raise ValueError("positions must lie in [0, 2^64), rows and columns in [0, 2^32)")
    return n, (ctypes.c_uint64 * n)(*at), (ctypes.c_uint32 * n)(*rows), (ctypes.c_uint32 * n)(*cols)


def _steps(steps: int, coefficients):
    a, b, c = coefficients
    if not 0 <= steps <= 64:
        raise ValueError("steps must lie in [0, 64]")
    return steps, a, b, c


def orthogonalize_workspace_bytes(N: int, matrices) -> int:
    """Bytes of the workspace that orthogonalize and orthogonal_step need."""
    if not 0 <= N < 1 << 64:
        raise ValueError("N must lie in [0, 2^64)")
    return int(_load().sparcml_orthogonalize_workspace(N, *_matrices(matrices)))


def _flat(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous tensor on a GPU")
    return _type(t.dtype, name)


def orthogonalize(update: torch.Tensor, matrices, dtype: Optional[torch.dtype] = None, steps: int = 5,
                  coefficients=NEWTON_SCHULZ, eps: float = 1e-7, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Orthogonalises every matrix of the flat `update` by Newton-Schulz steps.
    `matrices` is [(position, rows, cols)], ascending and disjoint, row-major.
    Returns `out`, like `update` in `dtype` (default: its own), written at the
    matrices' positions only (a new one is 0 elsewhere)."""
    kind = _flat(update, "update")
    N = update.numel()
    dev = update.device
    args = _matrices(matrices)
    L = _load()
    workspace = _workspace(workspace, L.sparcml_orthogonalize_workspace(N, *args), update)
    if out is None:
        whole = sum(m[1] * m[2] for m in matrices) == N
        out = (torch.empty_like if whole else torch.zeros_like)(update, dtype=dtype)
    okind = _flat(out, "out")
    if out.numel() != N or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must hold {N} elements of the dtype asked for")
    st = L.sparcml_orthogonalize(N, *args, *_steps(steps, coefficients), eps, kind, _ptr(update), okind, _ptr(out),
                                 _ptr(workspace), workspace.numel(), _stream(dev))
    _raise(st, "sparcml_orthogonalize")
    return out


def orthogonal_step(weight: torch.Tensor, update: torch.Tensor, matrices, lr: float, weight_decay: float = 0.0,
                    steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Moves the flat `weight` at every matrix's place, in place:
    w = (1 - lr * weight_decay) * w - lr * sqrt(max(1, rows / cols)) * o, o the
    orthogonalised matrix of `update` (see orthogonalize). Returns `weight`."""
    kind, wkind = _flat(update, "update"), _flat(weight, "weight")
    N = update.numel()
    if weight.numel() != N:
        raise ValueError(f"weight must hold {N} elements")
    args = _matrices(matrices)
    L = _load()
    workspace = _workspace(workspace, L.sparcml_orthogonalize_workspace(N, *args), weight)
    st = L.sparcml_orthogonal_step(N, *args, *_steps(steps, coefficients), eps, kind, _ptr(update), wkind,
                                   _ptr(weight), lr, weight_decay, _ptr(workspace), workspace.numel(),
                                   _stream(weight.device))
    _raise(st, "sparcml_orthogonal_step")
    return weight
