"""Thin ctypes binding of ``libhstu.so`` (the C ABI of ``include/hstu_attn.h``).

The functions keep the C names and only marshal arguments: torch tensors or
raw integer addresses become pointers, a torch stream becomes a
``cudaStream_t``, and a negative status becomes an ``HstuError``.  Every step
of the attention runs in the library's CUDA kernel; there is no Python or
CPU fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhstu.so")

HSTU_OK = 0
HSTU_ERR_INVALID_ARG = -1
HSTU_ERR_UNSUPPORTED = -2
HSTU_ERR_CUDA = -3
HSTU_ERR_TIMEOUT = -4
HSTU_ERR_NO_MEMORY = -5
HSTU_ERR_CAPACITY = -6
HSTU_NOALLOC_MAX_ITEMS = 65536
BLOCK_M = 128
HSTU_DEBUG_UNSIGNALLED_WAIT = 1
HSTU_DEBUG_TRACE = 2
HSTU_DEBUG_NO_PAIRS = 4
HSTU_DEBUG_BWD_ROWS = 8
TRACE_EVENTS = {1: "qk_issue", 2: "pv_issue", 3: "silu_start", 4: "silu_end", 5: "epi_start",
                6: "epi_end", 7: "load_k", 8: "load_v", 9: "load_q", 10: "mma_k_ready",
                11: "mma_qk_done", 12: "mma_p_ready", 13: "mma_pv_done"}

# name -> (restype, argtypes); the exported symbols of include/hstu_attn.h
_VP, _I32P, _IP = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int)


class _Rab(ctypes.Structure):
    """struct hstu_rab"""
    _fields_ = [("timestamps", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("num_pos", ctypes.c_int),
                ("time", ctypes.c_void_p), ("num_time", ctypes.c_int)]


class _NormGate(ctypes.Structure):
    """struct hstu_norm_gate"""
    _fields_ = [("u", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class _PagedBatch(ctypes.Structure):
    """struct hstu_paged_batch"""
    _fields_ = [("q_offsets", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("num_targets", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("batch", ctypes.c_int), ("max_pages", ctypes.c_int), ("max_q", ctypes.c_int),
                ("rows", ctypes.c_int)]


class _Rotary(ctypes.Structure):
    """struct hstu_rotary"""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int), ("dim", ctypes.c_int),
                ("pairs", ctypes.c_int)]


_RABP, _NGP = ctypes.POINTER(_Rab), ctypes.POINTER(_NormGate)
_PBP, _ROTP = ctypes.POINTER(_PagedBatch), ctypes.POINTER(_Rotary)
_I64, _F32, _INT = ctypes.c_int64, ctypes.c_float, ctypes.c_int
_SIGNATURES = {
    "hstu_attn_fwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_float, ctypes.c_float, _VP, _VP]),
    "hstu_attn_fwd_host": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                          _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP]),
    "hstu_attn_fwd_noalloc": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                             ctypes.c_float, _VP, _VP]),
    "hstu_plan_create": (ctypes.c_int, [_I32P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(_VP)]),
    "hstu_attn_fwd_plan": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP, _VP]),
    "hstu_plan_destroy": (ctypes.c_int, [_VP]),
    "hstu_plan_num_items": (ctypes.c_int, [_VP, _IP]),
    "hstu_plan_num_pairs": (ctypes.c_int, [_VP, _IP]),
    "hstu_worklist_build_pairs": (ctypes.c_int, [_I32P, ctypes.c_int, ctypes.c_int, _I32P, ctypes.c_int,
                                                 _IP]),
    "hstu_plan_worklist": (ctypes.c_int, [_VP, _I32P, ctypes.c_int, _IP]),
    "hstu_worklist_schedule": (ctypes.c_int, [_I32P, ctypes.c_int, ctypes.c_int, _I32P, _I32P,
                                              ctypes.POINTER(ctypes.c_longlong)]),
    "hstu_host_runs": (ctypes.c_int, [_I32P, ctypes.c_int, ctypes.c_int, _I32P, ctypes.c_int, _IP]),
    "hstu_worklist_build": (ctypes.c_int, [_I32P, ctypes.c_int, ctypes.c_int, _I32P, ctypes.c_int, _IP]),
    "hstu_launch_shape": (ctypes.c_int, [_VP, _IP, _IP, _IP]),
    "hstu_last_status": (ctypes.c_int, [_IP, _IP]),
    "hstu_set_wait_timeout_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "hstu_set_debug_flags": (ctypes.c_int, [ctypes.c_uint32]),
    "hstu_trace_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint64), ctypes.c_int, _IP]),
    "hstu_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "hstu_attn_fwd_targets": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32P, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                             ctypes.c_float, _VP, _VP]),
    "hstu_plan_create_targets": (ctypes.c_int, [_I32P, _I32P, ctypes.c_int, ctypes.c_int,
                                                ctypes.c_int, ctypes.c_int, ctypes.POINTER(_VP)]),
    "hstu_plan_item_hist": (ctypes.c_int, [_VP, _I32P, ctypes.c_int, _IP]),
    "hstu_worklist_build_targets": (ctypes.c_int, [_I32P, _I32P, ctypes.c_int, ctypes.c_int, _I32P,
                                                   _I32P, ctypes.c_int, _IP]),
    "hstu_worklist_build_candidates": (ctypes.c_int, [_I32P, _I32P, ctypes.c_int, ctypes.c_int,
                                                      _I32P, _I32P, ctypes.c_int, _IP]),
    "hstu_plan_create_ex": (ctypes.c_int, [_I32P, _I32P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_int, ctypes.c_uint32, ctypes.POINTER(_VP)]),
    "hstu_attn_fwd_norm_gate_plan": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_float,
                                                    ctypes.c_float, ctypes.c_float, _VP, _VP]),
    "hstu_attn_fwd_plan_ex": (ctypes.c_int, [_VP, _VP, _VP, _VP, _RABP, _NGP, ctypes.c_float,
                                             ctypes.c_float, _VP, _VP]),
    "hstu_attn_fwd_ex": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32P, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, _RABP, _NGP, ctypes.c_float,
                                        ctypes.c_float, _VP, _VP]),
    "hstu_attn_bwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_float, ctypes.c_float, _VP, _VP, _VP, _VP]),
    "hstu_attn_bwd_plan": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_float, ctypes.c_float, _VP,
                                          _VP, _VP, _VP]),
    "hstu_worklist_build_bwd": (ctypes.c_int, [_I32P, ctypes.c_int, ctypes.c_int, _I32P, ctypes.c_int,
                                               _IP]),
    "hstu_attn_bwd_ex": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _I32P, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, _RABP, ctypes.c_float,
                                        ctypes.c_float, _VP, _VP, _VP, _VP, _VP, _VP]),
    "hstu_worklist_build_bwd_targets": (ctypes.c_int, [_I32P, _I32P, ctypes.c_int, ctypes.c_int,
                                                       _I32P, _I32P, ctypes.c_int, _IP]),
    "hstu_attn_bwd_plan_ex": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _RABP, ctypes.c_float,
                                             ctypes.c_float, _VP, _VP, _VP, _VP, _VP, _VP]),
    "hstu_attn_fwd_norm_gate": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_float, _VP,
                                               _I32P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                               ctypes.c_int, ctypes.c_float, ctypes.c_float, _VP,
                                               _VP]),
    "hstu_cache_create": (_INT, [_VP, _VP, _INT, _INT, _INT, _INT, _I64, ctypes.POINTER(_VP)]),
    "hstu_cache_q4_page_bytes": (_INT, [_INT, _INT, _INT, ctypes.POINTER(ctypes.c_size_t)]),
    "hstu_cache_create_q4": (_INT, [_VP, _INT, _INT, _INT, _INT, _I64, ctypes.POINTER(_VP)]),
    "hstu_cache_read": (_INT, [_VP, _PBP, _VP, _I64, _VP, _I64, _VP]),
    "hstu_cache_destroy": (_INT, [_VP]),
    "hstu_cache_workspace": (_INT, [_VP, ctypes.POINTER(ctypes.c_size_t)]),
    "hstu_cache_slots": (_INT, [_PBP, _INT, _INT, ctypes.POINTER(_I64), _I32P]),
    "hstu_cache_worklist": (_INT, [_PBP, _INT, _INT, _INT, _INT, _INT, _INT, _INT, _INT, _I32P, _INT,
                                   _IP]),
    "hstu_cache_worklist_ex": (_INT, [_PBP, _INT, _INT, _INT, _INT, _INT, _INT, _INT, _INT, _INT, _I32P,
                                      _INT, _IP]),
    "hstu_cache_append": (_INT, [_VP, _PBP, _VP, _I64, _VP, _I64, _VP, _I64, _ROTP, _VP, _VP]),
    "hstu_attn_fwd_cache": (_INT, [_VP, _PBP, _VP, _I64, _F32, _F32, _VP, _VP, _VP]),
    "hstu_norm_fwd": (_INT, [_VP, _I64, _VP, _I64, _F32, _VP, _I64, _VP, _VP, _F32, _I64, _INT, _VP, _VP,
                             _VP]),
    "hstu_norm_bwd_workspace": (_INT, [_INT, ctypes.POINTER(ctypes.c_size_t)]),
    "hstu_norm_bwd": (_INT, [_VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _F32, _VP, _I64, _F32, _I64, _INT,
                             _VP, _VP, _VP, _I64, _VP, _VP, _VP, _VP]),
}

HSTU_PLAN_NORM_GATE = 1
HSTU_PLAN_BACKWARD = 2
HSTU_PLAN_CANDIDATES_ONLY = 4
HSTU_PLAN_PAIRS = 8

_lib = None


class HstuError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {hstu_status_string(code)} (status {code})")


def lib():
    """Load libhstu.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m hstu_jagged_attention_gb300.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def exported_symbols():
    return sorted(_SIGNATURES)


def _check(code: int, where: str):
    if code != HSTU_OK:
        raise HstuError(code, where)


def _addr(x) -> int | None:
    """Device/host address of a tensor or an integer address."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x).__name__}")


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream or None
        return None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _host_offsets(offsets) -> np.ndarray:
    if hasattr(offsets, "detach"):
        offsets = offsets.detach().to("cpu").numpy()
    return np.ascontiguousarray(np.asarray(offsets), dtype=np.int32)


def hstu_status_string(code: int) -> str:
    return lib().hstu_status_string(int(code)).decode()


def hstu_attn_fwd(q, k, v, offsets, batch: int, heads: int, d: int, max_seqlen: int, alpha: float,
                  inv_n: float, out, stream=None) -> None:
    """Enqueue the forward on ``stream`` (default: torch's current stream).

    ``offsets`` may be a CUDA int32 tensor, a CPU tensor / numpy array (host),
    or a raw address.
    """
    keep = None
    if isinstance(offsets, int):
        off_ptr = offsets
    elif hasattr(offsets, "is_cuda") and offsets.is_cuda:
        if offsets.dtype.itemsize != 4 or not offsets.is_contiguous():
            raise ValueError("device offsets must be contiguous int32")
        off_ptr = offsets.data_ptr()
    else:
        keep = _host_offsets(offsets)
        off_ptr = keep.ctypes.data
    _check(lib().hstu_attn_fwd(_addr(q), _addr(k), _addr(v), off_ptr, int(batch), int(heads), int(d),
                               int(max_seqlen), float(alpha), float(inv_n), _addr(out),
                               _stream(stream)), "hstu_attn_fwd")


def hstu_attn_fwd_host(q, k, v, offsets, batch: int, heads: int, d: int, max_seqlen: int,
                       alpha: float, inv_n: float, out, q_dev, k_dev, v_dev, out_dev,
                       n_chunks: int = 0, stream=None) -> None:
    """The forward from host q, k, v to host out (CPU tensors, page-locked
    for overlap), staged through the caller's device tensors q_dev, k_dev,
    v_dev, out_dev, in n_chunks runs of whole sequences (0: automatic) whose
    copies overlap the kernel.  ``offsets``: host int32.  Enqueued on
    ``stream``; out is valid once the stream reaches the call's end."""
    for t in (q, k, v, out):
        if hasattr(t, "is_cuda") and t.is_cuda:
            raise ValueError("q, k, v and out must be host tensors")
    off = _host_offsets(offsets)
    _check(lib().hstu_attn_fwd_host(_addr(q), _addr(k), _addr(v), off.ctypes.data, int(batch),
                                    int(heads), int(d), int(max_seqlen), float(alpha),
                                    float(inv_n), _addr(out), _addr(q_dev), _addr(k_dev),
                                    _addr(v_dev), _addr(out_dev), int(n_chunks), _stream(stream)),
           "hstu_attn_fwd_host")


def _host_targets(num_targets, batch: int) -> np.ndarray:
    nt = _host_offsets(num_targets)
    if nt.shape != (batch,):
        raise ValueError("num_targets needs one entry per sequence")
    return nt


def hstu_attn_fwd_targets(q, k, v, offsets, num_targets, batch: int, heads: int, d: int,
                          max_seqlen: int, alpha: float, inv_n: float, out, stream=None) -> None:
    """hstu_attn_fwd with the M-FALCON candidate mask: the last num_targets[b]
    tokens of sequence b see the history and themselves only.  ``num_targets``
    is host memory (CPU tensor or numpy array), one entry per sequence."""
    keep = None
    if isinstance(offsets, int):
        off_ptr = offsets
    elif hasattr(offsets, "is_cuda") and offsets.is_cuda:
        if offsets.dtype.itemsize != 4 or not offsets.is_contiguous():
            raise ValueError("device offsets must be contiguous int32")
        off_ptr = offsets.data_ptr()
    else:
        keep = _host_offsets(offsets)
        off_ptr = keep.ctypes.data
    nt = _host_targets(num_targets, int(batch))
    _check(lib().hstu_attn_fwd_targets(_addr(q), _addr(k), _addr(v), off_ptr,
                                       nt.ctypes.data_as(_I32P), int(batch), int(heads), int(d),
                                       int(max_seqlen), float(alpha), float(inv_n), _addr(out),
                                       _stream(stream)), "hstu_attn_fwd_targets")


def _offsets_arg(offsets):
    """(address, keep-alive) for offsets given as a CUDA tensor, host data or an address."""
    if isinstance(offsets, int):
        return offsets, None
    if hasattr(offsets, "is_cuda") and offsets.is_cuda:
        if offsets.dtype.itemsize != 4 or not offsets.is_contiguous():
            raise ValueError("device offsets must be contiguous int32")
        return offsets.data_ptr(), None
    keep = _host_offsets(offsets)
    return keep.ctypes.data, keep


def _rab_struct(rab):
    """rab = (timestamps int32 device tensor, pos fp32 table, time fp32 table) or None."""
    if rab is None:
        return None
    ts, pos, time = rab
    n_pos = int(pos.numel()) if hasattr(pos, "numel") else len(pos)
    n_time = int(time.numel()) if hasattr(time, "numel") else len(time)
    return ctypes.pointer(_Rab(_addr(ts), _addr(pos), n_pos, _addr(time), n_time))


def _ng_struct(norm_gate):
    """norm_gate = (u, gamma, beta, eps) or None."""
    if norm_gate is None:
        return None
    u, gamma, beta, eps = norm_gate
    return ctypes.pointer(_NormGate(_addr(u), _addr(gamma), _addr(beta), float(eps)))


def hstu_attn_fwd_plan_ex(plan: Plan, q, k, v, alpha: float, inv_n: float, out, rab=None,
                          norm_gate=None, stream=None) -> None:
    """Every option on a plan: ``rab`` = (timestamps, pos, time), ``norm_gate`` =
    (u, gamma, beta, eps) (the plan needs HSTU_PLAN_NORM_GATE)."""
    _check(lib().hstu_attn_fwd_plan_ex(plan.handle, _addr(q), _addr(k), _addr(v), _rab_struct(rab),
                                       _ng_struct(norm_gate), float(alpha), float(inv_n), _addr(out),
                                       _stream(stream)), "hstu_attn_fwd_plan_ex")


def hstu_attn_fwd_ex(q, k, v, offsets, batch: int, heads: int, d: int, max_seqlen: int, alpha: float,
                     inv_n: float, out, num_targets=None, rab=None, norm_gate=None,
                     stream=None) -> None:
    """Every option in one call (see hstu_attn_fwd_plan_ex; num_targets host memory or None)."""
    off_ptr, keep = _offsets_arg(offsets)
    nt = None if num_targets is None else _host_targets(num_targets, int(batch))
    _check(lib().hstu_attn_fwd_ex(_addr(q), _addr(k), _addr(v), off_ptr,
                                  None if nt is None else nt.ctypes.data_as(_I32P), int(batch),
                                  int(heads), int(d), int(max_seqlen), _rab_struct(rab),
                                  _ng_struct(norm_gate), float(alpha), float(inv_n), _addr(out),
                                  _stream(stream)), "hstu_attn_fwd_ex")
    del keep


def hstu_attn_bwd(q, k, v, dout, offsets, batch: int, heads: int, d: int, max_seqlen: int,
                  alpha: float, inv_n: float, dq, dk, dv, stream=None) -> None:
    """Gradients of the forward for ``dout``: dq, dk, dv (bf16, like q) are written."""
    off_ptr, keep = _offsets_arg(offsets)
    _check(lib().hstu_attn_bwd(_addr(q), _addr(k), _addr(v), _addr(dout), off_ptr, int(batch),
                               int(heads), int(d), int(max_seqlen), float(alpha), float(inv_n),
                               _addr(dq), _addr(dk), _addr(dv), _stream(stream)), "hstu_attn_bwd")
    del keep


def hstu_attn_bwd_plan(plan: Plan, q, k, v, dout, alpha: float, inv_n: float, dq, dk, dv,
                       stream=None) -> None:
    _check(lib().hstu_attn_bwd_plan(plan.handle, _addr(q), _addr(k), _addr(v), _addr(dout),
                                    float(alpha), float(inv_n), _addr(dq), _addr(dk), _addr(dv),
                                    _stream(stream)), "hstu_attn_bwd_plan")


def hstu_attn_bwd_ex(q, k, v, dout, offsets, batch: int, heads: int, d: int, max_seqlen: int,
                     alpha: float, inv_n: float, dq, dk, dv, num_targets=None, rab=None, dpos=None,
                     dtime=None, stream=None) -> None:
    """hstu_attn_bwd with candidates (``num_targets``, host memory) and the
    bias ``rab`` = (timestamps, pos, time): dpos and dtime (fp32 device, one
    entry per table entry) receive the tables' gradients."""
    off_ptr, keep = _offsets_arg(offsets)
    nt = None if num_targets is None else _host_targets(num_targets, int(batch))
    _check(lib().hstu_attn_bwd_ex(_addr(q), _addr(k), _addr(v), _addr(dout), off_ptr,
                                  None if nt is None else nt.ctypes.data_as(_I32P), int(batch),
                                  int(heads), int(d), int(max_seqlen), _rab_struct(rab),
                                  float(alpha), float(inv_n), _addr(dq), _addr(dk), _addr(dv),
                                  _addr(dpos), _addr(dtime), _stream(stream)), "hstu_attn_bwd_ex")
    del keep


def hstu_attn_bwd_plan_ex(plan: Plan, q, k, v, dout, alpha: float, inv_n: float, dq, dk, dv,
                          rab=None, dpos=None, dtime=None, stream=None) -> None:
    _check(lib().hstu_attn_bwd_plan_ex(plan.handle, _addr(q), _addr(k), _addr(v), _addr(dout),
                                       _rab_struct(rab), float(alpha), float(inv_n), _addr(dq),
                                       _addr(dk), _addr(dv), _addr(dpos), _addr(dtime),
                                       _stream(stream)), "hstu_attn_bwd_plan_ex")


def hstu_worklist_build_bwd(host_offsets, heads: int) -> np.ndarray:
    """Host-only work list of the backward: int32 (n, 4) items (first token, length, head, kt)."""
    off = _host_offsets(host_offsets)
    batch = len(off) - 1
    n = ctypes.c_int()
    _check(lib().hstu_worklist_build_bwd(off.ctypes.data_as(_I32P), batch, int(heads), None, 0,
                                         ctypes.byref(n)), "hstu_worklist_build_bwd")
    buf = np.zeros((max(n.value, 1), 4), dtype=np.int32)
    _check(lib().hstu_worklist_build_bwd(off.ctypes.data_as(_I32P), batch, int(heads),
                                         buf.ctypes.data_as(_I32P), n.value, ctypes.byref(n)),
           "hstu_worklist_build_bwd")
    return buf[:n.value]


def hstu_attn_fwd_norm_gate(q, k, v, u, gamma, beta, eps: float, offsets, num_targets, batch: int,
                            heads: int, d: int, max_seqlen: int, alpha: float, inv_n: float, y,
                            stream=None) -> None:
    """y = Norm(attention output) (.) u: a layer norm over each token's
    heads * d outputs with affine gamma, beta (fp32, heads * d), times u
    (bf16, like q).  ``num_targets`` is None (causal) or host memory with one
    entry per sequence (the candidate mask)."""
    off_ptr, keep = _offsets_arg(offsets)
    nt = None if num_targets is None else _host_targets(num_targets, int(batch))
    _check(lib().hstu_attn_fwd_norm_gate(_addr(q), _addr(k), _addr(v), _addr(u), _addr(gamma),
                                         _addr(beta), float(eps), off_ptr,
                                         None if nt is None else nt.ctypes.data_as(_I32P),
                                         int(batch), int(heads), int(d), int(max_seqlen),
                                         float(alpha), float(inv_n), _addr(y), _stream(stream)),
           "hstu_attn_fwd_norm_gate")
    del keep


def hstu_attn_fwd_noalloc(q, k, v, offsets, batch: int, heads: int, d: int, max_seqlen: int,
                          alpha: float, inv_n: float, out, stream=None) -> None:
    """As hstu_attn_fwd, for callers that cannot let the library allocate.

    The work list goes into a fixed device array inside the library instead
    of a per-call allocation; ``offsets`` must be host memory (a CPU tensor,
    a numpy array or a host address).  Calls in flight on the GPU at the same
    time share that array and must not overlap.
    """
    keep = None
    if isinstance(offsets, int):
        off_ptr = offsets
    else:
        if hasattr(offsets, "is_cuda") and offsets.is_cuda:
            raise ValueError("hstu_attn_fwd_noalloc takes host offsets only")
        keep = _host_offsets(offsets)
        off_ptr = keep.ctypes.data
    _check(lib().hstu_attn_fwd_noalloc(_addr(q), _addr(k), _addr(v), off_ptr, int(batch), int(heads),
                                       int(d), int(max_seqlen), float(alpha), float(inv_n),
                                       _addr(out), _stream(stream)), "hstu_attn_fwd_noalloc")


class Plan:
    """Owner of an ``hstu_plan*``; call ``hstu_plan_destroy`` or use as a context manager."""

    def __init__(self, handle: int, batch: int, heads: int, d: int, max_seqlen: int, total: int):
        self.handle = handle
        self.batch, self.heads, self.d, self.max_seqlen, self.total = batch, heads, d, max_seqlen, total

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        hstu_plan_destroy(self)

    def __del__(self):
        try:
            hstu_plan_destroy(self)
        except Exception:
            pass


def hstu_plan_create(host_offsets, batch: int, heads: int, d: int, max_seqlen: int) -> Plan:
    off = _host_offsets(host_offsets)
    if len(off) < batch + 1:
        raise ValueError("offsets needs batch + 1 entries")
    h = _VP()
    _check(lib().hstu_plan_create(off.ctypes.data_as(_I32P), int(batch), int(heads), int(d),
                                  int(max_seqlen), ctypes.byref(h)), "hstu_plan_create")
    return Plan(h.value, batch, heads, d, max_seqlen, int(off[batch]) if batch else 0)


def hstu_plan_create_targets(host_offsets, num_targets, batch: int, heads: int, d: int,
                             max_seqlen: int) -> Plan:
    """A plan with the M-FALCON candidate mask (see hstu_attn_fwd_targets)."""
    off = _host_offsets(host_offsets)
    if len(off) < batch + 1:
        raise ValueError("offsets needs batch + 1 entries")
    nt = _host_targets(num_targets, int(batch))
    h = _VP()
    _check(lib().hstu_plan_create_targets(off.ctypes.data_as(_I32P), nt.ctypes.data_as(_I32P),
                                          int(batch), int(heads), int(d), int(max_seqlen),
                                          ctypes.byref(h)), "hstu_plan_create_targets")
    return Plan(h.value, batch, heads, d, max_seqlen, int(off[batch]) if batch else 0)


def hstu_plan_create_ex(host_offsets, num_targets, batch: int, heads: int, d: int, max_seqlen: int,
                        flags: int = 0) -> Plan:
    """A plan with optional candidates (``num_targets`` None or one entry per
    sequence) and flags (HSTU_PLAN_NORM_GATE: the output stage's scratch)."""
    off = _host_offsets(host_offsets)
    if len(off) < batch + 1:
        raise ValueError("offsets needs batch + 1 entries")
    nt = None if num_targets is None else _host_targets(num_targets, int(batch))
    h = _VP()
    _check(lib().hstu_plan_create_ex(off.ctypes.data_as(_I32P),
                                     None if nt is None else nt.ctypes.data_as(_I32P), int(batch),
                                     int(heads), int(d), int(max_seqlen), int(flags),
                                     ctypes.byref(h)), "hstu_plan_create_ex")
    return Plan(h.value, batch, heads, d, max_seqlen, int(off[batch]) if batch else 0)


def hstu_attn_fwd_norm_gate_plan(plan: Plan, q, k, v, u, gamma, beta, eps: float, alpha: float,
                                 inv_n: float, y, stream=None) -> None:
    _check(lib().hstu_attn_fwd_norm_gate_plan(plan.handle, _addr(q), _addr(k), _addr(v), _addr(u),
                                              _addr(gamma), _addr(beta), float(eps), float(alpha),
                                              float(inv_n), _addr(y), _stream(stream)),
           "hstu_attn_fwd_norm_gate_plan")


def hstu_plan_item_hist(plan: Plan) -> np.ndarray:
    n = hstu_plan_num_items(plan)
    buf = np.zeros(max(n, 1), dtype=np.int32)
    got = ctypes.c_int()
    _check(lib().hstu_plan_item_hist(plan.handle, buf.ctypes.data_as(_I32P), max(n, 1),
                                     ctypes.byref(got)), "hstu_plan_item_hist")
    return buf[:got.value]


def _worklist_with_hist(name: str, host_offsets, num_targets, heads: int):
    off = _host_offsets(host_offsets)
    batch = len(off) - 1
    nt = _host_targets(num_targets, batch)
    fn = getattr(lib(), name)
    n = ctypes.c_int()
    _check(fn(off.ctypes.data_as(_I32P), nt.ctypes.data_as(_I32P), batch, int(heads), None, None, 0,
              ctypes.byref(n)), name)
    items = np.zeros((max(n.value, 1), 4), dtype=np.int32)
    hist = np.zeros(max(n.value, 1), dtype=np.int32)
    _check(fn(off.ctypes.data_as(_I32P), nt.ctypes.data_as(_I32P), batch, int(heads),
              items.ctypes.data_as(_I32P), hist.ctypes.data_as(_I32P), n.value, ctypes.byref(n)), name)
    return items[:n.value], hist[:n.value]


def hstu_worklist_build_targets(host_offsets, num_targets, heads: int):
    """Host-only candidate work list: (items int32 (n, 4), hist int32 (n,))."""
    return _worklist_with_hist("hstu_worklist_build_targets", host_offsets, num_targets, heads)


def hstu_worklist_build_bwd_targets(host_offsets, num_targets, heads: int):
    """Host-only work list of the backward with candidates: (items, hist)."""
    return _worklist_with_hist("hstu_worklist_build_bwd_targets", host_offsets, num_targets, heads)


def hstu_worklist_build_candidates(host_offsets, num_targets, heads: int):
    """Host-only work list of a HSTU_PLAN_CANDIDATES_ONLY plan: the candidate
    work list's items whose query block holds a candidate row."""
    return _worklist_with_hist("hstu_worklist_build_candidates", host_offsets, num_targets, heads)


def hstu_attn_fwd_plan(plan: Plan, q, k, v, alpha: float, inv_n: float, out, stream=None) -> None:
    _check(lib().hstu_attn_fwd_plan(plan.handle, _addr(q), _addr(k), _addr(v), float(alpha),
                                    float(inv_n), _addr(out), _stream(stream)), "hstu_attn_fwd_plan")


def hstu_plan_destroy(plan: Plan) -> None:
    if plan.handle:
        h, plan.handle = plan.handle, None
        _check(lib().hstu_plan_destroy(h), "hstu_plan_destroy")


def hstu_plan_num_items(plan: Plan) -> int:
    n = ctypes.c_int()
    _check(lib().hstu_plan_num_items(plan.handle, ctypes.byref(n)), "hstu_plan_num_items")
    return n.value


def hstu_plan_num_pairs(plan: Plan) -> int:
    """Pair items of the plan (0: one CTA per work item)."""
    n = ctypes.c_int()
    _check(lib().hstu_plan_num_pairs(plan.handle, ctypes.byref(n)), "hstu_plan_num_pairs")
    return n.value


def hstu_worklist_build_pairs(host_offsets, heads: int) -> np.ndarray:
    """Host-only work list of CTA pairs (no CUDA call): int32 (n_items, 4),
    rows (first token, length, head, qp)."""
    off = _host_offsets(host_offsets)
    batch = len(off) - 1
    n = ctypes.c_int()
    _check(lib().hstu_worklist_build_pairs(off.ctypes.data_as(_I32P), batch, int(heads), None, 0,
                                           ctypes.byref(n)), "hstu_worklist_build_pairs")
    buf = np.zeros((max(n.value, 1), 4), dtype=np.int32)
    _check(lib().hstu_worklist_build_pairs(off.ctypes.data_as(_I32P), batch, int(heads),
                                           buf.ctypes.data_as(_I32P), n.value, ctypes.byref(n)),
           "hstu_worklist_build_pairs")
    return buf[:n.value]


def hstu_worklist_schedule(cost, grid: int):
    """Host-only list schedule of a longest-first work list (no CUDA call):
    (order int32 (n,), first int32 (grid + 1,), makespan)."""
    c = np.ascontiguousarray(cost, dtype=np.int32).reshape(-1)
    order = np.zeros(max(len(c), 1), dtype=np.int32)
    first = np.zeros(max(int(grid), 0) + 1, dtype=np.int32)
    span = ctypes.c_longlong()
    _check(lib().hstu_worklist_schedule(c.ctypes.data_as(_I32P), len(c), int(grid),
                                        order.ctypes.data_as(_I32P), first.ctypes.data_as(_I32P),
                                        ctypes.byref(span)),
           "hstu_worklist_schedule")
    return order[:len(c)], first, span.value


def hstu_host_runs(offsets, n_chunks: int = 0) -> np.ndarray:
    """Host-only (no CUDA call): the runs of whole sequences
    hstu_attn_fwd_host takes, as first (int32, n_runs + 1): run c is
    sequences first[c] .. first[c + 1] - 1."""
    off = _host_offsets(offsets)
    batch = len(off) - 1
    n = ctypes.c_int()
    _check(lib().hstu_host_runs(off.ctypes.data_as(_I32P), batch, int(n_chunks), None, 0,
                                ctypes.byref(n)), "hstu_host_runs")
    first = np.zeros(n.value + 1, dtype=np.int32)
    _check(lib().hstu_host_runs(off.ctypes.data_as(_I32P), batch, int(n_chunks),
                                first.ctypes.data_as(_I32P), len(first), ctypes.byref(n)),
           "hstu_host_runs")
    return first


def hstu_plan_worklist(plan: Plan) -> np.ndarray:
    n = hstu_plan_num_items(plan)
    buf = np.zeros((max(n, 1), 4), dtype=np.int32)
    got = ctypes.c_int()
    _check(lib().hstu_plan_worklist(plan.handle, buf.ctypes.data_as(_I32P), max(n, 1),
                                    ctypes.byref(got)), "hstu_plan_worklist")
    return buf[:got.value]


def hstu_worklist_build(host_offsets, heads: int) -> np.ndarray:
    """Host-only work list (no CUDA call): int32 (n_items, 4)."""
    off = _host_offsets(host_offsets)
    batch = len(off) - 1
    n = ctypes.c_int()
    _check(lib().hstu_worklist_build(off.ctypes.data_as(_I32P), batch, int(heads), None, 0,
                                     ctypes.byref(n)), "hstu_worklist_build")
    buf = np.zeros((max(n.value, 1), 4), dtype=np.int32)
    _check(lib().hstu_worklist_build(off.ctypes.data_as(_I32P), batch, int(heads),
                                     buf.ctypes.data_as(_I32P), n.value, ctypes.byref(n)),
           "hstu_worklist_build")
    return buf[:n.value]


def hstu_launch_shape(plan: Plan) -> tuple[int, int, int]:
    g, b, s = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().hstu_launch_shape(plan.handle, ctypes.byref(g), ctypes.byref(b), ctypes.byref(s)),
           "hstu_launch_shape")
    return g.value, b.value, s.value


def hstu_last_status() -> tuple[int, int]:
    """(device status, site) -- reads and clears the device status word; synchronises."""
    st, site = ctypes.c_int(), ctypes.c_int()
    _check(lib().hstu_last_status(ctypes.byref(st), ctypes.byref(site)), "hstu_last_status")
    return st.value, site.value


def hstu_set_wait_timeout_ns(ns: int) -> None:
    _check(lib().hstu_set_wait_timeout_ns(int(ns)), "hstu_set_wait_timeout_ns")


def hstu_set_debug_flags(flags: int) -> None:
    _check(lib().hstu_set_debug_flags(int(flags)), "hstu_set_debug_flags")


def hstu_trace_read(capacity: int = 32768) -> np.ndarray:
    """Pipeline trace of CTA 0 (see include/hstu_attn.h): structured array
    with fields clock, event, warp, index; read and cleared."""
    buf = np.zeros(2 * capacity, dtype=np.uint64)
    n = ctypes.c_int()
    _check(lib().hstu_trace_read(buf.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), capacity,
                                 ctypes.byref(n)), "hstu_trace_read")
    raw = buf[: 2 * n.value].reshape(-1, 2)
    out = np.zeros(n.value, dtype=[("clock", np.int64), ("event", np.int32), ("warp", np.int32),
                                   ("index", np.int64)])
    out["clock"] = raw[:, 0].astype(np.int64)
    out["event"] = (raw[:, 1] >> np.uint64(48)).astype(np.int32)
    out["warp"] = ((raw[:, 1] >> np.uint64(40)) & np.uint64(0xFF)).astype(np.int32)
    out["index"] = (raw[:, 1] & np.uint64((1 << 40) - 1)).astype(np.int64)
    return out


# ------------------------------------------------------- the paged K/V cache
# A decode step's kernels take a few microseconds, so these calls check their
# tensors by comparing attributes and build nothing that they can keep.
_torch = None


def _load_torch():
    global _torch, _bf16, _f32
    import torch
    _torch, _bf16, _f32 = torch, torch.bfloat16, torch.float32


def _cuda_stream(stream, device):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device.index) or None
    return _stream(stream)


def _refuse(t, dtype, shape, device, what: str):
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")


def _row_stride(t, shape, device, what: str) -> int:
    """Elements between rows of a bf16 device tensor of ``shape`` (rows, width)
    or (rows, heads, d), whose rows are packed (a slice of a wider projection
    has a larger row stride)."""
    if t.dtype is not _bf16 or t.device != device or t.shape != shape:
        _refuse(t, _bf16, shape, device, what)
    step = t.stride()
    if step[-1] != 1 or (len(step) > 2 and step[-2] != shape[-1]) or shape[0] <= 1:
        return _odd_row_stride(step, shape, what)
    return step[0]


def _odd_row_stride(step, shape, what: str) -> int:
    """As _row_stride, where a dimension of one entry may have any stride."""
    width = 1
    for i in range(len(shape) - 1, 0, -1):
        if step[i] != width and shape[i] != 1:
            raise ValueError(f"{what}: the values of a row must be packed")
        width *= shape[i]
    return step[0] if shape[0] > 1 else width


def _packed(t, shape, device, what: str) -> int:
    if t.dtype is not _bf16 or t.device != device or t.shape != shape:
        _refuse(t, _bf16, shape, device, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _space(t, device, size: int, what: str):
    if t is None:
        return None
    if t.device != device or not t.is_contiguous() or t.numel() * t.element_size() < size:
        raise ValueError(f"{what} needs {size} contiguous bytes on {device}")
    return t.data_ptr()


class Cache:
    """Owner of an ``hstu_cache*`` over the caller's page pools, which it keeps
    alive: ``k_pages`` and ``v_pages``, or the codes' ``pages``."""

    def __init__(self, handle: int, shape, k_pages=None, v_pages=None, pages=None):
        self.handle, self.k_pages, self.v_pages, self.pages = handle, k_pages, v_pages, pages
        self.num_pages, self.page_size, self.heads, self.d = (int(n) for n in shape)
        self.device = (k_pages if pages is None else pages).device
        n = ctypes.c_size_t()
        _check(lib().hstu_cache_workspace(handle, ctypes.byref(n)), "hstu_cache_workspace")
        self.workspace_bytes = n.value

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        hstu_cache_destroy(self)

    def __del__(self):
        try:
            hstu_cache_destroy(self)
        except Exception:
            pass


class PagedBatch:
    """A batch of new tokens against a cache (struct hstu_paged_batch): int32
    device tensors ``q_offsets`` (batch + 1), ``kv_lens`` (batch),
    ``page_table`` (batch, max_pages) and optionally ``num_targets`` (batch).
    The kernels read them when they run, so a captured call follows their
    contents.  ``max_q`` bounds the new tokens of every sequence.  With
    numpy arrays the batch serves the host-only functions."""

    def __init__(self, q_offsets, kv_lens, page_table, max_q: int, num_targets=None):
        arrays = dict(q_offsets=q_offsets, kv_lens=kv_lens, page_table=page_table)
        if num_targets is not None:
            arrays["num_targets"] = num_targets
        batch = int(q_offsets.shape[0]) - 1
        shapes = dict(q_offsets=(batch + 1,), kv_lens=(batch,), num_targets=(batch,),
                      page_table=(batch, int(page_table.shape[1]) if page_table.ndim == 2 else -1))
        self.host = isinstance(q_offsets, np.ndarray)
        self.device = None if self.host else q_offsets.device
        for name, a in arrays.items():
            if isinstance(a, np.ndarray) != self.host:
                raise ValueError("the batch's arrays must all be device tensors, or all numpy arrays")
            if str(a.dtype).replace("torch.", "") != "int32":
                raise ValueError(f"{name} must be int32, not {a.dtype}")
            if batch < 0 or tuple(a.shape) != shapes[name]:
                raise ValueError(f"{name} has shape {tuple(a.shape)}, not {shapes[name]}")
            if not (a.flags.c_contiguous if self.host else a.is_contiguous()):
                raise ValueError(f"{name} must be contiguous")
            if not self.host:
                if not a.is_cuda:
                    raise ValueError(f"{name} must be a device tensor (or a numpy array)")
                if a.device != self.device:
                    raise ValueError(f"{name} is on {a.device}, not on {self.device}")
        if max_q < 0:
            raise ValueError(f"max_q must not be negative, not {max_q}")
        # (the struct's field has 32 bits)
        self.keep, self.batch, self.max_q = arrays, batch, min(int(max_q), 2 ** 31 - 1)
        at = {n: (a.ctypes.data if self.host else a.data_ptr()) for n, a in arrays.items()}
        self._fields = (at["q_offsets"], at["kv_lens"], at.get("num_targets"), at["page_table"], batch,
                        shapes["page_table"][1], self.max_q)
        self._structs = {}

    def struct(self, rows: int):
        """A pointer to the C struct for tensors of ``rows`` rows."""
        s = self._structs.get(rows)
        if s is None:
            if rows >= 2 ** 31:
                raise ValueError(f"{rows} rows: a call takes at most 2^31 - 1")
            if len(self._structs) >= 8:  # a batch is called with a few row counts, if not one
                self._structs.clear()
            s = self._structs[rows] = ctypes.byref(_PagedBatch(*self._fields, int(rows)))
        return s


def hstu_cache_create(k_pages, v_pages) -> Cache:
    """A cache over the pools ``k_pages`` and ``v_pages``: bf16 device tensors
    (num_pages, page_size, heads, d) with packed pages (pages may lie further
    apart, as in a pool that interleaves K and V)."""
    _load_torch()
    shape = k_pages.shape
    if len(shape) != 4 or not k_pages.is_cuda:
        raise ValueError("k_pages must be a device tensor (num_pages, page_size, heads, d)")
    if k_pages.device.index != _torch._C._cuda_getDevice():  # the cache is the current device's
        raise ValueError(f"k_pages is on {k_pages.device}, which is not the current device")
    _refuse(k_pages, _bf16, shape, k_pages.device, "k_pages")
    _refuse(v_pages, _bf16, shape, k_pages.device, "v_pages")
    stride = _odd_row_stride(k_pages.stride(), shape, "k_pages")
    if _odd_row_stride(v_pages.stride(), shape, "v_pages") != stride:
        raise ValueError("k_pages and v_pages must have the same page stride")
    if stride == 0:  # which the library takes for packed pages
        raise ValueError("k_pages and v_pages must not share memory between pages")
    h = _VP()
    _check(lib().hstu_cache_create(k_pages.data_ptr(), v_pages.data_ptr(), *shape, stride,
                                   ctypes.byref(h)), "hstu_cache_create")
    return Cache(h.value, shape, k_pages, v_pages)


def hstu_cache_q4_page_bytes(page_size: int, heads: int, d: int) -> int:
    """Bytes of a page of 4-bit codes."""
    n = ctypes.c_size_t()
    _check(lib().hstu_cache_q4_page_bytes(int(page_size), int(heads), int(d), ctypes.byref(n)),
           "hstu_cache_q4_page_bytes")
    return n.value


def hstu_cache_create_q4(pages, page_size: int, heads: int, d: int) -> Cache:
    """A cache of 4-bit codes over the pool ``pages``: a uint8 device tensor
    (num_pages, hstu_cache_q4_page_bytes(...)), whose rows may lie further
    apart.  Zeroed pages hold zeros."""
    _load_torch()
    if pages.ndim != 2 or not pages.is_cuda:
        raise ValueError("pages must be a device tensor (num_pages, page bytes)")
    if pages.device.index != _torch._C._cuda_getDevice():  # the cache is the current device's
        raise ValueError(f"pages is on {pages.device}, which is not the current device")
    shape = (pages.shape[0], hstu_cache_q4_page_bytes(page_size, heads, d))
    _refuse(pages, _torch.uint8, shape, pages.device, "pages")
    stride = _odd_row_stride(pages.stride(), shape, "pages")
    if stride == 0:  # which the library takes for packed pages
        raise ValueError("pages must not share memory")
    h = _VP()
    _check(lib().hstu_cache_create_q4(pages.data_ptr(), shape[0], int(page_size), int(heads), int(d), stride,
                                      ctypes.byref(h)), "hstu_cache_create_q4")
    return Cache(h.value, (shape[0], page_size, heads, d), pages=pages)


def hstu_cache_destroy(cache: Cache) -> None:
    if cache.handle:
        h, cache.handle = cache.handle, None
        _check(lib().hstu_cache_destroy(h), "hstu_cache_destroy")


def hstu_cache_workspace_bytes(cache: Cache) -> int:
    """Bytes of a workspace for hstu_attn_fwd_cache (zero it once)."""
    return cache.workspace_bytes


def _batch_on(batch: PagedBatch, device):
    if batch.device != device:
        raise ValueError(f"the batch is on {batch.device or 'the host'}, not on {device}")


def hstu_cache_append(cache: Cache, batch: PagedBatch, k, v, q=None, q_out=None, rotary=None,
                      rotary_pairs: bool = False, stream=None) -> None:
    """Write the new tokens' ``k`` and ``v`` (rows, heads, d) into the cache.

    ``rotary``: fp32 (positions, dim) table, cosines then sines: keys (and
    ``q``, into ``q_out``) are rotated by their position on the way, channels
    i and dim / 2 + i together, or with ``rotary_pairs`` 2 i and 2 i + 1."""
    dev, rows = cache.device, k.shape[0]
    shape = (rows, cache.heads, cache.d)
    _batch_on(batch, dev)
    ks = _row_stride(k, shape, dev, "k")
    vs = _row_stride(v, shape, dev, "v")
    qa, qs, qo, rot = None, 0, None, None
    if q is not None:
        qa, qs = q.data_ptr(), _row_stride(q, shape, dev, "q")
    if q_out is not None:
        qo = _packed(q_out, shape, dev, "q_out")
    if rotary is not None:
        if rotary.dtype is not _f32 or rotary.device != dev or rotary.ndim != 2 or \
                not rotary.is_contiguous():
            raise ValueError(f"rotary must be a contiguous fp32 (positions, dim) table on {dev}")
        rot = ctypes.byref(_Rotary(rotary.data_ptr(), rotary.shape[0], rotary.shape[1],
                                   1 if rotary_pairs else 0))
    code = lib().hstu_cache_append(cache.handle, batch.struct(rows), qa, qs, k.data_ptr(), ks,
                                   v.data_ptr(), vs, rot, qo, _cuda_stream(stream, dev))
    if code:
        _check(code, "hstu_cache_append")


def hstu_cache_read(cache: Cache, batch: PagedBatch, k, v, stream=None) -> None:
    """Copy the batch's tokens' keys (as held: rotated) and values out of the
    cache into ``k`` and ``v``, bf16 (rows, heads, d)."""
    dev, rows = cache.device, k.shape[0]
    shape = (rows, cache.heads, cache.d)
    _batch_on(batch, dev)
    ks = _row_stride(k, shape, dev, "k")
    vs = _row_stride(v, shape, dev, "v")
    code = lib().hstu_cache_read(cache.handle, batch.struct(rows), k.data_ptr(), ks, v.data_ptr(), vs,
                                 _cuda_stream(stream, dev))
    if code:
        _check(code, "hstu_cache_read")


def hstu_attn_fwd_cache(cache: Cache, batch: PagedBatch, q, alpha: float, inv_n: float, out,
                        workspace=None, stream=None) -> None:
    """The attention of the new tokens ``q`` (rows, heads, d) over the cache,
    which already holds their own keys and values, into ``out``.
    ``workspace``: a zeroed uint8 device tensor of hstu_cache_workspace_bytes,
    kept between calls (one call at a time); None allocates per call."""
    dev, rows = cache.device, q.shape[0]
    shape = (rows, cache.heads, cache.d)
    _batch_on(batch, dev)
    qs = _row_stride(q, shape, dev, "q")
    o = _packed(out, shape, dev, "out")
    ws = _space(workspace, dev, cache.workspace_bytes, "workspace")
    code = lib().hstu_attn_fwd_cache(cache.handle, batch.struct(rows), q.data_ptr(), qs, float(alpha),
                                     float(inv_n), o, ws, _cuda_stream(stream, dev))
    if code:
        _check(code, "hstu_attn_fwd_cache")


def hstu_cache_slots(batch: PagedBatch, num_pages: int, page_size: int, rows: int):
    """Host-only (no CUDA call; a batch of numpy arrays): (slots int64, positions
    int32, ok) of the rows; ok is False when the device would report the batch."""
    if not batch.host:
        raise ValueError("hstu_cache_slots takes a batch of numpy arrays")
    slot = np.full(max(rows, 1), -2, dtype=np.int64)
    pos = np.full(max(rows, 1), -2, dtype=np.int32)
    code = lib().hstu_cache_slots(batch.struct(rows), int(num_pages), int(page_size),
                                  slot.ctypes.data_as(ctypes.POINTER(_I64)), pos.ctypes.data_as(_I32P))
    if code != HSTU_OK and (rows == 0 or slot[0] == -2):
        raise HstuError(code, "hstu_cache_slots")
    return slot[:rows], pos[:rows], code == HSTU_OK


def hstu_cache_worklist(batch: PagedBatch, num_pages: int, page_size: int, rows: int, heads: int,
                        tile_rows: int, block_keys: int, grid: int, min_units: int = 1,
                        extra: int = 1, most_parts: int = 16) -> np.ndarray:
    """Host-only (no CUDA call; a batch of numpy arrays): the shares of
    hstu_attn_fwd_cache's CTAs, int32 (n, 8): CTA, sequence, head, tile, first
    block, blocks, first CTA of the item, CTAs that share it.  ``most_parts``:
    32 for 16-row tiles over a cache of 4-bit codes, else 16."""
    if not batch.host:
        raise ValueError("hstu_cache_worklist takes a batch of numpy arrays")
    args = (batch.struct(rows), int(num_pages), int(page_size), int(heads), int(tile_rows),
            int(block_keys), int(extra), int(grid), int(min_units), int(most_parts))
    n = ctypes.c_int()
    _check(lib().hstu_cache_worklist_ex(*args, None, 0, ctypes.byref(n)), "hstu_cache_worklist")
    buf = np.zeros((max(n.value, 1), 8), dtype=np.int32)
    _check(lib().hstu_cache_worklist_ex(*args, buf.ctypes.data_as(_I32P), n.value, ctypes.byref(n)),
           "hstu_cache_worklist")
    return buf[:n.value]


# ------------------------------------------- layer norm, its gate and residual
def _vector(t, width: int, device, what: str) -> int:
    if t.dtype is not _f32 or t.device != device or t.shape != (width,):
        _refuse(t, _f32, (width,), device, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows_of(t, what: str):
    if _torch is None:
        _load_torch()
    if t.ndim != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor (rows, width)")
    device = t.device
    if device.index != _torch._C._cuda_getDevice():
        raise ValueError(f"{what} is on {device}, which is not the current device")
    return t.shape, device


def hstu_norm_fwd(x, gamma, beta, eps: float, y, u=None, residual=None, scale: float = 1.0, z=None,
                  stream=None) -> None:
    """y = Norm(z) (.) u with z = residual + ``scale`` x (z = x without a
    ``residual``; then ``z`` is not given, else it receives the new residual
    stream).  x, u, residual, y, z: bf16 (rows, width), inputs with any row
    stride; gamma, beta: fp32 (width)."""
    shape, dev = _rows_of(x, "x")
    rows, width = shape
    xs = _row_stride(x, shape, dev, "x")
    ra, rs, ua, us, za = None, 0, None, 0, None
    if residual is not None:
        ra, rs = residual.data_ptr(), _row_stride(residual, shape, dev, "residual")
    if u is not None:
        ua, us = u.data_ptr(), _row_stride(u, shape, dev, "u")
    if z is not None:
        za = _packed(z, shape, dev, "z")
    code = lib().hstu_norm_fwd(x.data_ptr(), xs, ra, rs, float(scale), ua, us,
                               _vector(gamma, width, dev, "gamma"), _vector(beta, width, dev, "beta"),
                               float(eps), rows, width,
                               _packed(y, shape, dev, "y"), za, _cuda_stream(stream, dev))
    if code:
        _check(code, "hstu_norm_fwd")


def hstu_norm_bwd_workspace_bytes(width: int) -> int:
    """Bytes of a workspace for hstu_norm_bwd on the current device."""
    n = ctypes.c_size_t()
    _check(lib().hstu_norm_bwd_workspace(int(width), ctypes.byref(n)), "hstu_norm_bwd_workspace")
    return n.value


_norm_workspace = {}  # (device, width) -> bytes


def _norm_workspace_bytes(device, width: int) -> int:
    n = _norm_workspace.get((device.index, width))
    if n is None:
        with _torch.cuda.device(device):
            n = _norm_workspace[device.index, width] = hstu_norm_bwd_workspace_bytes(width)
    return n


def hstu_norm_bwd(dy, z, gamma, beta, eps: float, dz, dgamma, dbeta, u=None, du=None, dz_in=None,
                  dx=None, scale: float = 1.0, workspace=None, stream=None) -> None:
    """Gradients of hstu_norm_fwd for ``dy``: ``dz`` of the norm's input ``z``
    (x without a residual; with one also the residual's gradient), with
    ``dz_in`` (the gradient reaching z past the norm) added; ``dx`` = scale
    dz; ``du`` of the gate ``u``; ``dgamma``, ``dbeta`` (fp32, overwritten)."""
    shape, dev = _rows_of(dy, "dy")
    rows, width = shape
    dys = _row_stride(dy, shape, dev, "dy")
    zs = _row_stride(z, shape, dev, "z")
    ua, us, dua, dus, da, ds, dxa, ws = None, 0, None, 0, None, 0, None, None
    if u is not None:
        ua, us = u.data_ptr(), _row_stride(u, shape, dev, "u")
    if du is not None:
        dua, dus = du.data_ptr(), _row_stride(du, shape, dev, "du")
    if dz_in is not None:
        da, ds = dz_in.data_ptr(), _row_stride(dz_in, shape, dev, "dz_in")
    if dx is not None:
        dxa = _packed(dx, shape, dev, "dx")
    if workspace is not None:
        ws = _space(workspace, dev, _norm_workspace_bytes(dev, width), "workspace")
    code = lib().hstu_norm_bwd(dy.data_ptr(), dys, z.data_ptr(), zs, ua, us,
                               _vector(gamma, width, dev, "gamma"), _vector(beta, width, dev, "beta"),
                               float(eps), da, ds, float(scale), rows, width, _packed(dz, shape, dev, "dz"), dxa, dua, dus,
                               _vector(dgamma, width, dev, "dgamma"), _vector(dbeta, width, dev, "dbeta"),
                               ws, _cuda_stream(stream, dev))
    if code:
        _check(code, "hstu_norm_bwd")
