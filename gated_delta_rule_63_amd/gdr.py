"""Thin Python binding of libgdr.so (C ABI in include/gdr.h).

Argument marshalling only: every function checks that the torch tensors it is
given are contiguous device tensors of the documented shape and dtype, builds the
``gdr_problem`` struct, passes raw pointers and the current HIP stream, and raises
``GdrError`` on a non-success status.  All computation happens in the library's
HIP kernels.  If the library has not been built, loading it raises immediately.

Names follow the C entry points: ``gdr_recurrent_fwd``, ``gdr_chunk_fwd``,
``gdr_chunk_fwd_noalloc``, ``gdr_chunk_workspace_size``, ``gdr_decode_paged``,
``gdr_gating_prepass``, ``gdr_decode_paged_gated``, ``gdr_kda_decode_fused``, ``gdr_linear_scan_fwd``,
``gdr_linear_scan_bwd``, ``gdr_linear_decode_paged``, ``gdr_linear_workspace_size``, ``gdr_beam_select``,
``gdr_beam_workspace_size``, ``gdr_beam_reorder``, ``gdr_status_string``.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_DEFAULT_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdr.so")
_LIB_PATH = _DEFAULT_LIB_PATH
_lib = None

GDR_SUCCESS, GDR_ERROR_INVALID_VALUE, GDR_ERROR_NOT_SUPPORTED, GDR_ERROR_LAUNCH_FAILED = 0, 1, 2, 3
GDR_ERROR_SCRATCH_LIMIT = 4
GDR_NOALLOC_SCRATCH_BYTES = 64 << 20
GDR_F32, GDR_BF16 = 0, 1
GDR_GATE_SCALAR, GDR_GATE_PER_K = 0, 1
GDR_LINEAR_LOG_DECAY, GDR_LINEAR_SIGMOID = 0, 1
GDR_LINEAR_BLOCK = 64


class GdrError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {gdr_status_string(status)} ({status})")
        self.status = status


class Gating(ctypes.Structure):
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("A_log", ctypes.c_void_p),
        ("dt_bias", ctypes.c_void_p),
        ("l2norm_eps", ctypes.c_float),
        ("qk_l2norm", ctypes.c_int32),
        ("allow_neg_eigval", ctypes.c_int32),
    ]


class KdaFront(ctypes.Structure):
    _fields_ = [
        ("conv_width", ctypes.c_int32),
        ("conv_weight", ctypes.c_void_p),
        ("conv_bias", ctypes.c_void_p),
        ("conv_state", ctypes.c_void_p),
        ("gate_in", ctypes.c_void_p),
        ("gate_weight", ctypes.c_void_p),
        ("gate_rank", ctypes.c_int32),
        ("A_log", ctypes.c_void_p),
        ("dt_bias", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("l2norm_eps", ctypes.c_float),
        ("norm_weight", ctypes.c_void_p),
        ("norm_gate", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
    ]


class LinearProblem(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("num_channels", ctypes.c_int32),
        ("gate", ctypes.c_int),
        ("io_dtype", ctypes.c_int),
    ]


class BeamProblem(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("beams", ctypes.c_int32),
        ("vocab", ctypes.c_int32),
        ("num_out", ctypes.c_int32),
        ("row_stride", ctypes.c_int64),
        ("eos_token", ctypes.c_int32),
        ("io_dtype", ctypes.c_int),
    ]


class Problem(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("num_seqs", ctypes.c_int32),
        ("num_k_heads", ctypes.c_int32),
        ("num_v_heads", ctypes.c_int32),
        ("head_dim_k", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("gate", ctypes.c_int),
        ("io_dtype", ctypes.c_int),
    ]


def library_path() -> str:
    return _LIB_PATH


def use_library(path: Optional[str] = None) -> None:
    """Bind to another build of the library from here on (the measurement build libgdr_stamps.so
    exports the same entry points, with the flow kernel's clock counters compiled in); None binds
    to libgdr.so again."""
    global _lib, _LIB_PATH
    _lib = None
    _LIB_PATH = path if path is not None else _DEFAULT_LIB_PATH


def lib():
    """Load libgdr.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with `python -m gated_delta_rule_63_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        P = ctypes.POINTER(Problem)
        L.gdr_status_string.restype = ctypes.c_char_p
        L.gdr_status_string.argtypes = [ctypes.c_int]
        L.gdr_recurrent_fwd.restype = ctypes.c_int
        L.gdr_recurrent_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.gdr_chunk_workspace_size.restype = ctypes.c_size_t
        L.gdr_chunk_workspace_size.argtypes = [P, i32]
        L.gdr_chunk_fwd.restype = ctypes.c_int
        L.gdr_chunk_fwd.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.gdr_chunk_fwd_noalloc.restype = ctypes.c_int
        L.gdr_chunk_fwd_noalloc.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.gdr_decode_paged.restype = ctypes.c_int
        L.gdr_decode_paged.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, i32, vp, i32,
                                       vp, ctypes.c_int, i32, i32, vp, vp, vp]
        G = ctypes.POINTER(Gating)
        L.gdr_gating_prepass.restype = ctypes.c_int
        L.gdr_gating_prepass.argtypes = [P, vp, vp, G, vp, vp, vp, vp, vp]
        L.gdr_decode_paged_gated.restype = ctypes.c_int
        L.gdr_decode_paged_gated.argtypes = [P, i32, vp, vp, vp, G, vp, vp, ctypes.c_int, i32, vp, i32,
                                             vp, ctypes.c_int, i32, i32, vp, vp, vp]
        L.gdr_kda_decode_fused.restype = ctypes.c_int
        L.gdr_kda_decode_fused.argtypes = [P, i32, vp, vp, vp, ctypes.POINTER(KdaFront), vp, vp, ctypes.c_int, i32, vp,
                                           i32, vp, vp]
        LP, sz = ctypes.POINTER(LinearProblem), ctypes.c_size_t
        L.gdr_linear_workspace_size.restype = sz
        L.gdr_linear_workspace_size.argtypes = [LP]
        L.gdr_linear_scan_fwd.restype = ctypes.c_int
        L.gdr_linear_scan_fwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.gdr_linear_scan_bwd.restype = ctypes.c_int
        L.gdr_linear_scan_bwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.gdr_linear_decode_paged.restype = ctypes.c_int
        L.gdr_linear_decode_paged.argtypes = [LP, i32, vp, vp, vp, vp, ctypes.c_int, i32, vp, i32, vp, vp]
        BP = ctypes.POINTER(BeamProblem)
        L.gdr_beam_workspace_size.restype = sz
        L.gdr_beam_workspace_size.argtypes = [BP]
        L.gdr_beam_select.restype = ctypes.c_int
        L.gdr_beam_select.argtypes = [BP, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.gdr_beam_reorder.restype = ctypes.c_int
        L.gdr_beam_reorder.argtypes = [i32, i32, vp, vp, vp, vp, i32, i32, i64, vp]
        _lib = L
    return _lib


def gdr_status_string(status: int) -> str:
    return lib().gdr_status_string(int(status)).decode()


# ---------------------------------------------------------------------------
def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return GDR_F32
    if t == torch.bfloat16:
        return GDR_BF16
    raise TypeError(f"unsupported dtype {t}: use float32 or bfloat16")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: Optional[torch.Tensor], name: str, shape=None, dtype=None, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (the C ABI sees no strides)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _problem(q, k, v, g, num_seqs: int, scale: Optional[float]) -> Problem:
    T, HK, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    per_k = g.dim() == 3
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    return Problem(T, num_seqs, HK, HV, K, V, float(scale), GDR_GATE_PER_K if per_k else GDR_GATE_SCALAR,
                   _dtype_code(q.dtype))


def _check_tokens(q, k, v, g, beta):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k are [T, HK, K] and v is [T, HV, V]")
    T, HK, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _check(q, "q")
    _check(k, "k", (T, HK, K), q.dtype)
    _check(v, "v", (T, HV, V), q.dtype)
    _check(beta, "beta", (T, HV), q.dtype)
    if g.dim() == 3:
        _check(g, "g", (T, HV, K), torch.float32)
    else:
        _check(g, "g", (T, HV), torch.float32)
    return T, HK, HV, K, V


def _num_seqs(cu_seqlens, default: int) -> int:
    if cu_seqlens is None:
        return default
    _check(cu_seqlens, "cu_seqlens", dtype=torch.int32)
    return cu_seqlens.shape[0] - 1


def _raise(status: int, where: str):
    if status != GDR_SUCCESS:
        raise GdrError(status, where)


# ---------------------------------------------------------------------------
def gdr_recurrent_fwd(q, k, v, g, beta, cu_seqlens=None, scale=None, initial_state=None, o=None,
                      final_state=None, output_final_state: bool = True, stream=None):
    """Token-by-token recurrence.  Returns (o, final_state or None)."""
    T, HK, HV, K, V = _check_tokens(q, k, v, g, beta)
    N = _num_seqs(cu_seqlens, 1)
    _check(initial_state, "initial_state", (N, HV, V, K), torch.float32, optional=True)
    if o is None:
        o = torch.empty((T, HV, V), dtype=q.dtype, device=q.device)
    _check(o, "o", (T, HV, V), q.dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, HV, V, K), dtype=torch.float32, device=q.device)
    _check(final_state, "final_state", (N, HV, V, K), torch.float32, optional=True)
    p = _problem(q, k, v, g, N, scale)
    st = lib().gdr_recurrent_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                 _ptr(cu_seqlens), _ptr(initial_state), _ptr(o), _ptr(final_state), _stream(stream))
    _raise(st, "gdr_recurrent_fwd")
    return o, final_state


def gdr_chunk_workspace_size(q, v, g, num_seqs: int, chunk_size: int = 64) -> int:
    p = _problem(q, q, v, g, num_seqs, 1.0)
    return int(lib().gdr_chunk_workspace_size(ctypes.byref(p), int(chunk_size)))


def gdr_chunk_fwd(q, k, v, g, beta, cu_seqlens=None, scale=None, initial_state=None, o=None,
                  final_state=None, output_final_state: bool = True, workspace=None, chunk_size: int = 64,
                  stream=None, segmented: bool = True):
    """Chunked (64-token) forward.  Returns (o, final_state or None).  ``workspace`` is a
    uint8 device tensor of at least gdr_chunk_workspace_size bytes (allocated here if absent).
    ``segmented=False`` passes no workspace, which makes the library run every sequence in one
    pass even where it would cut few long sequences into segments."""
    T, HK, HV, K, V = _check_tokens(q, k, v, g, beta)
    N = _num_seqs(cu_seqlens, 1)
    _check(initial_state, "initial_state", (N, HV, V, K), torch.float32, optional=True)
    if o is None:
        o = torch.empty((T, HV, V), dtype=q.dtype, device=q.device)
    _check(o, "o", (T, HV, V), q.dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, HV, V, K), dtype=torch.float32, device=q.device)
    _check(final_state, "final_state", (N, HV, V, K), torch.float32, optional=True)
    p = _problem(q, k, v, g, N, scale)
    need = int(lib().gdr_chunk_workspace_size(ctypes.byref(p), int(chunk_size)))
    if not segmented:
        workspace = None
    elif workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", dtype=torch.uint8, optional=True)
    st = lib().gdr_chunk_fwd(ctypes.byref(p), int(chunk_size), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                             _ptr(cu_seqlens), _ptr(initial_state), _ptr(o), _ptr(final_state), _ptr(workspace),
                             0 if workspace is None else workspace.numel(), _stream(stream))
    _raise(st, "gdr_chunk_fwd")
    return o, final_state


def gdr_chunk_fwd_noalloc(q, k, v, g, beta, cu_seqlens=None, scale=None, initial_state=None, o=None,
                          final_state=None, chunk_size: int = 64, stream=None):
    """gdr_chunk_fwd without a workspace argument: the library's fixed per-GPU scratch array
    (GDR_NOALLOC_SCRATCH_BYTES) stands in for it.  ``o`` must be given; the C call allocates
    nothing.  Calls that overlap on one GPU race on the scratch."""
    T, HK, HV, K, V = _check_tokens(q, k, v, g, beta)
    N = _num_seqs(cu_seqlens, 1)
    _check(initial_state, "initial_state", (N, HV, V, K), torch.float32, optional=True)
    _check(o, "o", (T, HV, V), q.dtype)
    _check(final_state, "final_state", (N, HV, V, K), torch.float32, optional=True)
    p = _problem(q, k, v, g, N, scale)
    st = lib().gdr_chunk_fwd_noalloc(ctypes.byref(p), int(chunk_size), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                     _ptr(beta), _ptr(cu_seqlens), _ptr(initial_state), _ptr(o), _ptr(final_state),
                                     _stream(stream))
    _raise(st, "gdr_chunk_fwd_noalloc")
    return o, final_state


def gdr_decode_paged(q, k, v, g, beta, pool, state_indices, cu_seqlens=None, max_q_len: int = 1,
                     commit: bool = True, inter_states=None, inter_state_indices=None, scale=None, o=None,
                     stream=None):
    """Paged decode / speculative verify.  pool [num_slots, HV, V, K] (float32 or bfloat16),
    state_indices int32 [N] (-1 = padded).  inter_states [num_cache_slots, cache_steps, HV, V, K]
    or None.  Returns o (rows of padded sequences are left as they were)."""
    T, HK, HV, K, V = _check_tokens(q, k, v, g, beta)
    _check(state_indices, "state_indices", dtype=torch.int32)
    N = state_indices.shape[0]
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32)
    if pool.dim() != 4:
        raise ValueError("pool is [num_slots, HV, V, K]")
    _check(pool, "pool", (pool.shape[0], HV, V, K))
    pool_dt = _dtype_code(pool.dtype)
    ncs = steps = 0
    inter_dt = GDR_F32
    if inter_states is not None:
        if inter_states.dim() != 5:
            raise ValueError("inter_states is [num_cache_slots, cache_steps, HV, V, K]")
        ncs, steps = inter_states.shape[0], inter_states.shape[1]
        _check(inter_states, "inter_states", (ncs, steps, HV, V, K))
        inter_dt = _dtype_code(inter_states.dtype)
        _check(inter_state_indices, "inter_state_indices", (N,), torch.int32)
    if o is None:
        o = torch.empty((T, HV, V), dtype=q.dtype, device=q.device)
    _check(o, "o", (T, HV, V), q.dtype)
    p = _problem(q, k, v, g, N, scale)
    st = lib().gdr_decode_paged(ctypes.byref(p), int(max_q_len), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                _ptr(cu_seqlens), _ptr(pool), pool_dt, pool.shape[0], _ptr(state_indices),
                                1 if commit else 0, _ptr(inter_states), inter_dt, ncs, steps,
                                _ptr(inter_state_indices), _ptr(o), _stream(stream))
    _raise(st, "gdr_decode_paged")
    return o


# ---------------------------------------------------------------------------
def _gating(q, v, a, b, A_log, dt_bias, eps: float, qk_l2norm: bool, allow_neg_eigval: bool) -> Gating:
    T, HV = q.shape[0], v.shape[1] if v is not None else a.shape[1]
    _check(a, "a", (T, HV), q.dtype)
    _check(b, "b", (T, HV), q.dtype)
    _check(A_log, "A_log", (HV,), torch.float32)
    _check(dt_bias, "dt_bias", (HV,), torch.float32)
    return Gating(a.data_ptr(), b.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr(), float(eps),
                  1 if qk_l2norm else 0, 1 if allow_neg_eigval else 0)


def gdr_gating_prepass(q, k, a, b, A_log, dt_bias, l2norm_eps: float = 1e-6, qk_l2norm: bool = True,
                       allow_neg_eigval: bool = False, q_out=None, k_out=None, g_out=None, beta_out=None,
                       stream=None):
    """Gating front as one pass.  q, k [T, HK, K] raw; a, b [T, HV] (q's dtype); A_log, dt_bias
    [HV] fp32.  Returns (q_out, k_out, g [T, HV] fp32, beta [T, HV]); q_out/k_out may be q/k
    (in place) and are None when qk_l2norm is False."""
    if q.dim() != 3 or a.dim() != 2:
        raise ValueError("q, k are [T, HK, K]; a, b are [T, HV]")
    T, HK, K = q.shape
    HV = a.shape[1]
    _check(q, "q")
    _check(k, "k", (T, HK, K), q.dtype)
    gt = _gating(q, None, a, b, A_log, dt_bias, l2norm_eps, qk_l2norm, allow_neg_eigval)
    if qk_l2norm:
        q_out = torch.empty_like(q) if q_out is None else q_out
        k_out = torch.empty_like(k) if k_out is None else k_out
        _check(q_out, "q_out", (T, HK, K), q.dtype)
        _check(k_out, "k_out", (T, HK, K), q.dtype)
    else:
        q_out = k_out = None
    g_out = torch.empty((T, HV), dtype=torch.float32, device=q.device) if g_out is None else g_out
    beta_out = torch.empty((T, HV), dtype=q.dtype, device=q.device) if beta_out is None else beta_out
    _check(g_out, "g_out", (T, HV), torch.float32)
    _check(beta_out, "beta_out", (T, HV), q.dtype)
    # gdr_problem: V is not read by this pass; K is given as the value width to pass validation
    p = Problem(T, 1, HK, HV, K, K, 1.0, GDR_GATE_SCALAR, _dtype_code(q.dtype))
    st = lib().gdr_gating_prepass(ctypes.byref(p), _ptr(q), _ptr(k), ctypes.byref(gt), _ptr(q_out), _ptr(k_out),
                                  _ptr(g_out), _ptr(beta_out), _stream(stream))
    _raise(st, "gdr_gating_prepass")
    return q_out, k_out, g_out, beta_out


def gdr_decode_paged_gated(q, k, v, a, b, A_log, dt_bias, pool, state_indices, cu_seqlens=None,
                           max_q_len: int = 1, commit: bool = True, inter_states=None, inter_state_indices=None,
                           scale=None, l2norm_eps: float = 1e-6, qk_l2norm: bool = True,
                           allow_neg_eigval: bool = False, o=None, stream=None):
    """gdr_decode_paged with the gating front in the token loop: q, k raw; a, b [T, HV] (q's
    dtype); A_log, dt_bias [HV] fp32.  Returns o."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k are [T, HK, K] and v is [T, HV, V]")
    T, HK, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _check(q, "q")
    _check(k, "k", (T, HK, K), q.dtype)
    _check(v, "v", (T, HV, V), q.dtype)
    gt = _gating(q, v, a, b, A_log, dt_bias, l2norm_eps, qk_l2norm, allow_neg_eigval)
    _check(state_indices, "state_indices", dtype=torch.int32)
    N = state_indices.shape[0]
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32)
    if pool.dim() != 4:
        raise ValueError("pool is [num_slots, HV, V, K]")
    _check(pool, "pool", (pool.shape[0], HV, V, K))
    pool_dt = _dtype_code(pool.dtype)
    ncs = steps = 0
    inter_dt = GDR_F32
    if inter_states is not None:
        if inter_states.dim() != 5:
            raise ValueError("inter_states is [num_cache_slots, cache_steps, HV, V, K]")
        ncs, steps = inter_states.shape[0], inter_states.shape[1]
        _check(inter_states, "inter_states", (ncs, steps, HV, V, K))
        inter_dt = _dtype_code(inter_states.dtype)
        _check(inter_state_indices, "inter_state_indices", (N,), torch.int32)
    if o is None:
        o = torch.empty((T, HV, V), dtype=q.dtype, device=q.device)
    _check(o, "o", (T, HV, V), q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    p = Problem(T, N, HK, HV, K, V, float(scale), GDR_GATE_SCALAR, _dtype_code(q.dtype))
    st = lib().gdr_decode_paged_gated(ctypes.byref(p), int(max_q_len), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(gt),
                                      _ptr(cu_seqlens), _ptr(pool), pool_dt, pool.shape[0], _ptr(state_indices),
                                      1 if commit else 0, _ptr(inter_states), inter_dt, ncs, steps,
                                      _ptr(inter_state_indices), _ptr(o), _stream(stream))
    _raise(st, "gdr_decode_paged_gated")
    return o


def gdr_kda_decode_fused(q, k, v, conv_weight, conv_state, gate_in, gate_weight, A_log, dt_bias, b, pool,
                         state_indices, cu_seqlens=None, max_q_len: int = 1, commit: bool = True, scale=None,
                         conv_bias=None, l2norm_eps: float = 1e-6, norm_weight=None, norm_gate=None,
                         norm_eps: float = 1e-6, o=None, stream=None):
    """Fused KDA decode front (raw q, k, v [T, H, K|V]; conv_weight [C, W]; conv_state
    [slots, C, W-1]; gate_in [T, R]; gate_weight [H*K, R]; A_log [H]; dt_bias [H*K]; b [T, H];
    optional norm_weight [V] with norm_gate [T, H, V]).  Returns o."""
    T, H, K = q.shape
    V = v.shape[2]
    _check(q, "q", (T, H, K))
    _check(k, "k", (T, H, K), q.dtype)
    _check(v, "v", (T, H, V), q.dtype)
    C, W = conv_weight.shape
    assert C == 2 * H * K + H * V, "conv_weight rows: q | k | v channels"
    _check(conv_weight, "conv_weight", (C, W), q.dtype)
    _check(conv_bias, "conv_bias", (C,), q.dtype, optional=True)
    _check(conv_state, "conv_state", (pool.shape[0], C, W - 1), q.dtype, optional=(W == 1))
    R = gate_in.shape[1]
    _check(gate_in, "gate_in", (T, R), q.dtype)
    _check(gate_weight, "gate_weight", (H * K, R), q.dtype)
    _check(A_log, "A_log", (H,), torch.float32)
    _check(dt_bias, "dt_bias", (H * K,), torch.float32)
    _check(b, "b", (T, H), q.dtype)
    _check(norm_weight, "norm_weight", (V,), q.dtype, optional=True)
    _check(norm_gate, "norm_gate", (T, H, V), q.dtype, optional=True)
    N = int(state_indices.shape[0])
    _check(state_indices, "state_indices", (N,), torch.int32)
    _check(pool, "pool", (pool.shape[0], H, V, K))
    if o is None:
        o = torch.empty((T, H, V), dtype=q.dtype, device=q.device)
    _check(o, "o", (T, H, V), q.dtype)
    p = Problem(T, N, H, H, K, V, float(1.0 / math.sqrt(K) if scale is None else scale), GDR_GATE_PER_K,
                _dtype_code(q.dtype))
    f = KdaFront(W, _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state), _ptr(gate_in), _ptr(gate_weight), R,
                 _ptr(A_log), _ptr(dt_bias), _ptr(b), float(l2norm_eps), _ptr(norm_weight), _ptr(norm_gate),
                 float(norm_eps))
    st = lib().gdr_kda_decode_fused(ctypes.byref(p), int(max_q_len), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(f),
                                    _ptr(cu_seqlens), _ptr(pool), _dtype_code(pool.dtype), int(pool.shape[0]),
                                    _ptr(state_indices), int(bool(commit)), _ptr(o), _stream(stream))
    _raise(st, "gdr_kda_decode_fused")
    return o


# ---------------------------------------------------------------------------
# The entry points below are called once per layer and step, with tens of microseconds of device time at
# most: their checks are one pass per tensor, and pointers go to ctypes as plain integers.
def _arg(t: Optional[torch.Tensor], name: str, shape, dtype, device: int):
    """Checks a tensor and returns its address (None for None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _check(t, name, shape, dtype)
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    return t.data_ptr()


_INT32_MAX = 0x7FFFFFFF  # of the C ABI's 32-bit fields: ctypes would cut a larger size off


def _too_large(names: str, *sizes):
    raise ValueError(f"{names}: {sizes} do not fit into 32 bits")


def _required(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> int:
    if t is None:
        raise ValueError(f"{name} is required")
    return _arg(t, name, shape, dtype, device)


def _rows(n: int, m: int, dtype, device: int) -> torch.Tensor:
    return torch.empty_strided((n, m), (m, 1), dtype=dtype, device=device)


class _On:
    """The device and stream of a call: outputs and workspaces that the binding makes are allocated on the
    stream that uses them, and the launch goes to the tensors' device whatever the current one is."""
    __slots__ = ("raw", "ctx")

    def __init__(self, device: int, stream):
        self.ctx = None
        if stream is not None:
            if stream.device.index != device:
                raise ValueError(f"stream of {stream.device}, tensors on cuda:{device}")
            self.ctx = torch.cuda.stream(stream)
            self.raw = stream.cuda_stream
        else:
            self.raw = torch._C._cuda_getCurrentRawStream(device)
            if torch._C._cuda_getDevice() != device:
                self.ctx = torch.cuda.device(device)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _workspace(workspace, need: int, device: int):
    """(address, bytes, tensor to keep) of the caller's workspace, or of one made here."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    _check(workspace, "workspace", dtype=torch.uint8)
    if workspace.get_device() != device:
        raise ValueError(f"workspace is on {workspace.device}, expected cuda:{device}")
    return workspace.data_ptr(), workspace.numel(), workspace


def _linear_problem(x, gate, gate_kind: int, num_seqs: int):
    """(problem, device, shape, gate's dtype, x's and gate's address)"""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError("x is [T, D]")
    if gate_kind == GDR_LINEAR_LOG_DECAY:
        gate_dtype = torch.float32
    elif gate_kind == GDR_LINEAR_SIGMOID:
        gate_dtype = dtype
    else:
        raise ValueError("gate_kind is GDR_LINEAR_LOG_DECAY or GDR_LINEAR_SIGMOID")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    dev = x.get_device()
    if (num_seqs | shape[1]) > _INT32_MAX:
        _too_large("sequences, channels", num_seqs, shape[1])
    p = LinearProblem(shape[0], num_seqs, shape[1], gate_kind, _dtype_code(dtype))
    return p, dev, shape, gate_dtype, _required(x, "x", shape, dtype, dev), _required(gate, "gate", shape, gate_dtype, dev)


def _seqs(cu_seqlens) -> int:
    if cu_seqlens is None:
        return 1
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens is [N + 1]")
    return cu_seqlens.shape[0] - 1


def gdr_linear_workspace_size(x, gate, gate_kind: int, num_seqs: int) -> int:
    p = _linear_problem(x, gate, gate_kind, num_seqs)[0]
    return lib().gdr_linear_workspace_size(ctypes.byref(p))


def gdr_linear_scan_fwd(x, gate, gate_kind: int, cu_seqlens=None, initial_state=None, y=None, final_state=None,
                        output_final_state: bool = True, block_states=None, output_block_states: bool = False,
                        workspace=None, stream=None):
    """Gated linear recurrence over a packed batch: x [T, D], gate [T, D] (fp32 log-decay, or x's dtype
    before the sigmoid), initial_state [N, D] fp32 (not the same memory as final_state).  Returns (y,
    final_state or None), and block_states
    [ceil(T / GDR_LINEAR_BLOCK), D] for gdr_linear_scan_bwd as a third where it is asked for or given.
    ``workspace`` is a uint8 device tensor of at least gdr_linear_workspace_size bytes (allocated here if
    absent).  Like every function here it records nothing for autograd: a layer that trains calls this and
    gdr_linear_scan_bwd from a torch.autograd.Function's forward and backward."""
    N = _seqs(cu_seqlens)
    p, dev, shape, _, px, pg = _linear_problem(x, gate, gate_kind, N)
    T, D = shape
    states, f32 = (N, D), torch.float32
    with _On(dev, stream) as raw:
        if y is None:
            y = torch.empty_like(x)
        if final_state is None and output_final_state:
            final_state = _rows(N, D, f32, dev)
        blocks = (-(-T // GDR_LINEAR_BLOCK), D)
        want_blocks = output_block_states or block_states is not None
        if want_blocks and block_states is None:
            block_states = _rows(*blocks, f32, dev)
        ref = ctypes.byref(p)
        ws, nb, keep = _workspace(workspace, lib().gdr_linear_workspace_size(ref), dev)
        st = _lib.gdr_linear_scan_fwd(ref, px, pg, _arg(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev),
                                      _arg(initial_state, "initial_state", states, f32, dev),
                                      _required(y, "y", shape, x.dtype, dev),
                                      _arg(final_state, "final_state", states, f32, dev),
                                      _arg(block_states, "block_states", blocks, f32, dev), ws, nb, raw)
    _raise(st, "gdr_linear_scan_fwd")
    return (y, final_state, block_states) if want_blocks else (y, final_state)


def gdr_linear_scan_bwd(x, gate, gate_kind: int, dy, block_states, cu_seqlens=None, initial_state=None,
                        d_final_state=None, dx=None, dgate=None, d_initial_state=None,
                        output_d_initial_state: bool = True, workspace=None, stream=None):
    """Gradients of gdr_linear_scan_fwd: dy [T, D] (x's dtype), block_states as the forward call wrote
    them, d_final_state [N, D] fp32 or None.  Returns (dx, dgate, d_initial_state or None)."""
    N = _seqs(cu_seqlens)
    p, dev, shape, gate_dtype, px, pg = _linear_problem(x, gate, gate_kind, N)
    T, D = shape
    states, f32 = (N, D), torch.float32
    with _On(dev, stream) as raw:
        if dx is None:
            dx = torch.empty_like(x)
        if dgate is None:
            dgate = torch.empty_like(gate)
        if d_initial_state is None and output_d_initial_state:
            d_initial_state = _rows(N, D, f32, dev)
        ref = ctypes.byref(p)
        ws, nb, keep = _workspace(workspace, lib().gdr_linear_workspace_size(ref), dev)
        st = _lib.gdr_linear_scan_bwd(ref, px, pg, _arg(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev),
                                      _arg(initial_state, "initial_state", states, f32, dev),
                                      _required(block_states, "block_states", (-(-T // GDR_LINEAR_BLOCK), D), f32, dev),
                                      _required(dy, "dy", shape, x.dtype, dev),
                                      _arg(d_final_state, "d_final_state", states, f32, dev),
                                      _required(dx, "dx", shape, x.dtype, dev),
                                      _required(dgate, "dgate", shape, gate_dtype, dev),
                                      _arg(d_initial_state, "d_initial_state", states, f32, dev), ws, nb, raw)
    _raise(st, "gdr_linear_scan_bwd")
    return dx, dgate, d_initial_state


def gdr_linear_decode_paged(x, gate, gate_kind: int, pool, state_indices, cu_seqlens=None, max_q_len: int = 1,
                            commit: bool = True, y=None, stream=None):
    """Paged decode of the gated linear recurrence: pool [num_slots, D] (float32 or bfloat16),
    state_indices int32 [N] (negative = padded).  Returns y (rows of padded sequences are left as they
    were)."""
    if state_indices.dim() != 1:
        raise ValueError("state_indices is [N]")
    N = state_indices.shape[0]
    p, dev, shape, _, px, pg = _linear_problem(x, gate, gate_kind, N)
    if pool.dim() != 2:
        raise ValueError("pool is [num_slots, D]")
    with _On(dev, stream) as raw:
        if y is None:
            y = torch.empty_like(x)
        slots = pool.shape[0]
        if (slots | max_q_len) > _INT32_MAX:
            _too_large("slots, max_q_len", slots, max_q_len)
        st = lib().gdr_linear_decode_paged(ctypes.byref(p), max_q_len, px, pg,
                                           _arg(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev),
                                           _arg(pool, "pool", (slots, shape[1]), pool.dtype, dev),
                                           _dtype_code(pool.dtype), slots,
                                           _arg(state_indices, "state_indices", (N,), torch.int32, dev),
                                           1 if commit else 0, _required(y, "y", shape, x.dtype, dev), raw)
    _raise(st, "gdr_linear_decode_paged")
    return y


# ---------------------------------------------------------------------------
def _beam_problem(logits, num_out: int, eos_token: int) -> BeamProblem:
    if logits.dim() != 3:
        raise ValueError("logits is [batch, beams, vocab]")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    B, W, V = logits.shape
    sb, sw, sv = logits.stride()
    # axes of one entry may have any stride
    if (sv != 1 and V > 1) or (B > 1 and W > 1 and sb != W * sw):
        raise ValueError("logits: the rows must be contiguous and evenly spaced")
    row = sw if W > 1 else sb if B > 1 else V
    if max(B | W | V, num_out, eos_token) > _INT32_MAX:
        _too_large("batch, beams, vocab, num_out, eos_token", B, W, V, num_out, eos_token)
    return BeamProblem(B, W, V, num_out, row, eos_token, _dtype_code(logits.dtype))


def gdr_beam_workspace_size(logits, num_out: int) -> int:
    p = _beam_problem(logits, num_out, 0)
    return lib().gdr_beam_workspace_size(ctypes.byref(p))


def gdr_beam_select(logits, scores, num_out: int, finished=None, eos_token: int = -1, out_scores=None,
                    out_parents=None, out_tokens=None, workspace=None, stream=None):
    """The num_out best candidates of each batch row: logits [batch, beams, vocab] (rows may be padded:
    a view of wider rows is taken as it is), scores [batch, beams] fp32, finished [batch, beams] uint8 or
    bool or None.  Returns (scores fp32, parents int32, tokens int32), each [batch, num_out]."""
    p = _beam_problem(logits, num_out, eos_token)
    B, W, _ = logits.shape
    dev, i32 = logits.get_device(), torch.int32
    shape = (B, max(0, num_out))
    if finished is not None and finished.dtype is torch.bool:
        finished = finished.view(torch.uint8)
    with _On(dev, stream) as raw:
        if out_scores is None:
            out_scores = _rows(*shape, torch.float32, dev)
        if out_parents is None:
            out_parents = _rows(*shape, i32, dev)
        if out_tokens is None:
            out_tokens = _rows(*shape, i32, dev)
        ref = ctypes.byref(p)
        ws, nb, keep = _workspace(workspace, lib().gdr_beam_workspace_size(ref), dev)
        st = _lib.gdr_beam_select(ref, logits.data_ptr(), _required(scores, "scores", (B, W), torch.float32, dev),
                                  _arg(finished, "finished", (B, W), torch.uint8, dev),
                                  _required(out_scores, "out_scores", shape, torch.float32, dev),
                                  _required(out_parents, "out_parents", shape, i32, dev),
                                  _required(out_tokens, "out_tokens", shape, i32, dev), ws, nb, raw)
    _raise(st, "gdr_beam_select")
    return out_scores, out_parents, out_tokens


def gdr_beam_reorder(pool, state_indices, parents, slot_dim: int = 0, state_indices_out=None, stream=None):
    """Moves the parents' states to their children: pool [num_slots, ...] (slot_dim 0, as the decode entry
    points take it) or [layers, num_slots, ...] (slot_dim 1), state_indices and parents int32 [batch,
    beams].  Returns the new beams' slots, int32 [batch, beams]; give the old ones to the calls for all
    pools of a model."""
    shape = pool.shape
    if slot_dim not in (0, 1) or len(shape) < slot_dim + 1:
        raise ValueError("pool is [num_slots, ...] with slot_dim 0 or [layers, num_slots, ...] with slot_dim 1")
    if state_indices.dim() != 2:
        raise ValueError("state_indices is [batch, beams]")
    if not pool.is_cuda:
        raise ValueError("pool must be a device tensor")
    rows, dev, i32 = state_indices.shape, pool.get_device(), torch.int32
    slot_bytes = pool.element_size() * math.prod(shape[slot_dim + 1:])
    if (rows[0] | rows[1] | shape[0] | shape[slot_dim]) > _INT32_MAX:
        _too_large("batch, beams, layers, slots", *rows, shape[0], shape[slot_dim])
    with _On(dev, stream) as raw:
        out = _rows(*rows, i32, dev) if state_indices_out is None else state_indices_out
        st = lib().gdr_beam_reorder(rows[0], rows[1], _required(parents, "parents", rows, i32, dev),
                                    _arg(state_indices, "state_indices", rows, i32, dev),
                                    _arg(out, "state_indices_out", rows, i32, dev),
                                    _arg(pool, "pool", shape, pool.dtype, dev), shape[0] if slot_dim else 1,
                                    shape[slot_dim], slot_bytes, raw)
    _raise(st, "gdr_beam_reorder")
    return out
