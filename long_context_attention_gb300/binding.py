"""Thin ctypes binding over libdilution_attn.so (argument marshalling only).

Every function here has the name of the C entry point it forwards to (see
``include/dilution_attn.h``).  Tensors are torch tensors used only as device
memory; every step of the computation runs in the library's CUDA kernels.
The library is loaded on first use; if it cannot be loaded the call raises.
There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

from . import build as _build

DA_OK, DA_ERR_INVALID, DA_ERR_UNSUPPORTED, DA_ERR_CUDA, DA_ERR_TIMEOUT, DA_ERR_WORKSPACE = range(6)
DA_F32, DA_BF16 = 0, 1
DA_FLAG_EARLIER_DEMAND_ONLY = 1
DA_FLAG_KEEP_FOR_BACKWARD = 2
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dilution_attn.h")

_lib = None
_lock = threading.Lock()

_c_void_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_float = ctypes.c_float
_c_size_t = ctypes.c_size_t

_SIGNATURES = {
    "dilution_attn_status_string": (ctypes.c_char_p, [_c_int]),
    "dilution_attn_version": (_c_int, []),
    "dilution_attn_fwd_workspace_size": (_c_size_t, [_c_int] * 5),
    "dilution_attn_fwd": (_c_int, [_c_void_p] * 7 + [_c_int] * 4 + [_c_float, _c_float, _c_int, _c_void_p,
                                                                        _c_size_t, _c_void_p]),
    "dilution_attn_fwd_with_events": (_c_int, [_c_void_p] * 7 + [_c_int] * 4 + [_c_float, _c_float, _c_int,
                                                                                    _c_void_p, _c_size_t, _c_void_p,
                                                                                    _c_void_p]),
    "dilution_attn_fwd_ex": (_c_int, [_c_void_p] * 7 + [_c_int] * 4 + [_c_float, _c_void_p, _c_float, _c_int, _c_int,
                                                                       _c_void_p, _c_size_t, _c_void_p, _c_void_p]),
    "dilution_attn_bwd_workspace_size": (_c_size_t, [_c_int] * 5),
    "dilution_attn_bwd": (_c_int, [_c_void_p] * 8 + [_c_int] * 4 + [_c_float, _c_float, _c_int, _c_void_p, _c_size_t,
                                                                        _c_void_p]),
    "dilution_attn_bwd_ex": (_c_int, [_c_void_p] * 8 + [_c_int] * 4 + [_c_float, _c_void_p, _c_float, _c_int, _c_int,
                                                                       _c_void_p, _c_size_t, _c_void_p]),
    "dilution_attn_decode_workspace_size": (_c_size_t, [_c_int] * 4),
    "dilution_attn_decode_step": (_c_int, [_c_void_p] * 6 + [_c_int, _c_int, _c_void_p] + [_c_int] * 3 +
                                  [_c_float, _c_float, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "dilution_attn_decode_step_ex": (_c_int, [_c_void_p] * 6 + [_c_int, _c_int, _c_void_p] + [_c_int] * 3 +
                                     [_c_float, _c_void_p, _c_float, _c_int, _c_int, _c_void_p, _c_size_t,
                                      _c_void_p]),
    "dilution_attn_decode_step_noalloc": (_c_int, [_c_void_p] * 6 + [_c_int, _c_int, _c_void_p] + [_c_int] * 3 +
                                          [_c_float, _c_float, _c_int, _c_void_p]),
    "dilution_attn_decode_noalloc_scratch_bytes": (_c_size_t, []),
    "dilution_attn_decode_noalloc_get_error": (_c_int, [_c_void_p]),
    "dilution_attn_debug_decode_stall": (_c_int, [_c_void_p] * 6 + [_c_int, _c_int, _c_void_p] + [_c_int] * 3 +
                                         [_c_float, _c_float, _c_int, _c_void_p, _c_size_t, _c_void_p, _c_int, _c_int,
                                          ctypes.c_longlong]),
    "dilution_attn_rope": (_c_int, [_c_void_p] * 9 + [_c_int, _c_void_p] + [_c_int] * 6 + [_c_void_p]),
    "dilution_attn_rope_bwd": (_c_int, [_c_void_p] * 9 + [_c_int, _c_void_p] + [_c_int] * 6 + [_c_void_p]),
    "dilution_attn_paged_append_workspace_size": (_c_size_t, []),
    "dilution_attn_paged_append": (_c_int, [_c_void_p] * 10 + [_c_int] + [_c_void_p] * 4 + [_c_size_t, _c_void_p]),
    "dilution_attn_paged_decode_workspace_size": (_c_size_t, [_c_int] * 8),
    "dilution_attn_paged_decode": (_c_int, [_c_void_p] * 3 + [_c_int, _c_int, _c_void_p, _c_float, _c_void_p, _c_float,
                                                             _c_int, _c_void_p, _c_size_t, _c_void_p]),
    "dilution_attn_paged_decode_ex": (_c_int, [_c_void_p] * 3 + [_c_int, _c_int, _c_void_p, _c_float, _c_void_p, _c_float,
                                                                _c_int, _c_void_p, _c_size_t, _c_void_p, _c_void_p]),
    "dilution_attn_debug_paged_decode_stall": (_c_int, [_c_void_p] * 3 + [_c_int, _c_int, _c_void_p, _c_float, _c_float,
                                                                         _c_void_p, _c_size_t, _c_void_p, _c_int, _c_int,
                                                                         ctypes.c_longlong]),
    "dilution_attn_get_error": (_c_int, [_c_void_p, _c_void_p]),
    "dilution_attn_debug_last_timeout": (_c_int, [_c_void_p, _c_void_p]),
    "dilution_attn_debug_tile_schedule": (_c_int, [_c_int, _c_int, _c_int, _c_void_p, _c_size_t]),
    "dilution_attn_debug_tile_mask": (_c_int, [_c_int, _c_int, _c_int, _c_void_p]),
}


class DilutionAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)}")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load (building first if needed) and return the ctypes library handle."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if build_if_missing and not os.path.exists(path):
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"libdilution_attn.so not found at {path}; run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def header_functions() -> list[str]:
    """Names of every function the public header declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dilution_attn_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return load().dilution_attn_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != DA_OK:
        raise DilutionAttnError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DA_F32
    if t.dtype == torch.bfloat16:
        return DA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _need(t, name, shape=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device and takes its per-device
        # set-up (and the no-alloc scratch address) from it
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{torch.cuda.current_device()}; "
                         f"call inside torch.cuda.device({t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


# --------------------------------------------------------------------------- forward
def dilution_attn_fwd_workspace_size(B: int, H: int, T: int, d: int, dtype: int) -> int:
    return int(load().dilution_attn_fwd_workspace_size(B, H, T, d, dtype))


def dilution_attn_fwd(q, k, v, out=None, lse2_out=None, rowsum_out=None, demand_out=None, *,
                      tau: float = 1.0, eps: float = 1e-6, workspace=None, stream=None, check: bool = True):
    """Forward over [B, H, T, d] q/k/v (float32 or bfloat16, contiguous, CUDA).

    Returns ``out`` (allocated if not given).  Optional fp32 [B, H, T] side
    outputs are filled when passed.  ``workspace`` (uint8 CUDA tensor) is
    allocated when omitted.
    """
    return dilution_attn_fwd_with_events(q, k, v, out, lse2_out, rowsum_out, demand_out, tau=tau, eps=eps,
                                         workspace=workspace, stream=stream, check=check, events=None)


def _event_handle(e):
    if e is None:
        return None
    if e.cuda_event == 0:   # torch creates the CUDA event lazily, on first record
        e.record()
    return e.cuda_event


def _fwd_prepare(q, k, v, out, lse2_out, rowsum_out, demand_out, workspace, flags=0):
    _need(q, "q")
    B, H, T, d = q.shape
    _need(k, "k", q.shape, q.dtype)
    _need(v, "v", q.shape, q.dtype)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.shape, q.dtype)
    for name, t in (("lse2_out", lse2_out), ("rowsum_out", rowsum_out), ("demand_out", demand_out)):
        if t is not None:
            _need(t, name, (B, H, T), torch.float32)
    dt = _dtype_code(q)
    need = (dilution_attn_bwd_workspace_size(B, H, T, d, dt) if flags & DA_FLAG_KEEP_FOR_BACKWARD
            else dilution_attn_fwd_workspace_size(B, H, T, d, dt))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    return out, workspace, dt


def _events_array(events):
    if events is None:
        return None
    return (ctypes.c_void_p * 4)(*[_event_handle(e) for e in events])


def _tau_bh_ptr(tau_bh, B, H):
    """Marshal an optional per-(batch, head) multiplier tensor: fp32 CUDA, B*H elements."""
    if tau_bh is None:
        return None
    _need(tau_bh, "tau_bh", None, torch.float32)
    if tau_bh.numel() != B * H:
        raise ValueError(f"tau_bh has {tau_bh.numel()} elements, expected B*H = {B * H}")
    return _ptr(tau_bh)


def dilution_attn_fwd_with_events(q, k, v, out=None, lse2_out=None, rowsum_out=None, demand_out=None, *,
                                  tau: float = 1.0, eps: float = 1e-6, workspace=None, stream=None,
                                  check: bool = True, events=None):
    """dilution_attn_fwd that also records up to four torch.cuda.Event
    (timing-enabled) on the stream: before row statistics, before the sweep,
    before finalize, after finalize."""
    lib = load()
    out, workspace, dt = _fwd_prepare(q, k, v, out, lse2_out, rowsum_out, demand_out, workspace)
    B, H, T, d = q.shape
    st = lib.dilution_attn_fwd_with_events(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse2_out), _ptr(rowsum_out),
                                           _ptr(demand_out), B, H, T, d, float(tau), float(eps), dt,
                                           _ptr(workspace), workspace.numel(), _stream_handle(stream),
                                           _events_array(events))
    if check:
        _check(st, "dilution_attn_fwd")
    return out


def dilution_attn_fwd_ex(q, k, v, out=None, lse2_out=None, rowsum_out=None, demand_out=None, *,
                         tau: float = 1.0, tau_bh=None, eps: float = 1e-6, flags: int = 0, workspace=None,
                         stream=None, check: bool = True, events=None):
    """Forward with a per-(batch, head) multiplier tensor ``tau_bh`` (fp32 CUDA,
    B*H elements, index b*H + h; replaces ``tau``) and ``flags``
    (``DA_FLAG_EARLIER_DEMAND_ONLY``, ``DA_FLAG_KEEP_FOR_BACKWARD``: pass the
    same ``workspace`` to ``dilution_attn_bwd_ex`` with the same flags; it is
    allocated backward-sized when omitted)."""
    lib = load()
    out, workspace, dt = _fwd_prepare(q, k, v, out, lse2_out, rowsum_out, demand_out, workspace, int(flags))
    B, H, T, d = q.shape
    st = lib.dilution_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse2_out), _ptr(rowsum_out),
                                  _ptr(demand_out), B, H, T, d, float(tau), _tau_bh_ptr(tau_bh, B, H), float(eps),
                                  int(flags), dt, _ptr(workspace), workspace.numel(), _stream_handle(stream),
                                  _events_array(events))
    if check:
        _check(st, "dilution_attn_fwd_ex")
    return out


# -------------------------------------------------------------------------- backward
def dilution_attn_bwd_workspace_size(B: int, H: int, T: int, d: int, dtype: int) -> int:
    return int(load().dilution_attn_bwd_workspace_size(B, H, T, d, dtype))


def _bwd_prepare(q, k, v, dout, lse2, dq, dk, dv, workspace):
    _need(q, "q")
    B, H, T, d = q.shape
    for name, t in (("k", k), ("v", v), ("dout", dout)):
        _need(t, name, q.shape, q.dtype)
    _need(lse2, "lse2", (B, H, T), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, q.shape, q.dtype)
    dt = _dtype_code(q)
    if workspace is None:
        workspace = torch.empty(max(dilution_attn_bwd_workspace_size(B, H, T, d, dt), 256), dtype=torch.uint8,
                                device=q.device)
    return dq, dk, dv, workspace, dt


def dilution_attn_bwd(q, k, v, dout, lse2, dq=None, dk=None, dv=None, *, tau: float = 1.0, eps: float = 1e-6,
                      workspace=None, stream=None, check: bool = True):
    """Gradients (dq, dk, dv) of sum(dout * out); lse2 is the forward's lse2_out."""
    lib = load()
    dq, dk, dv, workspace, dt = _bwd_prepare(q, k, v, dout, lse2, dq, dk, dv, workspace)
    B, H, T, d = q.shape
    st = lib.dilution_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse2), _ptr(dq), _ptr(dk), _ptr(dv), B,
                               H, T, d, float(tau), float(eps), dt, _ptr(workspace), workspace.numel(),
                               _stream_handle(stream))
    if check:
        _check(st, "dilution_attn_bwd")
    return dq, dk, dv


def dilution_attn_bwd_ex(q, k, v, dout, lse2, dq=None, dk=None, dv=None, *, tau: float = 1.0, tau_bh=None,
                         eps: float = 1e-6, flags: int = 0, workspace=None, stream=None, check: bool = True):
    """dilution_attn_bwd with the ``tau_bh`` and ``flags`` of the matching forward."""
    lib = load()
    dq, dk, dv, workspace, dt = _bwd_prepare(q, k, v, dout, lse2, dq, dk, dv, workspace)
    B, H, T, d = q.shape
    st = lib.dilution_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse2), _ptr(dq), _ptr(dk), _ptr(dv),
                                  B, H, T, d, float(tau), _tau_bh_ptr(tau_bh, B, H), float(eps), int(flags), dt,
                                  _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if check:
        _check(st, "dilution_attn_bwd_ex")
    return dq, dk, dv


# ---------------------------------------------------------------------------- decode
def dilution_attn_decode_workspace_size(B: int, H: int, T_cap: int, d: int) -> int:
    return int(load().dilution_attn_decode_workspace_size(B, H, T_cap, d))


def _decode_prepare(q_new, k_new, v_new, k_cache, v_cache, demand, out):
    _need(q_new, "q_new")
    B, H, d = q_new.shape
    _need(k_new, "k_new", q_new.shape, q_new.dtype)
    _need(v_new, "v_new", q_new.shape, q_new.dtype)
    _need(k_cache, "k_cache", None, q_new.dtype)
    T_cap = k_cache.shape[2]
    _need(k_cache, "k_cache", (B, H, T_cap, d))
    _need(v_cache, "v_cache", (B, H, T_cap, d), q_new.dtype)
    _need(demand, "demand", (B, H, T_cap), torch.float32)
    if out is None:
        out = torch.empty_like(q_new)
    _need(out, "out", q_new.shape, q_new.dtype)
    return out, T_cap


def dilution_attn_decode_step(q_new, k_new, v_new, k_cache, v_cache, demand, n_ctx: int, out=None, *,
                              tau: float = 1.0, eps: float = 1e-6, workspace=None, stream=None,
                              check: bool = True):
    """One cached decode step; caches [B, H, T_cap, d], demand [B, H, T_cap] fp32.

    Appends k_new/v_new at position n_ctx, updates ``demand`` in place and
    returns ``out`` [B, H, d].
    """
    lib = load()
    out, T_cap = _decode_prepare(q_new, k_new, v_new, k_cache, v_cache, demand, out)
    B, H, d = q_new.shape
    if workspace is None:
        workspace = torch.empty(max(dilution_attn_decode_workspace_size(B, H, T_cap, d), 256), dtype=torch.uint8,
                                device=q_new.device)
    st = lib.dilution_attn_decode_step(_ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(demand), int(n_ctx), T_cap, _ptr(out), B, H, d, float(tau), float(eps),
                                       _dtype_code(q_new), _ptr(workspace), workspace.numel(),
                                       _stream_handle(stream))
    if check:
        _check(st, "dilution_attn_decode_step")
    return out


def dilution_attn_decode_step_ex(q_new, k_new, v_new, k_cache, v_cache, demand, n_ctx: int, out=None, *,
                                 tau: float = 1.0, tau_bh=None, eps: float = 1e-6, flags: int = 0, workspace=None,
                                 stream=None, check: bool = True):
    """dilution_attn_decode_step with ``tau_bh`` and ``flags`` (see dilution_attn_fwd_ex)."""
    lib = load()
    out, T_cap = _decode_prepare(q_new, k_new, v_new, k_cache, v_cache, demand, out)
    B, H, d = q_new.shape
    if workspace is None:
        workspace = torch.empty(max(dilution_attn_decode_workspace_size(B, H, T_cap, d), 256), dtype=torch.uint8,
                                device=q_new.device)
    st = lib.dilution_attn_decode_step_ex(_ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(demand), int(n_ctx), T_cap, _ptr(out), B, H, d, float(tau),
                                          _tau_bh_ptr(tau_bh, B, H), float(eps), int(flags), _dtype_code(q_new),
                                          _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if check:
        _check(st, "dilution_attn_decode_step_ex")
    return out


def dilution_attn_decode_step_noalloc(q_new, k_new, v_new, k_cache, v_cache, demand, n_ctx: int, out=None, *,
                                      tau: float = 1.0, eps: float = 1e-6, stream=None, check: bool = True):
    """dilution_attn_decode_step with the library's fixed scratch array instead of a workspace."""
    lib = load()
    out, T_cap = _decode_prepare(q_new, k_new, v_new, k_cache, v_cache, demand, out)
    B, H, d = q_new.shape
    st = lib.dilution_attn_decode_step_noalloc(_ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                               _ptr(demand), int(n_ctx), T_cap, _ptr(out), B, H, d, float(tau),
                                               float(eps), _dtype_code(q_new), _stream_handle(stream))
    if check:
        _check(st, "dilution_attn_decode_step_noalloc")
    return out


def dilution_attn_decode_noalloc_scratch_bytes() -> int:
    return int(load().dilution_attn_decode_noalloc_scratch_bytes())


def dilution_attn_decode_noalloc_get_error(stream=None) -> int:
    """Status of the no-alloc decode step's fixed array on the current
    device (synchronises the stream, then reads and clears the word)."""
    return int(load().dilution_attn_decode_noalloc_get_error(_stream_handle(stream)))


def dilution_attn_debug_decode_stall(q_new, k_new, v_new, k_cache, v_cache, demand, n_ctx: int, out=None, *,
                                     tau: float = 1.0, eps: float = 1e-6, workspace=None, stream=None,
                                     stall_chunk: int = 0, stall_bh: int = 0, wait_limit_ns: int = 2_000_000):
    """Test hook of the bounded waits: a decode step in which one block's ring
    slot is never handed back (see the header).  Returns (status, out); the
    kernel-side outcome is read with dilution_attn_debug_last_timeout /
    dilution_attn_get_error on ``workspace``."""
    lib = load()
    out, T_cap = _decode_prepare(q_new, k_new, v_new, k_cache, v_cache, demand, out)
    B, H, d = q_new.shape
    if workspace is None:
        workspace = torch.empty(max(dilution_attn_decode_workspace_size(B, H, T_cap, d), 256), dtype=torch.uint8,
                                device=q_new.device)
    st = lib.dilution_attn_debug_decode_stall(_ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                              _ptr(demand), int(n_ctx), T_cap, _ptr(out), B, H, d, float(tau),
                                              float(eps), _dtype_code(q_new), _ptr(workspace), workspace.numel(),
                                              _stream_handle(stream), int(stall_chunk), int(stall_bh),
                                              int(wait_limit_ns))
    return int(st), out


# --------------------------------------------------------------------- rotary positions
DA_MAX_ROPE_PAIRS, DA_MAX_ROPE_AXES = 64, 4


class _CRopeSpec(ctypes.Structure):
    _fields_ = [("inv_freq", _c_void_p), ("n_pairs", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("adjacent", ctypes.c_int32), ("pair_axis", ctypes.c_uint8 * DA_MAX_ROPE_PAIRS)]


class RopeSpec:
    """What ``rope_spec`` returns: the C struct, the frequencies it points to and its sizes."""

    __slots__ = ("inv_freq", "n_pairs", "n_axes", "adjacent", "_c", "_ref", "_dev")

    def __init__(self, inv_freq, pair_axis, n_axes, adjacent):
        self.inv_freq, self.n_pairs, self.n_axes, self.adjacent = inv_freq, len(pair_axis), n_axes, adjacent
        self._c = _CRopeSpec(inv_freq.data_ptr(), self.n_pairs, n_axes, int(adjacent),
                             (ctypes.c_uint8 * DA_MAX_ROPE_PAIRS)(*pair_axis))
        self._ref = ctypes.byref(self._c)
        self._dev = inv_freq.get_device()


def rope_spec(inv_freq, pair_axis=None, n_axes: int = 1, adjacent: bool = False) -> RopeSpec:
    """Rotation of ``inv_freq.numel()`` pairs of a head's elements (fp32 CUDA
    frequencies, radians per position).  ``pair_axis``: the position axis of
    each pair (axis 0 when omitted).  Pairs are (j, n_pairs + j), or
    (2j, 2j + 1) with ``adjacent``.  The tensor is read by every call that
    gets the spec: new frequencies written into it take effect."""
    _need(inv_freq, "inv_freq", None, torch.float32)
    n = inv_freq.numel()
    if inv_freq.dim() != 1 or n > DA_MAX_ROPE_PAIRS:
        raise ValueError(f"inv_freq must be one-dimensional with at most {DA_MAX_ROPE_PAIRS} entries")
    if not 1 <= n_axes <= DA_MAX_ROPE_AXES:
        raise ValueError(f"n_axes must be 1 .. {DA_MAX_ROPE_AXES}, got {n_axes}")
    pair_axis = [0] * n if pair_axis is None else [int(a) for a in pair_axis]
    if len(pair_axis) != n or any(not 0 <= a < n_axes for a in pair_axis):
        raise ValueError(f"pair_axis must hold {n} axes in 0 .. {n_axes - 1}")
    return RopeSpec(inv_freq, pair_axis, int(n_axes), bool(adjacent))


# The calls of a serving loop are short (a few microseconds on the GPU), so their
# checks are written for the case that passes: one condition per tensor, the
# device and the stream read once, strides kept as C arrays by their values.
_Tensor = torch.Tensor


def _fit(t, name, shape, dtype, dev):
    """_need for a contiguous tensor on device ``dev`` (the current one)."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, tuple(shape), dtype)


def _fit_rows(t, name, shape, dtype, dev):
    """The same for a tensor whose last dimension alone is contiguous; returns the
    strides of the others as a C array."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape):
        _need_any_strides(t, name, tuple(shape), dtype)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _stride_arrays.get(st) or _c_strides(st, len(st) - 1)


def _need_any_strides(t, name, shape, dtype):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.device.index == torch.cuda.current_device():
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    _need(t, name)


_stride_arrays: dict = {}   # of tensors of rows: strides -> all but the last as a C array


def _c_strides(st, n):
    """The first n of a tensor's strides as a C array, kept if they are all but the last."""
    got = (ctypes.c_int64 * n)(*st[:n])
    if n == len(st) - 1:
        if len(_stride_arrays) >= 4096:
            _stride_arrays.clear()
        _stride_arrays[st] = got
    return got


_cuda_up = False


def _current_device() -> int:
    global _cuda_up
    if not _cuda_up:
        if not torch.cuda.is_initialized():
            return torch.cuda.current_device()
        _cuda_up = True
    return _get_device()


# absent in a torch without CUDA, where every call fails its tensor checks before
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_id(stream, dev) -> int:
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _need_bytes(workspace, dev):
    if not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and workspace.get_device() == dev
            and workspace.is_contiguous()):
        _need(workspace, "workspace", None, torch.uint8)


def _need_table(table, dev):
    if not (isinstance(table, torch.Tensor) and table.dtype is torch.int32 and table.get_device() == dev
            and table.dim() == 1 and table.is_contiguous()):
        _need(table, "prefix_table", None, torch.int32)
        raise ValueError("prefix_table must be one-dimensional")


def _new(shape, dtype, device, stream):
    """A tensor for a call on ``stream`` (None: the current one), allocated on
    that stream: its memory is then not handed on before the call has used it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_CODES = {torch.float32: DA_F32, torch.bfloat16: DA_BF16}


def _rope_call(name, q, k, positions, rope, q_out, k_out, stream, check):
    lib = _lib or load()
    if type(rope) is not RopeSpec:
        raise TypeError("rope must be a RopeSpec (see rope_spec)")
    if not isinstance(q, _Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, H, T, d] tensor")
    shape, dtype = q.shape, q.dtype
    B, Hq, T, d = shape
    dt = _CODES.get(dtype)
    if dt is None:
        dt = _dtype_code(q)
    dev = _current_device()
    sq = _fit_rows(q, "q", shape, dtype, dev)
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=q.device) if stream is None else _new(shape, dtype, q.device, stream)
        so = None
    else:
        so = _fit_rows(q_out, "q_out", shape, dtype, dev)
    if k is not None:
        Hk = k.shape[1] if isinstance(k, _Tensor) and k.dim() == 4 else 0
        kshape = shape if Hk == Hq else (B, Hk, T, d)
        sk, kp = _fit_rows(k, "k", kshape, dtype, dev), k.data_ptr()
        if k_out is None:
            k_out = torch.empty(kshape, dtype=dtype, device=q.device) if stream is None else \
                _new(kshape, dtype, q.device, stream)
            sko = None
        else:
            sko = _fit_rows(k_out, "k_out", kshape, dtype, dev)
        kop = k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        Hk, sk, kp, sko, kop = 0, None, None, None, None
    if not (isinstance(positions, torch.Tensor) and positions.dtype is torch.int32 and positions.get_device() == dev
            and positions.is_contiguous()):
        _need(positions, "positions", None, torch.int32)
    ps = positions.shape
    pb = 1 if len(ps) == 2 else ps[1] if len(ps) == 3 else -1
    if pb not in (1, B) or ps[0] != rope.n_axes or ps[-1] != T:
        raise ValueError(f"positions has shape {tuple(ps)}, expected ({rope.n_axes}, [1 or {B},] {T})")
    if rope._dev != dev:
        _need(rope.inv_freq, "inv_freq")
    st = getattr(lib, name)(q.data_ptr(), sq, kp, sk, q_out.data_ptr(), so, kop, sko, positions.data_ptr(), pb,
                            rope._ref, B, Hq, Hk, T, d, dt, _stream_id(stream, dev))
    if check and st != DA_OK:
        _check(st, name)
    return q_out, k_out


def dilution_attn_rope(q, k, positions, rope, q_out=None, k_out=None, *, stream=None, check: bool = True):
    """Queries and keys turned by their positions: q [B, Hq, T, d], k [B, Hk, T, d]
    (views of a fused projection are fine; k may be None) -> (q_out, k_out),
    contiguous [B, H, T, d] when not given.  positions: int32 [n_axes, T] or
    [n_axes, B, T]; ``rope``: see rope_spec."""
    return _rope_call("dilution_attn_rope", q, k, positions, rope, q_out, k_out, stream, check)


def dilution_attn_rope_bwd(dq_out, dk_out, positions, rope, dq=None, dk=None, *, stream=None, check: bool = True):
    """Gradients (dq, dk) of dilution_attn_rope's inputs from those of its
    outputs; dq and dk may be views of a fused projection's gradient."""
    return _rope_call("dilution_attn_rope_bwd", dq_out, dk_out, positions, rope, dq, dk, stream, check)


# ---------------------------------------------------------------------------- paged cache
def _zeroed_status(device):
    """A status block that is zero for calls on every stream, whatever the current one still has to do."""
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(256, dtype=torch.uint8, device=device)
    side = torch.cuda.Stream(device)
    with torch.cuda.stream(side):
        t = torch.zeros(256, dtype=torch.uint8, device=device)
    side.synchronize()
    return t


_graph_status: dict = {}   # the status blocks of captured calls: a graph may outlive the cache object


def _own_status(cache, stream):
    """The cache's status block for a call on ``stream``: not handed on, if the cache goes, before the call has ended
    (of a captured call, not at all)."""
    cache.status.record_stream(torch.cuda.current_stream() if stream is None else stream)
    if torch.cuda.is_current_stream_capturing():
        _graph_status[id(cache.status)] = cache.status
    return cache.status


class _CPagedCache(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in ("k_pages", "v_pages", "demand_pages", "page_table", "demand_table", "seq_lens")] \
        + [(n, ctypes.c_int32) for n in ("S", "Hq", "Hkv", "d", "page_size", "num_pages", "num_demand_pages",
                                         "max_pages", "dtype")]


class PagedCache:
    """The tensors of a paged cache (see the header): k_pages, v_pages
    [num_pages, Hkv, page_size, d], demand_pages [num_demand_pages, Hq,
    page_size] fp32, page_table and demand_table [S, max_pages] int32, seq_lens
    [S] int32.  Checked once here; the tables and lengths are the caller's to
    update in place between calls.  ``status``: the status block of the calls
    that are given no workspace; dilution_attn_get_error(cache.status) reads and
    clears the first bad length or page that they found."""

    __slots__ = ("k_pages", "v_pages", "demand_pages", "page_table", "demand_table", "seq_lens", "status", "S", "Hq", "Hkv", "d",
                 "page_size", "max_pages", "dtype", "device", "_code", "_c", "_ref", "_dev", "_q_shape", "_cu_shape")

    def __init__(self, k_pages, v_pages, demand_pages, page_table, demand_table, seq_lens):
        _need(k_pages, "k_pages")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [num_pages, Hkv, page_size, d]")
        num_pages, Hkv, page_size, d = k_pages.shape
        _need(v_pages, "v_pages", k_pages.shape, k_pages.dtype)
        _need(demand_pages, "demand_pages", None, torch.float32)
        if demand_pages.dim() != 3 or demand_pages.shape[2] != page_size:
            raise ValueError(f"demand_pages must be [num_demand_pages, Hq, {page_size}]")
        num_demand_pages, Hq, _ = demand_pages.shape
        if Hkv < 1 or Hq < 1 or Hq % Hkv != 0:
            raise ValueError(f"{Hq} query heads over {Hkv} key heads: not a multiple")
        _need(page_table, "page_table", None, torch.int32)
        if page_table.dim() != 2:
            raise ValueError("page_table must be [S, max_pages]")
        S, max_pages = page_table.shape
        _need(demand_table, "demand_table", page_table.shape, torch.int32)
        _need(seq_lens, "seq_lens", (S,), torch.int32)
        self._code = _dtype_code(k_pages)
        self.k_pages, self.v_pages, self.demand_pages = k_pages, v_pages, demand_pages
        self.page_table, self.demand_table, self.seq_lens = page_table, demand_table, seq_lens
        self.S, self.Hq, self.Hkv, self.d, self.page_size, self.max_pages = S, Hq, Hkv, d, page_size, max_pages
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self._c = _CPagedCache(*(t.data_ptr() for t in (k_pages, v_pages, demand_pages, page_table, demand_table,
                                                        seq_lens)), S, Hq, Hkv, d, page_size, num_pages,
                               num_demand_pages, max_pages, self._code)
        self._ref = ctypes.byref(self._c)
        self.status = _zeroed_status(self.device)
        self._dev, self._q_shape, self._cu_shape = k_pages.get_device(), torch.Size((S, Hq, d)), torch.Size((S + 1,))


def _need_cache(cache) -> int:
    """The cache's device, which has to be the current one."""
    if type(cache) is not PagedCache:
        raise TypeError("cache must be a PagedCache")
    dev = _current_device()
    if cache._dev != dev:
        raise ValueError(f"the cache is on {cache.device} but the current device is cuda:{dev}; "
                         f"call inside torch.cuda.device({cache.device})")
    return dev


def dilution_attn_paged_append_workspace_size() -> int:
    return int(load().dilution_attn_paged_append_workspace_size())


def dilution_attn_paged_append_workspace(cache):
    """A workspace for dilution_attn_paged_append, its status block zeroed."""
    return torch.zeros(dilution_attn_paged_append_workspace_size(), dtype=torch.uint8, device=cache.device)


def dilution_attn_paged_append(q, k, v, cache, cu_tokens, q_out=None, *, rope=None, positions=None, demand=None,
                               workspace=None, stream=None, check: bool = True):
    """Append k, v [N, Hkv, d] (rows may be strided) as the last tokens of the
    cache's sequences: sequence s takes tokens cu_tokens[s] .. cu_tokens[s+1]-1
    (int32 [S+1]; seq_lens already counts them).  With ``rope`` the keys turn
    on the way, by ``positions`` (int32 [n_axes, N]) or by their place in the
    sequence.  ``demand`` [N, Hq] fp32: the keys' totals (a prompt's
    demand_out after prefill), 0 when omitted.  q [N, Hq, d] (or None) turns
    likewise into ``q_out`` (contiguous), which is returned.  Bad lengths or
    page ids are found on the device: read them with dilution_attn_get_error on
    ``workspace``, or on ``cache.status`` if none is given."""
    lib = _lib or load()
    dev = _need_cache(cache)
    Hq, Hkv, d, dtype = cache.Hq, cache.Hkv, cache.d, cache.dtype
    if not isinstance(k, _Tensor) or k.dim() != 3:
        raise ValueError("k must be [N, Hkv, d]")
    N = k.shape[0]
    kvshape = (N, Hkv, d)
    sk = _fit_rows(k, "k", kvshape, dtype, dev)
    sv = _fit_rows(v, "v", kvshape, dtype, dev)
    _fit(cu_tokens, "cu_tokens", cache._cu_shape, torch.int32, dev)
    qp = sq = qop = dp = sd = None
    if q is not None:
        qshape = (N, Hq, d)
        sq, qp = _fit_rows(q, "q", qshape, dtype, dev), q.data_ptr()
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dtype, device=cache.device) if stream is None else \
                _new(qshape, dtype, cache.device, stream)
        else:
            _fit(q_out, "q_out", qshape, dtype, dev)
        qop = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rope is not None:
        if type(rope) is not RopeSpec:
            raise TypeError("rope must be a RopeSpec (see rope_spec)")
        if rope._dev != dev:
            _need(rope.inv_freq, "inv_freq")
    if positions is not None:
        _fit(positions, "positions", (1 if rope is None else rope.n_axes, N), torch.int32, dev)
    if demand is not None:
        if not (isinstance(demand, torch.Tensor) and demand.dtype is torch.float32 and demand.get_device() == dev
                and demand.shape == (N, Hq)):
            _need_any_strides(demand, "demand", (N, Hq), torch.float32)
        dp, sd = demand.data_ptr(), _c_strides(demand.stride(), 2)
    if workspace is None:
        workspace = _own_status(cache, stream)     # an append needs nothing else
    else:
        _need_bytes(workspace, dev)
    st = lib.dilution_attn_paged_append(qp, sq, k.data_ptr(), sk, v.data_ptr(), sv, dp, sd, qop, cu_tokens.data_ptr(), N,
                                        cache._ref, None if rope is None else rope._ref,
                                        None if positions is None else positions.data_ptr(), workspace.data_ptr(),
                                        workspace.numel(), _stream_id(stream, dev))
    if check and st != DA_OK:
        _check(st, "dilution_attn_paged_append")
    return q_out


def dilution_attn_paged_decode_workspace_size(S: int, Hq: int, Hkv: int, d: int, max_len: int, n_prefix_pages: int,
                                              page_size: int, dtype: int) -> int:
    return int(load().dilution_attn_paged_decode_workspace_size(S, Hq, Hkv, d, max_len, n_prefix_pages, page_size,
                                                                dtype))


def dilution_attn_paged_decode_workspace(cache, max_len: int, n_prefix_pages=None):
    """A workspace for dilution_attn_paged_decode over ``cache`` up to
    ``max_len`` tokens, its status block zeroed.  n_prefix_pages: the prefix
    it will serve (omitted: large enough for any)."""
    args = (cache.S, cache.Hq, cache.Hkv, cache.d, int(max_len))
    # the size depends on whether there is a prefix, not on its length
    counts = (0, min(1, int(max_len) // cache.page_size)) if n_prefix_pages is None else (int(n_prefix_pages),)
    need = max(dilution_attn_paged_decode_workspace_size(*args, n, cache.page_size, cache._code) for n in counts)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=cache.device)
    ws[:256].zero_()
    return ws


def dilution_attn_paged_decode(q, cache, max_len: int, out=None, *, prefix_table=None, tau: float = 1.0, tau_bh=None,
                               eps: float = 1e-6, flags: int = 0, workspace=None, stream=None, check: bool = True):
    """One decode step of every sequence of ``cache`` (the new tokens are
    already appended): q [S, Hq, d] -> ``out`` [S, Hq, d]; each key's demand
    grows by its bid.  ``max_len``: upper bound of cache.seq_lens.
    ``prefix_table`` (int32 [n]): pages of the tokens that every sequence
    shares, read for many sequences at once.  Bad lengths or page ids are found on the
    device: read them with dilution_attn_get_error on ``workspace``, or on
    ``cache.status`` if none is given."""
    lib = _lib or load()
    dev = _need_cache(cache)
    shape, dtype = cache._q_shape, cache.dtype
    _fit(q, "q", shape, dtype, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=cache.device) if stream is None else \
            _new(shape, dtype, cache.device, stream)
    else:
        _fit(out, "out", shape, dtype, dev)
    n_prefix, pt = 0, None
    if prefix_table is not None:
        _need_table(prefix_table, dev)
        n_prefix, pt = prefix_table.numel(), prefix_table.data_ptr()
    if workspace is None:
        need = dilution_attn_paged_decode_workspace_size(cache.S, cache.Hq, cache.Hkv, cache.d, int(max_len), n_prefix,
                                                         cache.page_size, cache._code)
        workspace, status = _new(max(need, 256), torch.uint8, cache.device, stream), _own_status(cache, stream).data_ptr()
    else:
        _need_bytes(workspace, dev)
        status = workspace.data_ptr()
    st = lib.dilution_attn_paged_decode_ex(q.data_ptr(), cache._ref, pt, n_prefix, int(max_len), out.data_ptr(), float(tau),
                                           None if tau_bh is None else _tau_bh_ptr(tau_bh, cache.S, cache.Hq), float(eps),
                                           int(flags), workspace.data_ptr(), workspace.numel(), status,
                                           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if check and st != DA_OK:
        _check(st, "dilution_attn_paged_decode")
    return out


def dilution_attn_debug_paged_decode_stall(q, cache, max_len: int, *, workspace, prefix_table=None, tau: float = 1.0,
                                           eps: float = 1e-6, stream=None, stall_kernel: int = 0, stall_block: int = 0,
                                           wait_limit_ns: int = 2_000_000):
    """Test hook of the bounded waits: a paged decode step in which one block
    of one kernel keeps what another role waits for (see the header).  Returns
    (status, out); the kernel-side outcome is read with
    dilution_attn_debug_last_timeout / dilution_attn_get_error on ``workspace``."""
    lib = load()
    dev = _need_cache(cache)
    _fit(q, "q", cache._q_shape, cache.dtype, dev)
    _need_bytes(workspace, dev)
    n_prefix, pt = 0, None
    if prefix_table is not None:
        _need_table(prefix_table, dev)
        n_prefix, pt = prefix_table.numel(), prefix_table.data_ptr()
    out = _new(cache._q_shape, cache.dtype, cache.device, stream)
    st = lib.dilution_attn_debug_paged_decode_stall(q.data_ptr(), cache._ref, pt, n_prefix, int(max_len), out.data_ptr(),
                                                    float(tau), float(eps), workspace.data_ptr(), workspace.numel(),
                                                    _stream_id(stream, dev), int(stall_kernel), int(stall_block),
                                                    int(wait_limit_ns))
    return int(st), out


# ----------------------------------------------------------------------------- misc
def dilution_attn_get_error(workspace, stream=None) -> int:
    return int(load().dilution_attn_get_error(_ptr(workspace), _stream_handle(stream)))


def dilution_attn_status_string(status: int) -> str:
    return status_string(status)


def dilution_attn_version() -> int:
    return int(load().dilution_attn_version())


def dilution_attn_debug_last_timeout(workspace):
    """(status, mbarrier shared-memory offset, block, thread) of the workspace's status block."""
    import numpy as np
    buf = np.zeros(4, dtype=np.int32)
    _check(load().dilution_attn_debug_last_timeout(_ptr(workspace), buf.ctypes.data_as(ctypes.c_void_p)),
           "dilution_attn_debug_last_timeout")
    return tuple(int(x) for x in buf)


def dilution_attn_debug_tile_schedule(BH: int, T: int, kernel: int):
    """[n_ctas, 4] int32 array: (head, first query tile, query tiles, first key)."""
    import numpy as np
    lib = load()
    n = lib.dilution_attn_debug_tile_schedule(BH, T, kernel, None, 0)
    n = -n if n < 0 else n
    buf = np.zeros((max(n, 1), 4), dtype=np.int32)
    got = lib.dilution_attn_debug_tile_schedule(BH, T, kernel, buf.ctypes.data_as(ctypes.c_void_p), buf.size)
    if got < 0:
        raise RuntimeError("tile schedule export failed")
    return buf[:got]


def dilution_attn_debug_tile_mask(T: int, qt: int, kt: int):
    import numpy as np
    buf = np.zeros((128, 128), dtype=np.uint8)
    _check(load().dilution_attn_debug_tile_mask(T, qt, kt, buf.ctypes.data_as(ctypes.c_void_p)),
           "dilution_attn_debug_tile_mask")
    return buf
