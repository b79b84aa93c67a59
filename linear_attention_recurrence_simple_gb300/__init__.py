"""GB300 (sm_103a) Simple GLA mixer: a thin binding over the C ABI of ``libgla.so``.

The functions keep the C names (``include/gla.h``) and only marshal arguments: they check
torch tensors, allocate outputs with torch, and pass raw device pointers and the current CUDA
stream to the library.  Every step of the computation runs in the library's CUDA kernels; there
is no other code path, and a missing library raises instead of falling back.

Layouts (see ``include/gla.h``): q, k ``[B, T, H, 96]``; v ``[B, T, H, 192]``; packed inputs
``[T_total, H, d]`` (or ``[1, T_total, H, d]``) with ``cu_seqlens``; states ``[B, H, 96, 192]`` fp32.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

__all__ = [
    "GlaError", "load_library", "library_path", "gla_workspace_bytes", "gla_bwd_workspace_bytes",
    "gla_chunk_fwd",
    "gla_chunk_bwd", "gla_decode_step", "gla_chunk_fwd_noalloc", "gla_head_norm_gate", "gla_chunk_fwd_split",
    "gla_split_choose_seg_chunks", "gla_get_device_error",
    "gla_set_wait_limit_ns", "gla_debug_bounds", "gla_debug_give_up", "debug_bounds_library", "gla_chunk_fwd_host",
    "gla_chunk_fwd_host_workspace_bytes", "GlaTail", "gla_tail_alloc", "gla_tail_append", "gla_tail_read",
    "gla_tail_fold", "gla_prefix_decode_step", "gla_prefix_fwd", "gla_prefix_bwd", "gla_prefix_bwd_workspace_bytes",
    "gla_status_string", "DK", "DV", "CHUNK", "EXPORTS",
]

DK, DV, CHUNK = 96, 192, 128
GLA_BF16, GLA_F32 = 0, 1
EXPORTS = ("gla_workspace_bytes", "gla_bwd_workspace_bytes", "gla_chunk_fwd", "gla_chunk_bwd",
           "gla_decode_step", "gla_chunk_fwd_aug", "gla_decode_step_aug", "gla_head_norm_gate",
           "gla_decode_step_bf16_state", "gla_split_workspace_bytes", "gla_chunk_fwd_split",
           "gla_decode_step_norm_gate", "gla_decode_step_mxfp8_state", "gla_state_to_mxfp8",
           "gla_state_from_mxfp8",
           "gla_split_choose_seg_chunks", "gla_chunk_fwd_noalloc", "gla_get_device_error", "gla_set_wait_limit_ns",
           "gla_debug_bounds", "gla_chunk_fwd_host", "gla_chunk_fwd_host_workspace_bytes", "gla_status_string",
           "gla_prefix_decode_step", "gla_tail_append", "gla_tail_read", "gla_tail_fold", "gla_prefix_fwd",
           "gla_prefix_bwd", "gla_prefix_bwd_workspace_bytes", "gla_debug_give_up")
NOALLOC_MAX_SEQS = 16384

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libgla.so")
_LIB_DEBUG_PATH = os.path.join(_PKG, "libgla_debug.so")  # the debug-bounds build
_lock = threading.Lock()
_libs = {}          # False: release build, True: debug-bounds build
_use_debug = False  # which one the calls go to (see debug_bounds_library)


class GlaError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {gla_status_string(status)} ({status})" if where else
                         f"{gla_status_string(status)} ({status})")


def library_path(debug: bool = False) -> str:
    return _LIB_DEBUG_PATH if debug else _LIB_PATH


def load_library(build: bool = True, debug: bool | None = None):
    """Loads libgla.so, or with ``debug`` (default: inside :func:`debug_bounds_library`) its
    debug-bounds build libgla_debug.so, building it first if missing and ``build``; raises if it
    cannot."""
    if debug is None:
        debug = _use_debug
    with _lock:
        if debug in _libs:
            return _libs[debug]
        path = library_path(debug)
        if build:
            from . import _build
            _build.build(debug=debug)
        if not os.path.exists(path):
            raise RuntimeError(f"{os.path.basename(path)} is missing ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        P, I, F, Z, U = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                         ctypes.c_ulonglong)
        lib.gla_workspace_bytes.argtypes = [I, I]
        lib.gla_workspace_bytes.restype = Z
        lib.gla_bwd_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.gla_bwd_workspace_bytes.restype = Z
        lib.gla_chunk_fwd.argtypes = [P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, P, Z, P]
        lib.gla_chunk_fwd.restype = I
        lib.gla_chunk_bwd.argtypes = [P, P, P, P, P, F, P, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]
        lib.gla_chunk_bwd.restype = I
        lib.gla_chunk_fwd_noalloc.argtypes = [P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, P]
        lib.gla_chunk_fwd_noalloc.restype = I
        lib.gla_decode_step.argtypes = [P, P, P, P, F, P, P, I, P, I, I, I, I, I, P]
        lib.gla_decode_step.restype = I
        lib.gla_chunk_fwd_aug.argtypes = [P, P, P, P, P, F, P, P, P, P, I, I, I, I, I, I, P, Z, P]
        lib.gla_chunk_fwd_aug.restype = I
        lib.gla_decode_step_aug.argtypes = [P, P, P, P, F, P, P, P, I, P, I, I, I, I, I, P]
        lib.gla_decode_step_aug.restype = I
        lib.gla_head_norm_gate.argtypes = [P, P, P, P, I, F, P, ctypes.c_longlong, I, I, I, P]
        lib.gla_decode_step_bf16_state.argtypes = [P, P, P, P, F, P, P, P, I, P, I, I, I, I, I, P]
        lib.gla_decode_step_bf16_state.restype = I
        lib.gla_decode_step_norm_gate.argtypes = [P, P, P, P, F, P, P, P, I, P, P, P, I, F, P, I, I, I, I, I, P]
        lib.gla_decode_step_norm_gate.restype = I
        lib.gla_decode_step_mxfp8_state.argtypes = [P, P, P, P, F, P, P, P, P, I, P, I, I, I, I, I, P]
        lib.gla_decode_step_mxfp8_state.restype = I
        lib.gla_state_to_mxfp8.argtypes = [P, P, P, ctypes.c_longlong, P]
        lib.gla_state_to_mxfp8.restype = I
        lib.gla_state_from_mxfp8.argtypes = [P, P, P, ctypes.c_longlong, P]
        lib.gla_state_from_mxfp8.restype = I
        lib.gla_split_workspace_bytes.argtypes = [P, I, I, I]
        lib.gla_split_workspace_bytes.restype = Z
        lib.gla_chunk_fwd_split.argtypes = [P, P, P, P, P, F, P, P, P, P, I, I, I, I, I, I, I, P, Z, P]
        lib.gla_chunk_fwd_split.restype = I
        lib.gla_split_choose_seg_chunks.argtypes = [P, I, I]
        lib.gla_split_choose_seg_chunks.restype = I
        lib.gla_head_norm_gate.restype = I
        lib.gla_get_device_error.argtypes = [P]
        lib.gla_get_device_error.restype = I
        lib.gla_set_wait_limit_ns.argtypes = [U]
        lib.gla_set_wait_limit_ns.restype = I
        lib.gla_status_string.argtypes = [I]
        lib.gla_status_string.restype = ctypes.c_char_p
        lib.gla_debug_bounds.argtypes = []
        lib.gla_debug_bounds.restype = I
        lib.gla_debug_give_up.argtypes = [I, I]
        lib.gla_debug_give_up.restype = I
        lib.gla_chunk_fwd_host_workspace_bytes.argtypes = [I, I, I, I]
        lib.gla_chunk_fwd_host_workspace_bytes.restype = Z
        lib.gla_chunk_fwd_host.argtypes = [P, P, P, P, P, F, P, P, I, I, I, I, I, I, I, P, Z, P]
        lib.gla_chunk_fwd_host.restype = I
        lib.gla_prefix_decode_step.argtypes = [P, P, P, P, F, P, I, P, P, P, P, P, I, I, I, I, I, P]
        lib.gla_prefix_decode_step.restype = I
        lib.gla_tail_append.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P]
        lib.gla_tail_append.restype = I
        lib.gla_tail_read.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P]
        lib.gla_tail_read.restype = I
        lib.gla_tail_fold.argtypes = [P, P, I, P, P, P, P, P, I, P, I, I, I, I, I, P]
        lib.gla_tail_fold.restype = I
        lib.gla_prefix_fwd.argtypes = [P, P, P, P, P, I, P, F, P, P, P, I, I, I, I, I, I, P, Z, P]
        lib.gla_prefix_fwd.restype = I
        lib.gla_prefix_bwd_workspace_bytes.argtypes = [I, I, I, I]
        lib.gla_prefix_bwd_workspace_bytes.restype = Z
        lib.gla_prefix_bwd.argtypes = [P, P, P, P, P, I, P, F, P, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]
        lib.gla_prefix_bwd.restype = I
        _libs[debug] = lib
        return lib


@contextlib.contextmanager
def debug_bounds_library():
    """Within the block every call goes to the debug-bounds build (libgla_debug.so: device index
    checks that record GLA_ERR_BOUNDS and skip the access).  Not for concurrent use from several
    threads.  Each build keeps its own device error word."""
    global _use_debug
    lib = load_library(debug=True)
    prev, _use_debug = _use_debug, True
    try:
        yield lib
    finally:
        _use_debug = prev


def gla_debug_bounds() -> int:
    """1 when calls go to the debug-bounds build, 0 for the release build."""
    return int(load_library().gla_debug_bounds())


def gla_debug_give_up(role: int, chunk: int = 0) -> None:
    """Makes one warp of the tails' decode and fold kernels give up its wait for ``chunk`` (debug-bounds build
    only, for tests of the bounded waits; ``role`` -1: no more)."""
    _check(load_library().gla_debug_give_up(int(role), int(chunk)), "gla_debug_give_up")


def gla_status_string(status: int) -> str:
    return load_library().gla_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise GlaError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GLA_BF16
    if t.dtype == torch.float32:
        return GLA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None, device=None, numel=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _layout(q, k, v, cu_seqlens):
    """Returns (n_seq, T, H, packed_shape_prefix) for fixed-length or packed inputs."""
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("without cu_seqlens, q must be [B, T, H, 96]")
        B, T, H, dk = q.shape
        n_seq = B
    else:
        if q.dim() == 4:
            if q.shape[0] != 1:
                raise ValueError("packed inputs must be [T_total, H, d] or [1, T_total, H, d]")
            T, H, dk = q.shape[1:]
        elif q.dim() == 3:
            T, H, dk = q.shape
        else:
            raise ValueError("packed q must be [T_total, H, 96]")
        n_seq = cu_seqlens.numel() - 1
    if dk != DK or k.shape != q.shape or v.shape[:-1] != q.shape[:-1] or v.shape[-1] != DV:
        raise ValueError("expected q, k [..., H, 96] and v [..., H, 192] with matching leading dims")
    return n_seq, T, H


def gla_workspace_bytes(n_seq: int, H: int) -> int:
    return int(load_library().gla_workspace_bytes(int(n_seq), int(H)))


def gla_bwd_workspace_bytes(n_seq: int, T: int, H: int, packed: bool, dtype_code: int) -> int:
    return int(load_library().gla_bwd_workspace_bytes(int(n_seq), int(T), int(H), int(bool(packed)),
                                                      int(dtype_code)))


def _workspace(cu_seqlens, n_seq, H, device, workspace):
    if cu_seqlens is None:
        return None, 0
    need = gla_workspace_bytes(n_seq, H)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def gla_chunk_fwd(q, k, v, log_lambda, scale=None, h0=None, cu_seqlens=None,
                  output_final_state: bool = True, o=None, hT=None, workspace=None, aug=None):
    """Chunked forward.  Returns ``(o, hT)`` (``hT`` is None if not requested).

    ``aug`` (aug_balance, fp32 ``[H, 96]``) adds the self-augmentation copy
    ``sigmoid(q_t . (aug[h] * k_t)) v_t`` to each output row (``gla_chunk_fwd_aug``)."""
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n_seq, T, H = _layout(q, k, v, cu_seqlens)
    if log_lambda.numel() != H:
        raise ValueError("log_lambda must have H entries")
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev)
        if h0.shape != (n_seq, H, DK, DV):
            raise ValueError("h0 must be [n_seq, H, 96, 192]")
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "o", v.dtype, dev, v.numel())
    if output_final_state and hT is None:
        hT = torch.empty((n_seq, H, DK, DV), dtype=torch.float32, device=dev)
    if hT is not None:
        _need(hT, "hT", torch.float32, dev, n_seq * H * DK * DV)
    ws, ws_bytes = _workspace(cu_seqlens, n_seq, H, dev, workspace)
    s = float(DK ** -0.5) if scale is None else float(scale)
    if aug is not None:
        _need(aug, "aug", torch.float32, dev)
        if aug.shape != (H, DK):
            raise ValueError("aug must be [H, 96]")
    with torch.cuda.device(dev):
        if aug is None:
            rc = lib.gla_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), s, _ptr(o),
                                   _ptr(hT), _ptr(cu_seqlens), n_seq, T, H, DK, DV, dt, _ptr(ws),
                                   ws_bytes, _stream(dev))
        else:
            rc = lib.gla_chunk_fwd_aug(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), s,
                                       _ptr(aug), _ptr(o), _ptr(hT), _ptr(cu_seqlens), n_seq, T, H, DK,
                                       DV, dt, _ptr(ws), ws_bytes, _stream(dev))
    _check(rc, "gla_chunk_fwd" if aug is None else "gla_chunk_fwd_aug")
    return o, hT


def gla_chunk_fwd_noalloc(q, k, v, log_lambda, scale=None, h0=None, cu_seqlens=None, o=None, hT=None):
    """The forward with no device allocation inside the library and no workspace argument.

    For callers that cannot allocate device memory per call (for instance a serving engine that
    hands all device memory to its own pool at start-up): pass preallocated ``o`` and ``hT`` and
    nothing is allocated here either.  The packed schedule lives in a 64 KB library-owned device
    array, so ``cu_seqlens`` may describe at most ``NOALLOC_MAX_SEQS`` sequences, and calls that
    overlap on the GPU (unordered streams) race on it.  Returns ``(o, hT)``."""
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n_seq, T, H = _layout(q, k, v, cu_seqlens)
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev, n_seq * H * DK * DV)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "o", v.dtype, dev, v.numel())
    if hT is not None:
        _need(hT, "hT", torch.float32, dev, n_seq * H * DK * DV)
    s = float(DK ** -0.5) if scale is None else float(scale)
    with torch.cuda.device(dev):
        rc = lib.gla_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), s,
                                       _ptr(o), _ptr(hT), _ptr(cu_seqlens), n_seq, T, H, DK, DV, dt,
                                       _stream(dev))
    _check(rc, "gla_chunk_fwd_noalloc")
    return o, hT


def gla_chunk_fwd_host_workspace_bytes(n_seq: int, T: int, H: int, dtype_code: int) -> int:
    return int(load_library().gla_chunk_fwd_host_workspace_bytes(n_seq, T, H, dtype_code))


def gla_chunk_fwd_host(q, k, v, log_lambda, scale=None, h0=None, o=None, hT=None, pieces=16, workspace=None,
                       output_final_state: bool = True):
    """The forward on HOST tensors (``gla_chunk_fwd_host``): q, k ``[B, T, H, 96]``, v
    ``[B, T, H, 192]`` and h0 (fp32, optional) on the CPU (page-locked for overlapped copies);
    log_lambda on the device.  Returns host ``(o, hT)``, written once the current stream has run
    (synchronise it before reading).  The library copies ``pieces`` pieces in, runs them and
    copies them out, pipelined; ``workspace`` is a device buffer of at least
    :func:`gla_chunk_fwd_host_workspace_bytes` bytes (allocated when not given)."""
    lib = load_library()
    dev = log_lambda.device
    if dev.type != "cuda":
        raise ValueError("log_lambda must be on the device")
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.device.type != "cpu" or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor of q's dtype")
    if q.dim() != 4 or q.shape[3] != DK or k.shape != q.shape or v.shape != (*q.shape[:3], DV):
        raise ValueError("expected q, k [B, T, H, 96] and v [B, T, H, 192]")
    B, T, H = q.shape[:3]
    _need(log_lambda, "log_lambda", torch.float32, dev, H)
    if h0 is not None and (h0.device.type != "cpu" or h0.dtype != torch.float32 or not h0.is_contiguous()
                           or h0.shape != (B, H, DK, DV)):
        raise ValueError("h0 must be a contiguous CPU fp32 tensor [B, H, 96, 192]")
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype).pin_memory()
    if hT is None and output_final_state:
        hT = torch.empty((B, H, DK, DV), dtype=torch.float32).pin_memory()
    for name, t, shape, dtype in (("o", o, v.shape, v.dtype), ("hT", hT, (B, H, DK, DV), torch.float32)):
        if t is not None and (t.device.type != "cpu" or t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CPU tensor {tuple(shape)} of {dtype}")
    need = gla_chunk_fwd_host_workspace_bytes(B, T, H, dt)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if workspace.numel() < need:
        raise ValueError(f"workspace has {workspace.numel()} bytes, needs {need}")
    s = float(DK ** -0.5) if scale is None else float(scale)
    with torch.cuda.device(dev):
        rc = lib.gla_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), s, _ptr(o), _ptr(hT),
                                    B, T, H, DK, DV, dt, int(pieces), _ptr(workspace), workspace.numel(),
                                    _stream(dev))
    _check(rc, "gla_chunk_fwd_host")
    return o, hT


def gla_chunk_bwd(q, k, v, log_lambda, dO, scale=None, h0=None, dhT=None, cu_seqlens=None,
                  need_dh0: bool = True, workspace=None, dq=None, dk=None, dv=None, dh0=None):
    """Chunked backward.  Returns ``(dq, dk, dv, dh0)`` (``dh0`` None if not requested).
    ``dq``, ``dk``, ``dv``, ``dh0``: optional preallocated outputs (contiguous, sized like q, k, v
    and [n_seq, H, 96, 192] fp32)."""
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("dO", dO)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n_seq, T, H = _layout(q, k, v, cu_seqlens)
    if dO.shape != v.shape:
        raise ValueError("dO must have the shape of v")
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _need(t, name, torch.float32, dev)
            if t.shape != (n_seq, H, DK, DV):
                raise ValueError(f"{name} must be [n_seq, H, 96, 192]")
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev) if dq is None else dq
    dk = torch.empty(k.shape, dtype=k.dtype, device=dev) if dk is None else dk
    dv = torch.empty(v.shape, dtype=v.dtype, device=dev) if dv is None else dv
    if dh0 is None and need_dh0:
        dh0 = torch.empty((n_seq, H, DK, DV), dtype=torch.float32, device=dev)
    for name, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        _need(t, name, q.dtype, dev, ref.numel())
    if dh0 is not None:
        _need(dh0, "dh0", torch.float32, dev, n_seq * H * DK * DV)
    need = gla_bwd_workspace_bytes(n_seq, T, H, cu_seqlens is not None, dt)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    s = float(DK ** -0.5) if scale is None else float(scale)
    with torch.cuda.device(dev):
        rc = lib.gla_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), s, _ptr(dO),
                               _ptr(dhT), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dh0), _ptr(cu_seqlens),
                               n_seq, T, H, DK, DV, dt, _ptr(workspace), ws_bytes, _stream(dev))
    _check(rc, "gla_chunk_bwd")
    return dq, dk, dv, dh0


def gla_decode_step(q, k, v, log_lambda, state, scale=None, slot=None, o=None, aug=None):
    """One decode step on the state pool ``state [P, H, 96, 192]`` (updated in place).

    q, k ``[N, H, 96]``; v ``[N, H, 192]``; ``slot`` ``[N]`` int32 pool rows or None (row n).
    ``aug`` (fp32 ``[H, 96]``) adds the self-augmentation copy of v (``gla_decode_step_aug``).
    A bf16 ``state`` pool runs ``gla_decode_step_bf16_state`` (the state is rounded to bf16 when
    it is written back).  Returns ``o [N, H, 192]``."""
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    if state.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("state must be float32 or bfloat16")
    _need(state, "state", state.dtype, dev)
    if q.dim() != 3 or q.shape[2] != DK or k.shape != q.shape or v.shape != (*q.shape[:2], DV):
        raise ValueError("expected q, k [N, H, 96] and v [N, H, 192]")
    N, H = q.shape[:2]
    if state.dim() != 4 or state.shape[1:] != (H, DK, DV):
        raise ValueError("state must be [P, H, 96, 192]")
    if slot is not None:
        _need(slot, "slot", torch.int32, dev)
        if slot.shape != (N,):
            raise ValueError("slot must be [N]")
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "o", v.dtype, dev, v.numel())
    s = float(DK ** -0.5) if scale is None else float(scale)
    if aug is not None:
        _need(aug, "aug", torch.float32, dev)
        if aug.shape != (H, DK):
            raise ValueError("aug must be [H, 96]")
    with torch.cuda.device(dev):
        if state.dtype == torch.bfloat16:
            rc = lib.gla_decode_step_bf16_state(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), s, _ptr(aug),
                                                _ptr(state), _ptr(slot), state.shape[0], _ptr(o), N, H, DK,
                                                DV, dt, _stream(dev))
            _check(rc, "gla_decode_step_bf16_state")
            return o
        if aug is None:
            rc = lib.gla_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), s, _ptr(state),
                                     _ptr(slot), state.shape[0], _ptr(o), N, H, DK, DV, dt, _stream(dev))
        else:
            rc = lib.gla_decode_step_aug(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), s, _ptr(aug),
                                         _ptr(state), _ptr(slot), state.shape[0], _ptr(o), N, H, DK, DV,
                                         dt, _stream(dev))
    _check(rc, "gla_decode_step" if aug is None else "gla_decode_step_aug")
    return o


def gla_decode_step_norm_gate(q, k, v, log_lambda, state, g, weight, tier, scale=None, slot=None,
                              eps=1e-6, y=None, aug=None):
    """One decode step (fp32 state pool, updated in place) whose readout goes straight through the
    per-tier Head RMSNorm and the SiLU(g) gate: returns ``y [N, H, 192]``,
    ``y = o / sqrt(mean(o^2) + eps) * weight[tier[h]] * SiLU(g)`` with o the step's readout (plus
    the self-augmentation copy when ``aug`` is given).  ``g`` ``[N, H, 192]`` (dtype of q),
    ``weight`` fp32 ``[n_tiers, 192]``, ``tier`` int32 ``[H]``."""
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    _need(state, "state", torch.float32, dev)
    if q.dim() != 3 or q.shape[2] != DK or k.shape != q.shape or v.shape != (*q.shape[:2], DV):
        raise ValueError("expected q, k [N, H, 96] and v [N, H, 192]")
    N, H = q.shape[:2]
    if state.dim() != 4 or state.shape[1:] != (H, DK, DV):
        raise ValueError("state must be [P, H, 96, 192]")
    _need(g, "g", q.dtype, dev, v.numel())
    _need(weight, "weight", torch.float32, dev)
    _need(tier, "tier", torch.int32, dev, H)
    if weight.dim() != 2 or weight.shape[1] != DV:
        raise ValueError("weight must be [n_tiers, 192]")
    if slot is not None:
        _need(slot, "slot", torch.int32, dev, N)
    if aug is not None:
        _need(aug, "aug", torch.float32, dev, H * DK)
    if y is None:
        y = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(y, "y", v.dtype, dev, v.numel())
    s = float(DK ** -0.5) if scale is None else float(scale)
    with torch.cuda.device(dev):
        rc = lib.gla_decode_step_norm_gate(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), s, _ptr(aug),
                                           _ptr(state), _ptr(slot), state.shape[0], _ptr(g), _ptr(weight),
                                           _ptr(tier), weight.shape[0], float(eps), _ptr(y), N, H, DK, DV,
                                           dt, _stream(dev))
    _check(rc, "gla_decode_step_norm_gate")
    return y


def gla_state_to_mxfp8(x, codes=None, scales=None):
    """fp32 state rows ``x [..., 192]`` to MXFP8: returns ``(codes uint8 [..., 192],
    scales uint8 [..., 6])`` (the format of :func:`gla_decode_step_mxfp8_state`)."""
    lib = load_library()
    dev = x.device
    _need(x, "x", torch.float32, dev)
    if x.shape[-1] != DV:
        raise ValueError("x must be [..., 192]")
    rows = x.numel() // DV
    codes = torch.empty(x.shape, dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty(x.shape[:-1] + (DV // 32,), dtype=torch.uint8, device=dev) if scales is None else scales
    _need(codes, "codes", torch.uint8, dev, x.numel())
    _need(scales, "scales", torch.uint8, dev, rows * (DV // 32))
    with torch.cuda.device(dev):
        rc = lib.gla_state_to_mxfp8(_ptr(x), _ptr(codes), _ptr(scales), rows, _stream(dev))
    _check(rc, "gla_state_to_mxfp8")
    return codes, scales


def gla_state_from_mxfp8(codes, scales, x=None):
    """MXFP8 state rows back to fp32 (exact); returns ``x [..., 192]``."""
    lib = load_library()
    dev = codes.device
    _need(codes, "codes", torch.uint8, dev)
    if codes.shape[-1] != DV:
        raise ValueError("codes must be [..., 192]")
    rows = codes.numel() // DV
    _need(scales, "scales", torch.uint8, dev, rows * (DV // 32))
    x = torch.empty(codes.shape, dtype=torch.float32, device=dev) if x is None else x
    _need(x, "x", torch.float32, dev, codes.numel())
    with torch.cuda.device(dev):
        rc = lib.gla_state_from_mxfp8(_ptr(codes), _ptr(scales), _ptr(x), rows, _stream(dev))
    _check(rc, "gla_state_from_mxfp8")
    return x


def gla_decode_step_mxfp8_state(q, k, v, log_lambda, codes, scales, scale=None, slot=None, o=None, aug=None):
    """One decode step on an MXFP8 state pool (``codes`` uint8 ``[P, H, 96, 192]``, ``scales``
    uint8 ``[P, H, 96, 6]``, both updated in place).  Returns ``o [N, H, 192]``."""
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    if q.dim() != 3 or q.shape[2] != DK or k.shape != q.shape or v.shape != (*q.shape[:2], DV):
        raise ValueError("expected q, k [N, H, 96] and v [N, H, 192]")
    N, H = q.shape[:2]
    _need(codes, "codes", torch.uint8, dev)
    if codes.dim() != 4 or codes.shape[1:] != (H, DK, DV):
        raise ValueError("codes must be [P, H, 96, 192]")
    _need(scales, "scales", torch.uint8, dev, codes.shape[0] * H * DK * (DV // 32))
    if slot is not None:
        _need(slot, "slot", torch.int32, dev, N)
    if aug is not None:
        _need(aug, "aug", torch.float32, dev, H * DK)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "o", v.dtype, dev, v.numel())
    s = float(DK ** -0.5) if scale is None else float(scale)
    with torch.cuda.device(dev):
        rc = lib.gla_decode_step_mxfp8_state(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), s, _ptr(aug),
                                             _ptr(codes), _ptr(scales), _ptr(slot), codes.shape[0], _ptr(o), N,
                                             H, DK, DV, dt, _stream(dev))
    _check(rc, "gla_decode_step_mxfp8_state")
    return o


def _host_offsets(lengths):
    import numpy as np
    cu = np.zeros(len(lengths) + 1, np.int32)
    cu[1:] = np.cumsum(np.asarray(lengths, np.int64))
    return cu


def gla_split_choose_seg_chunks(lengths, H):
    """Chunks per segment that ``gla_chunk_fwd_split(..., seg_chunks=0)`` uses for these sequence
    lengths and H heads; 0 when every sequence stays one segment (the plain forward)."""
    cu = _host_offsets(lengths)
    rc = load_library().gla_split_choose_seg_chunks(cu.ctypes.data_as(ctypes.c_void_p), len(lengths), int(H))
    if rc < 0:
        _check(rc, "gla_split_choose_seg_chunks")
    return rc


def gla_chunk_fwd_split(q, k, v, log_lambda, lengths, seg_chunks=0, scale=None, h0=None, aug=None,
                        output_final_state: bool = True, o=None, hT=None, workspace=None):
    """Sequence-split forward (``gla_chunk_fwd_split``) for long sequences.

    ``lengths``: the sequences' token counts (host ints); q, k ``[T_total, H, 96]``, v
    ``[T_total, H, 192]`` packed in that order (a fixed-length batch may pass ``[B, T, H, d]``
    tensors with ``lengths = [T] * B``).  Segments hold at most ``seg_chunks`` chunks of 128
    tokens; 0 lets the library choose (:func:`gla_split_choose_seg_chunks`), which may keep every
    sequence whole.  Returns ``(o, hT)`` like :func:`gla_chunk_fwd`."""
    import numpy as np
    lib = load_library()
    dev = q.device
    dt = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(log_lambda, "log_lambda", torch.float32, dev)
    cu = np.zeros(len(lengths) + 1, np.int32)
    cu[1:] = np.cumsum(np.asarray(lengths, np.int64))
    n_seq, H = len(lengths), q.shape[-2]
    T = int(cu[-1])
    if q.numel() != T * H * DK or k.shape != q.shape or v.numel() != T * H * DV or q.shape[-1] != DK:
        raise ValueError("q, k, v must hold sum(lengths) tokens of H heads")
    if log_lambda.numel() != H:
        raise ValueError("log_lambda must have H entries")
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev, n_seq * H * DK * DV)
        if h0.shape != (n_seq, H, DK, DV):
            raise ValueError("h0 must be [n_seq, H, 96, 192]")
    if aug is not None:
        _need(aug, "aug", torch.float32, dev)
        if aug.shape != (H, DK):
            raise ValueError("aug must be [H, 96]")
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "o", v.dtype, dev, v.numel())
    if output_final_state and hT is None:
        hT = torch.empty((n_seq, H, DK, DV), dtype=torch.float32, device=dev)
    if hT is not None:
        _need(hT, "hT", torch.float32, dev, n_seq * H * DK * DV)
    cu_p = cu.ctypes.data_as(ctypes.c_void_p)
    need = lib.gla_split_workspace_bytes(cu_p, n_seq, H, int(seg_chunks))
    if need == 0 and n_seq > 0:
        raise ValueError("bad lengths or seg_chunks")
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    s = float(DK ** -0.5) if scale is None else float(scale)
    with torch.cuda.device(dev):
        rc = lib.gla_chunk_fwd_split(_ptr(q), _ptr(k), _ptr(v), _ptr(log_lambda), _ptr(h0), s, _ptr(aug),
                                     _ptr(o), _ptr(hT), cu_p, n_seq, T, H, DK, DV, dt, int(seg_chunks),
                                     _ptr(workspace), workspace.numel(), _stream(dev))
    _check(rc, "gla_chunk_fwd_split")
    return o, hT


def gla_head_norm_gate(o, g, weight, tier, eps=1e-6, y=None):
    """Per-tier Head RMSNorm of each head's output row and the SiLU(g) gate.

    o, g ``[..., H, 192]`` (same dtype, bf16 or fp32); weight fp32 ``[n_tiers, 192]``; tier int32
    ``[H]``.  Returns ``y`` like ``o``."""
    lib = load_library()
    dev = o.device
    dt = _dtype_code(o)
    _need(o, "o", o.dtype, dev)
    _need(g, "g", o.dtype, dev)
    _need(weight, "weight", torch.float32, dev)
    _need(tier, "tier", torch.int32, dev)
    if o.dim() < 2 or o.shape[-1] != DV or g.shape != o.shape:
        raise ValueError("expected o, g [..., H, 192] of one shape")
    H = o.shape[-2]
    rows = o.numel() // (H * DV)
    if weight.dim() != 2 or weight.shape[1] != DV or tier.shape != (H,):
        raise ValueError("weight must be [n_tiers, 192] and tier [H]")
    if y is None:
        y = torch.empty_like(o)
    _need(y, "y", o.dtype, dev)
    with torch.cuda.device(dev):
        rc = lib.gla_head_norm_gate(_ptr(o), _ptr(g), _ptr(weight), _ptr(tier), weight.shape[0], float(eps),
                                    _ptr(y), rows, H, DV, dt, _stream(dev))
    _check(rc, "gla_head_norm_gate")
    return y


class GlaTail(NamedTuple):
    """Tail caches of sequences that continue a shared prefix: keys ``[R, H, cap, 96]`` and values
    ``[R, H, cap, 192]`` in the type of the calls' q, k, v, or as MXFP8 (uint8 E4M3 codes of the same
    shapes, with uint8 E8M0 scales ``[R, H, cap, 3]`` and ``[R, H, cap, 6]``)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scales: Optional[torch.Tensor] = None
    v_scales: Optional[torch.Tensor] = None


class _CTail(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("rows", ctypes.c_int), ("cap", ctypes.c_int),
                ("format", ctypes.c_int)]


def gla_tail_alloc(rows: int, H: int, cap: int, dtype=torch.bfloat16, device="cuda") -> GlaTail:
    """Zeroed tails of ``rows`` rows with room for ``cap`` tokens (rounded up to a multiple of 16);
    ``dtype`` bfloat16 or float32, or ``torch.float8_e4m3fn`` for MXFP8."""
    cap = max(16, -(-int(cap) // 16) * 16)
    if dtype == torch.float8_e4m3fn:
        z = lambda d: torch.zeros((rows, H, cap, d), dtype=torch.uint8, device=device)  # noqa: E731
        return GlaTail(z(DK), z(DV), z(DK // 32), z(DV // 32))
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"tails are bfloat16, float32 or float8_e4m3fn (MXFP8), got {dtype}")
    z = lambda d: torch.zeros((rows, H, cap, d), dtype=dtype, device=device)  # noqa: E731
    return GlaTail(z(DK), z(DV))


# The calls below are made once per layer and token, where a microsecond on the host counts: a call tests
# its tensors in one expression and goes through them one by one (_need says what is wrong) only when
# that fails.
def _like(i, dtype, *tensors):
    """Whether the tensors are contiguous, of this type and on CUDA device i."""
    try:
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != i or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return True


def _good(t, name, dtype, dev, numel=None):
    if not _like(dev.index, dtype, t) or (numel is not None and t.numel() != numel):
        _need(t, name, dtype, dev, numel)


def _device_of(t, name):
    """The CUDA device of a call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _need(t, name)
    return t.device


# The current stream's handle without a Stream object around it, where torch has that call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(fn, where, dev, *args):
    """Calls the library with `dev` current, on its current stream."""
    i = dev.index
    if torch.cuda.current_device() == i:
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(i))
    if rc != 0:
        raise GlaError(rc, where)


def _addr(t):
    return None if t is None else t.data_ptr()


def _tail(tail, H, dtype, dev):
    """Checks the tails' tensors and returns the C struct."""
    k, v, ks, vs = tail
    mx = ks is not None or vs is not None
    if not (_like(dev.index, torch.uint8, k, v, ks, vs) if mx else _like(dev.index, dtype, k, v)):
        for name, t in (("k", k), ("v", v)) + ((("k_scales", ks), ("v_scales", vs)) if mx else ()):
            _need(t, "tail." + name, torch.uint8 if mx else dtype, dev)
    if k.dim() != 4:
        raise ValueError("the tail must be k [R, H, cap, 96] and v [R, H, cap, 192]")
    R, h, cap, d = k.shape
    if h != H or d != DK or v.shape != (R, H, cap, DV):
        raise ValueError("the tail must be k [R, H, cap, 96] and v [R, H, cap, 192]")
    if not mx:
        return _CTail(k.data_ptr(), v.data_ptr(), None, None, R, cap, 0)
    if ks.shape != (R, H, cap, DK // 32) or vs.shape != (R, H, cap, DV // 32):
        raise ValueError("tail scales must be [R, H, cap, 3] and [R, H, cap, 6]")
    return _CTail(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), R, cap, 1)


def _pool(pool, H, dev, name="pool"):
    _good(pool, name, torch.float32, dev)
    P = pool.shape[0] if pool.dim() == 4 else -1
    if pool.shape != (P, H, DK, DV):
        raise ValueError(f"{name} must be [P, H, 96, 192]")
    return P


def gla_prefix_decode_step(q, k, v, log_lambda, pool, prefix_row, tail, tail_len, tail_slot=None, scale=None, o=None):
    """One decode step of N sequences that continue shared states (``gla_prefix_decode_step``).

    q, k ``[N, H, 96]``; v ``[N, H, 192]``; ``pool`` fp32 ``[P, H, 96, 192]`` (read only);
    ``prefix_row`` ``[N]`` int32: the pool row each sequence continues (best sorted: neighbours with
    one row share its read); ``tail`` a :class:`GlaTail` with ``tail_len`` ``[N]`` int32 tokens in
    row ``tail_slot[n]`` (None: row n).  Returns ``o [N, H, 192]`` and writes k, v to place
    ``tail_len[n]``; the caller advances ``tail_len``."""
    lib = _libs.get(_use_debug) or load_library()
    dt, dtype = _dtype_code(q), q.dtype
    dev = _device_of(q, "q")
    i = dev.index
    if not _like(i, dtype, q, k, v):
        for name, t in (("q", q), ("k", k), ("v", v)):
            _need(t, name, dtype, dev)
    N, H, d = q.shape if q.dim() == 3 else (0, 0, 0)
    if d != DK or k.shape != q.shape or v.shape != (N, H, DV):
        raise ValueError("expected q, k [N, H, 96] and v [N, H, 192]")
    if not _like(i, torch.float32, log_lambda) or log_lambda.numel() != H:
        _need(log_lambda, "log_lambda", torch.float32, dev, H)
    rows = _pool(pool, H, dev)
    ct = _tail(tail, H, dtype, dev)
    slot = tail_len if tail_slot is None else tail_slot
    if (not _like(i, torch.int32, prefix_row, tail_len, slot) or prefix_row.numel() != N or tail_len.numel() != N
            or slot.numel() != N):
        for name, t in (("prefix_row", prefix_row), ("tail_len", tail_len), ("tail_slot", slot)):
            _need(t, name, torch.int32, dev, N)
    if o is None:
        o = torch.empty_like(v)
    else:
        _good(o, "o", dtype, dev, N * H * DV)
    _run(lib.gla_prefix_decode_step, "gla_prefix_decode_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
         log_lambda.data_ptr(), DK ** -0.5 if scale is None else float(scale), pool.data_ptr(), rows,
         prefix_row.data_ptr(), ctypes.byref(ct), _addr(tail_slot), tail_len.data_ptr(), o.data_ptr(), N, H, DK, DV, dt)
    return o


def _packed_offsets(cu_seqlens, pos, tail_slot, dev):
    _good(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n_seq = cu_seqlens.numel() - 1
    _good(pos, "pos", torch.int32, dev, n_seq)
    if tail_slot is not None:
        _good(tail_slot, "tail_slot", torch.int32, dev, n_seq)
    return n_seq


def gla_tail_append(k, v, tail, pos, cu_seqlens, tail_slot=None):
    """Writes packed tokens (k ``[T, H, 96]``, v ``[T, H, 192]``, offsets ``cu_seqlens``) to the
    tails: sequence n's to places ``pos[n]``, ``pos[n] + 1``, ... of row ``tail_slot[n]`` (None: row
    n), quantised where the tail is MXFP8."""
    lib = _libs.get(_use_debug) or load_library()
    dt = _dtype_code(k)
    dev = _device_of(k, "k")
    _good(k, "k", k.dtype, dev)
    _good(v, "v", k.dtype, dev)
    shape = tuple(k.shape)
    if len(shape) != 3 or shape[2] != DK or tuple(v.shape) != shape[:2] + (DV,):
        raise ValueError("expected packed k [T, H, 96] and v [T, H, 192]")
    T, H = shape[:2]
    ct = _tail(tail, H, k.dtype, dev)
    n_seq = _packed_offsets(cu_seqlens, pos, tail_slot, dev)
    _run(lib.gla_tail_append, "gla_tail_append", dev, k.data_ptr(), v.data_ptr(), ctypes.byref(ct), _addr(tail_slot),
         pos.data_ptr(), cu_seqlens.data_ptr(), n_seq, T, H, DK, DV, dt)


def gla_tail_read(tail, pos, cu_seqlens, T, tail_slot=None, dtype=None, k=None, v=None):
    """The tokens at places ``pos[n]``, ``pos[n] + 1``, ... of the tails as packed ``(k [T, H, 96],
    v [T, H, 192])`` with offsets ``cu_seqlens`` (``T`` their total), the reverse of
    :func:`gla_tail_append`.  ``dtype`` of the results: bfloat16 or float32 (default: the tail's
    own type, bfloat16 for MXFP8; a plain tail is read in its own type)."""
    lib = _libs.get(_use_debug) or load_library()
    dev = _device_of(tail[0], "tail.k")
    if dtype is None:
        dtype = k.dtype if k is not None else (torch.bfloat16 if tail[2] is not None else tail[0].dtype)
    if tail[0].dim() != 4:
        raise ValueError("the tail must be k [R, H, cap, 96] and v [R, H, cap, 192]")
    H, T = tail[0].shape[1], int(T)
    ct = _tail(tail, H, dtype, dev)
    if k is None:
        k = torch.empty((T, H, DK), dtype=dtype, device=dev)
    if v is None:
        v = torch.empty((T, H, DV), dtype=dtype, device=dev)
    dt = _dtype_code(k)
    _good(k, "k", dtype, dev, T * H * DK)
    _good(v, "v", dtype, dev, T * H * DV)
    n_seq = _packed_offsets(cu_seqlens, pos, tail_slot, dev)
    _run(lib.gla_tail_read, "gla_tail_read", dev, ctypes.byref(ct), _addr(tail_slot), pos.data_ptr(),
         cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr(), n_seq, T, H, DK, DV, dt)
    return k, v


def gla_tail_fold(log_lambda, pool, prefix_row, tail, tail_len, out=None, out_row=None, tail_slot=None):
    """Folds each sequence's tail into a state of its own (``gla_tail_fold``):
    ``out[out_row[n]] = lambda^L pool[prefix_row[n]] + sum_j lambda^(L-1-j) k_j v_j^T`` with
    L = ``tail_len[n]``.  ``out`` fp32 ``[P', H, 96, 192]`` (None: a new ``[N, H, 96, 192]``; may be
    ``pool`` itself, see the header), ``out_row`` None: row n.  Returns ``out``."""
    lib = _libs.get(_use_debug) or load_library()
    dev = _device_of(pool, "pool")
    _good(log_lambda, "log_lambda", torch.float32, dev)
    H = log_lambda.numel()
    rows = _pool(pool, H, dev)
    et = tail[0].dtype if tail[2] is None else torch.bfloat16
    if et not in (torch.bfloat16, torch.float32):
        raise TypeError("a tail without scales must be bfloat16 or float32")
    ct = _tail(tail, H, et, dev)
    _good(prefix_row, "prefix_row", torch.int32, dev)
    N = prefix_row.numel()
    _good(tail_len, "tail_len", torch.int32, dev, N)
    for name, t in (("tail_slot", tail_slot), ("out_row", out_row)):
        if t is not None:
            _good(t, name, torch.int32, dev, N)
    if out is None:
        if out_row is not None:
            raise ValueError("out_row needs out")
        out = torch.empty((N, H, DK, DV), dtype=torch.float32, device=dev)
    out_rows = _pool(out, H, dev, "out")
    _run(lib.gla_tail_fold, "gla_tail_fold", dev, log_lambda.data_ptr(), pool.data_ptr(), rows, prefix_row.data_ptr(),
         ctypes.byref(ct), _addr(tail_slot), tail_len.data_ptr(), out.data_ptr(), out_rows, _addr(out_row), N, H, DK, DV,
         GLA_F32 if et is torch.float32 else GLA_BF16)
    return out


def _prefix_call(q, k, v, log_lambda, pool, prefix_row, cu_seqlens):
    """Checks shared by the packed calls; returns (device, dtype code, n_seq, T, H, pool rows)."""
    dt, dtype = _dtype_code(q), q.dtype
    dev = _device_of(q, "q")
    _good(q, "q", dtype, dev)
    _good(k, "k", dtype, dev)
    _good(v, "v", dtype, dev)
    _good(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n_seq, T, H = _layout(q, k, v, cu_seqlens)
    _good(log_lambda, "log_lambda", torch.float32, dev, H)
    rows = _pool(pool, H, dev)
    _good(prefix_row, "prefix_row", torch.int32, dev, n_seq)
    return dev, dt, n_seq, T, H, rows


def gla_prefix_fwd(q, k, v, log_lambda, pool, prefix_row, cu_seqlens, scale=None, output_final_state: bool = True,
                   o=None, hT=None, workspace=None):
    """Chunked forward of packed sequences that continue shared states (``gla_prefix_fwd``): as
    :func:`gla_chunk_fwd` with ``cu_seqlens``, sequence n starting from ``pool[prefix_row[n]]``
    (``pool`` fp32 ``[P, H, 96, 192]``, ``prefix_row`` ``[n_seq]`` int32, rows may repeat).  Returns
    ``(o, hT)``."""
    lib = _libs.get(_use_debug) or load_library()
    dev, dt, n_seq, T, H, rows = _prefix_call(q, k, v, log_lambda, pool, prefix_row, cu_seqlens)
    if o is None:
        o = torch.empty_like(v)
    else:
        _good(o, "o", v.dtype, dev, T * H * DV)
    if hT is None:
        if output_final_state:
            hT = torch.empty((n_seq, H, DK, DV), dtype=torch.float32, device=dev)
    else:
        _good(hT, "hT", torch.float32, dev, n_seq * H * DK * DV)
    ws, ws_bytes = _workspace(cu_seqlens, n_seq, H, dev, workspace)
    _run(lib.gla_prefix_fwd, "gla_prefix_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_lambda.data_ptr(),
         pool.data_ptr(), rows, prefix_row.data_ptr(), DK ** -0.5 if scale is None else float(scale), o.data_ptr(),
         _addr(hT), cu_seqlens.data_ptr(), n_seq, T, H, DK, DV, dt, ws.data_ptr(), ws_bytes)
    return o, hT


def gla_prefix_bwd_workspace_bytes(n_seq: int, T: int, H: int, dtype_code: int) -> int:
    return int(load_library().gla_prefix_bwd_workspace_bytes(int(n_seq), int(T), int(H), int(dtype_code)))


def gla_prefix_bwd(q, k, v, log_lambda, dO, pool, prefix_row, cu_seqlens, scale=None, dhT=None,
                   need_dpool: bool = True, workspace=None, dq=None, dk=None, dv=None, dpool=None):
    """Backward of :func:`gla_prefix_fwd` (``gla_prefix_bwd``).  Returns ``(dq, dk, dv, dpool)``;
    ``dpool`` has the shape of ``pool``: row p is the sum of the initial-state gradients of the
    sequences that continue p, in their order, zeros where none does (None if not requested)."""
    lib = _libs.get(_use_debug) or load_library()
    dev, dt, n_seq, T, H, rows = _prefix_call(q, k, v, log_lambda, pool, prefix_row, cu_seqlens)
    _good(dO, "dO", q.dtype, dev)
    if dO.shape != v.shape:
        raise ValueError("dO must have the shape of v")
    if dhT is not None:
        _good(dhT, "dhT", torch.float32, dev)
        if tuple(dhT.shape) != (n_seq, H, DK, DV):
            raise ValueError("dhT must be [n_seq, H, 96, 192]")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dpool is None and need_dpool:
        dpool = torch.empty_like(pool)
    _good(dq, "dq", q.dtype, dev, q.numel())
    _good(dk, "dk", q.dtype, dev, k.numel())
    _good(dv, "dv", q.dtype, dev, v.numel())
    if dpool is not None:
        _good(dpool, "dpool", torch.float32, dev, pool.numel())
    if workspace is None:
        workspace = torch.empty(gla_prefix_bwd_workspace_bytes(n_seq, T, H, dt), dtype=torch.uint8, device=dev)
    _run(lib.gla_prefix_bwd, "gla_prefix_bwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_lambda.data_ptr(),
         pool.data_ptr(), rows, prefix_row.data_ptr(), DK ** -0.5 if scale is None else float(scale), dO.data_ptr(),
         _addr(dhT), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _addr(dpool), cu_seqlens.data_ptr(), n_seq, T, H, DK,
         DV, dt, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dv, dpool


def gla_get_device_error(device=None) -> int:
    """Synchronises the current stream; returns and clears the device's sticky error status."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(load_library().gla_get_device_error(_stream(dev)))


def gla_set_wait_limit_ns(ns: int) -> None:
    _check(load_library().gla_set_wait_limit_ns(int(ns)), "gla_set_wait_limit_ns")
