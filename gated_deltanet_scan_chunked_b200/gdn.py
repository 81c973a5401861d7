"""Thin Python binding of libgdn (see include/gdn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libgdn.so.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or the tensors are
not on a CUDA device, the call raises.

A call given ``stream=`` runs on that stream.  What it allocates is that
stream's memory, and neither that nor its arguments' memory goes to others
before both streams are done with it; but it is the caller who makes the
stream wait for whatever still produces the arguments.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "gdn.h")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT = range(5)
GDN_BF16, GDN_FP32 = 0, 1
PATHS = {"auto": 0, "tensor": 1, "simt": 2, "tensor_pair": 3, "tensor_single": 4,
         "tensor_split": 5}
# paths that may run the split layout, which needs a workspace
_WS_PATHS = ("auto", "tensor", "tensor_split")

_lib = None
_vp = ctypes.c_void_p


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))


def load(path: str = LIB_PATH):
    """Load libgdn.so (once).  Raises if it has not been built."""
    global _lib, _current_device, _current_stream
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            "libgdn.so not found at %s; build it with "
            "`python -m gated_deltanet_scan_chunked_b200.build`" % path)
    lib = ctypes.CDLL(path)
    f = lib.gdn_chunk_fwd_path
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 9 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp,
        ctypes.c_int, _vp]
    f = lib.gdn_chunk_fwd_ws
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 9 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp,
        ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    f = lib.gdn_chunk_fwd_static_ws
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 9 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp, _vp]
    f = lib.gdn_chunk_fwd_workspace_size
    f.restype = ctypes.c_size_t
    f.argtypes = [ctypes.c_int32] * 4 + [ctypes.c_int]
    f = lib.gdn_chunk_fwd
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 9 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp, _vp]
    f = lib.gdn_decode_step
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 8 + [ctypes.c_int32] * 6 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp]
    f = lib.gdn_decode_multi
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 10 + [ctypes.c_int32] * 7 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp]
    f = lib.gdn_chunk_bwd_workspace_size
    f.restype = ctypes.c_size_t
    f.argtypes = [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 4
    f = lib.gdn_chunk_bwd
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 9 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float] + [_vp] * 10 + [
        _vp, ctypes.c_size_t, _vp]
    f = lib.gdn_conv_frontend
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 7 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        _vp, _vp, _vp, _vp]
    f = lib.gdn_chunk_fwd_conv_workspace_size
    f.restype = ctypes.c_size_t
    f.argtypes = [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 4 + [ctypes.c_int]
    f = lib.gdn_chunk_fwd_conv
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 12 + [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 5 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp,
        ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    f = lib.gdn_decode_conv
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 12 + [ctypes.c_int32] * 7 + [
        ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, _vp]
    f = lib.gdn_gr_read_workspace_size
    f.restype = ctypes.c_size_t
    f.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    f = lib.gdn_gr_read
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 6 + [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                              ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    f = lib.gdn_gr_write
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 4 + [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _vp]
    f = lib.gdn_glr_fwd
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 3 + [ctypes.c_int, _vp, _vp, ctypes.c_int32, ctypes.c_int64,
                              ctypes.c_int32, ctypes.c_int] + [_vp] * 4
    f = lib.gdn_glr_bwd_workspace_size
    f.restype = ctypes.c_size_t
    f.argtypes = [ctypes.c_int64, ctypes.c_int32]
    f = lib.gdn_glr_bwd
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 3 + [ctypes.c_int, _vp, _vp, ctypes.c_int32, ctypes.c_int64,
                              ctypes.c_int32, ctypes.c_int] + [_vp] * 8 + [ctypes.c_size_t, _vp]
    f = lib.gdn_glr_step
    f.restype = ctypes.c_int
    f.argtypes = [_vp] * 3 + [ctypes.c_int, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
                              _vp, _vp]
    f = lib.gdn_beam_select
    f.restype = ctypes.c_int
    f.argtypes = [_vp, ctypes.c_int64, _vp, _vp] + [ctypes.c_int32] * 5 + [ctypes.c_int] + [
        _vp] * 5
    f = lib.gdn_state_reorder
    f.restype = ctypes.c_int
    f.argtypes = [_vp, _vp, ctypes.c_int32, _vp, ctypes.c_int32, ctypes.c_int32, _vp]
    lib.gdn_selftest_bounded_wait.restype = ctypes.c_int
    lib.gdn_selftest_bounded_wait.argtypes = [ctypes.c_int32, _vp]
    lib.gdn_check_device_error.restype = ctypes.c_int
    lib.gdn_check_device_error.argtypes = [_vp]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_version.restype = ctypes.c_int32
    lib.gdn_version.argtypes = []
    _current_device = getattr(torch._C, "_cuda_getDevice", None)
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _lib = lib
    return lib


def header_functions(path: str = HEADER_PATH):
    """Names of the functions declared in include/gdn.h."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _tensors(v):
    """The tensors of an argument or result, lists and dicts of them included."""
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (list, tuple)):
        for w in v:
            yield from _tensors(w)
    elif isinstance(v, dict):
        yield from _tensors(list(v.values()))


def _on_stream(stream, call, *args):
    """call(*args) with the given stream as torch's current one, so that what the
    call allocates comes from that stream's own memory: a block just freed on
    another stream may still be in use by work queued there.  The arguments must
    not go to others before the stream has done with them, nor the results
    before the caller's current stream has."""
    used = [t for t in _tensors(args) if t.is_cuda]
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, used[0].device if used else None)
    for t in used:
        if t.device != stream.device:
            raise ValueError("the stream is on %s, a tensor on %s" % (stream.device, t.device))
    outer = torch.cuda.current_stream(stream.device)
    for t in used:
        t.record_stream(stream)
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in _tensors(out):
        t.record_stream(outer)
    return out


def _dtype_code_of(dtype) -> int:
    if dtype == torch.bfloat16:
        return GDN_BF16
    if dtype == torch.float32:
        return GDN_FP32
    raise TypeError("q/k/v/g must be bfloat16 or float32, got %s" % dtype)


def _dtype_code(t: torch.Tensor) -> int:
    return _dtype_code_of(t.dtype)


def _check(t: Optional[torch.Tensor], name: str, dtype=None, device=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (libgdn has no CPU path)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def workspace_size(n_seq: int, H_v: int, d_k: int, d_v: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace the split prefill layout uses (0: not applicable)."""
    return int(load().gdn_chunk_fwd_workspace_size(n_seq, H_v, d_k, d_v, _dtype_code_of(dtype)))


def gdn_chunk_fwd(q, k, v, log_alpha, beta, g=None, norm_w=None,
                  initial_state=None, cu_seqlens=None, l2norm_qk=True,
                  eps_l2=1e-6, eps_norm=1e-6, scale=1.0, y=None,
                  final_state=None, output_final_state=True, path="auto",
                  workspace="auto", stream=None
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked prefill over packed sequences: returns (y, final_state).

    q, k [T, H_qk, d_k]; v [T, H_v, d_v]; log_alpha, beta [T, H_v] fp32;
    g [T, H_v, d_v] or None; norm_w [d_v] fp32 or None; initial_state
    [n_seq, H_v, d_k, d_v] fp32 or None; cu_seqlens [n_seq + 1] int32 (device)
    or None.  y / final_state may be passed in (final_state may be
    initial_state itself for an in-place update).  ``workspace``: a uint8
    CUDA tensor of at least ``workspace_size(...)`` bytes, None (no split
    layout), or "auto" (allocated here through torch when the path may use
    it).  A workspace must not be shared by calls that can overlap.
    """
    if stream is not None:
        return _on_stream(stream, gdn_chunk_fwd, q, k, v, log_alpha, beta, g, norm_w,
                          initial_state, cu_seqlens, l2norm_qk, eps_l2, eps_norm, scale, y,
                          final_state, output_final_state, path, workspace)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    n_seq = 1 if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        _check(t, name, q.dtype, dev)
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("norm_w", norm_w),
                    ("initial_state", initial_state)):
        _check(t, name, torch.float32, dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if y is None:
        y = torch.empty((T, Hv, dv), dtype=q.dtype, device=dev)
    _check(y, "y", q.dtype, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((n_seq, Hv, dk, dv), dtype=torch.float32, device=dev)
    _check(final_state, "final_state", torch.float32, dev)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, None or 'auto'")
        workspace = None
        if path in _WS_PATHS:
            nbytes = int(lib.gdn_chunk_fwd_workspace_size(n_seq, Hv, dk, dv, dt))
            if nbytes > 0:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    ws_bytes = 0 if workspace is None else workspace.numel()
    st = lib.gdn_chunk_fwd_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(g), _ptr(norm_w),
        _ptr(initial_state), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, dk, dv, dt,
        1 if l2norm_qk else 0, float(eps_l2), float(eps_norm), float(scale), _ptr(y),
        _ptr(final_state), PATHS[path], _ptr(workspace), ws_bytes, _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_chunk_fwd")
    return y, final_state


def gdn_chunk_fwd_static_ws(q, k, v, log_alpha, beta, g=None, norm_w=None,
                            initial_state=None, cu_seqlens=None, l2norm_qk=True,
                            eps_l2=1e-6, eps_norm=1e-6, scale=1.0, y=None,
                            final_state=None, output_final_state=True, stream=None
                            ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The split-layout prefill with the library's own fixed workspace (at
    most 48 sequence x head items); arguments and results as gdn_chunk_fwd.
    Calls that can overlap must not be made (they share that workspace)."""
    if stream is not None:
        return _on_stream(stream, gdn_chunk_fwd_static_ws, q, k, v, log_alpha, beta, g, norm_w,
                          initial_state, cu_seqlens, l2norm_qk, eps_l2, eps_norm, scale, y,
                          final_state, output_final_state)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    n_seq = 1 if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        _check(t, name, q.dtype, dev)
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("norm_w", norm_w),
                    ("initial_state", initial_state)):
        _check(t, name, torch.float32, dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if y is None:
        y = torch.empty((T, Hv, dv), dtype=q.dtype, device=dev)
    _check(y, "y", q.dtype, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((n_seq, Hv, dk, dv), dtype=torch.float32, device=dev)
    _check(final_state, "final_state", torch.float32, dev)
    st = lib.gdn_chunk_fwd_static_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(g), _ptr(norm_w),
        _ptr(initial_state), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, dk, dv, dt,
        1 if l2norm_qk else 0, float(eps_l2), float(eps_norm), float(scale), _ptr(y),
        _ptr(final_state), _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_chunk_fwd_static_ws")
    return y, final_state


def bwd_workspace_size(n_seq: int, total_T: int, H_qk: int, H_v: int, d_k: int,
                       d_v: int) -> int:
    """Bytes of workspace gdn_chunk_bwd needs (0: arguments it never accepts)."""
    return int(load().gdn_chunk_bwd_workspace_size(n_seq, total_T, H_qk, H_v, d_k, d_v))


def gdn_chunk_bwd(q, k, v, log_alpha, beta, dy, g=None, norm_w=None,
                  initial_state=None, d_final_state=None, cu_seqlens=None,
                  l2norm_qk=True, eps_l2=1e-6, eps_norm=1e-6, scale=1.0,
                  want_d_initial_state=True, want_dnorm_w=True, workspace=None,
                  stream=None) -> dict:
    """Gradients of a gdn_chunk_fwd call with the same inputs.

    dy [T, H_v, d_v] (dtype of q): gradient with respect to y; d_final_state
    [n_seq, H_v, d_k, d_v] fp32 or None.  Returns a dict of fp32 tensors: dq,
    dk [T, H_qk, d_k]; dv [T, H_v, d_v]; dlog_alpha, dbeta [T, H_v]; and
    d_initial_state [n_seq, H_v, d_k, d_v], dg [T, H_v, d_v], dnorm_w [d_v]
    when asked for / when g is given.  ``workspace``: a uint8 CUDA tensor of
    at least ``bwd_workspace_size(...)`` bytes, or None (allocated here
    through torch).
    """
    if stream is not None:
        return _on_stream(stream, gdn_chunk_bwd, q, k, v, log_alpha, beta, dy, g, norm_w,
                          initial_state, d_final_state, cu_seqlens, l2norm_qk, eps_l2, eps_norm,
                          scale, want_d_initial_state, want_dnorm_w, workspace)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    n_seq = 1 if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("dy", dy)):
        _check(t, name, q.dtype, dev)
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("norm_w", norm_w),
                    ("initial_state", initial_state), ("d_final_state", d_final_state)):
        _check(t, name, torch.float32, dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty((T, Hqk, dk), **f32), dk=torch.empty((T, Hqk, dk), **f32),
               dv=torch.empty((T, Hv, dv), **f32), dlog_alpha=torch.empty((T, Hv), **f32),
               dbeta=torch.empty((T, Hv), **f32))
    if want_d_initial_state:
        out["d_initial_state"] = torch.empty((n_seq, Hv, dk, dv), **f32)
    if g is not None:
        out["dg"] = torch.empty((T, Hv, dv), **f32)
        if want_dnorm_w:
            out["dnorm_w"] = torch.empty((dv,), **f32)
    nbytes = int(lib.gdn_chunk_bwd_workspace_size(n_seq, T, Hqk, Hv, dk, dv))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    st = lib.gdn_chunk_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(g), _ptr(norm_w),
        _ptr(initial_state), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, dk, dv, dt,
        1 if l2norm_qk else 0, float(eps_l2), float(eps_norm), float(scale), _ptr(dy),
        _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
        _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]), _ptr(out.get("dg")),
        _ptr(out.get("dnorm_w")), _ptr(out.get("d_initial_state")), _ptr(workspace),
        workspace.numel(), _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_chunk_bwd")
    return out


def gdn_decode_step(q, k, v, log_alpha, beta, state, g=None, norm_w=None,
                    l2norm_qk=True, eps_l2=1e-6, eps_norm=1e-6, scale=1.0,
                    y=None, stream=None) -> torch.Tensor:
    """One token per sequence; ``state`` [N, H_v, d_k, d_v] fp32 is updated
    in place.  q, k [N, H_qk, d_k]; v [N, H_v, d_v]; gates [N, H_v].
    Returns y [N, H_v, d_v]."""
    if stream is not None:
        return _on_stream(stream, gdn_decode_step, q, k, v, log_alpha, beta, state, g, norm_w,
                          l2norm_qk, eps_l2, eps_norm, scale, y)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    N, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        _check(t, name, q.dtype, dev)
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("norm_w", norm_w),
                    ("state", state)):
        _check(t, name, torch.float32, dev)
    if y is None:
        y = torch.empty((N, Hv, dv), dtype=q.dtype, device=dev)
    _check(y, "y", q.dtype, dev)
    st = lib.gdn_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(g), _ptr(norm_w),
        _ptr(state), N, Hqk, Hv, dk, dv, dt, 1 if l2norm_qk else 0, float(eps_l2),
        float(eps_norm), float(scale), _ptr(y), _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_decode_step")
    return y


def gdn_decode_multi(q, k, v, log_alpha, beta, state_in, state_out="in_place",
                     snapshots=None, g=None, norm_w=None, l2norm_qk=True, eps_l2=1e-6,
                     eps_norm=1e-6, scale=1.0, y=None, stream=None) -> torch.Tensor:
    """T_s tokens per sequence in one launch.  q, k [N, T_s, H_qk, d_k];
    v [N, T_s, H_v, d_v]; gates [N, T_s, H_v]; state_in [N, H_v, d_k, d_v]
    fp32.  state_out: "in_place" (default: state_in is updated), a tensor, or
    None (not written).  snapshots: None, True (allocated here), or a
    [T_s, N, H_v, d_k, d_v] fp32 tensor receiving the state after each
    token.  Returns (y, snapshots)."""
    if stream is not None:
        return _on_stream(stream, gdn_decode_multi, q, k, v, log_alpha, beta, state_in, state_out,
                          snapshots, g, norm_w, l2norm_qk, eps_l2, eps_norm, scale, y)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    N, T_s, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        _check(t, name, q.dtype, dev)
    if isinstance(state_out, str):
        if state_out != "in_place":
            raise ValueError("state_out must be a tensor, None or 'in_place'")
        state_out = state_in
    if snapshots is True:
        snapshots = torch.empty((T_s, N, Hv, dk, dv), dtype=torch.float32, device=dev)
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("norm_w", norm_w),
                    ("state_in", state_in), ("state_out", state_out),
                    ("snapshots", snapshots)):
        _check(t, name, torch.float32, dev)
    if y is None:
        y = torch.empty((N, T_s, Hv, dv), dtype=q.dtype, device=dev)
    _check(y, "y", q.dtype, dev)
    st = lib.gdn_decode_multi(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(g), _ptr(norm_w),
        _ptr(state_in), _ptr(state_out), _ptr(snapshots), N, T_s, Hqk, Hv, dk, dv, dt,
        1 if l2norm_qk else 0, float(eps_l2), float(eps_norm), float(scale), _ptr(y),
        _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_decode_multi")
    return y, snapshots


def conv_state_shape(n_seq: int, H_v: int, d_k: int, d_v: int):
    """Shape of the carried conv state: [n_seq, H_v, 3, 2 d_k + d_v]."""
    return (n_seq, H_v, 3, 2 * d_k + d_v)


def gdn_conv_frontend(q, k, v, conv_w, conv_state_in=None, cu_seqlens=None,
                      conv_state_out=True, out=None, stream=None):
    """Causal depthwise conv (kernel 4) + SiLU over q, k, v (pre-conv, shapes
    as gdn_chunk_fwd).  conv_w [2 H_qk d_k + H_v d_v, 4] fp32 (channels q |
    k | v); conv_state_in [n_seq, H_v, 3, 2 d_k + d_v] fp32 or None;
    conv_state_out: True (allocated here), a tensor, or None (not written).
    Returns (q', k', v', conv_state_out)."""
    if stream is not None:
        return _on_stream(stream, gdn_conv_frontend, q, k, v, conv_w, conv_state_in, cu_seqlens,
                          conv_state_out, out)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    n_seq = 1 if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, q.dtype, dev)
    if conv_state_out is True:
        conv_state_out = torch.empty(conv_state_shape(n_seq, Hv, dk, dv), dtype=torch.float32,
                                     device=dev)
    for name, t in (("conv_w", conv_w), ("conv_state_in", conv_state_in),
                    ("conv_state_out", conv_state_out)):
        _check(t, name, torch.float32, dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    qo, ko, vo = out if out is not None else (torch.empty_like(q), torch.empty_like(k),
                                              torch.empty_like(v))
    st = lib.gdn_conv_frontend(
        _ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(conv_state_in), _ptr(conv_state_out),
        _ptr(cu_seqlens), n_seq, T, Hqk, Hv, dk, dv, dt, _ptr(qo), _ptr(ko), _ptr(vo),
        _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_conv_frontend")
    return qo, ko, vo, conv_state_out


def conv_workspace_size(n_seq: int, total_T: int, H_qk: int, H_v: int, d_k: int, d_v: int,
                        dtype=torch.bfloat16) -> int:
    """Bytes of workspace gdn_chunk_fwd_conv needs (0: never accepted)."""
    return int(load().gdn_chunk_fwd_conv_workspace_size(n_seq, total_T, H_qk, H_v, d_k, d_v,
                                                        _dtype_code_of(dtype)))


def gdn_chunk_fwd_conv(q, k, v, conv_w, log_alpha, beta, conv_state_in=None,
                       conv_state_out=True, g=None, norm_w=None, initial_state=None,
                       cu_seqlens=None, l2norm_qk=True, eps_l2=1e-6, eps_norm=1e-6,
                       scale=1.0, y=None, final_state=None, output_final_state=True,
                       path="auto", workspace=None, stream=None):
    """Prefill on pre-conv q, k, v: the front end, then gdn_chunk_fwd.
    Returns (y, final_state, conv_state_out).  ``workspace``: a uint8 CUDA
    tensor of at least conv_workspace_size(...) bytes, or None (allocated)."""
    if stream is not None:
        return _on_stream(stream, gdn_chunk_fwd_conv, q, k, v, conv_w, log_alpha, beta,
                          conv_state_in, conv_state_out, g, norm_w, initial_state, cu_seqlens,
                          l2norm_qk, eps_l2, eps_norm, scale, y, final_state, output_final_state,
                          path, workspace)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    n_seq = 1 if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        _check(t, name, q.dtype, dev)
    if conv_state_out is True:
        conv_state_out = torch.empty(conv_state_shape(n_seq, Hv, dk, dv), dtype=torch.float32,
                                     device=dev)
    for name, t in (("conv_w", conv_w), ("conv_state_in", conv_state_in),
                    ("conv_state_out", conv_state_out), ("log_alpha", log_alpha),
                    ("beta", beta), ("norm_w", norm_w), ("initial_state", initial_state)):
        _check(t, name, torch.float32, dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if y is None:
        y = torch.empty((T, Hv, dv), dtype=q.dtype, device=dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((n_seq, Hv, dk, dv), dtype=torch.float32, device=dev)
    _check(y, "y", q.dtype, dev)
    _check(final_state, "final_state", torch.float32, dev)
    nbytes = int(lib.gdn_chunk_fwd_conv_workspace_size(n_seq, T, Hqk, Hv, dk, dv, dt))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    st = lib.gdn_chunk_fwd_conv(
        _ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(conv_state_in), _ptr(conv_state_out),
        _ptr(log_alpha), _ptr(beta), _ptr(g), _ptr(norm_w), _ptr(initial_state),
        _ptr(cu_seqlens), n_seq, T, Hqk, Hv, dk, dv, dt, 1 if l2norm_qk else 0,
        float(eps_l2), float(eps_norm), float(scale), _ptr(y), _ptr(final_state), PATHS[path],
        _ptr(workspace), workspace.numel(), _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_chunk_fwd_conv")
    return y, final_state, conv_state_out


def gdn_decode_conv(q, k, v, conv_w, log_alpha, beta, state_in, conv_state,
                    state_out="in_place", snapshots=None, g=None, norm_w=None,
                    l2norm_qk=True, eps_l2=1e-6, eps_norm=1e-6, scale=1.0, y=None,
                    stream=None):
    """gdn_decode_multi on pre-conv q, k, v with the front end fused: q, k
    [N, T_s, H_qk, d_k]; v [N, T_s, H_v, d_v]; conv_state [N, H_v, 3,
    2 d_k + d_v] fp32, updated in place (None: zeros, not written).  Returns
    (y, snapshots)."""
    if stream is not None:
        return _on_stream(stream, gdn_decode_conv, q, k, v, conv_w, log_alpha, beta, state_in,
                          conv_state, state_out, snapshots, g, norm_w, l2norm_qk, eps_l2, eps_norm,
                          scale, y)
    lib = load()
    dev = q.device
    dt = _dtype_code(q)
    N, T_s, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        _check(t, name, q.dtype, dev)
    if isinstance(state_out, str):
        if state_out != "in_place":
            raise ValueError("state_out must be a tensor, None or 'in_place'")
        state_out = state_in
    if snapshots is True:
        snapshots = torch.empty((T_s, N, Hv, dk, dv), dtype=torch.float32, device=dev)
    for name, t in (("conv_w", conv_w), ("conv_state", conv_state), ("log_alpha", log_alpha),
                    ("beta", beta), ("norm_w", norm_w), ("state_in", state_in),
                    ("state_out", state_out), ("snapshots", snapshots)):
        _check(t, name, torch.float32, dev)
    if y is None:
        y = torch.empty((N, T_s, Hv, dv), dtype=q.dtype, device=dev)
    _check(y, "y", q.dtype, dev)
    st = lib.gdn_decode_conv(
        _ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(conv_state), _ptr(log_alpha),
        _ptr(beta), _ptr(g), _ptr(norm_w), _ptr(state_in), _ptr(state_out), _ptr(snapshots),
        N, T_s, Hqk, Hv, dk, dv, dt, 1 if l2norm_qk else 0, float(eps_l2), float(eps_norm),
        float(scale), _ptr(y), _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_decode_conv")
    return y, snapshots


def gr_read_workspace_size(T: int, n_r: int, d: int, rank: int) -> int:
    return int(load().gdn_gr_read_workspace_size(T, n_r, d, rank))


def gdn_gr_read(codes, scales, gamma, W_d, W_u, W_w, eps=1e-6, x=None, s=None,
                workspace=None, stream=None):
    """Gated Residual read: codes [T, n_r, d] uint8 (E4M3), scales [T, n_r]
    fp32, gamma [n_r, d] fp32, W_d [rank, n_r d], W_u [n_r d, rank], W_w
    [n_r, n_r d] bf16.  Returns (x [T, d] bf16, s [T, n_r] fp32)."""
    if stream is not None:
        return _on_stream(stream, gdn_gr_read, codes, scales, gamma, W_d, W_u, W_w, eps, x, s,
                          workspace)
    lib = load()
    dev = codes.device
    T, n_r, d = codes.shape
    rank = W_d.shape[0]
    _check(codes, "codes", torch.uint8, dev)
    for name, t in (("scales", scales), ("gamma", gamma)):
        _check(t, name, torch.float32, dev)
    for name, t in (("W_d", W_d), ("W_u", W_u), ("W_w", W_w)):
        _check(t, name, torch.bfloat16, dev)
    if x is None:
        x = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
    if s is None:
        s = torch.empty((T, n_r), dtype=torch.float32, device=dev)
    nbytes = int(lib.gdn_gr_read_workspace_size(T, n_r, d, rank))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    st = lib.gdn_gr_read(_ptr(codes), _ptr(scales), _ptr(gamma), _ptr(W_d), _ptr(W_u),
                         _ptr(W_w), T, n_r, d, rank, float(eps), _ptr(x), _ptr(s),
                         _ptr(workspace), workspace.numel(), _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_gr_read")
    return x, s


def gdn_gr_write(codes, scales, y, s, stream=None):
    """Gated Residual write, in place: R'_i = R_i + s_i y, requantised."""
    if stream is not None:
        return _on_stream(stream, gdn_gr_write, codes, scales, y, s)
    lib = load()
    dev = codes.device
    T, n_r, d = codes.shape
    _check(codes, "codes", torch.uint8, dev)
    _check(scales, "scales", torch.float32, dev)
    _check(y, "y", torch.bfloat16, dev)
    _check(s, "s", torch.float32, dev)
    st = lib.gdn_gr_write(_ptr(codes), _ptr(scales), _ptr(y), _ptr(s), T, n_r, d,
                          _stream_handle())
    if st != GDN_OK:
        raise GdnError(st, "gdn_gr_write")
    return codes, scales


# --- gated linear recurrence, beam search -------------------------------------

GLR_TILE = 32  # tokens between two checkpoints
_GATE_NONE, _GATE_BETA, _GATE_COMPLEMENT = 0, 1, 2


# These calls may be as short as a few microseconds, so the binding asks torch
# for the device and the stream by its cheapest ways.  (load() looks them up: a
# torch without CUDA has neither, and what needs no GPU must import there.)
_current_device = _current_stream = None
_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_FP32}


def _device_of(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (libgdn has no CPU path)" % name)
    return t.get_device()


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_INT32_MAX = (1 << 31) - 1


def _int32(v: int, name: str) -> int:
    """v, which goes to an int32 argument (ctypes would cut it to its low 32 bits)."""
    if not -_INT32_MAX - 1 <= v <= _INT32_MAX:
        raise ValueError("%s = %d does not fit in 32 bits" % (name, v))
    return v


def _need(t: torch.Tensor, name: str, dtype, shape, i: int):
    """t is a dense CUDA tensor on device i of that type and shape."""
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == i):
        _check(t, name, dtype, torch.device("cuda", i))
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _glr_inputs(x, log_alpha, beta, i):
    """(dtype code, gate code, beta tensor) of a call on x's device i."""
    dtype, shape = x.dtype, x.shape
    dt = _CODES.get(dtype)
    if dt is None:
        raise TypeError("x must be bfloat16 or float32, got %s" % dtype)
    if len(shape) != 2 or not x.is_contiguous():
        raise ValueError("x must be contiguous [tokens, channels], got %s" % (tuple(shape),))
    if shape[1] > _INT32_MAX:
        _int32(shape[1], "channels")
    _need(log_alpha, "log_alpha", dtype, shape, i)
    if beta is None:
        return dt, _GATE_NONE, None
    if isinstance(beta, str):
        if beta != "complement":
            raise ValueError("beta must be a tensor, None or 'complement'")
        return dt, _GATE_COMPLEMENT, None
    _need(beta, "beta", dtype, shape, i)
    return dt, _GATE_BETA, beta


def _glr_sequences(cu_seqlens, i):
    if cu_seqlens is None:
        return 1
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    _need(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, i)
    return _int32(cu_seqlens.shape[0] - 1, "sequences")


def glr_checkpoint_shape(total_T: int, C: int):
    """Shape of the recurrence's checkpoints: [ceil(total_T / 32), C]."""
    return ((total_T + GLR_TILE - 1) // GLR_TILE, C)


def gdn_glr_fwd(x, log_alpha, beta=None, initial_state=None, cu_seqlens=None, y=None,
                final_state=None, output_final_state=True, checkpoints=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + b_t x_t per channel, a =
    exp(log_alpha), over packed sequences: returns (y, final_state,
    checkpoints).

    x, log_alpha [T, C] (bf16 or fp32); beta: the input gate b as a tensor [T,
    C], None (b = 1) or "complement" (b = 1 - a); initial_state [n_seq, C]
    fp32 or None; cu_seqlens [n_seq + 1] int32 (device) or None.  y /
    final_state may be passed in (final_state may be initial_state itself).
    checkpoints: None (not written), True (allocated here) or a tensor of
    glr_checkpoint_shape(T, C) fp32, for gdn_glr_bwd.
    """
    if stream is not None:
        return _on_stream(stream, gdn_glr_fwd, x, log_alpha, beta, initial_state, cu_seqlens, y,
                          final_state, output_final_state, checkpoints)
    lib = _lib or load()
    i = _device_of(x, "x")
    if i != _current_device():
        with torch.cuda.device(i):
            return gdn_glr_fwd(x, log_alpha, beta, initial_state, cu_seqlens, y, final_state,
                               output_final_state, checkpoints)
    dt, gate, beta = _glr_inputs(x, log_alpha, beta, i)
    T, C = x.shape
    n_seq = _glr_sequences(cu_seqlens, i)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (n_seq, C), i)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", x.dtype, x.shape, i)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, (n_seq, C), i)
    elif output_final_state:
        if initial_state is not None:
            final_state = torch.empty_like(initial_state)
        else:
            final_state = x.new_empty((n_seq, C), dtype=torch.float32)
    if checkpoints is True:
        checkpoints = x.new_empty(glr_checkpoint_shape(T, C), dtype=torch.float32)
    elif checkpoints is not None:
        _need(checkpoints, "checkpoints", torch.float32, glr_checkpoint_shape(T, C), i)
    st = lib.gdn_glr_fwd(x.data_ptr(), log_alpha.data_ptr(), _addr(beta), gate,
                         _addr(initial_state), _addr(cu_seqlens), n_seq, T, C, dt, y.data_ptr(),
                         _addr(final_state), _addr(checkpoints), _current_stream(i))
    if st != GDN_OK:
        raise GdnError(st, "gdn_glr_fwd")
    return y, final_state, checkpoints


def glr_bwd_workspace_size(total_T: int, C: int) -> int:
    """Bytes of workspace gdn_glr_bwd needs when it is given no checkpoints."""
    return int(load().gdn_glr_bwd_workspace_size(total_T, C))


def gdn_glr_bwd(x, log_alpha, dy, beta=None, initial_state=None, d_final_state=None,
                cu_seqlens=None, checkpoints=None, want_d_initial_state=True, workspace=None,
                stream=None) -> dict:
    """Gradients of a gdn_glr_fwd call with the same inputs: dx, dlog_alpha
    (and dbeta for a tensor beta) [T, C] in x's dtype, d_initial_state [n_seq,
    C] fp32 when asked for.  dy [T, C]; d_final_state [n_seq, C] fp32 or None.
    ``checkpoints``: what the forward returned for them; without it they are
    computed again into ``workspace`` (a uint8 CUDA tensor of at least
    glr_bwd_workspace_size(T, C) bytes, or None: allocated here)."""
    if stream is not None:
        return _on_stream(stream, gdn_glr_bwd, x, log_alpha, dy, beta, initial_state,
                          d_final_state, cu_seqlens, checkpoints, want_d_initial_state, workspace)
    lib = _lib or load()
    i = _device_of(x, "x")
    if i != _current_device():
        with torch.cuda.device(i):
            return gdn_glr_bwd(x, log_alpha, dy, beta, initial_state, d_final_state, cu_seqlens,
                               checkpoints, want_d_initial_state, workspace)
    dt, gate, beta = _glr_inputs(x, log_alpha, beta, i)
    T, C = x.shape
    n_seq = _glr_sequences(cu_seqlens, i)
    _need(dy, "dy", x.dtype, x.shape, i)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, (n_seq, C), i)
    if d_final_state is not None:
        _need(d_final_state, "d_final_state", torch.float32, (n_seq, C), i)
    if checkpoints is not None:
        _need(checkpoints, "checkpoints", torch.float32, glr_checkpoint_shape(T, C), i)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, workspace.shape, i)
    elif checkpoints is None:
        workspace = x.new_empty(max(int(lib.gdn_glr_bwd_workspace_size(T, C)), 1),
                                dtype=torch.uint8)
    out = dict(dx=torch.empty_like(x), dlog_alpha=torch.empty_like(x))
    if gate == _GATE_BETA:
        out["dbeta"] = torch.empty_like(x)
    if want_d_initial_state:
        out["d_initial_state"] = x.new_empty((n_seq, C), dtype=torch.float32)
    st = lib.gdn_glr_bwd(x.data_ptr(), log_alpha.data_ptr(), _addr(beta), gate,
                         _addr(initial_state), _addr(cu_seqlens), n_seq, T, C, dt, dy.data_ptr(),
                         _addr(d_final_state), _addr(checkpoints), out["dx"].data_ptr(),
                         out["dlog_alpha"].data_ptr(), _addr(out.get("dbeta")),
                         _addr(out.get("d_initial_state")), _addr(workspace),
                         0 if workspace is None else workspace.numel(), _current_stream(i))
    if st != GDN_OK:
        raise GdnError(st, "gdn_glr_bwd")
    return out


def gdn_glr_step(x, log_alpha, state, beta=None, y=None, stream=None) -> torch.Tensor:
    """One token per sequence of the gated linear recurrence: x, log_alpha [N,
    C]; beta as for gdn_glr_fwd; ``state`` [N, C] fp32 is updated in place.
    Returns y [N, C]."""
    if stream is not None:
        return _on_stream(stream, gdn_glr_step, x, log_alpha, state, beta, y)
    lib = _lib or load()
    i = _device_of(x, "x")
    if i != _current_device():
        with torch.cuda.device(i):
            return gdn_glr_step(x, log_alpha, state, beta, y)
    dt, gate, beta = _glr_inputs(x, log_alpha, beta, i)
    shape = x.shape
    if shape[0] > _INT32_MAX:
        _int32(shape[0], "rows")
    _need(state, "state", torch.float32, shape, i)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", x.dtype, shape, i)
    st = lib.gdn_glr_step(x.data_ptr(), log_alpha.data_ptr(), _addr(beta), gate,
                          state.data_ptr(), shape[0], shape[1], dt, y.data_ptr(),
                          _current_stream(i))
    if st != GDN_OK:
        raise GdnError(st, "gdn_glr_step")
    return y


def gdn_beam_select(logits, scores, n_candidates, finished=None, end_token=-1, out=None,
                    stream=None):
    """Beam search's choice: the ``n_candidates`` (M) best continuations of each
    group over its K beams and the vocabulary, by scores[g, k] + log softmax of
    logits[g, k], best first; ties go to the lowest k V + v.

    logits [G, K, V] bf16 or fp32 with a contiguous last dimension and rows at
    one distance (a slice of a padded vocabulary may be given as it is);
    scores [G, K] fp32; finished [G, K] uint8 or bool or None: those beams are
    continued by ``end_token`` alone, at their own score.  Returns (scores,
    parents, tokens, finished), [G, M] fp32, int32, int32 and uint8, or writes
    them into ``out``, four such tensors (with M = K, out[0] may be scores and
    out[3] finished)."""
    if stream is not None:
        return _on_stream(stream, gdn_beam_select, logits, scores, n_candidates, finished,
                          end_token, out)
    lib = _lib or load()
    i = _device_of(logits, "logits")
    if i != _current_device():
        with torch.cuda.device(i):
            return gdn_beam_select(logits, scores, n_candidates, finished, end_token, out)
    dt = _CODES.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be bfloat16 or float32, got %s" % logits.dtype)
    if logits.dim() != 3:
        raise ValueError("logits must be [groups, beams, vocabulary], got %s"
                         % (tuple(logits.shape),))
    G, K, V = logits.shape
    M, end_token = int(n_candidates), int(end_token)
    if max(G, K, V, M, end_token) > _INT32_MAX or end_token < -1:
        for v, name in ((G, "groups"), (K, "beams"), (V, "vocabulary"), (M, "n_candidates"),
                        (end_token, "end_token")):
            _int32(v, name)
    sg, ld, sv = logits.stride()
    if K == 1:
        ld = sg
    if G * K == 1:
        ld = V
    if (V > 1 and sv != 1) or (G > 1 and sg != K * ld):
        raise ValueError("logits must have a contiguous vocabulary and equally spaced rows, got "
                         "strides %s" % (logits.stride(),))
    _need(scores, "scores", torch.float32, (G, K), i)
    if finished is not None:
        if finished.dtype is torch.bool:
            finished = finished.view(torch.uint8)
        _need(finished, "finished", torch.uint8, (G, K), i)
    if out is None:
        best = torch.empty_like(scores) if M == K else scores.new_empty((G, M))
        parents = torch.empty_like(best, dtype=torch.int32)
        out = (best, parents, torch.empty_like(parents), torch.empty_like(best, dtype=torch.uint8))
    else:
        out = tuple(out)
        for t, name, dtype in zip(out, ("out scores", "out parents", "out tokens", "out finished"),
                                  (torch.float32, torch.int32, torch.int32, torch.uint8)):
            _need(t, name, dtype, (G, M), i)
    st = lib.gdn_beam_select(logits.data_ptr(), ld, scores.data_ptr(), _addr(finished),
                             end_token, G, K, V, M, dt, out[0].data_ptr(),
                             out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                             _current_stream(i))
    if st != GDN_OK:
        raise GdnError(st, "gdn_beam_select")
    return out


def gdn_state_reorder(states, parents, stream=None):
    """The states of the chosen beams, in place: with parents [G, K] int32, row
    g K + j of every tensor becomes what row g K + parents[g, j] was.
    ``states``: a tensor or a list of up to 16, each contiguous with G * K rows
    (recurrent states, conv states, token histories; any type)."""
    if stream is not None:
        return _on_stream(stream, gdn_state_reorder, states, parents)
    lib = _lib or load()
    i = _device_of(parents, "parents")
    if i != _current_device():
        with torch.cuda.device(i):
            return gdn_state_reorder(states, parents)
    if parents.dim() != 2:
        raise ValueError("parents must be [groups, beams], got %s" % (tuple(parents.shape),))
    _need(parents, "parents", torch.int32, parents.shape, i)
    many = [states] if isinstance(states, torch.Tensor) else states
    G, K = parents.shape
    rows, n = _int32(G, "groups") * _int32(K, "beams"), len(many)
    if n == 0:
        raise ValueError("there must be a state to reorder")
    ptrs, sizes = (ctypes.c_void_p * n)(), (ctypes.c_size_t * n)()
    for j, t in enumerate(many):
        if t.get_device() != i or not t.is_contiguous():
            _check(t, "states[%d]" % j, None, parents.device)
        if t.dim() < 1 or t.shape[0] != rows:
            raise ValueError("states[%d] must have %d rows, got %s" % (j, rows, tuple(t.shape)))
        ptrs[j] = t.data_ptr()
        sizes[j] = t.nbytes // rows if rows else 0
    st = lib.gdn_state_reorder(ptrs, sizes, n, parents.data_ptr(), G, K, _current_stream(i))
    if st != GDN_OK:
        raise GdnError(st, "gdn_state_reorder")
    return states


def gdn_check_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(load().gdn_check_device_error(_stream_handle(stream)))
