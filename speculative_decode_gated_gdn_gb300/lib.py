"""Python binding of libgdn_gb300.so (ctypes; argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of the method: it turns torch tensors into device pointers and the
current torch stream into a cudaStream_t, calls the library, and raises
GdnError on a nonzero return code.  There is no CPU fallback: if the library
cannot be built or loaded, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_MISALIGNED = -3
GDN_ERR_WORKSPACE = -4
GDN_ERR_CUDA = -5
GDN_ACT_NONE = 0
GDN_ACT_SILU = 1
GDN_COMMIT_RECOMPUTE = 0
GDN_COMMIT_SNAPSHOT = 1
GDN_COMMIT_DEFERRED = 2
GDN_VERIFY_OVERLAP = 0x100
GDN_VERIFY_OVERLAP_STATE = 0x200
GDN_STATUS_TIMEOUT = 2
GDN_STATUS_BAD_KEEP = 1
GDN_STATUS_BAD_ROW = 4
GDN_STATUS_NO_PAGES = 8
GDN_STATUS_BAD_INDEX = 16
GDN_STATUS_BAD_LEN = 32
GDN_ROPE_HALF = 0
GDN_ROPE_PAIRS = 1
GDN_MAX_LAYERS = 256
GDN_NOALLOC_WS_BYTES = 4 << 20

EXPORTS = ("gdn_version", "gdn_last_error", "gdn_layer_workspace_bytes", "gdn_conv_verify",
           "gdn_commit", "gdn_prefill_workspace_bytes", "gdn_prefill_chunked", "gdn_get_status",
           "gdn_conv_verify_noalloc", "gdn_flush", "gdn_accept_workspace_bytes", "gdn_accept_greedy",
           "gdn_conv_verify_gated", "gdn_move_rows", "gdn_kv4_page_bytes", "gdn_kv_plan", "gdn_kv_plan_shared",
           "gdn_kv_fork", "gdn_kv_compact", "gdn_kv_copy_pages", "gdn_kv4_append",
           "gdn_kv4_read", "gdn_sample", "gdn_accept_sampled",
           "gdn_accept_sampled_workspace_bytes", "gdn_kv4_attend_workspace_bytes", "gdn_kv4_attend", "gdn_test_verify_timeout",
           "gdn_test_kv4_attend_timeout")


class GdnError(RuntimeError):
    def __init__(self, code: int, fn: str, msg: str):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


class gdn_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "T_max", "H_k", "H_v", "d_k", "d_v", "width", "act")]


def dims(B, T, H_k, H_v, d, T_max=None, width=4, act=GDN_ACT_SILU) -> gdn_dims:
    """gdn_dims for one cohort: B rows, T positions per verify (T_max >= T sizes
    the conv ring), H_k key and H_v value heads of size d, width-4 conv."""
    return gdn_dims(B, T, T if T_max is None else T_max, H_k, H_v, d, d, width, act)


def dims_of(geom) -> gdn_dims:
    """gdn_dims from a synth.Geometry."""
    return dims(geom.B, geom.T, geom.H_k, geom.H_v, geom.d, geom.tmax, geom.width, geom.act)


class gdn_kv4_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H_q", "H_kv", "d", "page", "max_pages", "n_pages")]


def kv4_dims(B, H_q, H_kv, d, page, max_pages, n_pages) -> gdn_kv4_dims:
    """gdn_kv4_dims of a paged 4-bit cache: B rows, H_q query heads over H_kv
    key/value heads of size d, pages of `page` tokens, a block table of
    max_pages columns, n_pages pages."""
    return gdn_kv4_dims(B, H_q, H_kv, d, page, max_pages, n_pages)


_P = ctypes.c_void_p
_lock = threading.Lock()
_lib = None


def _declare(lib):
    D = ctypes.POINTER(gdn_dims)
    lib.gdn_version.restype = ctypes.c_char_p
    lib.gdn_version.argtypes = []
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_last_error.argtypes = []
    lib.gdn_layer_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_layer_workspace_bytes.argtypes = [D, ctypes.c_int]
    lib.gdn_conv_verify.restype = ctypes.c_int
    lib.gdn_conv_verify.argtypes = [D, ctypes.c_int] + [_P] * 10 + [ctypes.c_size_t, _P]
    lib.gdn_commit.restype = ctypes.c_int
    lib.gdn_commit.argtypes = [D, ctypes.c_int, ctypes.c_int, ctypes.POINTER(_P), ctypes.POINTER(_P),
                               ctypes.POINTER(_P), _P, _P, _P, _P]
    lib.gdn_flush.restype = ctypes.c_int
    lib.gdn_flush.argtypes = [D, ctypes.c_int, ctypes.c_int, ctypes.POINTER(_P), ctypes.POINTER(_P), _P]
    lib.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_prefill_workspace_bytes.argtypes = [D, ctypes.c_int]
    lib.gdn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_prefill_chunked.argtypes = [D, ctypes.c_int] + [_P] * 9 + [ctypes.c_size_t, _P]
    lib.gdn_conv_verify_noalloc.restype = ctypes.c_int
    lib.gdn_conv_verify_noalloc.argtypes = [D, ctypes.c_int] + [_P] * 9 + [ctypes.POINTER(_P), _P]
    lib.gdn_test_verify_timeout.restype = ctypes.c_int
    lib.gdn_test_verify_timeout.argtypes = [D, ctypes.c_int] + [_P] * 10 + [ctypes.c_size_t, ctypes.c_uint32, _P]
    lib.gdn_get_status.restype = ctypes.c_int
    lib.gdn_get_status.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_uint32)]
    lib.gdn_conv_verify_gated.restype = ctypes.c_int
    lib.gdn_conv_verify_gated.argtypes = [D, ctypes.c_int] + [_P] * 10 + [ctypes.c_float, _P, _P, ctypes.c_size_t, _P]
    PP = ctypes.POINTER(_P)
    lib.gdn_move_rows.restype = ctypes.c_int
    lib.gdn_move_rows.argtypes = [D, D, ctypes.c_int, ctypes.c_int, PP, PP, _P, PP, PP, _P, PP, _P, _P,
                                  ctypes.c_int, _P]
    lib.gdn_accept_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_accept_workspace_bytes.argtypes = [ctypes.c_int] * 3
    lib.gdn_accept_greedy.restype = ctypes.c_int
    lib.gdn_accept_greedy.argtypes = [ctypes.c_int] * 3 + [_P] * 6 + [ctypes.c_size_t, _P]
    lib.gdn_sample.restype = ctypes.c_int
    lib.gdn_sample.argtypes = [ctypes.c_int] * 2 + [_P, ctypes.c_longlong] + [_P] * 9
    lib.gdn_accept_sampled_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_accept_sampled_workspace_bytes.argtypes = [ctypes.c_int] * 3
    lib.gdn_accept_sampled.restype = ctypes.c_int
    lib.gdn_accept_sampled.argtypes = ([ctypes.c_int] * 3 + [_P, ctypes.c_longlong] + [_P] * 12 + [ctypes.c_size_t, _P])
    K, I, LL = ctypes.POINTER(gdn_kv4_dims), ctypes.c_int, ctypes.c_longlong
    lib.gdn_kv4_page_bytes.restype = ctypes.c_size_t
    lib.gdn_kv4_page_bytes.argtypes = [K]
    lib.gdn_kv_plan.restype = ctypes.c_int
    lib.gdn_kv_plan.argtypes = [K, I, I] + [_P] * 13
    lib.gdn_kv_plan_shared.restype = ctypes.c_int
    lib.gdn_kv_plan_shared.argtypes = [K, I, I] + [_P] * 14
    lib.gdn_kv_fork.restype = ctypes.c_int
    lib.gdn_kv_fork.argtypes = [K, I] + [_P] * 11
    lib.gdn_kv_compact.restype = ctypes.c_int
    lib.gdn_kv_compact.argtypes = [K] + [_P] * 12
    lib.gdn_kv_copy_pages.restype = ctypes.c_int
    lib.gdn_kv_copy_pages.argtypes = [K, I, PP, I] + [_P] * 4
    lib.gdn_kv4_append.restype = ctypes.c_int
    lib.gdn_kv4_append.argtypes = [K, I, _P, LL, _P, LL, _P, LL, _P, I, _P, I, I, ctypes.c_char_p, I, _P, _P, _P, _P]
    lib.gdn_kv4_read.restype = ctypes.c_int
    lib.gdn_kv4_read.argtypes = [K, I] + [_P] * 5
    lib.gdn_kv4_attend_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_kv4_attend_workspace_bytes.argtypes = [K, I, I]
    lib.gdn_kv4_attend.restype = ctypes.c_int
    lib.gdn_kv4_attend.argtypes = [K, I, I] + [_P] * 6 + [ctypes.c_float, _P, _P, ctypes.c_size_t, _P]
    lib.gdn_test_kv4_attend_timeout.restype = ctypes.c_int
    lib.gdn_test_kv4_attend_timeout.argtypes = lib.gdn_kv4_attend.argtypes[:-1] + [ctypes.c_uint32, _P]


def library_path() -> str:
    """Where build() puts libgdn_gb300.so."""
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load (building first if missing or stale) and return the ctypes library."""
    global _lib
    if path is None and _lib is not None:  # every call comes through here
        return _lib
    with _lock:
        if _lib is None or path is not None:
            p = path or _build.build()
            if not os.path.exists(p):
                raise RuntimeError(f"libgdn_gb300.so not found at {p}")
            lib = ctypes.CDLL(p)
            _declare(lib)
            if path is not None:
                return lib
            _lib = lib
    return _lib


# ------------------------------------------------------------------ marshalling
def _ptr(t, what, dtype=None):
    """Device pointer of a tensor (or a raw int pointer / None)."""
    if t is None or isinstance(t, int):
        return t
    torch = _t()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor or an int pointer")
    if not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


_device_number = None


def _here():
    """The current CUDA device's number: what get_device() of a call's tensors
    has to be (-1 is the host); -2 where there is none."""
    global _device_number
    if _device_number is None:  # torch's own question behind current_device, without its look at the state of CUDA
        torch = _t()
        _device_number = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
    try:
        return _device_number()
    except (RuntimeError, AssertionError):
        return -2


def _elsewhere(t, what):
    """Refuses a tensor that is on another CUDA device than the current one,
    whose address the call's kernels could not follow."""
    if t.is_cuda and t.get_device() != _here():
        raise ValueError(f"{what}: tensor is on {t.device}, the current CUDA device is {_here()}")


def _ptr_here(t, what, dtype=None):
    """_ptr of a tensor that has to be on the current device."""
    p = _ptr(t, what, dtype)
    if p is not t:  # (not a raw pointer, or None)
        _elsewhere(t, what)
    return p


_raw_stream = None


def _stream(stream):
    """The stream's handle; by default torch's current stream of the current
    device, asked for without making a Stream object (2.9 us of a small call's
    10, 0.2 this way)."""
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            torch = _t()
            handle = torch.cuda.current_stream().cuda_stream  # initialises CUDA, or says why it cannot
            device, raw = (getattr(torch._C, name, None) for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))
            _raw_stream = (lambda: raw(device())) if device and raw else (lambda: torch.cuda.current_stream().cuda_stream)
            return handle
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc, fn):
    if rc != GDN_OK:
        raise GdnError(rc, fn, load().gdn_last_error().decode())


_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def gdn_version() -> str:
    """Library name, version and target architecture."""
    return load().gdn_version().decode()


def gdn_last_error() -> str:
    """Text of the last error returned on this thread."""
    return load().gdn_last_error().decode()


def gdn_layer_workspace_bytes(d: gdn_dims, mode: int) -> int:
    """Bytes of per-layer workspace gdn_conv_verify fills and gdn_commit reads
    in commit mode `mode` (0 for invalid dims or mode)."""
    return int(load().gdn_layer_workspace_bytes(ctypes.byref(d), mode))


def gdn_conv_verify(d: gdn_dims, mode, x, conv_w, g, beta, state, ring, offsets, active, out,
                    layer_ws, layer_ws_bytes=None, stream=None):
    """Verify one layer (gdn.h, gdn_conv_verify).  CUDA tensors: x [B][T][C]
    bf16, conv_w [C][4] bf16, g and beta [B][T][H_v] fp32, state
    [B][H_v][d][d] fp32, ring [B][R][C] bf16, offsets [B] int32 (may be
    None), active [B] uint8, out [B][T][H_v][d] bf16, layer_ws uint8 of
    gdn_layer_workspace_bytes.  `mode` may carry GDN_VERIFY_OVERLAP.
    Runs on `stream` (default: torch's current stream)."""
    torch = _t()
    if layer_ws_bytes is None:
        layer_ws_bytes = layer_ws.numel() * layer_ws.element_size()
    rc = load().gdn_conv_verify(
        ctypes.byref(d), mode, _ptr(x, "x", torch.bfloat16), _ptr(conv_w, "conv_w", torch.bfloat16),
        _ptr(g, "g", torch.float32), _ptr(beta, "beta", torch.float32), _ptr(state, "state", torch.float32),
        _ptr(ring, "ring", torch.bfloat16), _ptr(offsets, "offsets", torch.int32),
        _ptr(active, "active", torch.uint8), _ptr(out, "out", torch.bfloat16), _ptr(layer_ws, "layer_ws"),
        int(layer_ws_bytes), _stream(stream))
    _check(rc, "gdn_conv_verify")


def gdn_conv_verify_gated(d: gdn_dims, mode, x, conv_w, g, beta, state, ring, offsets, active, gate_z, norm_w,
                          eps, out, layer_ws, layer_ws_bytes=None, stream=None):
    """gdn_conv_verify with the gated RMSNorm of the output fused in:
    out = o / sqrt(mean(o^2) + eps) * norm_w * silu(gate_z) per (row, position, head)."""
    torch = _t()
    if layer_ws_bytes is None:
        layer_ws_bytes = layer_ws.numel() * layer_ws.element_size()
    rc = load().gdn_conv_verify_gated(
        ctypes.byref(d), mode, _ptr(x, "x", torch.bfloat16), _ptr(conv_w, "conv_w", torch.bfloat16),
        _ptr(g, "g", torch.float32), _ptr(beta, "beta", torch.float32), _ptr(state, "state", torch.float32),
        _ptr(ring, "ring", torch.bfloat16), _ptr(offsets, "offsets", torch.int32),
        _ptr(active, "active", torch.uint8), _ptr(gate_z, "gate_z", torch.bfloat16),
        _ptr(norm_w, "norm_w", torch.bfloat16), float(eps), _ptr(out, "out", torch.bfloat16),
        _ptr(layer_ws, "layer_ws"), int(layer_ws_bytes), _stream(stream))
    _check(rc, "gdn_conv_verify_gated")


def gdn_conv_verify_noalloc(d: gdn_dims, mode, x, conv_w, g, beta, state, ring, offsets, active, out,
                            stream=None) -> int:
    """gdn_conv_verify with the library's built-in scratch as the workspace.

    For callers that cannot allocate device memory.  Returns the scratch's
    device address, to be passed as this layer's workspace to gdn_commit
    before the next call of this function on the device.
    """
    torch = _t()
    used = _P(0)
    rc = load().gdn_conv_verify_noalloc(
        ctypes.byref(d), mode, _ptr(x, "x", torch.bfloat16), _ptr(conv_w, "conv_w", torch.bfloat16),
        _ptr(g, "g", torch.float32), _ptr(beta, "beta", torch.float32), _ptr(state, "state", torch.float32),
        _ptr(ring, "ring", torch.bfloat16), _ptr(offsets, "offsets", torch.int32),
        _ptr(active, "active", torch.uint8), _ptr(out, "out", torch.bfloat16), ctypes.byref(used),
        _stream(stream))
    _check(rc, "gdn_conv_verify_noalloc")
    return int(used.value)


def gdn_test_verify_timeout(d: gdn_dims, mode, x, conv_w, g, beta, state, ring, offsets, active, out, layer_ws,
                            wait_limit, layer_ws_bytes=None, stream=None):
    """gdn_conv_verify with its bounded-wait failure path forced for the CTA of
    (row 0, head 0), giving up after `wait_limit` polls (gdn.h, test hook)."""
    torch = _t()
    if layer_ws_bytes is None:
        layer_ws_bytes = layer_ws.numel() * layer_ws.element_size()
    rc = load().gdn_test_verify_timeout(
        ctypes.byref(d), mode, _ptr(x, "x", torch.bfloat16), _ptr(conv_w, "conv_w", torch.bfloat16),
        _ptr(g, "g", torch.float32), _ptr(beta, "beta", torch.float32), _ptr(state, "state", torch.float32),
        _ptr(ring, "ring", torch.bfloat16), _ptr(offsets, "offsets", torch.int32),
        _ptr(active, "active", torch.uint8), _ptr(out, "out", torch.bfloat16), _ptr(layer_ws, "layer_ws"),
        int(layer_ws_bytes), int(wait_limit), _stream(stream))
    _check(rc, "gdn_test_verify_timeout")


def _layer_ptrs(seq, what, dtype=None):
    return (_P * max(len(seq), 1))(*[_ptr(t, f"{what}[{i}]", dtype) for i, t in enumerate(seq)])


def gdn_commit(d: gdn_dims, mode, states, rings, layer_ws, keep, active, offsets, stream=None):
    """states / rings / layer_ws: sequences (one per layer) of tensors or int device pointers."""
    torch = _t()
    n = len(states)
    if len(layer_ws) != n or len(rings) != n:
        raise ValueError("states, rings and layer_ws must have one entry per layer")
    rc = load().gdn_commit(ctypes.byref(d), mode, n, _layer_ptrs(states, "state", torch.float32),
                           _layer_ptrs(rings, "ring", torch.bfloat16), _layer_ptrs(layer_ws, "layer_ws"),
                           _ptr(keep, "keep", torch.int32), _ptr(active, "active", torch.uint8),
                           _ptr(offsets, "offsets", torch.int32), _stream(stream))
    _check(rc, "gdn_commit")


def gdn_flush(d: gdn_dims, mode, states, layer_ws, stream=None):
    """Materialise commits a DEFERRED cycle left pending (no-op in other modes)."""
    torch = _t()
    if len(layer_ws) != len(states):
        raise ValueError("states and layer_ws must have one entry per layer")
    rc = load().gdn_flush(ctypes.byref(d), mode, len(states), _layer_ptrs(states, "state", torch.float32),
                          _layer_ptrs(layer_ws, "layer_ws"), _stream(stream))
    _check(rc, "gdn_flush")


def gdn_prefill_workspace_bytes(d: gdn_dims, L: int) -> int:
    """Bytes of scratch gdn_prefill_chunked needs for an L-token prompt."""
    return int(load().gdn_prefill_workspace_bytes(ctypes.byref(d), L))


def gdn_prefill_chunked(d: gdn_dims, L, x, conv_w, g, beta, state, ring, offsets, out, ws,
                        ws_bytes=None, stream=None):
    """Prime state, ring and offsets over an L-token prompt (gdn.h,
    gdn_prefill_chunked): x [B][L][C] bf16, g and beta [B][L][H_v] fp32,
    out [B][L][H_v][d] bf16, ws of gdn_prefill_workspace_bytes; the other
    tensors as in gdn_conv_verify."""
    torch = _t()
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().gdn_prefill_chunked(
        ctypes.byref(d), L, _ptr(x, "x", torch.bfloat16), _ptr(conv_w, "conv_w", torch.bfloat16),
        _ptr(g, "g", torch.float32), _ptr(beta, "beta", torch.float32), _ptr(state, "state", torch.float32),
        _ptr(ring, "ring", torch.bfloat16), _ptr(offsets, "offsets", torch.int32),
        _ptr(out, "out", torch.bfloat16), _ptr(ws, "ws"), int(ws_bytes), _stream(stream))
    _check(rc, "gdn_prefill_chunked")


def gdn_move_rows(src_d: gdn_dims, dst_d: gdn_dims, mode, src_states, src_rings, src_offsets, dst_states,
                  dst_rings, dst_offsets, dst_layer_ws, src_rows, dst_rows, stream=None):
    """Copy rows src_rows[i] of one cohort into rows dst_rows[i] of another,
    every layer: state, conv cache and committed offset (device index arrays)."""
    torch = _t()
    n = len(src_states)
    ws = None if dst_layer_ws is None else _layer_ptrs(dst_layer_ws, "dst_layer_ws")
    rc = load().gdn_move_rows(
        ctypes.byref(src_d), ctypes.byref(dst_d), mode, n, _layer_ptrs(src_states, "src_state", torch.float32),
        _layer_ptrs(src_rings, "src_ring", torch.bfloat16), _ptr(src_offsets, "src_offsets", torch.int32),
        _layer_ptrs(dst_states, "dst_state", torch.float32), _layer_ptrs(dst_rings, "dst_ring", torch.bfloat16),
        _ptr(dst_offsets, "dst_offsets", torch.int32), ws, _ptr(src_rows, "src_rows", torch.int32),
        _ptr(dst_rows, "dst_rows", torch.int32), int(src_rows.numel()), _stream(stream))
    _check(rc, "gdn_move_rows")


def gdn_accept_workspace_bytes(B: int, T: int, V: int) -> int:
    """Bytes of workspace gdn_accept_greedy needs (0 for invalid sizes)."""
    return int(load().gdn_accept_workspace_bytes(B, T, V))


def gdn_accept_greedy(logits, draft, active, keep, nxt, ws, stream=None):
    """Greedy acceptance on the device: logits [B][T][V] bf16, draft [B][T]
    int32, active [B] uint8 -> keep [B], nxt [B] int32 (written in place).
    ws: gdn_accept_workspace_bytes(B, T, V) bytes, zero-filled once."""
    torch = _t()
    B, T, V = logits.shape
    rc = load().gdn_accept_greedy(B, T, V, _ptr_here(logits, "logits", torch.bfloat16), _ptr_here(draft, "draft", torch.int32),
                                  _ptr_here(active, "active", torch.uint8), _ptr_here(keep, "keep", torch.int32),
                                  _ptr_here(nxt, "next", torch.int32), _ptr_here(ws, "ws"),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "gdn_accept_greedy")


def _logits(t, dims, here):
    """Pointer and position stride of [B][V] or [B][T][V] bf16 logits whose
    positions lie at equal distances (a slice of a padded vocabulary serves)."""
    torch = _t()
    try:
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"logits: expected {torch.bfloat16}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError("logits: tensor must be on a CUDA device")
        if t.get_device() != here:
            _elsewhere(t, "logits")
        shape, stride = t.shape, t.stride()
    except AttributeError:
        _need(logits=t)
        raise
    if len(shape) != dims:
        raise ValueError(f"logits: expected {dims} dimensions, got {tuple(shape)}")
    V = shape[-1]
    if stride[-1] != 1 and V > 1:
        raise ValueError("logits: a position's logits must be densely packed")
    B, T = shape[0], shape[1] if dims == 3 else 1
    s = stride[1] if T > 1 else stride[0] if B > 1 else max(V, 1)
    if T > 1 and B > 1 and stride[0] != T * s:
        raise ValueError("logits: positions must lie at equal distances")
    return t.data_ptr(), s


def _some_ptrs(here, *args):
    """_ptrs of arguments that may be None, which stays None."""
    p = []
    for t, what, n, dtype in args:
        if t is None:
            p.append(None)
        else:
            try:
                if t.numel() == n and t.dtype is dtype and t.get_device() == here and t.is_contiguous():
                    p.append(t.data_ptr())
                    continue
            except AttributeError:
                pass
            _count(t, what, n)
            p.append(_ptr_here(t, what, dtype))
    return p


def gdn_sample(logits, u, token, logp=None, temperature=None, top_k=None, top_p=None, min_p=None, active=None,
               stream=None):
    """One token a row from its logits (gdn.h, gdn_sample): logits [B][V] bf16
    (row stride free), u [B] fp32 -> token [B] int32, logp [B] fp32, written in
    place.  temperature, top_p, min_p [B] fp32, top_k [B] int32, active [B]
    uint8; None: 1, off, off, off, all."""
    torch = _t()
    f32, i32, here = torch.float32, torch.int32, _here()
    lp, stride = _logits(logits, 2, here)
    B, V = logits.shape
    p = _some_ptrs(here, (active, "active", B, torch.uint8), (temperature, "temperature", B, f32), (top_k, "top_k", B, i32),
                   (top_p, "top_p", B, f32), (min_p, "min_p", B, f32), (u, "u", B, f32), (token, "token", B, i32), (logp, "logp", B, f32))
    rc = load().gdn_sample(B, V, lp, stride, *p, _stream(stream))
    if rc:
        _check(rc, "gdn_sample")


def gdn_accept_sampled_workspace_bytes(B: int, T: int, V: int) -> int:
    """Bytes of workspace gdn_accept_sampled needs (0 for invalid sizes)."""
    return int(load().gdn_accept_sampled_workspace_bytes(B, T, V))


def gdn_accept_sampled(logits, draft, active, u, keep, nxt, token, logp, ws, temperature=None, top_k=None, top_p=None,
                       min_p=None, stream=None):
    """Sampled acceptance on the device (gdn.h, gdn_accept_sampled): logits
    [B][T][V] bf16 (position stride free), draft [B][T] int32, active [B] uint8
    (None: all), u [B][T] fp32 -> keep [B], nxt [B] int32, token [B][T] int32 and
    logp [B][T] fp32 (each may be None), written in place.  ws:
    gdn_accept_sampled_workspace_bytes(B, T, V) bytes, zero-filled once."""
    torch = _t()
    f32, i32, here = torch.float32, torch.int32, _here()
    lp, stride = _logits(logits, 3, here)
    B, T, V = logits.shape
    N = B * T
    try:
        bytes_ = ws.numel() * ws.element_size()
    except AttributeError:
        _need(ws=ws)
        raise
    p = _some_ptrs(here, (draft, "draft", N, i32), (active, "active", B, torch.uint8), (temperature, "temperature", B, f32),
                   (top_k, "top_k", B, i32), (top_p, "top_p", B, f32), (min_p, "min_p", B, f32), (u, "u", N, f32), (keep, "keep", B, i32),
                   (nxt, "next", B, i32), (token, "token", N, i32), (logp, "logp", N, f32), (ws, "ws", ws.numel(), ws.dtype))
    rc = load().gdn_accept_sampled(B, T, V, lp, stride, *p, bytes_, _stream(stream))
    if rc:
        _check(rc, "gdn_accept_sampled")


def gdn_kv4_page_bytes(kd: gdn_kv4_dims) -> int:
    """Bytes of one page (all kv heads) of one layer's cache (0 for invalid dims)."""
    return int(load().gdn_kv4_page_bytes(ctypes.byref(kd)))


def _tokens(t, what, heads, d):
    """Pointer and token stride of a [N][heads][d] bf16 tensor whose heads are
    densely packed (a slice of a fused projection serves)."""
    torch = _t()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    _elsewhere(t, what)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what}: expected {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{what}: expected [N][{heads}][{d}], got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and heads > 1):
        raise ValueError(f"{what}: a token's heads must be densely packed")
    return t.data_ptr(), (s0 if t.shape[0] > 1 else max(heads * d, 8))


def _need(**args):
    """Names the first argument that is no tensor; called where one turned out
    to lack a tensor's methods, so that calls that are right do not wait for it."""
    for what, t in args.items():
        if not isinstance(t, _t().Tensor):
            raise TypeError(f"{what}: expected a torch.Tensor")


def _count(t, what, n):
    _need(**{what: t})
    if t.numel() != n:
        raise ValueError(f"{what}: expected {n} elements, got {t.numel()}")


def _ptrs(*args):
    """Device pointers of contiguous CUDA tensors, each (tensor, name, elements,
    dtype).  What they are is asked for in one pass, because small calls wait
    for the host; the checks that name what is wrong run when something is."""
    here = _here()
    try:
        p = [t.data_ptr() for t, _, n, dtype in args if t.numel() == n and t.dtype is dtype and t.get_device() == here and t.is_contiguous()]
        if len(p) == len(args):
            return p
    except AttributeError:
        pass
    for t, what, n, _ in args:
        _count(t, what, n)
    return [_ptr_here(t, what, dtype) for t, what, _, dtype in args]


def gdn_kv_plan(kd: gdn_kv4_dims, lens, add, active, held, table, free_list, free_count, q_start, q_count, kv_len,
                slots, positions, T=0, stream=None):
    """Block table, slots and positions of a cycle's new tokens (gdn.h,
    gdn_kv_plan): int32 CUDA tensors, active uint8; N = slots.numel().  T > 0
    puts row b's tokens at b*T, T = 0 packs them."""
    torch = _t()
    try:
        i32, B, N = torch.int32, kd.B, slots.numel()
    except AttributeError:
        _need(slots=slots)
        raise
    p = _ptrs((lens, "lens", B, i32), (add, "add", B, i32), (active, "active", B, torch.uint8), (held, "held", B, i32),
              (table, "table", B * kd.max_pages, i32), (free_list, "free_list", kd.n_pages, i32),
              (free_count, "free_count", 1, i32), (q_start, "q_start", B + 1, i32), (q_count, "q_count", B, i32),
              (kv_len, "kv_len", B, i32), (slots, "slots", N, i32), (positions, "positions", N, i32))
    rc = load().gdn_kv_plan(ctypes.byref(kd), T, N, *p, _stream(stream))
    _check(rc, "gdn_kv_plan")


def gdn_kv_plan_shared(kd: gdn_kv4_dims, lens, add, active, held, table, free_list, free_count, refs, q_start, q_count,
                       kv_len, slots, positions, T=0, stream=None):
    """gdn_kv_plan for a cache whose pages several rows may hold (gdn.h,
    gdn_kv_plan_shared): refs [n_pages] int32, the holders of each page."""
    torch = _t()
    try:
        i32, B, N = torch.int32, kd.B, slots.numel()
    except AttributeError:
        _need(slots=slots)
        raise
    p = _ptrs((lens, "lens", B, i32), (add, "add", B, i32), (active, "active", B, torch.uint8), (held, "held", B, i32),
              (table, "table", B * kd.max_pages, i32), (free_list, "free_list", kd.n_pages, i32),
              (free_count, "free_count", 1, i32), (refs, "refs", kd.n_pages, i32), (q_start, "q_start", B + 1, i32),
              (q_count, "q_count", B, i32), (kv_len, "kv_len", B, i32), (slots, "slots", N, i32),
              (positions, "positions", N, i32))
    rc = load().gdn_kv_plan_shared(ctypes.byref(kd), T, N, *p, _stream(stream))
    _check(rc, "gdn_kv_plan_shared")


def gdn_kv_fork(kd: gdn_kv4_dims, src_rows, dst_rows, lens, held, table, free_list, free_count, refs, copy_src, copy_dst,
                stream=None):
    """Rows dst_rows continue the first lens tokens of rows src_rows (gdn.h,
    gdn_kv_fork): int32 CUDA tensors; copy_src and copy_dst [n] are written, for
    gdn_kv_copy_pages."""
    i32 = _t().int32
    try:
        n, B = src_rows.numel(), kd.B
    except AttributeError:
        _need(src_rows=src_rows)
        raise
    p = _ptrs((src_rows, "src_rows", n, i32), (dst_rows, "dst_rows", n, i32), (lens, "lens", n, i32),
              (held, "held", B, i32), (table, "table", B * kd.max_pages, i32), (free_list, "free_list", kd.n_pages, i32),
              (free_count, "free_count", 1, i32), (refs, "refs", kd.n_pages, i32), (copy_src, "copy_src", n, i32),
              (copy_dst, "copy_dst", n, i32))
    _check(load().gdn_kv_fork(ctypes.byref(kd), n, *p, _stream(stream)), "gdn_kv_fork")


def gdn_kv_compact(kd: gdn_kv4_dims, held, table, refs, new_table, new_refs, new_free_list, new_free_count, page_map,
                   copy_src, copy_dst, copy_count, stream=None):
    """Places for the pages in use at the cache's front (gdn.h, gdn_kv_compact):
    int32 CUDA tensors; new_table and new_refs may be table and refs, copy_src and
    copy_dst have n_pages / 2 elements or more."""
    i32, B, n = _t().int32, kd.B, kd.n_pages
    try:
        size = copy_src.numel()
    except AttributeError:
        _need(copy_src=copy_src)
        raise
    if size < max(n // 2, 1):
        raise ValueError(f"copy_src: {size} elements, needs {max(n // 2, 1)}")
    p = _ptrs((held, "held", B, i32), (table, "table", B * kd.max_pages, i32), (refs, "refs", n, i32),
              (new_table, "new_table", B * kd.max_pages, i32), (new_refs, "new_refs", n, i32),
              (new_free_list, "new_free_list", n, i32), (new_free_count, "new_free_count", 1, i32),
              (page_map, "page_map", n, i32), (copy_src, "copy_src", size, i32), (copy_dst, "copy_dst", size, i32),
              (copy_count, "copy_count", 1, i32))
    _check(load().gdn_kv_compact(ctypes.byref(kd), *p, _stream(stream)), "gdn_kv_compact")


def gdn_kv_copy_pages(kd: gdn_kv4_dims, caches, src, dst, count=None, stream=None):
    """Page src[i] to page dst[i] in every layer's cache (gdn.h,
    gdn_kv_copy_pages): caches, a sequence of uint8 CUDA tensors; src, dst [n]
    int32; count [1] int32, or None for all n."""
    i32 = _t().int32
    try:
        n = src.numel()
    except AttributeError:
        _need(src=src)
        raise
    sp, dp = _ptrs((src, "src", n, i32), (dst, "dst", n, i32))
    u8, need = _t().uint8, _cache_bytes(kd)
    try:  # one pass, as in _ptrs
        here = _here()
        p = [t.data_ptr() for t in caches if t.dtype is u8 and t.get_device() == here and t.is_contiguous() and t.numel() >= need]
    except AttributeError:
        p = ()
    if len(p) != len(caches):
        p = [_cache(kd, t, f"caches[{i}]") for i, t in enumerate(caches)]
    rc = load().gdn_kv_copy_pages(ctypes.byref(kd), len(p), (_P * max(len(p), 1))(*p), n, sp, dp,
                                  None if count is None else _ptrs((count, "count", 1, i32))[0], _stream(stream))
    _check(rc, "gdn_kv_copy_pages")


def _cache_bytes(kd):
    """Bytes of a cache of these dims; a page's size is asked for once."""
    key = (kd.H_kv, kd.d, kd.page)
    if kd.__dict__.get("_key") != key:
        kd._page_bytes = gdn_kv4_page_bytes(kd)
        kd._key = key if kd._page_bytes else None  # (0: dims that the call will refuse, which says nothing of others)
    return kd.n_pages * kd._page_bytes


def _cache(kd, pages, what="pages"):
    """Pointer of a cache; it may be larger than its dims say, never smaller."""
    need = _cache_bytes(kd)
    try:
        size = pages.numel()
    except AttributeError:
        _need(**{what: pages})
        raise
    p = _ptr_here(pages, what, _t().uint8)
    if size < need:
        raise ValueError(f"{what}: {size} bytes, needs {need}")
    return p


def gdn_kv4_append(kd: gdn_kv4_dims, q, k, v, positions, rope, axis, slots, pages, q_out, style=GDN_ROPE_HALF,
                   stream=None):
    """Rotate q and k, write k and v into the cache (gdn.h, gdn_kv4_append).
    q [N][H_q][d], k and v [N][H_kv][d] bf16 (token stride free), positions
    [axes][N] int32, rope [max_pos][rot/2][2] fp32 (None: no rotation), axis:
    bytes, the axis of each pair, slots [N] int32, pages uint8, q_out
    [N][H_q][d] bf16."""
    torch = _t()
    qp, qs = _tokens(q, "q", kd.H_q, kd.d)
    kp, ks = _tokens(k, "k", kd.H_kv, kd.d)
    vp, vs = _tokens(v, "v", kd.H_kv, kd.d)
    N = q.shape[0]
    if k.shape[0] != N or v.shape[0] != N:
        raise ValueError("q, k and v must have the same number of tokens")
    sp, op = _ptrs((slots, "slots", N, torch.int32), (q_out, "q_out", N * kd.H_q * kd.d, torch.bfloat16))
    rot, max_pos, n_axes = 0, 0, 0
    if rope is not None:
        try:
            if rope.dim() != 3 or rope.shape[2] != 2:
                raise ValueError("rope: expected [max_pos][rot/2][2]")
            if positions.dim() != 2 or positions.shape[1] != N:
                raise ValueError("positions: expected [axes][N]")
        except AttributeError:
            _need(rope=rope, positions=positions)
            raise
        if not isinstance(axis, (bytes, ctypes.Array)):
            raise TypeError("axis: expected bytes")
        max_pos, rot, n_axes = rope.shape[0], 2 * rope.shape[1], positions.shape[0]
        if len(axis) != rot // 2:
            raise ValueError(f"axis: expected {rot // 2} bytes, got {len(axis)}")
    rc = load().gdn_kv4_append(
        ctypes.byref(kd), N, qp, qs, kp, ks, vp, vs, _ptr_here(positions, "positions", torch.int32) if rot else None,
        n_axes, _ptr_here(rope, "rope", torch.float32), max_pos, rot, axis if rot else None, style,
        sp, _cache(kd, pages), op, _stream(stream))
    _check(rc, "gdn_kv4_append")


def gdn_kv4_read(kd: gdn_kv4_dims, slots, pages, k, v, stream=None):
    """The cached keys and values at the given slots in bf16 (gdn.h,
    gdn_kv4_read): k and v [N][H_kv][d] bf16, written."""
    torch = _t()
    try:
        N = slots.numel()
    except AttributeError:
        _need(slots=slots)
        raise
    size, bf16 = N * kd.H_kv * kd.d, torch.bfloat16
    sp, kp, vp = _ptrs((slots, "slots", N, torch.int32), (k, "k", size, bf16), (v, "v", size, bf16))
    rc = load().gdn_kv4_read(ctypes.byref(kd), N, sp, _cache(kd, pages), kp, vp, _stream(stream))
    _check(rc, "gdn_kv4_read")


def gdn_kv4_attend_workspace_bytes(kd: gdn_kv4_dims, N: int, max_q: int) -> int:
    """Bytes of workspace gdn_kv4_attend needs (0 for invalid arguments)."""
    return int(load().gdn_kv4_attend_workspace_bytes(ctypes.byref(kd), N, max_q))


def _attend_args(kd, q, pages, table, q_start, q_count, kv_len, scale, out, ws, max_q):
    torch = _t()
    try:
        i32, bf16, B, N, ws_bytes = torch.int32, torch.bfloat16, kd.B, q.shape[0], ws.numel() * ws.element_size()
    except AttributeError:
        _need(q=q, ws=ws)
        raise
    size = N * kd.H_q * kd.d
    qp, op, tp, sp, cp, lp = _ptrs((q, "q", size, bf16), (out, "out", size, bf16), (table, "table", B * kd.max_pages, i32),
                                   (q_start, "q_start", B + 1, i32), (q_count, "q_count", B, i32), (kv_len, "kv_len", B, i32))
    return ctypes.byref(kd), N, max_q, qp, _cache(kd, pages), tp, sp, cp, lp, scale, op, _ptr_here(ws, "ws"), ws_bytes


def gdn_kv4_attend(kd: gdn_kv4_dims, q, pages, table, q_start, q_count, kv_len, scale, out, ws, max_q, stream=None):
    """Causal attention of the new tokens over the cache (gdn.h,
    gdn_kv4_attend): q and out [N][H_q][d] bf16, pages uint8, table, q_start,
    q_count, kv_len as gdn_kv_plan leaves them, ws zero-filled once."""
    args = _attend_args(kd, q, pages, table, q_start, q_count, kv_len, scale, out, ws, max_q)
    _check(load().gdn_kv4_attend(*args, _stream(stream)), "gdn_kv4_attend")


def gdn_test_kv4_attend_timeout(kd: gdn_kv4_dims, q, pages, table, q_start, q_count, kv_len, scale, out, ws, max_q,
                                wait_limit=4000, stream=None):
    """Test hook: gdn_kv4_attend with its bounded-wait failure path forced (gdn.h)."""
    args = _attend_args(kd, q, pages, table, q_start, q_count, kv_len, scale, out, ws, max_q)
    _check(load().gdn_test_kv4_attend_timeout(*args, wait_limit, _stream(stream)), "gdn_test_kv4_attend_timeout")


def gdn_get_status(clear: bool = False) -> int:
    """The sticky device status word (GDN_STATUS_* bits); synchronises the
    device.  clear=True resets it after reading."""
    v = ctypes.c_uint32(0)
    rc = load().gdn_get_status(1 if clear else 0, ctypes.byref(v))
    _check(rc, "gdn_get_status")
    return int(v.value)
