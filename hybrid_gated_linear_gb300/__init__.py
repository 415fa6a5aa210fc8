"""GB300 (sm_103a) Lizard-attention operator: a thin Python binding of ``include/lizard.h``.

Every function below has the name of a C entry point and only marshals arguments:
tensors become device pointers, the stream becomes a ``cudaStream_t``, and a non-OK
status raises :class:`LizardError`.  All arithmetic runs in the library's CUDA kernels;
there is no Python or CPU fallback.  Call :func:`build`
once to compile ``_build/liblizard.so``; importing works without it, but every call
raises until the library is present.
"""
from __future__ import annotations

import ctypes
import os
import threading

from .build_lib import LIB as LIB_PATH
from .build_lib import build as _build

__all__ = [
    "LizardError", "build", "library", "lizard_dims", "lizard_decode_dims",
    "lizard_attn_fwd", "lizard_attn_bwd", "lizard_decode_step", "lizard_chunk_cumsum",
    "lizard_fwd_workspace_bytes", "lizard_bwd_workspace_bytes", "lizard_decode_workspace_bytes",
    "lizard_workspace_init", "lizard_check_device_errors", "lizard_status_string",
    "lizard_abi_version", "lizard_last_launch_count", "lizard_trace_enable", "lizard_trace_read",
    "lizard_decode_step_noalloc", "LIZARD_NOALLOC_MAX_SEQUENCES",
    "lizard_attn_fwd_bwd_host", "lizard_fwd_bwd_host_workspace_bytes",
    "lizard_decode_ring_fill", "lizard_state_combine", "lizard_fmap_dims",
    "lizard_feature_map_fwd", "lizard_feature_map_bwd", "lizard_feature_map_workspace_bytes",
    "lizard_attn_fwd_fmap", "lizard_selftest_wait_timeout", "lizard_gate_dims",
    "lizard_gate_fwd", "lizard_gate_bwd", "lizard_gate_workspace_bytes", "lizard_gla_std_fwd",
    "lizard_gla_std_workspace_bytes",
    "lizard_rope_spec", "lizard_rope", "lizard_rope_dims", "lizard_rope_table", "lizard_rope_fwd",
    "lizard_rope_bwd", "LIZARD_ROPE_HALF", "LIZARD_ROPE_INTERLEAVED", "LIZARD_ROPE_PLAIN",
    "LIZARD_ROPE_LINEAR", "LIZARD_ROPE_PARTS", "lizard_strides", "lizard_cache", "lizard_cache_io",
    "lizard_cache_workspace_bytes", "lizard_cache_write", "lizard_cache_read",
    "lizard_cache_attn_dims", "lizard_cache_attn_workspace_bytes", "lizard_cache_attn",
    "LIZARD_KV_E4M3", "LIZARD_KV_I8", "LIZARD_F32", "LIZARD_BF16", "EXPORTED_SYMBOLS",
]

LIZARD_F32 = 0
LIZARD_BF16 = 1
LIZARD_NOALLOC_MAX_SEQUENCES = 16384
LIZARD_ROPE_HALF = 0
LIZARD_ROPE_INTERLEAVED = 1
LIZARD_ROPE_PLAIN = 0
LIZARD_ROPE_LINEAR = 1
LIZARD_ROPE_PARTS = 2
LIZARD_KV_E4M3 = 0
LIZARD_KV_I8 = 1

EXPORTED_SYMBOLS = (
    "lizard_attn_fwd", "lizard_attn_bwd", "lizard_decode_step", "lizard_chunk_cumsum",
    "lizard_fwd_workspace_bytes", "lizard_bwd_workspace_bytes", "lizard_decode_workspace_bytes",
    "lizard_workspace_init", "lizard_check_device_errors", "lizard_status_string",
    "lizard_abi_version", "lizard_last_launch_count", "lizard_trace_enable", "lizard_trace_read",
    "lizard_decode_step_noalloc", "lizard_attn_fwd_bwd_host", "lizard_fwd_bwd_host_workspace_bytes",
    "lizard_decode_ring_fill", "lizard_state_combine", "lizard_feature_map_fwd",
    "lizard_feature_map_bwd", "lizard_feature_map_workspace_bytes", "lizard_attn_fwd_fmap",
    "lizard_selftest_wait_timeout", "lizard_gate_fwd", "lizard_gate_bwd",
    "lizard_gate_workspace_bytes", "lizard_gla_std_fwd", "lizard_gla_std_workspace_bytes",
    "lizard_rope_table", "lizard_rope_fwd", "lizard_rope_bwd", "lizard_cache_workspace_bytes",
    "lizard_cache_write", "lizard_cache_read", "lizard_cache_attn_workspace_bytes",
    "lizard_cache_attn",
)

STATUS_NAMES = {0: "LIZARD_OK", 1: "LIZARD_ERR_INVALID_ARG", 2: "LIZARD_ERR_UNSUPPORTED",
                3: "LIZARD_ERR_CUDA", 4: "LIZARD_ERR_TIMEOUT", 5: "LIZARD_ERR_DEVICE_CHECK",
                6: "LIZARD_ERR_WORKSPACE"}


class LizardError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{what}: {name} ({lizard_status_string(status)})")


class lizard_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("L", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("M", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class lizard_decode_dims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("M", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class lizard_gate_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("L", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dk", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("tau", ctypes.c_float)]


class lizard_fmap_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("L", ctypes.c_int32),
                ("D", ctypes.c_int32), ("F", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class lizard_strides(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class lizard_rope_spec(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("original", ctypes.c_int64)]


class lizard_rope(ctypes.Structure):
    """A rotary table on the device; keeps its tensor alive."""
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("attn_factor", ctypes.c_float)]

    def __init__(self, turns, rot: int, layout: int, attn_factor: float = 1.0):
        if (turns.element_size() != 8 or turns.is_floating_point() or turns.is_complex()
                or turns.numel() != rot // 2 or not turns.is_contiguous()):
            raise ValueError("turns must be the rot/2 words of lizard_rope_table")
        super().__init__(turns.data_ptr(), rot, layout, attn_factor)
        self._keep = turns


class lizard_rope_dims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("Hk", ctypes.c_int32),
                ("T", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class lizard_cache(ctypes.Structure):
    """The pools and the page table of an 8-bit cache; keeps their tensors alive.
    k_codes, v_codes [pages,Hk,page_tokens,d] of one byte per element, k_scale, v_scale
    [pages,Hk] fp32, table [N,max_pages] int32, all contiguous on one device."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("N", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("Hk", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("d", ctypes.c_int32), ("format", ctypes.c_int32)]

    def __init__(self, k_codes, v_codes, k_scale, v_scale, table, format: int):
        import torch
        pages, hk, page_tokens, d = k_codes.shape
        if v_codes.shape != k_codes.shape or k_codes.element_size() != 1 or v_codes.element_size() != 1:
            raise ValueError("k_codes and v_codes must be [pages, Hk, page_tokens, d] bytes")
        for s in (k_scale, v_scale):
            if tuple(s.shape) != (pages, hk) or s.dtype != torch.float32:
                raise ValueError("k_scale and v_scale must be [pages, Hk] float32")
        if table.dim() != 2 or table.dtype != torch.int32:
            raise ValueError("table must be [N, max_pages] int32")
        keep = (k_codes, v_codes, k_scale, v_scale, table)
        if not all(t.is_contiguous() and t.device == table.device for t in keep):
            raise ValueError("the cache's tensors must be contiguous and on one device")
        super().__init__(*(t.data_ptr() for t in keep), table.shape[0], table.shape[1], pages, hk,
                         page_tokens, d, format)
        self._keep = keep


class lizard_cache_io(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class lizard_cache_attn_dims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("T", ctypes.c_int32), ("M", ctypes.c_int32),
                ("W", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("alpha", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile the CUDA library for sm_103a (see build_lib.py)."""
    return _build(force=force)


def library():
    """The loaded ctypes library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library {LIB_PATH} is missing: run hybrid_gated_linear_gb300.build()")
            lib = ctypes.CDLL(LIB_PATH)
            P, I32, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
            DP, DDP = ctypes.POINTER(lizard_dims), ctypes.POINTER(lizard_decode_dims)
            FMP = ctypes.POINTER(lizard_fmap_dims)
            GDP = ctypes.POINTER(lizard_gate_dims)
            sig = {
                "lizard_attn_fwd": (I32, [DP] + [P] * 8 + [I32, F, P, P, P, P, SZ, P]),
                "lizard_attn_bwd": (I32, [DP] + [P] * 8 + [I32, F] + [P] * 12 + [P, SZ, P]),
                "lizard_decode_step": (I32, [DDP] + [P] * 8 + [I32, F] + [P] * 5 + [P, SZ, P]),
                "lizard_chunk_cumsum": (I32, [I32, I32, I32, I32, P, P, P, P]),
                "lizard_fwd_workspace_bytes": (SZ, [DP, I32]),
                "lizard_bwd_workspace_bytes": (SZ, [DP, I32]),
                "lizard_decode_workspace_bytes": (SZ, [DDP]),
                "lizard_workspace_init": (I32, [P, SZ, P]),
                "lizard_check_device_errors": (I32, [P, P]),
                "lizard_status_string": (ctypes.c_char_p, [I32]),
                "lizard_abi_version": (I32, []),
                "lizard_last_launch_count": (I32, []),
                "lizard_trace_enable": (I32, [I32]),
                "lizard_trace_read": (I32, [ctypes.c_char_p, I32, ctypes.POINTER(F), I32]),
                "lizard_decode_step_noalloc": (I32, [DDP] + [P] * 8 + [I32, F] + [P] * 5 + [P]),
                "lizard_fwd_bwd_host_workspace_bytes": (SZ, [DP, I32]),
                "lizard_decode_ring_fill": (I32, [DDP, I32, I32] + [P] * 5 + [P]),
                "lizard_state_combine": (I32, [I32, I32, I32] + [P] * 6 + [P]),
                "lizard_feature_map_workspace_bytes": (SZ, [FMP, I32]),
                "lizard_attn_fwd_fmap": (I32, [DP] + [P] * 10 + [I32, F, P, P, P, P, SZ, P]),
                "lizard_feature_map_fwd": (I32, [FMP, P, P, P, P, SZ, P]),
                "lizard_feature_map_bwd": (I32, [FMP, P, P, P, P, P, P, SZ, P]),
                "lizard_attn_fwd_bwd_host": (I32, [DP] + [P] * 8 + [I32, F] + [P] * 13 + [P, SZ, P]),
                "lizard_selftest_wait_timeout": (I32, [P, SZ, ctypes.c_int64, P]),
                "lizard_gate_workspace_bytes": (SZ, [GDP]),
                "lizard_gate_fwd": (I32, [GDP, P, P, P, P]),
                "lizard_gate_bwd": (I32, [GDP, P, P, P, P, P, P, SZ, P]),
                "lizard_gla_std_workspace_bytes": (SZ, [DP]),
                "lizard_gla_std_fwd": (I32, [DP] + [P] * 8 + [SZ, P]),
                "lizard_rope_table": (I32, [P, P]),
                "lizard_rope_fwd": (I32, [P] * 12),
                "lizard_rope_bwd": (I32, [P] * 12),
                "lizard_cache_workspace_bytes": (SZ, []),
                "lizard_cache_write": (I32, [P] * 10 + [SZ, P]),
                "lizard_cache_read": (I32, [P] * 9 + [SZ, P]),
                "lizard_cache_attn_workspace_bytes": (SZ, [P, P]),
                "lizard_cache_attn": (I32, [P] * 15 + [SZ, P]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            _lib = lib
    return _lib


# ------------------------------------------------------------------------------------
# marshalling helpers
# ------------------------------------------------------------------------------------
def _ptr(t):
    """Device pointer of a tensor (None -> NULL).  Requires a contiguous tensor."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        # the current stream's handle; where torch offers it, without the Stream object around it
        try:
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            stream = torch.cuda.current_stream()
    handle = getattr(stream, "cuda_stream", stream)
    return ctypes.c_void_p(int(handle))


_dtype_codes: dict = {}


def _dtype_code(t) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float32: LIZARD_F32, torch.bfloat16: LIZARD_BF16})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _check(status: int, what: str):
    if status != 0:
        raise LizardError(status, what)


def lizard_status_string(status: int) -> str:
    try:
        return library().lizard_status_string(status).decode()
    except RuntimeError:
        return STATUS_NAMES.get(status, "unknown")


def lizard_abi_version() -> int:
    return library().lizard_abi_version()


def lizard_last_launch_count() -> int:
    return library().lizard_last_launch_count()


def make_dims(B, H, L, dk, dv, M, dtype, scale=0.0) -> lizard_dims:
    return lizard_dims(B, H, L, dk, dv, M, dtype, scale)


def lizard_fwd_workspace_bytes(dims: lizard_dims, W: int) -> int:
    return library().lizard_fwd_workspace_bytes(ctypes.byref(dims), W)


def lizard_bwd_workspace_bytes(dims: lizard_dims, W: int) -> int:
    return library().lizard_bwd_workspace_bytes(ctypes.byref(dims), W)


def lizard_fwd_bwd_host_workspace_bytes(dims: lizard_dims, W: int) -> int:
    return library().lizard_fwd_bwd_host_workspace_bytes(ctypes.byref(dims), W)


def lizard_decode_workspace_bytes(dims: lizard_decode_dims) -> int:
    return library().lizard_decode_workspace_bytes(ctypes.byref(dims))


def lizard_workspace_init(workspace, stream=None):
    _check(library().lizard_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream)), "lizard_workspace_init")


def lizard_check_device_errors(workspace, stream=None) -> int:
    """Synchronises the stream and returns the device status (0 = OK); does not raise."""
    return library().lizard_check_device_errors(_ptr(workspace), _stream(stream))


def lizard_selftest_wait_timeout(workspace, wait_cycles: int, stream=None):
    """Makes one bounded device wait run out on purpose (see include/lizard.h)."""
    _check(library().lizard_selftest_wait_timeout(_ptr(workspace), _ws_bytes(workspace),
                                                  int(wait_cycles), _stream(stream)),
           "lizard_selftest_wait_timeout")


def lizard_gate_workspace_bytes(dims: lizard_gate_dims) -> int:
    return library().lizard_gate_workspace_bytes(ctypes.byref(dims))


def lizard_gate_fwd(dims: lizard_gate_dims, x, w, log_gamma, stream=None):
    """log_gamma = logsigmoid(x W) / tau into preallocated ``log_gamma``."""
    _check(library().lizard_gate_fwd(ctypes.byref(dims), _ptr(x), _ptr(w), _ptr(log_gamma),
                                     _stream(stream)), "lizard_gate_fwd")


def lizard_gate_bwd(dims: lizard_gate_dims, x, w, d_log_gamma, d_x, d_w, workspace, stream=None):
    """d_x and d_w of the gate projection from d_log_gamma."""
    _check(library().lizard_gate_bwd(ctypes.byref(dims), _ptr(x), _ptr(w), _ptr(d_log_gamma),
                                     _ptr(d_x), _ptr(d_w), _ptr(workspace), _ws_bytes(workspace),
                                     _stream(stream)), "lizard_gate_bwd")


def _ws_bytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def lizard_attn_fwd(dims: lizard_dims, phi_q, phi_k, v, log_gamma, q, k, meta_k, meta_v, W: int,
                    alpha: float, y, h0, h_final, workspace, stream=None):
    """Forward pass into preallocated ``y`` (and ``h_final`` if given)."""
    st = library().lizard_attn_fwd(ctypes.byref(dims), _ptr(phi_q), _ptr(phi_k), _ptr(v),
                                   _ptr(log_gamma), _ptr(q), _ptr(k), _ptr(meta_k), _ptr(meta_v),
                                   int(W), float(alpha), _ptr(y), _ptr(h0), _ptr(h_final),
                                   _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    _check(st, "lizard_attn_fwd")


def lizard_gla_std_workspace_bytes(dims: lizard_dims) -> int:
    return library().lizard_gla_std_workspace_bytes(ctypes.byref(dims))


def lizard_gla_std_fwd(dims: lizard_dims, phi_q, phi_k, v, log_gamma, y, h0, h_final, workspace,
                       stream=None):
    """The standard fp32 chunkwise GLA forward (GLA branch only) into preallocated ``y``."""
    st = library().lizard_gla_std_fwd(ctypes.byref(dims), _ptr(phi_q), _ptr(phi_k), _ptr(v),
                                      _ptr(log_gamma), _ptr(y), _ptr(h0), _ptr(h_final),
                                      _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    _check(st, "lizard_gla_std_fwd")


def lizard_attn_bwd(dims: lizard_dims, phi_q, phi_k, v, log_gamma, q, k, meta_k, meta_v, W: int,
                    alpha: float, h0, dy, d_phi_q, d_phi_k, d_v, d_log_gamma, d_q, d_k,
                    d_meta_k, d_meta_v, d_h0, workspace, stream=None, fwd_workspace=None):
    """Backward pass into preallocated gradient tensors.  ``fwd_workspace``: the workspace
    of the matching lizard_attn_fwd call, whose chunk features and states are reused."""
    st = library().lizard_attn_bwd(ctypes.byref(dims), _ptr(phi_q), _ptr(phi_k), _ptr(v),
                                   _ptr(log_gamma), _ptr(q), _ptr(k), _ptr(meta_k), _ptr(meta_v),
                                   int(W), float(alpha), _ptr(h0), _ptr(dy), _ptr(d_phi_q),
                                   _ptr(d_phi_k), _ptr(d_v), _ptr(d_log_gamma), _ptr(d_q),
                                   _ptr(d_k), _ptr(d_meta_k), _ptr(d_meta_v), _ptr(d_h0),
                                   _ptr(fwd_workspace), _ptr(workspace), _ws_bytes(workspace),
                                   _stream(stream))
    _check(st, "lizard_attn_bwd")


def lizard_decode_step(dims: lizard_decode_dims, phi_q, phi_k, v, log_gamma, q, k, meta_k,
                       meta_v, W: int, alpha: float, h, k_ring, v_ring, pos, y, workspace,
                       stream=None):
    """One decode step; h, rings and pos are updated in place."""
    st = library().lizard_decode_step(ctypes.byref(dims), _ptr(phi_q), _ptr(phi_k), _ptr(v),
                                      _ptr(log_gamma), _ptr(q), _ptr(k), _ptr(meta_k),
                                      _ptr(meta_v), int(W), float(alpha), _ptr(h), _ptr(k_ring),
                                      _ptr(v_ring), _ptr(pos), _ptr(y), _ptr(workspace),
                                      _ws_bytes(workspace), _stream(stream))
    _check(st, "lizard_decode_step")


def lizard_chunk_cumsum(units: int, L: int, dk: int, chunk: int, log_gamma, b, gamma_chunk=None,
                        stream=None):
    st = library().lizard_chunk_cumsum(int(units), int(L), int(dk), int(chunk), _ptr(log_gamma),
                                       _ptr(b), _ptr(gamma_chunk), _stream(stream))
    _check(st, "lizard_chunk_cumsum")


def lizard_trace_enable(enable: bool = True):
    """Turn per-kernel event timing on or off for the calling host thread."""
    _check(library().lizard_trace_enable(1 if enable else 0), "lizard_trace_enable")


def lizard_trace_read(max_records: int = 4096):
    """Wait for the traced kernels and return [(kernel_name, milliseconds), ...]."""
    name_len = 64
    names = ctypes.create_string_buffer(name_len * max_records)
    ms = (ctypes.c_float * max_records)()
    n = library().lizard_trace_read(names, name_len, ms, max_records)
    raw = names.raw
    return [(raw[i * name_len:(i + 1) * name_len].split(b"\0", 1)[0].decode(), float(ms[i]))
            for i in range(n)]


def lizard_decode_step_noalloc(dims: lizard_decode_dims, phi_q, phi_k, v, log_gamma, q, k,
                               meta_k, meta_v, W: int, alpha: float, h, k_ring, v_ring, pos, y,
                               stream=None):
    """lizard_decode_step without a workspace, for callers that cannot allocate device
    memory: the library's own fixed device array holds the per-sequence counters (N at
    most LIZARD_NOALLOC_MAX_SEQUENCES).  Calls that overlap on the GPU race on that array."""
    st = library().lizard_decode_step_noalloc(ctypes.byref(dims), _ptr(phi_q), _ptr(phi_k),
                                              _ptr(v), _ptr(log_gamma), _ptr(q), _ptr(k),
                                              _ptr(meta_k), _ptr(meta_v), int(W), float(alpha),
                                              _ptr(h), _ptr(k_ring), _ptr(v_ring), _ptr(pos),
                                              _ptr(y), _stream(stream))
    _check(st, "lizard_decode_step_noalloc")


def lizard_attn_fwd_bwd_host(dims: lizard_dims, phi_q, phi_k, v, log_gamma, q, k, meta_k, meta_v,
                             W: int, alpha: float, h0, dy, y, h_final, d_phi_q, d_phi_k, d_v,
                             d_log_gamma, d_q, d_k, d_meta_k, d_meta_v, d_h0, workspace,
                             stream=None):
    """Forward + backward with every tensor in host memory (CPU tensors, pinned for overlap);
    ``workspace`` is a device tensor of lizard_fwd_bwd_host_workspace_bytes bytes.  Returns
    once the work is queued; synchronise the stream before reading the outputs."""
    st = library().lizard_attn_fwd_bwd_host(
        ctypes.byref(dims), _ptr(phi_q), _ptr(phi_k), _ptr(v), _ptr(log_gamma), _ptr(q), _ptr(k),
        _ptr(meta_k), _ptr(meta_v), int(W), float(alpha), _ptr(h0), _ptr(dy), _ptr(y),
        _ptr(h_final), _ptr(d_phi_q), _ptr(d_phi_k), _ptr(d_v), _ptr(d_log_gamma), _ptr(d_q),
        _ptr(d_k), _ptr(d_meta_k), _ptr(d_meta_v), _ptr(d_h0), _ptr(workspace),
        _ws_bytes(workspace), _stream(stream))
    _check(st, "lizard_attn_fwd_bwd_host")


def lizard_decode_ring_fill(dims: lizard_decode_dims, L: int, W: int, k, v, k_ring, v_ring, pos,
                            stream=None):
    """Fills the decode rings and positions from a prefill's last W keys and values."""
    st = library().lizard_decode_ring_fill(ctypes.byref(dims), int(L), int(W), _ptr(k), _ptr(v),
                                           _ptr(k_ring), _ptr(v_ring), _ptr(pos), _stream(stream))
    _check(st, "lizard_decode_ring_fill")


def lizard_state_combine(units: int, dk: int, dv: int, gamma_a, h_a, gamma_b, h_b, gamma_out,
                         h_out, stream=None):
    """(gamma_out, h_out) = (gamma_a, h_a) o (gamma_b, h_b): segment a followed by segment b."""
    st = library().lizard_state_combine(int(units), int(dk), int(dv), _ptr(gamma_a), _ptr(h_a),
                                        _ptr(gamma_b), _ptr(h_b), _ptr(gamma_out), _ptr(h_out),
                                        _stream(stream))
    _check(st, "lizard_state_combine")


def lizard_feature_map_workspace_bytes(dims: lizard_fmap_dims, is_bwd: bool) -> int:
    return int(library().lizard_feature_map_workspace_bytes(ctypes.byref(dims), int(bool(is_bwd))))


def lizard_feature_map_fwd(dims: lizard_fmap_dims, x, w, phi, workspace, stream=None):
    """phi = [exp(x W), exp(-x W)] per head (Hedgehog feature map)."""
    st = library().lizard_feature_map_fwd(ctypes.byref(dims), _ptr(x), _ptr(w), _ptr(phi),
                                          _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    _check(st, "lizard_feature_map_fwd")


def lizard_feature_map_bwd(dims: lizard_fmap_dims, x, w, d_phi, d_x, d_w, workspace, stream=None):
    """Gradients of the feature map: d_x [B,H,L,D] and d_w [H,D,F] (fp32)."""
    st = library().lizard_feature_map_bwd(ctypes.byref(dims), _ptr(x), _ptr(w), _ptr(d_phi),
                                          _ptr(d_x), _ptr(d_w), _ptr(workspace), _ws_bytes(workspace),
                                          _stream(stream))
    _check(st, "lizard_feature_map_bwd")


def lizard_attn_fwd_fmap(dims: lizard_dims, x_q, x_k, w_q, w_k, v, log_gamma, q, k, meta_k,
                         meta_v, W: int, alpha: float, y, h0, h_final, workspace, stream=None):
    """Forward pass from the raw projections with the Hedgehog feature map fused into the
    log-space gate absorption (phi is never formed)."""
    st = library().lizard_attn_fwd_fmap(
        ctypes.byref(dims), _ptr(x_q), _ptr(x_k), _ptr(w_q), _ptr(w_k), _ptr(v), _ptr(log_gamma),
        _ptr(q), _ptr(k), _ptr(meta_k), _ptr(meta_v), int(W), float(alpha), _ptr(y), _ptr(h0),
        _ptr(h_final), _ptr(workspace), _ws_bytes(workspace), _stream(stream))
    _check(st, "lizard_attn_fwd_fmap")


# ------------------------------------------------------------------------------------
# rotary positions, the 8-bit paged cache and the attention over it
# ------------------------------------------------------------------------------------
def _rows(t, shape, dtype: int):
    """Pointer and strides (None when contiguous) of a [N,H,T,d] device tensor."""
    if t is None:
        return None, None
    if t.shape != shape or not t.is_cuda or _dtype_code(t) != dtype:
        raise ValueError(f"expected a device tensor of shape {shape} and element type {dtype}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), None
    s = t.stride()
    if s[3] != 1:
        raise ValueError("the channels of a row must be contiguous")
    return t.data_ptr(), ctypes.byref(lizard_strides(s[0], s[1], s[2]))


def _ints(t, shape, size: int):
    """Pointer of a contiguous device tensor of integers of `size` bytes (None -> NULL)."""
    if t is None:
        return None
    if (t.shape != shape or not t.is_cuda or not t.is_contiguous() or t.element_size() != size
            or t.is_floating_point() or t.is_complex()):
        raise ValueError(f"expected a contiguous int{8 * size} device tensor of shape {shape}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _held(x):
    """A handle (None -> NULL) whose tensors are on a device: a host pointer would fault."""
    if x is None:
        return None
    keep = x._keep
    if not (keep[0] if isinstance(keep, tuple) else keep).is_cuda:
        raise ValueError(f"{type(x).__name__}'s tensors must be on the device")
    return ctypes.byref(x)


def _workspace(ws):
    if ws is not None and not ws.is_cuda:
        raise ValueError("the workspace must be on the device")
    return _ptr(ws), _ws_bytes(ws)


def lizard_rope_table(spec: lizard_rope_spec):
    """The rotary table of ``spec`` as an int64 CPU tensor of rot/2 words (64-bit fixed-point
    turns per token); move it to the device and pass it to :class:`lizard_rope`."""
    import torch
    table = torch.zeros(max(spec.rot // 2, 1), dtype=torch.int64)
    _check(library().lizard_rope_table(ctypes.byref(spec), table.data_ptr()), "lizard_rope_table")
    return table


def _rope_call(name, dims, rope, a_q, a_k, positions, b_q, b_k, stream):
    sq = (dims.N, dims.H, dims.T, dims.d)
    sk = (dims.N, dims.Hk, dims.T, dims.d)
    aq, bq = _rows(a_q, sq, dims.dtype), _rows(b_q, sq, dims.dtype)
    ak, bk = _rows(a_k, sk, dims.dtype), _rows(b_k, sk, dims.dtype)
    st = getattr(library(), name)(_ref(dims), _held(rope), *aq, *ak,
                                  _ints(positions, (dims.N, dims.T), 8), *bq, *bk, _stream(stream))
    _check(st, name)


def lizard_rope_fwd(dims: lizard_rope_dims, rope: lizard_rope, x_q, x_k, positions, y_q, y_k,
                    stream=None):
    """Rotates queries [N,H,T,d] and keys [N,Hk,T,d] (or None) into y_q, y_k (which may be
    the inputs); the tensors may be strided."""
    _rope_call("lizard_rope_fwd", dims, rope, x_q, x_k, positions, y_q, y_k, stream)


def lizard_rope_bwd(dims: lizard_rope_dims, rope: lizard_rope, dy_q, dy_k, positions, dx_q, dx_k,
                    stream=None):
    """Gradients of lizard_rope_fwd's inputs from those of its outputs."""
    _rope_call("lizard_rope_bwd", dims, rope, dy_q, dy_k, positions, dx_q, dx_k, stream)


def lizard_cache_workspace_bytes() -> int:
    return library().lizard_cache_workspace_bytes()


def lizard_cache_write(cache: lizard_cache, io: lizard_cache_io, k, v, rope, pos, count, workspace,
                       stream=None):
    """Quantises tokens k, v [N,Hk,T,d] (may be strided) into positions pos[n] + j, j < count[n]
    (None: T) of the cache, the keys rotated first if ``rope`` is given."""
    shape = (cache.N, cache.Hk, io.T, cache.d)
    st = library().lizard_cache_write(
        _held(cache), _ref(io), *_rows(k, shape, io.dtype), *_rows(v, shape, io.dtype), _held(rope),
        _ints(pos, (cache.N,), 8), _ints(count, (cache.N,), 4), *_workspace(workspace),
        _stream(stream))
    _check(st, "lizard_cache_write")


def lizard_cache_read(cache: lizard_cache, io: lizard_cache_io, pos, count, k, v, workspace,
                      stream=None):
    """Values of positions pos[n] + j, j < count[n] (None: T) into k, v [N,Hk,T,d]; other rows 0."""
    shape = (cache.N, cache.Hk, io.T, cache.d)
    st = library().lizard_cache_read(
        _held(cache), _ref(io), _ints(pos, (cache.N,), 8), _ints(count, (cache.N,), 4),
        *_rows(k, shape, io.dtype), *_rows(v, shape, io.dtype),
        *_workspace(workspace), _stream(stream))
    _check(st, "lizard_cache_read")


def lizard_cache_attn_workspace_bytes(cache: lizard_cache, dims: lizard_cache_attn_dims) -> int:
    return library().lizard_cache_attn_workspace_bytes(_ref(cache), _ref(dims))


def lizard_cache_attn(cache: lizard_cache, dims: lizard_cache_attn_dims, q, rope, pos, count, first,
                      meta_k, meta_v, y_add, y, workspace, stream=None):
    """y = y_add + alpha * attention of q [N,H,T,d] over the cache and the meta tokens
    (meta_k, meta_v [H,M,d]); q, y_add and y may be strided, y_add may be None or y."""
    shape = (cache.N, dims.H, dims.T, cache.d)
    for m in (meta_k, meta_v):
        if m is not None and (m.shape != (dims.H, dims.M, cache.d) or not m.is_cuda
                              or _dtype_code(m) != dims.dtype):
            raise ValueError("meta_k and meta_v must be [H, M, d] in the call's element type, on the device")
    st = library().lizard_cache_attn(
        _held(cache), _ref(dims), *_rows(q, shape, dims.dtype), _held(rope), _ints(pos, (cache.N,), 8),
        _ints(count, (cache.N,), 4), _ints(first, (cache.N,), 8), _ptr(meta_k), _ptr(meta_v),
        *_rows(y_add, shape, dims.dtype), *_rows(y, shape, dims.dtype),
        *_workspace(workspace), _stream(stream))
    _check(st, "lizard_cache_attn")
