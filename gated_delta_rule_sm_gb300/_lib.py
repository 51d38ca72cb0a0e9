"""Thin Python binding of the KDA C ABI (``include/kda.h``).

Argument marshalling only: torch provides device memory and the current CUDA
stream, every step of the computation runs in the library's CUDA kernels.
There is no fallback: if ``libkda_gb300.so`` is missing or CUDA is not
available the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda_gb300.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_WORKSPACE = range(6)
KDA_BF16, KDA_FP32 = 0, 1

# Every symbol include/kda.h declares.
EXPORTS = ("kda_fwd_workspace_size", "kda_bwd_workspace_size", "kda_fwd", "kda_fwd_simt", "kda_bwd",
           "kda_status_string", "kda_device_status", "kda_version", "kda_timing_begin", "kda_timing_end",
           "kda_kernel_name", "kda_fwd_noalloc", "kda_saved_size", "kda_fwd_save", "kda_bwd_saved",
           "kda_short_conv_fwd", "kda_short_conv_bwd_workspace_size", "kda_short_conv_bwd",
           "kda_fwd_segmented_workspace_size", "kda_fwd_segmented", "kda_bwd_segmented_workspace_size",
           "kda_bwd_segmented", "kda_selftest_wait_timeout",
           "kda_gated_norm_fwd", "kda_gated_norm_bwd_workspace_size", "kda_gated_norm_bwd",
           "kda_decode_step", "kda_ssm_fwd_workspace_size", "kda_ssm_fwd", "kda_ssm_step",
           "kda_short_conv_prompt", "kda_short_conv_step", "kda_pages_workspace_size", "kda_pages_copy",
           "kda_pages_fork", "kda_pages_extend", "kda_pages_free", "kda_pages_compact")
NOALLOC_SCRATCH_BYTES = 32 << 20
GATES = {"lower_bounded": 0, "softplus": 1}   # kda_gate


class KdaDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("K", ctypes.c_int),
                ("V", ctypes.c_int), ("dtype", ctypes.c_int), ("num_seqs", ctypes.c_int), ("Hk", ctypes.c_int),
                ("gate", ctypes.c_int)]


class SsmDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("G", ctypes.c_int),
                ("N", ctypes.c_int), ("P", ctypes.c_int), ("dtype", ctypes.c_int), ("num_seqs", ctypes.c_int),
                ("x_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64)]


class PagesDims(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int), ("num_pages", ctypes.c_int), ("num_seqs", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("page_tokens", ctypes.c_int), ("page_bytes", ctypes.c_int64),
                ("layer_stride", ctypes.c_int64)]


class KdaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} (status {code})")
        self.code = code


_lock = threading.Lock()
_lib = None
_vp = ctypes.c_void_p


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (build it first with ``gated_delta_rule_sm_gb300.build.build()``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ImportError(f"KDA CUDA library not built: {path} is missing "
                              "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
        lib = ctypes.CDLL(path)
        dims_p = ctypes.POINTER(KdaDims)
        lib.kda_fwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_fwd_workspace_size.argtypes = [dims_p, ctypes.c_int]
        lib.kda_bwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_bwd_workspace_size.argtypes = [dims_p, ctypes.c_int]
        # ... chunk_size, cu_seqlens, cu_seqlens_host, initial_state, out, final_state, workspace, bytes, stream
        fwd_args = [dims_p] + [_vp] * 7 + [ctypes.c_float, ctypes.c_float, ctypes.c_int] + [_vp] * 5 + \
            [_vp, ctypes.c_size_t, _vp]
        for name in ("kda_fwd", "kda_fwd_simt"):
            f = getattr(lib, name)
            f.restype = ctypes.c_int
            f.argtypes = fwd_args
        lib.kda_fwd_segmented_workspace_size.restype = ctypes.c_size_t
        lib.kda_fwd_segmented_workspace_size.argtypes = [dims_p, ctypes.c_int, ctypes.c_int]
        lib.kda_fwd_segmented.restype = ctypes.c_int
        # ... chunk_size, segments, cu_seqlens, cu_seqlens_host, initial_state, out, final_state, ws, bytes, stream
        lib.kda_fwd_segmented.argtypes = [dims_p] + [_vp] * 7 + [ctypes.c_float, ctypes.c_float, ctypes.c_int,
                                                                  ctypes.c_int] + [_vp] * 5 + [_vp, ctypes.c_size_t, _vp]
        gn = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, ctypes.c_float]
        lib.kda_gated_norm_fwd.restype = ctypes.c_int
        lib.kda_gated_norm_fwd.argtypes = gn + [_vp, _vp]
        lib.kda_gated_norm_bwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_gated_norm_bwd_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int]
        lib.kda_gated_norm_bwd.restype = ctypes.c_int
        lib.kda_gated_norm_bwd.argtypes = gn + [_vp] * 4 + [_vp, ctypes.c_size_t, _vp]
        lib.kda_selftest_wait_timeout.restype = ctypes.c_int
        lib.kda_selftest_wait_timeout.argtypes = [_vp]
        lib.kda_fwd_noalloc.restype = ctypes.c_int
        lib.kda_fwd_noalloc.argtypes = [dims_p] + [_vp] * 7 + [ctypes.c_float, ctypes.c_float, ctypes.c_int] + \
            [_vp] * 5 + [_vp]
        lib.kda_bwd.restype = ctypes.c_int
        lib.kda_bwd.argtypes = [dims_p] + [_vp] * 7 + [ctypes.c_float, ctypes.c_float, ctypes.c_int] + \
            [_vp] * 3 + [_vp] * 2 + [_vp] * 8 + [_vp, ctypes.c_size_t, _vp]
        lib.kda_bwd_segmented_workspace_size.restype = ctypes.c_size_t
        lib.kda_bwd_segmented_workspace_size.argtypes = [dims_p, ctypes.c_int, ctypes.c_int]
        lib.kda_bwd_segmented.restype = ctypes.c_int
        lib.kda_bwd_segmented.argtypes = [dims_p] + [_vp] * 7 + [ctypes.c_float, ctypes.c_float, ctypes.c_int,
                                                                  ctypes.c_int] + [_vp] * 3 + [_vp] * 2 + [_vp] * 8 + \
            [_vp, ctypes.c_size_t, _vp]
        lib.kda_saved_size.restype = ctypes.c_size_t
        lib.kda_saved_size.argtypes = [dims_p, ctypes.c_int]
        lib.kda_fwd_save.restype = ctypes.c_int
        lib.kda_fwd_save.argtypes = fwd_args[:-3] + [_vp, ctypes.c_size_t] + fwd_args[-3:]
        lib.kda_bwd_saved.restype = ctypes.c_int
        lib.kda_bwd_saved.argtypes = lib.kda_bwd.argtypes[:-3] + [_vp, ctypes.c_size_t] + lib.kda_bwd.argtypes[-3:]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [ctypes.c_int]
        lib.kda_device_status.restype = ctypes.c_int
        lib.kda_device_status.argtypes = [ctypes.c_int]
        lib.kda_version.restype = ctypes.c_int
        lib.kda_version.argtypes = []
        lib.kda_timing_begin.restype = ctypes.c_int
        lib.kda_timing_begin.argtypes = [ctypes.c_int]
        lib.kda_timing_end.restype = ctypes.c_int
        lib.kda_timing_end.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), ctypes.c_int]
        lib.kda_kernel_name.restype = ctypes.c_char_p
        lib.kda_kernel_name.argtypes = [ctypes.c_int]
        conv = [ctypes.c_int] * 5 + [_vp] * 4 + [ctypes.c_int]
        lib.kda_short_conv_fwd.restype = ctypes.c_int
        lib.kda_short_conv_fwd.argtypes = conv + [_vp, _vp]
        lib.kda_short_conv_bwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_short_conv_bwd_workspace_size.argtypes = [ctypes.c_int] * 4
        lib.kda_short_conv_bwd.restype = ctypes.c_int
        lib.kda_short_conv_bwd.argtypes = conv + [_vp] * 5 + [ctypes.c_size_t, _vp]
        i, i64, sz, f = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        ssm_p, pages_p = ctypes.POINTER(SsmDims), ctypes.POINTER(PagesDims)
        serving = {   # argument types; the two sizes return size_t, the others a status
            "kda_decode_step": [dims_p] + [_vp] * 7 + [f, f, _vp, i] + [_vp] * 4,
            "kda_ssm_fwd_workspace_size": [ssm_p],
            "kda_ssm_fwd": [ssm_p] + [_vp] * 12 + [_vp, sz, _vp],
            "kda_ssm_step": [ssm_p] + [_vp] * 8 + [i] + [_vp] * 4,
            "kda_short_conv_prompt": [i] * 5 + [_vp, i64] + [_vp] * 4 + [i] + [_vp] * 4,
            "kda_short_conv_step": [i] * 4 + [_vp, i64] + [_vp] * 3 + [i] + [_vp] * 4,
            "kda_pages_workspace_size": [pages_p, i],
            "kda_pages_copy": [i, i64, _vp, i64, i, _vp, i64, i, _vp, _vp, i, _vp],
            "kda_pages_fork": [pages_p] + [_vp] * 6 + [i] + [_vp] * 4 + [_vp, sz, _vp],
            "kda_pages_extend": [pages_p] + [_vp] * 5 + [i] + [_vp] * 4 + [_vp, sz, _vp],
            "kda_pages_free": [pages_p] + [_vp] * 4 + [i] + [_vp] * 4,
            "kda_pages_compact": [pages_p] + [_vp] * 6 + [_vp, sz, _vp],
        }
        for name, types in serving.items():
            fn = getattr(lib, name)
            fn.restype = sz if name.endswith("_workspace_size") else i
            fn.argtypes = types
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().kda_status_string(int(code)).decode()


def device_status(reset: bool = True) -> int:
    """The device status word (synchronises the device)."""
    return load().kda_device_status(1 if reset else 0)


def timing_begin(max_launches: int) -> None:
    """Start recording per-kernel CUDA events inside the library (see kda_timing_begin)."""
    _check(load().kda_timing_begin(int(max_launches)), "kda_timing_begin")


def timing_end(cap: int = 1 << 16) -> list[tuple[str, float]]:
    """Stop recording; returns [(kernel name, milliseconds)] in launch order."""
    lib = load()
    ms = (ctypes.c_float * cap)()
    ids = (ctypes.c_int * cap)()
    n = lib.kda_timing_end(ms, ids, cap)
    if n < 0:
        raise KdaError(KDA_ERR_CUDA, "kda_timing_end")
    return [(lib.kda_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(n)]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def host_offsets(cu_seqlens_host, n_expected: Optional[int] = None):
    """A host copy of packed-document offsets as a ctypes int32 array (None stays None).

    Accepts a CPU tensor or any sequence of ints.  ``n_expected``: the entry count the call needs
    (num_seqs + 1); a copy of another length is refused here, since the library reads exactly that
    many entries."""
    if cu_seqlens_host is None:
        return None
    if isinstance(cu_seqlens_host, torch.Tensor):
        if cu_seqlens_host.is_cuda:
            raise ValueError("cu_seqlens_host must live in host memory")
        vals = [int(x) for x in cu_seqlens_host.reshape(-1).tolist()]
    else:
        vals = [int(x) for x in cu_seqlens_host]
    if n_expected is not None and len(vals) != n_expected:
        raise ValueError(f"cu_seqlens_host has {len(vals)} entries, the call needs {n_expected}")
    return (ctypes.c_int32 * len(vals))(*vals)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_FP32
    raise TypeError(f"unsupported activation dtype {t.dtype} (bf16 or fp32)")


def _gate_code(gate: str) -> int:
    if gate not in GATES:
        raise ValueError(f"gate must be one of {sorted(GATES)}, got {gate!r}")
    return GATES[gate]


def make_dims(q: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor],
              gate: str = "lower_bounded") -> KdaDims:
    """Shape of a call: q [B, T, Hk, K] (key heads), v [B, T, H, V] (value heads)."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[-1]
    n = int(cu_seqlens.numel() - 1) if cu_seqlens is not None else 0
    return KdaDims(B, T, H, K, V, _dtype_code(q), n, Hk, _gate_code(gate))


def _check_shapes(q, k, v, g_raw, beta_raw, a_log, dt_bias):
    B, T, Hk, K = q.shape
    if k.shape != q.shape or v.dim() != 4 or tuple(v.shape[:2]) != (B, T):
        raise ValueError("q, k must share [B, T, Hk, K] and v must be [B, T, H, V]")
    H = v.shape[2]
    if H % Hk:
        raise ValueError(f"value heads ({H}) must be a multiple of key heads ({Hk})")
    if tuple(g_raw.shape) != (B, T, H, K) or tuple(beta_raw.shape) != (B, T, H):
        raise ValueError("g_raw must be [B, T, H, K] and beta_raw [B, T, H] (value heads)")
    if a_log.numel() != H or dt_bias.numel() != H * K:
        raise ValueError("a_log must hold H values and dt_bias H * K (value heads)")


class _Workspace:
    """Caches one device workspace per (device, kind); grows on demand."""

    def __init__(self):
        self.buf: dict = {}

    def get(self, device: torch.device, kind: str, nbytes: int) -> torch.Tensor:
        key = (device.index, kind)
        b = self.buf.get(key)
        if b is None or b.numel() < nbytes:
            b = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
            self.buf[key] = b
        return b

    def clear(self):
        self.buf.clear()


workspace_cache = _Workspace()


def _check(code: int, what: str):
    if code != KDA_OK:
        raise KdaError(code, what)


def _contig(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("KDA inputs must be contiguous CUDA tensors")


def forward(q, k, v, g_raw, beta_raw, a_log, dt_bias, *, scale: float, lower_bound: float = -5.0,
            gate: str = "lower_bounded", chunk_size: int = 64, cu_seqlens=None, cu_seqlens_host=None,
            initial_state=None, output_final_state: bool = False, out=None, final_state=None, simt: bool = False,
            saved: Optional[torch.Tensor] = None, segments: int = 0, stream: Optional[torch.cuda.Stream] = None):
    """KDA forward through ``kda_fwd`` (or ``kda_fwd_simt``).  Returns (out, final_state or None).

    ``gate``: "lower_bounded" (g = lower_bound * sigmoid(exp(a_log) * (g_raw + dt_bias))) or
    "softplus" (g = -exp(a_log) * softplus(g_raw + dt_bias), unbounded below).
    ``saved``: a device byte buffer of ``saved_size(...)`` bytes; the forward then runs
    ``kda_fwd_save`` and keeps the per-chunk quantities there for ``backward(..., saved=...)``.
    ``segments`` > 0: run ``kda_fwd_segmented``, the chain cut into pieces of about 1 / segments of a
    row (of the longest possible document with ``cu_seqlens``); for long rows with few rows x heads.
    ``cu_seqlens_host``: optional host copy of ``cu_seqlens`` (CPU tensor or sequence); the library then
    checks the offsets before it launches anything and a bad one raises ``KdaError`` (invalid argument).
    """
    lib = load()
    _contig(q, k, v, g_raw, beta_raw, a_log, dt_bias, cu_seqlens, initial_state)
    _check_shapes(q, k, v, g_raw, beta_raw, a_log, dt_bias)
    dims = make_dims(q, v, cu_seqlens, gate)
    B, T, _, K = q.shape
    H, V = v.shape[2], v.shape[-1]
    N = dims.num_seqs if cu_seqlens is not None else B
    if out is None:
        out = torch.empty((B, T, H, V), dtype=q.dtype, device=q.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    if not output_final_state:
        final_state = None
    st = stream if stream is not None else torch.cuda.current_stream(q.device)
    cu_h = host_offsets(cu_seqlens_host, N + 1 if cu_seqlens is not None else None)
    if segments:
        if saved is not None or simt:
            raise ValueError("segments= runs without saved= or simt=")
        ws_bytes = lib.kda_fwd_segmented_workspace_size(ctypes.byref(dims), int(chunk_size), int(segments))
        ws = workspace_cache.get(q.device, "fwd", ws_bytes)
        code = lib.kda_fwd_segmented(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(beta_raw),
                                     _ptr(a_log), _ptr(dt_bias), float(scale), float(lower_bound), int(chunk_size),
                                     int(segments), _ptr(cu_seqlens), cu_h, _ptr(initial_state), _ptr(out),
                                     _ptr(final_state), _ptr(ws), ctypes.c_size_t(ws.numel()),
                                     ctypes.c_void_p(st.cuda_stream))
        _check(code, "kda_fwd_segmented")
        return out, final_state
    ws_bytes = lib.kda_fwd_workspace_size(ctypes.byref(dims), chunk_size)
    ws = workspace_cache.get(q.device, "fwd", ws_bytes)
    head = (ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(beta_raw), _ptr(a_log),
            _ptr(dt_bias), float(scale), float(lower_bound), int(chunk_size), _ptr(cu_seqlens), cu_h,
            _ptr(initial_state), _ptr(out), _ptr(final_state))
    tail = (_ptr(ws), ctypes.c_size_t(ws.numel()), ctypes.c_void_p(st.cuda_stream))
    if saved is not None:
        if simt:
            raise ValueError("saved= needs the tensor-core forward")
        code = lib.kda_fwd_save(*head, _ptr(saved), ctypes.c_size_t(saved.numel() * saved.element_size()), *tail)
        _check(code, "kda_fwd_save")
        return out, final_state
    fn = lib.kda_fwd_simt if simt else lib.kda_fwd
    code = fn(*head, *tail)
    _check(code, "kda_fwd_simt" if simt else "kda_fwd")
    return out, final_state


def saved_size(q, v, cu_seqlens=None, chunk_size: int = 64, gate: str = "lower_bounded") -> int:
    """Bytes of the buffer ``forward(..., saved=...)`` fills (0: the shape has no saved path)."""
    lib = load()
    dims = make_dims(q, v, cu_seqlens, gate)
    return int(lib.kda_saved_size(ctypes.byref(dims), int(chunk_size)))


def backward(q, k, v, g_raw, beta_raw, a_log, dt_bias, dout, *, scale: float, lower_bound: float = -5.0,
             gate: str = "lower_bounded", chunk_size: int = 64, cu_seqlens=None, cu_seqlens_host=None,
             initial_state=None, dfinal_state=None,
             want_dinitial_state: bool = True, grads: Optional[dict] = None,
             saved: Optional[torch.Tensor] = None, segments: int = 0,
             stream: Optional[torch.cuda.Stream] = None) -> dict:
    """KDA backward through ``kda_bwd``.  Returns a dict of fp32 gradients.

    ``saved``: the buffer a ``forward(..., saved=...)`` on the same inputs filled; the backward then
    runs ``kda_bwd_saved`` and skips rebuilding the per-chunk quantities.
    ``segments`` > 0: run ``kda_bwd_segmented``, both state chains cut into the pieces of
    ``forward(..., segments=...)``.
    """
    lib = load()
    _contig(q, k, v, g_raw, beta_raw, a_log, dt_bias, dout, cu_seqlens, initial_state, dfinal_state)
    _check_shapes(q, k, v, g_raw, beta_raw, a_log, dt_bias)
    dims = make_dims(q, v, cu_seqlens, gate)
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[-1]
    N = dims.num_seqs if cu_seqlens is not None else B
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    if grads is None:
        grads = dict(dq=torch.empty((B, T, Hk, K), **f32), dk=torch.empty((B, T, Hk, K), **f32),
                     dv=torch.empty((B, T, H, V), **f32), dg_raw=torch.empty((B, T, H, K), **f32),
                     dbeta_raw=torch.empty((B, T, H), **f32), da_log=torch.empty((H,), **f32),
                     ddt_bias=torch.empty((H * K,), **f32),
                     dinitial_state=torch.empty((N, H, K, V), **f32) if want_dinitial_state else None)
    if segments and saved is not None:
        raise ValueError("segments= runs without saved=")
    ws_bytes = (lib.kda_bwd_segmented_workspace_size(ctypes.byref(dims), int(chunk_size), int(segments))
                if segments else lib.kda_bwd_workspace_size(ctypes.byref(dims), chunk_size))
    ws = workspace_cache.get(dev, "bwd", ws_bytes)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    cu_h = host_offsets(cu_seqlens_host, N + 1 if cu_seqlens is not None else None)
    head = (ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(beta_raw), _ptr(a_log),
            _ptr(dt_bias), float(scale), float(lower_bound), int(chunk_size), _ptr(cu_seqlens), cu_h,
            _ptr(initial_state), _ptr(dout), _ptr(dfinal_state), _ptr(grads["dq"]), _ptr(grads["dk"]),
            _ptr(grads["dv"]), _ptr(grads["dg_raw"]), _ptr(grads["dbeta_raw"]), _ptr(grads["da_log"]),
            _ptr(grads["ddt_bias"]), _ptr(grads.get("dinitial_state")))
    tail = (_ptr(ws), ctypes.c_size_t(ws.numel()), ctypes.c_void_p(st.cuda_stream))
    if saved is not None:
        code = lib.kda_bwd_saved(*head, _ptr(saved), ctypes.c_size_t(saved.numel() * saved.element_size()), *tail)
        _check(code, "kda_bwd_saved")
        return grads
    if segments:
        # kda_bwd_segmented takes `segments` right after chunk_size
        code = lib.kda_bwd_segmented(*head[:11], int(segments), *head[11:], *tail)
        _check(code, "kda_bwd_segmented")
        return grads
    code = lib.kda_bwd(*head, *tail)
    _check(code, "kda_bwd")
    return grads


def short_conv(x, weight, bias=None, *, cu_seqlens=None, out=None, stream: Optional[torch.cuda.Stream] = None):
    """Causal depthwise short convolution + SiLU through ``kda_short_conv_fwd``.

    x: [B, T, C] (bf16 or fp32); weight: [C, W] fp32; bias: [C] fp32 or None.  Returns y like x.
    """
    lib = load()
    _contig(x, weight, bias, cu_seqlens)
    B, T, C = x.shape
    W = weight.shape[-1]
    if weight.numel() != C * W or (bias is not None and bias.numel() != C):
        raise ValueError("weight must be [C, W] and bias [C]")
    if out is None:
        out = torch.empty_like(x)
    st = stream if stream is not None else torch.cuda.current_stream(x.device)
    n = int(cu_seqlens.numel() - 1) if cu_seqlens is not None else 0
    code = lib.kda_short_conv_fwd(B, T, C, W, _dtype_code(x), _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens),
                                  n, _ptr(out), ctypes.c_void_p(st.cuda_stream))
    _check(code, "kda_short_conv_fwd")
    return out


def short_conv_backward(x, weight, bias, dy, *, cu_seqlens=None, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Reverse mode of :func:`short_conv`: dict(dx [B, T, C], dweight [C, W], dbias [C] or None), fp32."""
    lib = load()
    _contig(x, weight, bias, dy, cu_seqlens)
    B, T, C = x.shape
    W = weight.shape[-1]
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty((B, T, C), **f32), dweight=torch.empty((C, W), **f32),
             dbias=torch.empty((C,), **f32) if bias is not None else None)
    ws = workspace_cache.get(dev, "conv", int(lib.kda_short_conv_bwd_workspace_size(B, T, C, W)))
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    n = int(cu_seqlens.numel() - 1) if cu_seqlens is not None else 0
    code = lib.kda_short_conv_bwd(B, T, C, W, _dtype_code(x), _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens), n,
                                  _ptr(dy), _ptr(g["dx"]), _ptr(g["dweight"]), _ptr(g["dbias"]), _ptr(ws),
                                  ctypes.c_size_t(ws.numel()), ctypes.c_void_p(st.cuda_stream))
    _check(code, "kda_short_conv_bwd")
    return g


def _norm_types(o, *others):
    """The norm kernels read every activation with o's element size and the weight as fp32: refuse
    anything else before it reaches them (a bf16 weight, or a bf16 gate beside fp32 o, would be read
    past its end).  ``others``: gate, weight[, dy]."""
    gate, weight = others[0], others[1]
    acts = [gate] + list(others[2:])
    if any(t.dtype != o.dtype for t in acts):
        raise ValueError(f"gate and dy must have o's dtype ({o.dtype})")
    if weight.dtype != torch.float32:
        raise ValueError(f"weight must be float32, got {weight.dtype}")
    if any(t.device != o.device for t in others):
        raise ValueError("o, gate, weight and dy must be on one device")


def gated_norm(o, gate, weight, *, eps: float = 1e-6, out=None, stream: Optional[torch.cuda.Stream] = None):
    """The output epilogue through ``kda_gated_norm_fwd``: o / sqrt(mean(o^2) + eps) * weight * sigmoid(gate)
    over the last axis.  o, gate: [..., V] (bf16 or fp32, same dtype); weight: [V] fp32.  Returns y like o."""
    lib = load()
    _contig(o, gate, weight)
    if gate.shape != o.shape or weight.numel() != o.shape[-1]:
        raise ValueError("gate must match o, and weight must hold o.shape[-1] values")
    _norm_types(o, gate, weight)
    V = o.shape[-1]
    if out is None:
        out = torch.empty_like(o)
    st = stream if stream is not None else torch.cuda.current_stream(o.device)
    _check(lib.kda_gated_norm_fwd(o.numel() // V, V, _dtype_code(o), _ptr(o), _ptr(gate), _ptr(weight), float(eps),
                                  _ptr(out), ctypes.c_void_p(st.cuda_stream)), "kda_gated_norm_fwd")
    return out


def gated_norm_backward(o, gate, weight, dy, *, eps: float = 1e-6, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Reverse mode through ``kda_gated_norm_bwd``: dict(do, dgate [..., V], dweight [V]), all fp32."""
    lib = load()
    _contig(o, gate, weight, dy)
    if gate.shape != o.shape or dy.shape != o.shape or weight.numel() != o.shape[-1]:
        raise ValueError("gate and dy must match o, and weight must hold o.shape[-1] values")
    _norm_types(o, gate, weight, dy)
    V = o.shape[-1]
    rows = o.numel() // V
    f32 = dict(dtype=torch.float32, device=o.device)
    g = dict(do=torch.empty(o.shape, **f32), dgate=torch.empty(o.shape, **f32), dweight=torch.empty((V,), **f32))
    nb = lib.kda_gated_norm_bwd_workspace_size(rows, V)
    ws = workspace_cache.get(o.device, "norm", nb)
    st = stream if stream is not None else torch.cuda.current_stream(o.device)
    _check(lib.kda_gated_norm_bwd(rows, V, _dtype_code(o), _ptr(o), _ptr(gate), _ptr(weight), float(eps), _ptr(dy),
                                  _ptr(g["do"]), _ptr(g["dgate"]), _ptr(g["dweight"]), _ptr(ws),
                                  ctypes.c_size_t(ws.numel()), ctypes.c_void_p(st.cuda_stream)), "kda_gated_norm_bwd")
    return g


# ---- serving: states carried from prompts to single tokens ----
#
# A step's kernel takes a few microseconds, so these calls keep their own time short: one test per tensor, plain
# integers for pointers, dimension structures kept by their values.

_F32, _I32 = torch.float32, torch.int32
_DTYPE_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}


def _refuse(name: str, t, dtype, shape, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: all tensors of a call must be on one CUDA device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _need(name: str, t, dtype, shape, dev):
    """t's address, once it is a contiguous tensor of the dtype and shape on the device (None: no tensor)."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev):
        _refuse(name, t, dtype, shape, dev)
    return t.data_ptr()


def _first(name: str, t, dims: int):
    """The device index and dtype code of a call's leading tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} axes, got {list(t.shape)}")
    code = _DTYPE_CODES.get(t.dtype)
    return t.get_device(), _dtype_code(t) if code is None else code


@functools.lru_cache(maxsize=4096)
def _token_stride(name: str, shape, strides, lead: int) -> int:
    """Elements between neighbouring tokens of a tensor whose first ``lead`` axes are tokens ([B, T] or [B]) and
    whose other axes are one token's contiguous values: it may be a slice of a wider projection."""
    want = 1
    for k in range(len(shape) - 1, lead - 1, -1):
        if strides[k] != want and shape[k] > 1:
            raise ValueError(f"{name}: the values of one token must be contiguous")
        want *= shape[k]
    step = span = None
    for k in range(lead - 1, -1, -1):
        if shape[k] > 1:
            if step is None:
                step = strides[k]
            elif strides[k] != span:
                raise ValueError(f"{name}: tokens must be evenly spaced over the leading axes")
            span = strides[k] * shape[k]
    return want if step is None else step


def _raw_stream(dev: int, stream) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _empty(like, shape, dtype, stream):
    """A new tensor, allocated for the stream the call runs on."""
    # (half the time of new_empty)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _result(name: str, out, like, dev: int, stream):
    """The output tensor of like's shape and dtype, given or new, and its address."""
    if out is not None:
        return out, _need(name, out, like.dtype, like.shape, dev)
    if stream is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:
        out = _empty(like, like.shape, like.dtype, stream)
    return out, out.data_ptr()


def _scratch(like, dev: int, kind: str, ptr: int, nbytes: int, stream):
    """One workspace per device, kind and stream: calls on different streams may overlap."""
    buf = workspace_cache.buf.get((dev, kind, ptr))
    if buf is None or buf.numel() < nbytes:
        buf = _empty(like, (max(nbytes, 256),), torch.uint8, stream)
        workspace_cache.buf[(dev, kind, ptr)] = buf
    return buf


@functools.lru_cache(maxsize=4096)
def _ssm_layout(lead: int, code: int, n: int, x, xs, b, bs, c, cs, dt, ds):
    """Checks of the shapes and strides of x, b, c and dt_raw: (dims reference, bytes of workspace of the scan, H)."""
    tokens, H = x[:lead], x[lead]
    if len(b) != lead + 2 or b[:lead] != tokens or c != b or dt != x[:lead + 1]:
        raise ValueError("x must be [..., H, P], b and c [..., G, N] and dt_raw [..., H] over the same tokens")
    G = b[lead]
    if G < 1 or H % G:
        raise ValueError(f"heads ({H}) must be a multiple of the groups of b and c ({G})")
    dims = SsmDims(tokens[0], tokens[1] if lead == 2 else 1, H, G, b[-1], x[-1], code, n, _token_stride("x", x, xs, lead),
                   _token_stride("b", b, bs, lead), _token_stride("c", c, cs, lead), _token_stride("dt_raw", dt, ds, lead))
    ref = ctypes.byref(dims)
    return ref, int(load().kda_ssm_fwd_workspace_size(ref)), H


def _ssm_args(x, dt_raw, b, c, a_log, dt_bias, d_skip, lead: int, n: int, dev: int, code: int):
    """Checks of the arguments that the scan and the step share: (dims reference, workspace bytes, addresses)."""
    ref, nbytes, H = _ssm_layout(lead, code, n, x.shape, x.stride(), b.shape, b.stride(), c.shape, c.stride(), dt_raw.shape,
                                 dt_raw.stride())
    dtype = x.dtype
    if b.dtype is not dtype or c.dtype is not dtype or dt_raw.dtype is not dtype:
        raise ValueError("x, b, c and dt_raw must have one dtype")
    if b.get_device() != dev or c.get_device() != dev or dt_raw.get_device() != dev:
        raise ValueError("all tensors of a call must be on one CUDA device")
    per_head = (H,)
    return ref, nbytes, (x.data_ptr(), dt_raw.data_ptr(), b.data_ptr(), c.data_ptr(),
                         _need("a_log", a_log, _F32, per_head, dev), _need("dt_bias", dt_bias, _F32, per_head, dev),
                         _need("d_skip", d_skip, _F32, per_head, dev))


def _offsets(cu_seqlens, cu_seqlens_host, B: int, dev: int):
    """(documents, rows, device address, host copy) of a call's packed-document offsets."""
    if cu_seqlens is None:
        return 0, B, None, host_offsets(cu_seqlens_host)
    n = cu_seqlens.numel() - 1
    return n, n, _need("cu_seqlens", cu_seqlens, _I32, (n + 1,), dev), host_offsets(cu_seqlens_host, n + 1)


def ssm_scan(x, dt_raw, b, c, a_log, dt_bias, d_skip=None, *, cu_seqlens=None, cu_seqlens_host=None,
             initial_state=None, output_final_state: bool = False, out=None, final_state=None,
             stream: Optional[torch.cuda.Stream] = None):
    """Selective state space scan over prompts through ``kda_ssm_fwd``.  Returns (y, final_state or None).

    x [B, T, H, P], b and c [B, T, G, N], dt_raw [B, T, H] (bf16 or fp32, one dtype; slices of a wider
    projection are taken as they are); a_log, dt_bias, d_skip [H] fp32; states [rows, H, N, P] fp32 with
    rows = B, or one per document of ``cu_seqlens`` (int32).
        S_t = exp(D_t a) S_{t-1} + D_t b_t x_t^T,  y_t = S_t^T c_t + d_skip x_t,
        D = softplus(dt_raw + dt_bias), a = -exp(a_log)."""
    lib = _lib or load()
    dev, code = _first("x", x, 4)
    n, rows, cu, cu_h = _offsets(cu_seqlens, cu_seqlens_host, x.shape[0], dev)
    ref, nbytes, args = _ssm_args(x, dt_raw, b, c, a_log, dt_bias, d_skip, 2, n, dev, code)
    state_shape = (rows, x.shape[2], b.shape[3], x.shape[3])
    s0 = _need("initial_state", initial_state, _F32, state_shape, dev)
    st = _raw_stream(dev, stream)
    out, po = _result("out", out, x, dev, stream)
    if not output_final_state:
        final_state = pf = None
    elif final_state is None:
        final_state = _empty(a_log, state_shape, _F32, stream)
        pf = final_state.data_ptr()
    else:
        pf = _need("final_state", final_state, _F32, state_shape, dev)
    ws = _scratch(x, dev, "ssm", st, nbytes, stream)
    _check(lib.kda_ssm_fwd(ref, *args, cu, cu_h, s0, po, pf, ws.data_ptr(), ws.numel(), st), "kda_ssm_fwd")
    return out, final_state


def _pool_args(name: str, pool, slots, B: int, cell, dtype, pool_out, dev: int):
    """Checks of a slot pool [slots, *cell]: (slots address, number of slots, pool address, address written, pool written)."""
    n = pool.shape[0] if pool.dim() else 0
    shape = (n, *cell)
    if pool_out is None:
        pool_out = pool
    return (_need("slots", slots, _I32, (B,), dev), n, _need(name, pool, dtype, shape, dev),
            _need(f"{name}_out", pool_out, dtype, shape, dev)), pool_out


def ssm_step(x, dt_raw, b, c, a_log, dt_bias, d_skip=None, *, state, slots=None, state_out=None, out=None,
             stream: Optional[torch.cuda.Stream] = None):
    """One token per row through ``kda_ssm_step``: x [B, H, P], b, c [B, G, N], dt_raw [B, H].

    ``state`` [slots, H, N, P] fp32 is the pool, row r works on slot ``slots[r]`` (int32; None: slot r; negative:
    the row is idle and gets zeros).  The pool is updated in place, or into ``state_out`` (only the named slots
    are written).  Returns (y, the pool written)."""
    lib = _lib or load()
    dev, code = _first("x", x, 3)
    ref, _, args = _ssm_args(x, dt_raw, b, c, a_log, dt_bias, d_skip, 1, 0, dev, code)
    B, H, P = x.shape
    pool, state_out = _pool_args("state", state, slots, B, (H, b.shape[2], P), _F32, state_out, dev)
    out, po = _result("out", out, x, dev, stream)
    _check(lib.kda_ssm_step(ref, *args, *pool, po, _raw_stream(dev, stream)), "kda_ssm_step")
    return out, state_out


@functools.lru_cache(maxsize=4096)
def _step_dims(*fields):
    dims = KdaDims(*fields)
    return dims, ctypes.byref(dims)


def decode_step(q, k, v, g_raw, beta_raw, a_log, dt_bias, *, scale: float, lower_bound: float = -5.0,
                gate: str = "lower_bounded", state, slots=None, state_out=None, out=None,
                stream: Optional[torch.cuda.Stream] = None):
    """The delta rule for one token per row through ``kda_decode_step``: :func:`forward` at T = 1 on a pool.

    q, k [B, Hk, K], v [B, H, V], g_raw [B, H, K], beta_raw [B, H]; ``state`` [slots, H, K, V] fp32, ``slots``,
    ``state_out`` as for :func:`ssm_step`.  Returns (out, the pool written)."""
    lib = _lib or load()
    dev, code = _first("q", q, 3)
    if v.dim() != 3:
        raise ValueError("v must be [B, H, V]")
    B, Hk, K = q.shape
    H, V = v.shape[1:]
    dtype, key, gates = q.dtype, (B, Hk, K), (B, H, K)
    args = (_need("q", q, dtype, key, dev), _need("k", k, dtype, key, dev), _need("v", v, dtype, (B, H, V), dev),
            _need("g_raw", g_raw, dtype, gates, dev), _need("beta_raw", beta_raw, dtype, (B, H), dev),
            _need("a_log", a_log, _F32, (H,), dev), _need("dt_bias", dt_bias, _F32, (H * K,), dev))
    pool, state_out = _pool_args("state", state, slots, B, (H, K, V), _F32, state_out, dev)
    out, po = _result("out", out, v, dev, stream)
    _, ref = _step_dims(B, 1, H, K, V, code, 0, Hk, _gate_code(gate))
    _check(lib.kda_decode_step(ref, *args, scale, lower_bound, *pool, po, _raw_stream(dev, stream)), "kda_decode_step")
    return out, state_out


def _conv_args(x, weight, bias, dev: int, C: int):
    W = weight.shape[-1]
    return W, (_need("weight", weight, _F32, (C, 1, W) if weight.dim() == 3 else (C, W), dev),
               _need("bias", bias, _F32, (C,), dev))


def short_conv_prompt(x, weight, bias=None, *, cu_seqlens=None, cu_seqlens_host=None, initial_history=None, out=None,
                      final_history=None, stream: Optional[torch.cuda.Stream] = None):
    """:func:`short_conv` with a carried history, through ``kda_short_conv_prompt``.  Returns (y, final_history).

    x [B, T, C] (a slice of a wider projection is taken as it is); histories [rows, W - 1, C] like x, oldest input
    first: the last W - 1 inputs before the row (None: zeros) and at its end."""
    lib = _lib or load()
    dev, code = _first("x", x, 3)
    B, T, C = x.shape
    W, params = _conv_args(x, weight, bias, dev, C)
    n, rows, cu, cu_h = _offsets(cu_seqlens, cu_seqlens_host, B, dev)
    hist = (rows, W - 1, C)
    h0 = _need("initial_history", initial_history, x.dtype, hist, dev)
    out, po = _result("out", out, x, dev, stream)
    if final_history is None:
        final_history = _empty(x, hist, x.dtype, stream)
    _check(lib.kda_short_conv_prompt(B, T, C, W, code, x.data_ptr(), _token_stride("x", x.shape, x.stride(), 2), *params,
                                     cu, cu_h, n, h0, po,
                                     _need("final_history", final_history, x.dtype, hist, dev), _raw_stream(dev, stream)),
           "kda_short_conv_prompt")
    return out, final_history


def short_conv_step(x, weight, bias=None, *, history, slots=None, history_out=None, out=None,
                    stream: Optional[torch.cuda.Stream] = None):
    """One token per row through ``kda_short_conv_step``: x [B, C], ``history`` [slots, W - 1, C] like x; ``slots``
    and ``history_out`` as for :func:`ssm_step`.  Returns (y, the pool written)."""
    lib = _lib or load()
    dev, code = _first("x", x, 2)
    B, C = x.shape
    W, params = _conv_args(x, weight, bias, dev, C)
    pool, history_out = _pool_args("history", history, slots, B, (W - 1, C), x.dtype, history_out, dev)
    out, po = _result("out", out, x, dev, stream)
    _check(lib.kda_short_conv_step(B, C, W, code, x.data_ptr(), _token_stride("x", x.shape, x.stride(), 1), *params, *pool,
                                   po, _raw_stream(dev, stream)), "kda_short_conv_step")
    return out, history_out


@functools.lru_cache(maxsize=4096)
def _pool_layers(name: str, shape, strides, es: int):
    """(layers, pages, bytes of a page, bytes between layers) of a pool [layers, pages, ...]."""
    if len(shape) < 2 or 0 in shape:
        raise ValueError(f"{name} must be [layers, pages, ...]")
    want = 1
    for k in range(len(shape) - 1, 0, -1):
        if strides[k] != want and shape[k] > 1:
            raise ValueError(f"{name}: the pages of a layer must be contiguous")
        want *= shape[k]
    return shape[0], shape[1], want // shape[1] * es, strides[0] * es


@functools.lru_cache(maxsize=4096)
def _pages_dims(n: int, *fields):
    """(the structure, its reference, bytes of workspace for n requests)."""
    dims = PagesDims(*fields)
    ref = ctypes.byref(dims)
    return dims, ref, int(load().kda_pages_workspace_size(ref, n))


def _pages_args(pool, table, lengths, refs, table_out, lengths_out, refs_out, page_tokens: int, n: int):
    """Checks of a cache's arrays: (device, dims reference, workspace bytes, inputs, outputs); lengths may be None."""
    dev = table.get_device()
    if (not table.is_cuda) or table.dim() != 2:
        raise ValueError("table must be a CUDA tensor [sequences, pages of a row]")
    shape = table.shape
    rows, pages = (shape[0],), (refs.numel(),)
    ins = (_need("table", table, _I32, shape, dev), _need("lengths", lengths, _I32, rows, dev),
           _need("refs", refs, _I32, pages, dev))
    outs = (ins[0] if table_out is None else _need("table_out", table_out, _I32, shape, dev),
            ins[1] if lengths_out is None else _need("lengths_out", lengths_out, _I32, rows, dev),
            ins[2] if refs_out is None else _need("refs_out", refs_out, _I32, pages, dev))
    if pool is None:
        layers, page, stride = 1, 1, 0
    else:
        layers, held, page, stride = _pool_layers("pool", pool.shape, pool.stride(), pool.element_size())
        if pool.get_device() != dev:
            raise ValueError("all tensors of a call must be on one CUDA device")
        if held != pages[0]:
            raise ValueError(f"refs must hold one count per page ({held}), got {pages[0]}")
    _, ref, nbytes = _pages_dims(n, layers, pages[0], shape[0], shape[1], int(page_tokens), page, stride)
    return dev, ref, nbytes, ins, outs


def _requests(dev: int, n: int, **named):
    return tuple(_need(name, t, _I32, (n,), dev) for name, t in named.items())


def pages_copy(pool, src, dst, *, src_pool=None, stream: Optional[torch.cuda.Stream] = None):
    """Page ``src[i]`` of ``src_pool`` (default: ``pool``) to page ``dst[i]`` of ``pool`` [layers, pages, ...], every
    layer, through ``kda_pages_copy``.  Pairs out of range are skipped; dst must not repeat nor meet src in one pool."""
    lib = _lib or load()
    src_pool = pool if src_pool is None else src_pool
    dev = pool.get_device()
    if not pool.is_cuda or src_pool.get_device() != dev:
        raise ValueError("both pools must be on one CUDA device")
    layers, pages, page, stride = _pool_layers("pool", pool.shape, pool.stride(), pool.element_size())
    s_layers, s_pages, s_page, s_stride = _pool_layers("src_pool", src_pool.shape, src_pool.stride(),
                                                       src_pool.element_size())
    if layers != s_layers or page != s_page:
        raise ValueError("both pools must have the same layers and page size")
    n = src.numel()
    ps, pd = _requests(dev, n, src=src, dst=dst)
    _check(lib.kda_pages_copy(layers, page, pool.data_ptr(), stride, pages, src_pool.data_ptr(), s_stride, s_pages, ps, pd,
                              n, _raw_stream(dev, stream)), "kda_pages_copy")
    return pool


def pages_fork(pool, table, lengths, refs, parents, children, *, page_tokens: int, table_out=None, lengths_out=None,
               refs_out=None, ok=None, stream: Optional[torch.cuda.Stream] = None):
    """Row ``children[i]`` becomes a copy of row ``parents[i]`` through ``kda_pages_fork``: full pages are shared, a
    partly filled last page is copied into a free one.  pool [layers, pages, ...], table [sequences, M], lengths
    [sequences], refs [pages] int32, updated in place or into the ``*_out`` arrays.  Returns ok [n] int32."""
    lib = _lib or load()
    n = parents.numel()
    dev, ref, nbytes, ins, outs = _pages_args(pool, table, lengths, refs, table_out, lengths_out, refs_out, page_tokens, n)
    req = _requests(dev, n, parents=parents, children=children)
    st = _raw_stream(dev, stream)
    if ok is None:
        ok = _empty(table, (n,), _I32, stream)
    ws = _scratch(table, dev, "pages", st, nbytes, stream)
    _check(lib.kda_pages_fork(ref, pool.data_ptr(), *ins, *req, n, *outs, _need("ok", ok, _I32, (n,), dev), ws.data_ptr(),
                              ws.numel(), st), "kda_pages_fork")
    return ok


def pages_extend(table, lengths, refs, seqs, new_lengths, *, page_tokens: int, table_out=None, lengths_out=None,
                 refs_out=None, ok=None, stream: Optional[torch.cuda.Stream] = None):
    """Row ``seqs[i]`` grows to ``new_lengths[i]`` tokens through ``kda_pages_extend``.  Returns ok [n] int32."""
    lib = _lib or load()
    n = seqs.numel()
    dev, ref, nbytes, ins, outs = _pages_args(None, table, lengths, refs, table_out, lengths_out, refs_out, page_tokens, n)
    req = _requests(dev, n, seqs=seqs, new_lengths=new_lengths)
    st = _raw_stream(dev, stream)
    if ok is None:
        ok = _empty(table, (n,), _I32, stream)
    ws = _scratch(table, dev, "pages", st, nbytes, stream)
    _check(lib.kda_pages_extend(ref, *ins, *req, n, *outs, _need("ok", ok, _I32, (n,), dev), ws.data_ptr(), ws.numel(), st),
           "kda_pages_extend")
    return ok


def pages_free(table, lengths, refs, seqs, *, table_out=None, lengths_out=None, refs_out=None,
               stream: Optional[torch.cuda.Stream] = None):
    """Rows ``seqs`` give up their pages through ``kda_pages_free``."""
    lib = _lib or load()
    n = seqs.numel()
    dev, ref, _, ins, outs = _pages_args(None, table, lengths, refs, table_out, lengths_out, refs_out, 1, n)
    _check(lib.kda_pages_free(ref, *ins, *_requests(dev, n, seqs=seqs), n, *outs, _raw_stream(dev, stream)),
           "kda_pages_free")


def pages_compact(pool, table, refs, *, table_out=None, refs_out=None, page_map=None,
                  stream: Optional[torch.cuda.Stream] = None):
    """Moves the live pages of pool [layers, pages, ...] to the lowest indices through ``kda_pages_compact``; table
    and refs follow.  Returns page_map [pages] int32: the new index of each page, -1 for a free one."""
    lib = _lib or load()
    dev, ref, nbytes, ins, outs = _pages_args(pool, table, None, refs, table_out, None, refs_out, 1, 0)
    st = _raw_stream(dev, stream)
    if page_map is None:
        page_map = _empty(refs, refs.shape, _I32, stream)
    ws = _scratch(table, dev, "pages", st, nbytes, stream)
    _check(lib.kda_pages_compact(ref, pool.data_ptr(), ins[0], ins[2], outs[0], outs[2],
                                 _need("page_map", page_map, _I32, refs.shape, dev), ws.data_ptr(), ws.numel(), st),
           "kda_pages_compact")
    return page_map
