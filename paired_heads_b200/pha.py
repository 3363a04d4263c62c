"""ctypes binding of libpha (include/pha.h, include/pha_sinks.h, include/pha_cache.h). Argument
marshalling only: every step runs in the library's CUDA kernels. Importing this module loads libpha.so and raises if it is missing -- there
is no fallback.

Functions keep the C names. Tensor arguments may be torch tensors (their device pointer is
passed) or plain integers (raw device addresses). ``stream`` defaults to torch's current stream
on the tensors' device. A negative status raises :class:`PhaError`.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpha.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pha.h")
HEADERS = [HEADER] + [os.path.join(os.path.dirname(HERE), "include", n)
                      for n in ("pha_sinks.h", "pha_cache.h")]

PHA_BF16 = 0
PHA_F32 = 1
STATUS = {0: "PHA_OK", -1: "PHA_ERR_INVALID", -2: "PHA_ERR_UNSUPPORTED", -3: "PHA_ERR_WORKSPACE",
          -4: "PHA_ERR_CUDA"}
DEVICE_STATUS = {0: "ok", 1: "malformed cu_seqlens", 2: "work list overflow", 3: "wait timeout",
                 4: "page table entry is no page", 5: "not enough free pages"}


class PhaError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(code, code)} ({msg})")
        self.code = code


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libpha.so is not built ({LIB_PATH}); run `python -m paired_heads_b200.build`")

_lib = ctypes.CDLL(LIB_PATH)
_p = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

_lib.pha_status_string.argtypes = [_i]
_lib.pha_status_string.restype = ctypes.c_char_p
_lib.pha_rope_tables.argtypes = [_p, _p, _i, _i, _i, ctypes.c_double, _p]
_lib.pha_rope.argtypes = [_p, _p, _p, _p, _i, _i, _p, _i, _i, _i, _i, _i, _i, _i, _p]
_lib.pha_attn_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
_lib.pha_attn_workspace_bytes.restype = _sz
_lib.pha_attn_fwd.argtypes = [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                              ctypes.c_float, _p, _p, _p, _sz, _p]
_lib.pha_attn_status.argtypes = [_p, ctypes.POINTER(_i), ctypes.POINTER(_i), _p]
_lib.pha_attn_fwd_noalloc.argtypes = [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                      ctypes.c_float, _p, _p, _p]
_lib.pha_attn_fwd_fp8.argtypes = [_p, _p, _p, ctypes.c_float, ctypes.c_float, ctypes.c_float, _p,
                                  _i, _i, _i, _i, _i, _i, _i, _i, _i, ctypes.c_float, _p, _p, _p,
                                  _sz, _p]
_lib.pha_test_attn_fwd_stalled.argtypes = [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                           _i, ctypes.c_float, _p, _p, _p, _sz, _i, _p]
_lib.pha_attn_fwd_aux_v.argtypes = [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                    ctypes.c_float, _p, _p, _p, _sz, _p]
_lib.pha_rope_bwd.argtypes = [_p, _p, _p, _p, _i, _i, _p, _i, _i, _i, _i, _i, _i, _i, _p]
_lib.pha_attn_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.pha_attn_bwd_workspace_bytes.restype = _sz
_lib.pha_attn_bwd.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                              _i, ctypes.c_float, _p, _p, _p, _p, _sz, _p]
_lib.pha_qk_norm_rope.argtypes = [_p, _p, _p, _p, ctypes.c_float, _p, _p, _i, _i, _p, _i, _i, _i,
                                  _i, _i, _i, _i, _p]
_lib.pha_rope_factor_bytes.argtypes = [_i, _i, _i]
_lib.pha_rope_factor_bytes.restype = _sz
_lib.pha_rope_factor_tables.argtypes = [_p, _sz, _i, _i, _i, ctypes.c_double, _p]
_lib.pha_rope_factored.argtypes = [_p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i, _p]
_lib.pha_rope_bwd_factored.argtypes = [_p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i, _p]
_lib.pha_qk_norm_rope_factored.argtypes = [_p, _p, _p, _p, ctypes.c_float, _p, _i, _p, _i, _i, _i,
                                           _i, _i, _i, _i, _p]
_f32 = ctypes.c_float
_lib.pha_attn_sinks_workspace_bytes.argtypes = [_i] * 8
_lib.pha_attn_sinks_workspace_bytes.restype = _sz
_lib.pha_attn_sinks_bwd_workspace_bytes.argtypes = [_i] * 9
_lib.pha_attn_sinks_bwd_workspace_bytes.restype = _sz
_lib.pha_attn_sinks_fwd.argtypes = [_p] * 4 + [_i] * 10 + [_f32, _p, _p, _p, _sz, _p]
_lib.pha_attn_sinks_bwd.argtypes = [_p] * 7 + [_i] * 10 + [_f32, _p, _p, _p, _p, _sz, _p]
_lib.pha_attn_paged_workspace_bytes.argtypes = [_i] * 11
_lib.pha_attn_paged_workspace_bytes.restype = _sz
_lib.pha_attn_paged_fwd.argtypes = [_p] * 4 + [_i] * 3 + [_p, _p] + [_i] * 11 + [_f32, _p, _p, _p,
                                                                               _sz, _p, _p]
_lib.pha_test_attn_sinks_fwd_stalled.argtypes = [_p] * 4 + [_i] * 10 + [_f32, _p, _p, _p, _sz, _i, _p]
_lib.pha_test_attn_sinks_bwd_stalled.argtypes = [_p] * 7 + [_i] * 10 + [_f32, _p, _p, _p, _p, _sz, _i, _p]
_lib.pha_test_attn_paged_fwd_stalled.argtypes = [_p] * 4 + [_i] * 3 + [_p, _p] + [_i] * 11 + [
    _f32, _p, _p, _p, _sz, _p, _i, _p]
_lib.pha_cache_append.argtypes = [_p] * 5 + [_i] * 3 + [_p, _p] + [_i] * 5 + [_p, _p]
_lib.pha_cache_workspace_bytes.argtypes = [_i, _i]
_lib.pha_cache_workspace_bytes.restype = _sz
_lib.pha_cache_fork.argtypes = [_p, _i, _p, _i, _p, _i, _p, _p, _i, _p, _sz, _p, _p]
_lib.pha_cache_reserve.argtypes = [_p, _i, _p, _i, _p, _i, _i, _p, _p, _i, _p, _p, _i, _sz, _p, _sz,
                                   _p, _p]
_lib.pha_cache_free.argtypes = [_p, _i, _p, _i, _p, _i, _p, _i, _p, _sz, _p, _p]
_lib.pha_cache_trim.argtypes = [_p, _i, _p, _i, _p] + [_i] * 5 + [_p, _p]
_lib.pha_cache_compact.argtypes = [_p, _i, _i, _p, _i, _p, _p, _i, _sz, _p, _sz, _p, _p]
for _f in ("pha_attn_sinks_fwd", "pha_attn_sinks_bwd", "pha_attn_paged_fwd", "pha_cache_append",
           "pha_cache_fork", "pha_cache_reserve", "pha_cache_free", "pha_cache_trim",
           "pha_cache_compact", "pha_test_attn_sinks_fwd_stalled", "pha_test_attn_sinks_bwd_stalled",
          "pha_test_attn_paged_fwd_stalled"):
    getattr(_lib, _f).restype = _i
for _f in ("pha_rope_tables", "pha_rope", "pha_attn_fwd", "pha_attn_status",
           "pha_attn_fwd_noalloc", "pha_test_attn_fwd_stalled", "pha_attn_fwd_fp8", "pha_qk_norm_rope", "pha_attn_fwd_aux_v", "pha_rope_bwd",
           "pha_attn_bwd", "pha_rope_factor_tables", "pha_rope_factored", "pha_rope_bwd_factored",
           "pha_qk_norm_rope_factored"):
    getattr(_lib, _f).restype = _i


def exported_symbols() -> list:
    """Names of the functions the headers declare."""
    names = set()
    for path in HEADERS:
        with open(path) as f:
            text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
        names.update(re.findall(r"^\s*(?:const\s+)?[\w\s\*]+?\b(pha_\w+)\s*\(", text, re.M))
    return sorted(names)


def library():
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream, *tensors):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch

    for t in tensors:
        if t is not None and not isinstance(t, int) and t.is_cuda:
            return torch.cuda.current_stream(t.device).cuda_stream
    return torch.cuda.current_stream().cuda_stream


def _check(fn: str, rc: int):
    if rc != 0:
        raise PhaError(fn, rc, _lib.pha_status_string(rc).decode())


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return PHA_BF16
    if t.dtype == torch.float32:
        return PHA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def pha_status_string(code: int) -> str:
    return _lib.pha_status_string(code).decode()


def pha_rope_tables(cos_tab, sin_tab, rows: int, head_dim: int, paired: bool, base: float = 10000.0,
                    stream=None):
    _check("pha_rope_tables", _lib.pha_rope_tables(_ptr(cos_tab), _ptr(sin_tab), rows, head_dim,
                                                   int(paired), float(base),
                                                   _stream(stream, cos_tab)))


def pha_rope(q, k, cos_tab, sin_tab, positions, paired: bool = False, stagger_offset: int = 0,
             stream=None, *, tab_rows=None, tab_width=None, total_tokens=None, n_heads=None,
             n_kv_heads=None, head_dim=None, dtype=None):
    """In-place RoPE of q [T][H][hd] and k [T][Hkv][hd]. Shapes are taken from the tensors unless
    given explicitly (needed when raw addresses are passed)."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = q.shape
        n_kv_heads = 0 if k is None else k.shape[1]
        tab_rows, tab_width = cos_tab.shape
        dtype = _dtype_code(q)
    _check("pha_rope", _lib.pha_rope(_ptr(q), _ptr(k), _ptr(cos_tab), _ptr(sin_tab), tab_rows,
                                     tab_width, _ptr(positions), total_tokens, n_heads, n_kv_heads,
                                     head_dim, dtype, int(paired), stagger_offset,
                                     _stream(stream, q)))


def pha_qk_norm_rope(q, k, cos_tab, sin_tab, positions, q_weight=None, k_weight=None,
                     eps: float = 1e-6, paired: bool = False, stagger_offset: int = 0, stream=None,
                     *, tab_rows=None, tab_width=None, total_tokens=None, n_heads=None,
                     n_kv_heads=None, head_dim=None, dtype=None):
    """In-place QK RMS-norm (per head row, optional float32 weights of length head_dim) followed
    by RoPE of q [T][H][hd] and k [T][Hkv][hd]."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = q.shape
        n_kv_heads = 0 if k is None else k.shape[1]
        tab_rows, tab_width = cos_tab.shape
        dtype = _dtype_code(q)
    _check("pha_qk_norm_rope",
           _lib.pha_qk_norm_rope(_ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), float(eps),
                                 _ptr(cos_tab), _ptr(sin_tab), tab_rows, tab_width, _ptr(positions),
                                 total_tokens, n_heads, n_kv_heads, head_dim, dtype, int(paired),
                                 stagger_offset, _stream(stream, q)))


def pha_rope_bwd(dq, dk, cos_tab, sin_tab, positions, paired: bool = False, stagger_offset: int = 0,
                 stream=None, *, tab_rows=None, tab_width=None, total_tokens=None, n_heads=None,
                 n_kv_heads=None, head_dim=None, dtype=None):
    """In place: gradients with respect to the rotated q, k -> with respect to the unrotated ones."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = dq.shape
        n_kv_heads = 0 if dk is None else dk.shape[1]
        tab_rows, tab_width = cos_tab.shape
        dtype = _dtype_code(dq)
    _check("pha_rope_bwd", _lib.pha_rope_bwd(_ptr(dq), _ptr(dk), _ptr(cos_tab), _ptr(sin_tab),
                                             tab_rows, tab_width, _ptr(positions), total_tokens,
                                             n_heads, n_kv_heads, head_dim, dtype, int(paired),
                                             stagger_offset, _stream(stream, dq)))


def pha_rope_factor_bytes(rows: int, head_dim: int, paired: bool) -> int:
    return int(_lib.pha_rope_factor_bytes(rows, head_dim, int(paired)))


def pha_rope_factor_tables(factors, rows: int, head_dim: int, paired: bool,
                           base: float = 10000.0, stream=None, *, nbytes=None):
    """Factored rotary tables for table rows [0, rows) into the device buffer `factors`."""
    if nbytes is None:
        nbytes = factors.numel() * factors.element_size()
    _check("pha_rope_factor_tables",
           _lib.pha_rope_factor_tables(_ptr(factors), nbytes, rows, head_dim, int(paired),
                                       float(base), _stream(stream, factors)))


def _rope_shape(q, k):
    total_tokens, n_heads, head_dim = q.shape
    return total_tokens, n_heads, 0 if k is None else k.shape[1], head_dim, _dtype_code(q)


def pha_rope_factored(q, k, factors, rows: int, positions, paired: bool = False,
                      stagger_offset: int = 0, stream=None):
    """pha_rope with factored tables (pha_rope_factor_tables for `rows` rows)."""
    t, h, hkv, hd, dt = _rope_shape(q, k)
    _check("pha_rope_factored",
           _lib.pha_rope_factored(_ptr(q), _ptr(k), _ptr(factors), rows, _ptr(positions), t, h,
                                  hkv, hd, dt, int(paired), stagger_offset, _stream(stream, q)))


def pha_qk_norm_rope_factored(q, k, factors, rows: int, positions, q_weight=None, k_weight=None,
                              eps: float = 1e-6, paired: bool = False, stagger_offset: int = 0,
                              stream=None):
    """pha_qk_norm_rope with factored tables."""
    t, h, hkv, hd, dt = _rope_shape(q, k)
    _check("pha_qk_norm_rope_factored",
           _lib.pha_qk_norm_rope_factored(_ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                          float(eps), _ptr(factors), rows, _ptr(positions), t, h,
                                          hkv, hd, dt, int(paired), stagger_offset,
                                          _stream(stream, q)))


def pha_rope_bwd_factored(dq, dk, factors, rows: int, positions, paired: bool = False,
                          stagger_offset: int = 0, stream=None):
    """pha_rope_bwd with factored tables."""
    t, h, hkv, hd, dt = _rope_shape(dq, dk)
    _check("pha_rope_bwd_factored",
           _lib.pha_rope_bwd_factored(_ptr(dq), _ptr(dk), _ptr(factors), rows, _ptr(positions), t,
                                      h, hkv, hd, dt, int(paired), stagger_offset,
                                      _stream(stream, dq)))


def pha_attn_bwd_workspace_bytes(batch: int, max_len: int, total_tokens: int, n_heads: int,
                                 head_dim: int, paired: bool) -> int:
    return int(_lib.pha_attn_bwd_workspace_bytes(batch, max_len, total_tokens, n_heads, head_dim,
                                                 int(paired)))


def pha_attn_bwd(q, k, v, o, lse, dout, cu_seqlens, max_len: int, dq, dk, dv, workspace, *,
                 causal: bool = True, window: int = 0, paired: bool = False, scale: float = 0.0,
                 stream=None, batch=None, total_tokens=None, n_heads=None, n_kv_heads=None,
                 head_dim=None, dtype=None, workspace_bytes=None):
    """Backward of pha_attn_fwd (o, lse: its outputs): writes dq, dk, dv for the upstream
    gradient dout."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = q.shape
        n_kv_heads = k.shape[1]
        batch = cu_seqlens.shape[0] - 1
        dtype = _dtype_code(q)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pha_attn_bwd",
           _lib.pha_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                             _ptr(cu_seqlens), batch, max_len, total_tokens, n_heads, n_kv_heads,
                             head_dim, dtype, int(causal), int(window), int(paired), float(scale),
                             _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes,
                             _stream(stream, q)))


def pha_attn_workspace_bytes(batch: int, max_len: int, n_heads: int, head_dim: int,
                             paired: bool) -> int:
    return int(_lib.pha_attn_workspace_bytes(batch, max_len, n_heads, head_dim, int(paired)))


def pha_attn_fwd(q, k, v, cu_seqlens, max_len: int, o, lse, workspace, *, causal: bool = True,
                 window: int = 0, paired: bool = False, scale: float = 0.0, stream=None,
                 batch=None, total_tokens=None, n_heads=None, n_kv_heads=None, head_dim=None,
                 dtype=None, workspace_bytes=None):
    """Varlen attention forward into o (like q) and lse [T][H] float32 (or None)."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = q.shape
        n_kv_heads = k.shape[1]
        batch = cu_seqlens.shape[0] - 1
        dtype = _dtype_code(q)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pha_attn_fwd", _lib.pha_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), batch,
                                             max_len, total_tokens, n_heads, n_kv_heads, head_dim,
                                             dtype, int(causal), int(window), int(paired),
                                             float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
                                             workspace_bytes, _stream(stream, q)))


def pha_attn_fwd_aux_v(q, k, v, aux_v, cu_seqlens, max_len: int, o, lse, workspace, *,
                       causal: bool = True, window: int = 0, paired: bool = False,
                       scale: float = 0.0, stream=None, batch=None, total_tokens=None,
                       n_heads=None, n_kv_heads=None, head_dim=None, dtype=None,
                       workspace_bytes=None):
    """Varlen attention forward over (q, k, v + aux_v) into o and lse (v, aux_v unchanged)."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = q.shape
        n_kv_heads = k.shape[1]
        batch = cu_seqlens.shape[0] - 1
        dtype = _dtype_code(q)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pha_attn_fwd_aux_v",
           _lib.pha_attn_fwd_aux_v(_ptr(q), _ptr(k), _ptr(v), _ptr(aux_v), _ptr(cu_seqlens), batch,
                                   max_len, total_tokens, n_heads, n_kv_heads, head_dim, dtype,
                                   int(causal), int(window), int(paired), float(scale), _ptr(o),
                                   _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream, q)))


def pha_attn_fwd_noalloc(q, k, v, cu_seqlens, max_len: int, o, lse, *, causal: bool = True,
                         window: int = 0, paired: bool = False, scale: float = 0.0, stream=None,
                         batch=None, total_tokens=None, n_heads=None, n_kv_heads=None,
                         head_dim=None, dtype=None):
    """pha_attn_fwd with the library's built-in 1 MiB scratch instead of a workspace (for callers
    that cannot allocate device memory; calls that can overlap on the GPU must be ordered)."""
    if total_tokens is None:
        total_tokens, n_heads, head_dim = q.shape
        n_kv_heads = k.shape[1]
        batch = cu_seqlens.shape[0] - 1
        dtype = _dtype_code(q)
    _check("pha_attn_fwd_noalloc",
           _lib.pha_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), batch, max_len,
                                     total_tokens, n_heads, n_kv_heads, head_dim, dtype,
                                     int(causal), int(window), int(paired), float(scale), _ptr(o),
                                     _ptr(lse), _stream(stream, q)))


def pha_attn_fwd_fp8(q8, k8, v8, q_scale: float, k_scale: float, v_scale: float, cu_seqlens,
                     max_len: int, o, lse, workspace, *, causal: bool = True, window: int = 0,
                     paired: bool = False, scale: float = 0.0, stream=None):
    """Attention forward over e4m3 q8, k8, v8 (torch.float8_e4m3fn or uint8 tensors) with
    per-tensor scales, into o (bf16, q's shape) and lse [T][H] float32 (or None)."""
    total_tokens, n_heads, head_dim = q8.shape
    _check("pha_attn_fwd_fp8",
           _lib.pha_attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), float(q_scale), float(k_scale),
                                 float(v_scale), _ptr(cu_seqlens), cu_seqlens.shape[0] - 1,
                                 max_len, total_tokens, n_heads, k8.shape[1], head_dim,
                                 int(causal), int(window), int(paired), float(scale), _ptr(o),
                                 _ptr(lse), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream, q8)))


def pha_test_attn_fwd_stalled(q, k, v, cu_seqlens, max_len: int, o, lse, workspace, stall_us: int,
                              *, causal: bool = True, window: int = 0, paired: bool = False,
                              scale: float = 0.0, stream=None):
    """Failure-detection test hook: pha_attn_fwd whose band-kernel softmax first waits stall_us
    microseconds on a barrier nothing signals (device status 3 afterwards, no output written)."""
    total_tokens, n_heads, head_dim = q.shape
    _check("pha_test_attn_fwd_stalled",
           _lib.pha_test_attn_fwd_stalled(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens),
                                          cu_seqlens.shape[0] - 1, max_len, total_tokens, n_heads,
                                          k.shape[1], head_dim, _dtype_code(q), int(causal),
                                          int(window), int(paired), float(scale), _ptr(o),
                                          _ptr(lse), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          int(stall_us), _stream(stream, q)))


def pha_attn_status(workspace, stream=None):
    """(device status, scheduled work items) recorded in the workspace; synchronises."""
    st, n = _i(0), _i(0)
    _check("pha_attn_status", _lib.pha_attn_status(_ptr(workspace), ctypes.byref(st),
                                                   ctypes.byref(n), _stream(stream, workspace)))
    return st.value, n.value


# ---------------------------------------------------------------- sinks and the paged cache
#
# These take torch tensors only, and check what the C side cannot see: types, shapes, devices and
# that the elements are contiguous. A tensor on another device than the current one is fine: the
# call is made on the tensor's device.

_torch = None
_raw_stream = None


def _lazy_torch():
    global _torch, _raw_stream
    if _torch is None:
        import torch

        # (building a torch Stream object to ask for its handle takes 3 us of every call)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    return _torch


def _explain(fn, index, name, t, dtype, shape):
    """Raises what is wrong with a tensor that _run found wanting."""
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {name}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name}: not contiguous")
    raise ValueError(f"{fn}: {name}: on {t.device}, others on device {index}")


def _run(fn, wanted, args, stream):
    """Calls the library. wanted: (name, tensor, dtype, shape) of each tensor argument (the first one's
    device is everybody's); None for one that is left out."""
    index = wanted[0][1].get_device()
    for w in wanted:
        if w is not None:
            t = w[1]
            if (t.dtype is not w[2] or t.shape != w[3] or not t.is_contiguous()
                    or t.get_device() != index):
                _explain(fn, index, *w)
    if index < 0:
        raise ValueError(f"{fn}: tensors not on a CUDA device")
    cuda = _lazy_torch().cuda
    if cuda.current_device() != index:
        with cuda.device(index):
            return _check(fn, getattr(_lib, fn)(*args, _stream(stream, wanted[0][1])))
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    rc = getattr(_lib, fn)(*args, stream)
    if rc != 0:
        _check(fn, rc)


def _scratch(workspace):
    """What _run wants of a workspace: contiguous bytes of any type and shape, on the device."""
    return ("workspace", workspace, workspace.dtype, workspace.shape)


def _status(status):
    return None if status is None else ("status", status, _int32(), (1,))


def _int32():
    return _lazy_torch().int32


def _dims(q, k):
    """(tokens, heads, kv heads, head_dim, dtype, dtype code) of a call."""
    dt = q.dtype
    t, h, hd = q.shape
    return t, h, k.shape[-2], hd, dt, PHA_BF16 if dt is _lazy_torch().bfloat16 else _dtype_code(q)


def _nbytes(t) -> int:
    return t.nbytes


_MOST = 2 ** 31


def _cut(*counts):
    """Counts of slots within the C side's 32 bits. ctypes would wrap them without a word (a window of 2^32 + 5
    would be one of 5); the nearest count that fits means the same or is refused by the library."""
    return [max(-_MOST, min(x, _MOST - 1)) for x in counts]


def pha_attn_sinks_workspace_bytes(batch: int, max_len: int, n_heads: int, n_kv_heads: int,
                                   head_dim: int, *, window: int, sinks: int,
                                   paired: bool = False) -> int:
    if not (-_MOST <= window < _MOST and -_MOST <= sinks < _MOST):
        window, sinks = _cut(window, sinks)
    return int(_lib.pha_attn_sinks_workspace_bytes(batch, max_len, n_heads, n_kv_heads, head_dim,
                                                   window, sinks, int(paired)))


def pha_attn_sinks_bwd_workspace_bytes(batch: int, max_len: int, total_tokens: int, n_heads: int,
                                       n_kv_heads: int, head_dim: int, *, window: int, sinks: int,
                                       paired: bool = False) -> int:
    if not (-_MOST <= window < _MOST and -_MOST <= sinks < _MOST):
        window, sinks = _cut(window, sinks)
    return int(_lib.pha_attn_sinks_bwd_workspace_bytes(batch, max_len, total_tokens, n_heads,
                                                       n_kv_heads, head_dim, window, sinks,
                                                       int(paired)))


def pha_attn_sinks_fwd(q, k, v, cu_seqlens, max_len: int, o, lse, workspace, *, window: int,
                       sinks: int, paired: bool = False, scale: float = 0.0, stream=None):
    """Causal varlen attention with a sliding window and `sinks` visible first slots per document,
    into o (like q) and lse [T][H] float32 (or None). pha_attn_status(workspace) reports."""
    if not (-_MOST <= window < _MOST and -_MOST <= sinks < _MOST):
        window, sinks = _cut(window, sinks)
    t, h, hkv, hd, dt, code = _dims(q, k)
    n = cu_seqlens.shape[0]
    _run("pha_attn_sinks_fwd",
         (("q", q, dt, (t, h, hd)), ("k", k, dt, (t, hkv, hd)), ("v", v, dt, (t, hkv, hd)),
          ("cu_seqlens", cu_seqlens, _int32(), (n,)), ("o", o, dt, (t, h, hd)),
          None if lse is None else ("lse", lse, _torch.float32, (t, h)), _scratch(workspace)),
         (q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), n - 1, max_len, t, h,
          hkv, hd, code, window, sinks, paired, scale, o.data_ptr(), _ptr(lse),
          workspace.data_ptr(), _nbytes(workspace)), stream)


def pha_attn_sinks_bwd(q, k, v, o, lse, dout, cu_seqlens, max_len: int, dq, dk, dv, workspace, *,
                       window: int, sinks: int, paired: bool = False, scale: float = 0.0,
                       stream=None):
    """Backward of pha_attn_sinks_fwd (o, lse: its outputs): dq, dk, dv for dout."""
    if not (-_MOST <= window < _MOST and -_MOST <= sinks < _MOST):
        window, sinks = _cut(window, sinks)
    t, h, hkv, hd, dt, code = _dims(q, k)
    n = cu_seqlens.shape[0]
    like_q, like_k = (t, h, hd), (t, hkv, hd)
    _run("pha_attn_sinks_bwd",
         (("q", q, dt, like_q), ("k", k, dt, like_k), ("v", v, dt, like_k), ("o", o, dt, like_q),
          ("lse", lse, _torch.float32, (t, h)), ("dout", dout, dt, like_q), ("dq", dq, dt, like_q),
          ("dk", dk, dt, like_k), ("dv", dv, dt, like_k),
          ("cu_seqlens", cu_seqlens, _int32(), (n,)), _scratch(workspace)),
         (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
          cu_seqlens.data_ptr(), n - 1, max_len, t, h, hkv, hd, code, window, sinks, paired, scale,
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), _nbytes(workspace)),
         stream)


def pha_attn_paged_workspace_bytes(batch: int, max_q: int, max_kv: int, total_q: int, n_heads: int,
                                   n_kv_heads: int, head_dim: int, dtype, *, window: int = 0,
                                   sinks: int = 0, paired: bool = False) -> int:
    """dtype: torch.bfloat16 or torch.float32."""
    if not (-_MOST <= window < _MOST and -_MOST <= sinks < _MOST):
        window, sinks = _cut(window, sinks)
    import torch

    code = PHA_BF16 if dtype == torch.bfloat16 else PHA_F32
    return int(_lib.pha_attn_paged_workspace_bytes(batch, max_q, max_kv, total_q, n_heads,
                                                   n_kv_heads, head_dim, code, window, sinks,
                                                   int(paired)))


def pha_attn_paged_fwd(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens, max_q: int,
                       max_kv: int, o, lse, workspace, *, window: int = 0, sinks: int = 0,
                       paired: bool = False, scale: float = 0.0, status=None, stream=None):
    """Attention of each sequence's new tokens q over its paged cache (k_pages, v_pages
    [pages][page_size][Hkv][hd], page_table [batch][max_pages], kv_lens [batch] with the new tokens
    included) into o and lse (or None). status: int32[1], raised on bad lengths or pages."""
    if not (-_MOST <= window < _MOST and -_MOST <= sinks < _MOST):
        window, sinks = _cut(window, sinks)
    t, h, hkv, hd, dt, code = _dims(q, k_pages)
    pool = k_pages.shape
    n_pages, page = pool[0], pool[1]
    batch, max_pages = page_table.shape
    i32 = _int32()
    _run("pha_attn_paged_fwd",
         (("q", q, dt, (t, h, hd)), ("k_pages", k_pages, dt, (n_pages, page, hkv, hd)),
          ("v_pages", v_pages, dt, pool), ("page_table", page_table, i32, (batch, max_pages)),
          ("cu_seqlens", cu_seqlens, i32, (batch + 1,)), ("kv_lens", kv_lens, i32, (batch,)),
          ("o", o, dt, (t, h, hd)),
          None if lse is None else ("lse", lse, _torch.float32, (t, h)), _scratch(workspace),
          _status(status)),
         (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), max_pages,
          n_pages, page, cu_seqlens.data_ptr(), kv_lens.data_ptr(), batch, max_q, max_kv, t, h,
          hkv, hd, code, window, sinks, paired, scale, o.data_ptr(), _ptr(lse),
          workspace.data_ptr(), _nbytes(workspace), _ptr(status)), stream)


def pha_test_attn_sinks_fwd_stalled(q, k, v, cu_seqlens, max_len: int, o, lse, workspace, stall_us: int,
                                    *, window: int, sinks: int, paired: bool = False, scale: float = 0.0,
                                    stream=None):
    """Failure-detection test hook: pha_attn_sinks_fwd whose softmax warps first wait stall_us
    microseconds on a barrier that nothing signals (device status 3, no row written)."""
    t, h, hkv, hd, _, code = _dims(q, k)
    _check("pha_test_attn_sinks_fwd_stalled",
           _lib.pha_test_attn_sinks_fwd_stalled(
               _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), cu_seqlens.shape[0] - 1, max_len, t, h, hkv, hd,
               code, window, sinks, int(paired), float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
               _nbytes(workspace), int(stall_us), _stream(stream, q)))


def pha_test_attn_sinks_bwd_stalled(q, k, v, o, lse, dout, cu_seqlens, max_len: int, dq, dk, dv,
                                    workspace, stall_us: int, *, window: int, sinks: int,
                                    paired: bool = False, scale: float = 0.0, stream=None):
    """The same of pha_attn_sinks_bwd."""
    t, h, hkv, hd, _, code = _dims(q, k)
    _check("pha_test_attn_sinks_bwd_stalled",
           _lib.pha_test_attn_sinks_bwd_stalled(
               _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(cu_seqlens),
               cu_seqlens.shape[0] - 1, max_len, t, h, hkv, hd, code, window, sinks, int(paired), float(scale),
               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), _nbytes(workspace), int(stall_us),
               _stream(stream, q)))


def pha_test_attn_paged_fwd_stalled(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens, max_q: int,
                                    max_kv: int, o, lse, workspace, stall_us: int, *, window: int = 0,
                                    sinks: int = 0, paired: bool = False, scale: float = 0.0,
                                    status=None, stream=None):
    """The same of pha_attn_paged_fwd (more than 16 rows a sequence)."""
    t, h, hkv, hd, _, code = _dims(q, k_pages)
    batch, max_pages = page_table.shape
    _check("pha_test_attn_paged_fwd_stalled",
           _lib.pha_test_attn_paged_fwd_stalled(
               _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), max_pages, k_pages.shape[0],
               k_pages.shape[1], _ptr(cu_seqlens), _ptr(kv_lens), batch, max_q, max_kv, t, h, hkv, hd, code,
               window, sinks, int(paired), float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
               _nbytes(workspace), _ptr(status), int(stall_us), _stream(stream, q)))


def pha_cache_append(k, v, k_pages, v_pages, page_table, cu_seqlens, kv_lens, *, status=None,
                     stream=None):
    """Writes the new tokens' k, v [T][Hkv][hd] to their places in k_pages, v_pages (one layer)."""
    shape, dt = k.shape, k.dtype
    t, hkv, hd = shape
    pool = k_pages.shape
    n_pages, page = pool[0], pool[1]
    batch, max_pages = page_table.shape
    i32 = _int32()
    _run("pha_cache_append",
         (("k", k, dt, shape), ("v", v, dt, shape), ("k_pages", k_pages, dt, (n_pages, page, hkv, hd)),
          ("v_pages", v_pages, dt, pool), ("page_table", page_table, i32, (batch, max_pages)),
          ("cu_seqlens", cu_seqlens, i32, (batch + 1,)), ("kv_lens", kv_lens, i32, (batch,)),
          _status(status)),
         (k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
          page_table.data_ptr(), max_pages, n_pages, page, cu_seqlens.data_ptr(),
          kv_lens.data_ptr(), batch, t, hkv, hd, k.element_size(), _ptr(status)), stream)


def pha_cache_workspace_bytes(n_pages: int, n_seqs: int) -> int:
    return int(_lib.pha_cache_workspace_bytes(n_pages, n_seqs))


def _cache_tensors(page_table, kv_lens, page_refs, status):
    """What _run wants of the bookkeeping tensors; (max_pages, sequences, pages)."""
    i32 = _int32()
    shape = page_table.shape
    n_seqs, max_pages = shape
    n_pages = page_refs.shape[0]
    wanted = (("page_table", page_table, i32, shape),
              None if kv_lens is None else ("kv_lens", kv_lens, i32, (n_seqs,)),
              ("page_refs", page_refs, i32, (n_pages,)), _status(status))
    return wanted, max_pages, n_seqs, n_pages


def _cache_pools(k_cache, v_cache, n_pages):
    """The same of pools [layers][pages][page_size][Hkv][hd]; (layers, bytes of one page)."""
    shape, dt = k_cache.shape, k_cache.dtype
    layers, _, page, hkv, hd = shape
    wanted = (("k_cache", k_cache, dt, (layers, n_pages, page, hkv, hd)), ("v_cache", v_cache, dt, shape))
    return wanted, layers, page * hkv * hd * k_cache.element_size()


def pha_cache_fork(page_table, kv_lens, page_refs, src, dst, workspace, *, status=None,
                   stream=None):
    """Empty sequences dst[i] become further holders of src[i]'s pages (nothing is copied)."""
    wanted, mp, ns, npg = _cache_tensors(page_table, kv_lens, page_refs, status)
    n, i32 = src.shape[0], _int32()
    _run("pha_cache_fork",
         wanted + (("src", src, i32, (n,)), ("dst", dst, i32, (n,)), _scratch(workspace)),
         (page_table.data_ptr(), mp, kv_lens.data_ptr(), ns, page_refs.data_ptr(), npg,
          src.data_ptr(), dst.data_ptr(), n, workspace.data_ptr(), _nbytes(workspace),
          _ptr(status)), stream)


def pha_cache_reserve(page_table, kv_lens, page_refs, seqs, new_tokens, k_cache, v_cache, workspace,
                      *, status=None, stream=None):
    """Room for new_tokens[i] more tokens of sequence seqs[i]; a shared last page that a sequence
    grows into is copied (k_cache, v_cache [layers][pages][page_size][Hkv][hd])."""
    wanted, mp, ns, npg = _cache_tensors(page_table, kv_lens, page_refs, status)
    pools, layers, page_bytes = _cache_pools(k_cache, v_cache, npg)
    n, i32 = seqs.shape[0], _int32()
    _run("pha_cache_reserve",
         wanted + pools + (("seqs", seqs, i32, (n,)), ("new_tokens", new_tokens, i32, (n,)),
                           _scratch(workspace)),
         (page_table.data_ptr(), mp, kv_lens.data_ptr(), ns, page_refs.data_ptr(), npg,
          k_cache.shape[2], seqs.data_ptr(), new_tokens.data_ptr(), n, k_cache.data_ptr(),
          v_cache.data_ptr(), layers, page_bytes, workspace.data_ptr(), _nbytes(workspace),
          _ptr(status)), stream)


def pha_cache_free(page_table, kv_lens, page_refs, seqs, workspace, *, status=None, stream=None):
    """Sequences seqs[i] let go of their pages and become empty."""
    wanted, mp, ns, npg = _cache_tensors(page_table, kv_lens, page_refs, status)
    n = seqs.shape[0]
    _run("pha_cache_free", wanted + (("seqs", seqs, _int32(), (n,)), _scratch(workspace)),
         (page_table.data_ptr(), mp, kv_lens.data_ptr(), ns, page_refs.data_ptr(), npg,
          seqs.data_ptr(), n, workspace.data_ptr(), _nbytes(workspace), _ptr(status)), stream)


def pha_cache_trim(page_table, kv_lens, page_refs, page_size: int, *, window: int, sinks: int = 0,
                   paired: bool = False, status=None, stream=None):
    """Every sequence lets go of the pages that no later token sees with this window and sinks."""
    window, sinks, page_size = _cut(window, sinks, page_size)
    wanted, mp, ns, npg = _cache_tensors(page_table, kv_lens, page_refs, status)
    _run("pha_cache_trim", wanted,
         (page_table.data_ptr(), mp, kv_lens.data_ptr(), ns, page_refs.data_ptr(), npg, page_size,
          window, sinks, paired, _ptr(status)), stream)


def pha_cache_compact(page_table, page_refs, k_cache, v_cache, workspace, *, status=None,
                      stream=None):
    """Moves the pages in use together at the front of the pool, in all layers."""
    wanted, mp, ns, npg = _cache_tensors(page_table, None, page_refs, status)
    pools, layers, page_bytes = _cache_pools(k_cache, v_cache, npg)
    _run("pha_cache_compact", wanted + pools + (_scratch(workspace),),
         (page_table.data_ptr(), mp, ns, page_refs.data_ptr(), npg, k_cache.data_ptr(),
          v_cache.data_ptr(), layers, page_bytes, workspace.data_ptr(), _nbytes(workspace),
          _ptr(status)), stream)
