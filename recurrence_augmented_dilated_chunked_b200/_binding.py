"""ctypes binding of ``libratp.so`` (the C ABI declared in ``include/ratp.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  There is no CPU fallback -- if the library is missing the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# RATP_LIBRARY may name another build of the same C ABI (the guarded debug
# build, libratp_guarded.so, for bounds-checked test runs)
LIB_PATH = os.environ.get("RATP_LIBRARY") or os.path.join(_PKG, "libratp.so")
MAX_HEADS = 256

RATP_F32, RATP_BF16 = 0, 1
_DTYPE = {torch.float32: RATP_F32, torch.bfloat16: RATP_BF16}

STATUS = {0: "OK", 1: "ERR_ARG", 2: "ERR_SHAPE", 3: "ERR_ALIGN", 4: "ERR_CAPACITY",
          5: "ERR_TIMEOUT", 6: "ERR_CUDA", 7: "ERR_UNSUPPORTED", 8: "ERR_BOUNDS"}


class RatpError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (fn, STATUS.get(code, "?"), code))


class CacheStruct(ctypes.Structure):
    """Mirror of ``struct ratp_cache``."""
    _fields_ = [
        ("Kc", ctypes.c_void_p), ("Vc", ctypes.c_void_p),
        ("Kw", ctypes.c_void_p), ("Vw", ctypes.c_void_p),
        ("len", ctypes.c_void_p), ("partial", ctypes.c_void_p), ("counters", ctypes.c_void_p),
        ("in_ring", ctypes.c_void_p),
        ("rows_per_b", ctypes.c_int64),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Dh", ctypes.c_int32),
        ("T_max", ctypes.c_int32), ("D", ctypes.c_int32), ("W", ctypes.c_int32),
        ("split_keys", ctypes.c_int32), ("max_splits", ctypes.c_int32),
        ("reset_L", ctypes.c_int32), ("window_L", ctypes.c_int32), ("kv_bits", ctypes.c_int32),
        ("dense", ctypes.c_uint8 * MAX_HEADS),
    ]


class DecodeLayerStruct(ctypes.Structure):
    """Mirror of ``struct ratp_decode_layer``."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("xk", ctypes.c_void_p), ("xv", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("state", ctypes.c_void_p),
        ("cache", ctypes.POINTER(CacheStruct)), ("o", ctypes.c_void_p),
    ]


# struct ratp_view {data, stride_b, stride_t, stride_h, heads}, as bytes
_VIEW = struct.Struct("=QqqqiI")


_lib = None
_lock = threading.Lock()

_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "ratp_status_string": ([_I], ctypes.c_char_p),
    "ratp_last_error": ([_P], _I),
    "ratp_device_sm_count": ([ctypes.POINTER(_I)], _I),
    "ratp_debug_fault": ([_I, ctypes.c_longlong], _I),
    "ratp_guard_line": ([ctypes.POINTER(_I)], _I),
    "ratp_debug_guard_probe": ([_P], _I),
    "ratp_scan_workspace_bytes": ([_I, _I, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "ratp_scan_prefill": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "ratp_scan_prefill_kv": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "ratp_scan_prefill_chunk_local": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "ratp_scan_prefill_kv_chunk_local": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "ratp_scan_prefill_kv_window": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P], _I),
    "ratp_scan_prefill_kv_noalloc": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P], _I),
    "ratp_dilated_attn_prefill": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P], _I),
    "ratp_dilated_attn_prefill_simt": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P], _I),
    "ratp_dilated_attn_prefill_per_sample": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P, _I, _P], _I),
    "ratp_dilated_attn_prefill_ws": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P], _I),
    "ratp_dilated_attn_prefill_per_sample_ws": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P, _I, _P, _P], _I),
    "ratp_prefill_fused_workspace_bytes": ([_I, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "ratp_prefill_fused": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _SZ, _P], _I),
    "ratp_qk_norm_rope": ([ctypes.c_char_p] * 4 + [_P] * 4 + [_I] * 6 + [ctypes.c_float, _I, _P], _I),
    "ratp_linear_attn_workspace_bytes": ([_I, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "ratp_linear_attn_prefill": ([_P] * 7 + [_I] * 4 + [ctypes.c_float, _I, _P, _SZ, _P], _I),
    "ratp_linear_attn_step": ([_P] * 6 + [_I] * 3 + [ctypes.c_float, _I, _P], _I),
    "ratp_cache_bytes_q4": ([_I, _I, _I, _I, _I, _I, _P, ctypes.POINTER(_SZ)], _I),
    "ratp_cache_init_q4": ([ctypes.POINTER(CacheStruct), _P, _SZ, _I, _I, _I, _I, _I, _I, _P, _P], _I),
    "ratp_cache_read_q4": ([ctypes.POINTER(CacheStruct), _P, _P, _P], _I),
    "ratp_cache_bytes": ([_I, _I, _I, _I, _I, _I, _P, ctypes.POINTER(_SZ)], _I),
    "ratp_cache_init": ([ctypes.POINTER(CacheStruct), _P, _SZ, _I, _I, _I, _I, _I, _I, _P, _P], _I),
    "ratp_cache_pack": ([ctypes.POINTER(CacheStruct), _P, _P, _I, _P], _I),
    "ratp_cache_set_chunk_local": ([ctypes.POINTER(CacheStruct), _I], _I),
    "ratp_cache_window_bytes": ([_I, _I, _I, _I, ctypes.POINTER(_SZ)], _I),
    "ratp_cache_set_window": ([ctypes.POINTER(CacheStruct), _P, _SZ, _I], _I),
    "ratp_cache_pack_inputs": ([ctypes.POINTER(CacheStruct), _P, _P, _P, _I, _P], _I),
    "ratp_decode_step": ([_P, _P, _P, _P, _P, ctypes.POINTER(CacheStruct), _P, _I, _I, _P, _P], _I),
    "ratp_decode_step_layers": ([ctypes.POINTER(DecodeLayerStruct), _I, _P], _I),
}


def load_library(path: str = LIB_PATH):
    """Load ``libratp.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    "CUDA library %s is missing; build it with "
                    "`python -m recurrence_augmented_dilated_chunked_b200.build`" % path)
            lib = ctypes.CDLL(path)
            for name, (args, res) in _SIGS.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def exported_symbols():
    return sorted(_SIGS)


def _check(fn, code):
    if code != 0:
        raise RatpError(fn, code)


# handle of a device's current stream without a Stream object (2.4 -> 0.2 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


_HERE = contextlib.nullcontext()


def _on(index):
    """Context with device ``index`` current (nothing to do, and next to nothing
    paid, where it is already)."""
    return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


def _addr(t):
    return None if t is None else t.data_ptr()


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _mask_buf(head_mask, H):
    if head_mask is None:
        return None, None
    m = bytes(1 if v else 0 for v in list(head_mask))
    if len(m) != H:
        raise ValueError("head_mask must have H = %d entries" % H)
    buf = (ctypes.c_uint8 * H).from_buffer_copy(m)
    return buf, ctypes.cast(buf, ctypes.c_void_p)


_ws_cache = {}


def scan_workspace(B, T, H, Dh, dtype, device, stream=None) -> torch.Tensor:
    """Device scratch for one scan call of this shape on ``stream`` (default:
    the device's current stream).

    A workspace may only be shared by calls ordered on one stream, so the
    cache holds one per (device, stream, size): scans of the same shape on two
    unordered streams get different workspaces."""
    lib = load_library()
    n = ctypes.c_size_t()
    _check("ratp_scan_workspace_bytes",
           lib.ratp_scan_workspace_bytes(B, T, H, Dh, _DTYPE[dtype], ctypes.byref(n)))
    device = torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    key = (str(device), stream.cuda_stream, n.value)
    with _lock:
        ws = _ws_cache.get(key)
        if ws is None:
            ws = torch.zeros(max(n.value, 256), dtype=torch.uint8, device=device)   # zero before first use
            if stream.cuda_stream != torch.cuda.current_stream(device).cuda_stream:
                torch.cuda.current_stream(device).synchronize()   # the zero fill precedes its first use
            _ws_cache[key] = ws
    return ws


def scan_prefill(x, g, out=None, final_state=None, workspace=None, L=0):
    """h = forget-gate scan of x with gates g over axis 1 of [B, T, H, Dh].

    L >= 1: chunk-local recurrence (the state restarts at t mod L == 0)."""
    lib = load_library()
    _need(x, "x")
    _need(g, "g", x.dtype)
    B, T, H, Dh = x.shape
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32)
    ws = workspace if workspace is not None else scan_workspace(B, T, H, Dh, x.dtype, x.device)
    if L:
        _check("ratp_scan_prefill_chunk_local", lib.ratp_scan_prefill_chunk_local(
            _ptr(x), _ptr(g), _ptr(out), _ptr(final_state), B, T, H, Dh, _DTYPE[x.dtype], int(L),
            _ptr(ws), ws.numel(), _stream(x)))
    else:
        _check("ratp_scan_prefill", lib.ratp_scan_prefill(
            _ptr(x), _ptr(g), _ptr(out), _ptr(final_state), B, T, H, Dh, _DTYPE[x.dtype],
            _ptr(ws), ws.numel(), _stream(x)))
    return out


def scan_prefill_kv(xk, xv, g, hk=None, hv=None, final_state=None, workspace=None, L=0):
    """(hk, hv) = scans of xk and xv sharing the gate tensor g (one pass).

    L >= 1: chunk-local recurrence (the state restarts at t mod L == 0)."""
    lib = load_library()
    _need(xk, "xk")
    _need(xv, "xv", xk.dtype)
    _need(g, "g", xk.dtype)
    B, T, H, Dh = xk.shape
    hk = torch.empty_like(xk) if hk is None else hk
    hv = torch.empty_like(xv) if hv is None else hv
    _need(hk, "hk", xk.dtype)
    _need(hv, "hv", xk.dtype)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32)
    ws = workspace if workspace is not None else scan_workspace(B, T, H, Dh, xk.dtype, xk.device)
    if L:
        _check("ratp_scan_prefill_kv_chunk_local", lib.ratp_scan_prefill_kv_chunk_local(
            _ptr(xk), _ptr(xv), _ptr(g), _ptr(hk), _ptr(hv), _ptr(final_state),
            B, T, H, Dh, _DTYPE[xk.dtype], int(L), _ptr(ws), ws.numel(), _stream(xk)))
    else:
        _check("ratp_scan_prefill_kv", lib.ratp_scan_prefill_kv(
            _ptr(xk), _ptr(xv), _ptr(g), _ptr(hk), _ptr(hv), _ptr(final_state),
            B, T, H, Dh, _DTYPE[xk.dtype], _ptr(ws), ws.numel(), _stream(xk)))
    return hk, hv


def scan_prefill_kv_window(xk, xv, g, L, hk=None, hv=None):
    """(hk, hv) with the fixed look-back recurrence: h_t runs from zero over the
    last L positions up to t (L = 16, 32 or 64)."""
    lib = load_library()
    _need(xk, "xk")
    _need(xv, "xv", xk.dtype)
    _need(g, "g", xk.dtype)
    B, T, H, Dh = xk.shape
    hk = torch.empty_like(xk) if hk is None else hk
    hv = torch.empty_like(xv) if hv is None else hv
    _need(hk, "hk", xk.dtype)
    _need(hv, "hv", xk.dtype)
    _check("ratp_scan_prefill_kv_window", lib.ratp_scan_prefill_kv_window(
        _ptr(xk), _ptr(xv), _ptr(g), _ptr(hk), _ptr(hv), B, T, H, Dh, _DTYPE[xk.dtype], int(L),
        _stream(xk)))
    return hk, hv


def scan_prefill_kv_noalloc(xk, xv, g, hk, hv, final_state=None):
    """(hk, hv) like ``scan_prefill_kv``, but the library supplies the scratch
    from its fixed device array, so nothing is allocated for the call (the
    outputs hk and hv must be passed in)."""
    lib = load_library()
    _need(xk, "xk")
    _need(xv, "xv", xk.dtype)
    _need(g, "g", xk.dtype)
    _need(hk, "hk", xk.dtype)
    _need(hv, "hv", xk.dtype)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32)
    B, T, H, Dh = xk.shape
    _check("ratp_scan_prefill_kv_noalloc", lib.ratp_scan_prefill_kv_noalloc(
        _ptr(xk), _ptr(xv), _ptr(g), _ptr(hk), _ptr(hv), _ptr(final_state),
        B, T, H, Dh, _DTYPE[xk.dtype], _stream(xk)))
    return hk, hv


ATTN_WORKSPACE_BYTES = 256
_attn_ws_cache = {}


def attn_workspace(device, stream=None) -> torch.Tensor:
    """The attention's small device workspace for ``stream`` (default: the
    device's current stream), cached per (device, stream): calls sharing one
    must be ordered on one stream.  It needs no initialisation."""
    device = torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    key = (str(device), stream.cuda_stream)
    with _lock:
        ws = _attn_ws_cache.get(key)
        if ws is None:
            ws = torch.empty(ATTN_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
            _attn_ws_cache[key] = ws
    return ws


def _attn(fn_name, q, hk, hv, D, W, head_mask, out, workspace=False):
    lib = load_library()
    _need(q, "q")
    _need(hk, "hk", q.dtype)
    _need(hv, "hv", q.dtype)
    B, T, H, Dh = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype)
    _buf, mp = _mask_buf(head_mask, H)
    args = [_ptr(q), _ptr(hk), _ptr(hv), _ptr(out), B, T, H, Dh, int(D), int(W), mp, _DTYPE[q.dtype]]
    if workspace is not False:
        args.append(_ptr(workspace) if workspace is not None else None)
    _check(fn_name, getattr(lib, fn_name)(*args, _stream(q)))
    return out


def dilated_attn_prefill(q, hk, hv, D, W=0, head_mask=None, out=None, workspace=None):
    """Dilated (+ windowed) causal attention of q over recurrent hk, hv.
    ``workspace``: an ``attn_workspace`` (default: the cached one of q's
    device and current stream), with which launches that mix dense and
    dilated items deal them dynamically."""
    if workspace is None and q.is_cuda:
        workspace = attn_workspace(q.device)
    return _attn("ratp_dilated_attn_prefill_ws", q, hk, hv, D, W, head_mask, out, workspace)


def dilated_attn_prefill_simt(q, hk, hv, D, W=0, head_mask=None, out=None):
    """Same operation on the CUDA-core kernel (fp32/bf16, Dh 64/128)."""
    return _attn("ratp_dilated_attn_prefill_simt", q, hk, hv, D, W, head_mask, out)


def dilated_attn_prefill_per_sample(q, hk, hv, D_per_sample, W=0, head_mask=None, out=None, workspace=None):
    """Dilated attention with one dilation per sample (``D_per_sample``: B
    ints >= 1; 1 = the sample runs dense) in one launch; bf16, Dh = 128.
    ``workspace`` as for ``dilated_attn_prefill``."""
    lib = load_library()
    _need(q, "q")
    _need(hk, "hk", q.dtype)
    _need(hv, "hv", q.dtype)
    B, T, H, Dh = q.shape
    if hk.shape != q.shape or hv.shape != q.shape:
        raise ValueError("q, hk, hv must have one shape")
    ds = [int(d) for d in D_per_sample]
    if len(ds) != B:
        raise ValueError("D_per_sample must have B = %d entries" % B)
    dbuf = (ctypes.c_int32 * max(B, 1))(*ds)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype)
    mbuf, mp = _mask_buf(head_mask, H)
    if q.dtype not in _DTYPE:
        raise ValueError("unsupported dtype %s" % q.dtype)
    if workspace is None and q.is_cuda:
        workspace = attn_workspace(q.device)
    _check("ratp_dilated_attn_prefill_per_sample_ws", lib.ratp_dilated_attn_prefill_per_sample_ws(
        _ptr(q), _ptr(hk), _ptr(hv), _ptr(out), B, T, H, Dh, ctypes.cast(dbuf, ctypes.c_void_p),
        int(W), mp, _DTYPE[q.dtype], _ptr(workspace) if workspace is not None else None, _stream(q)))
    return out


_fused_ws_cache = {}


def prefill_fused_workspace(B, T, H, Dh, device, stream=None) -> torch.Tensor:
    """Device scratch for one fused prefill of this shape on ``stream`` (default:
    the device's current stream), cached per (device, stream, size) like the
    scan workspace."""
    lib = load_library()
    n = ctypes.c_size_t()
    _check("ratp_prefill_fused_workspace_bytes",
           lib.ratp_prefill_fused_workspace_bytes(B, T, H, Dh, ctypes.byref(n)))
    device = torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    key = (str(device), stream.cuda_stream, n.value)
    with _lock:
        ws = _fused_ws_cache.get(key)
        if ws is None:
            ws = torch.zeros(max(n.value, 256), dtype=torch.uint8, device=device)   # zero before first use
            if stream.cuda_stream != torch.cuda.current_stream(device).cuda_stream:
                torch.cuda.current_stream(device).synchronize()
            _fused_ws_cache[key] = ws
    return ws


def prefill_fused(q, xk, xv, g, D, W=0, head_mask=None, hk=None, hv=None, out=None, final_state=None,
                  workspace=None):
    """(o, hk, hv): the key/value recurrence and the dilated (+ windowed)
    attention over it in one launch; bf16, head dim 128."""
    lib = load_library()
    _need(q, "q")
    for t, nm in ((xk, "xk"), (xv, "xv"), (g, "g")):
        _need(t, nm, q.dtype)
    B, T, H, Dh = q.shape
    if xk.shape != q.shape or xv.shape != q.shape or g.shape != q.shape:
        raise ValueError("q, xk, xv, g must have one shape")
    hk = torch.empty_like(xk) if hk is None else hk
    hv = torch.empty_like(xv) if hv is None else hv
    out = torch.empty_like(q) if out is None else out
    for t, nm in ((hk, "hk"), (hv, "hv"), (out, "out")):
        _need(t, nm, q.dtype)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32)
    if q.dtype not in _DTYPE:
        raise ValueError("unsupported dtype %s" % q.dtype)
    ws = workspace if workspace is not None else prefill_fused_workspace(B, T, H, Dh, q.device)
    _buf, mp = _mask_buf(head_mask, H)
    _check("ratp_prefill_fused", lib.ratp_prefill_fused(
        _ptr(q), _ptr(xk), _ptr(xv), _ptr(g), _ptr(hk), _ptr(hv), _ptr(out), _ptr(final_state),
        B, T, H, Dh, int(D), int(W), mp, _DTYPE[q.dtype], _ptr(ws), ws.numel(), _stream(q)))
    return out, hk, hv


def _head_view(t, name, dtype, device, shape=None):
    """(shape, packed ratp_view) of a [B, T, H, Dh] or [B, H, Dh] view whose
    channels are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype or t.get_device() != device:
        raise ValueError("%s must be %s on cuda:%d, got %s on %s" % (name, dtype, device, t.dtype, t.device))
    sz, st = t.shape, t.stride()
    n = len(sz)
    if shape is not None and sz != shape:
        raise ValueError("%s must have the shape %s" % (name, tuple(shape)))
    if n != 4 and n != 3:
        raise ValueError("%s must be [B, T, H, Dh] or [B, H, Dh]" % name)
    if st[-1] != 1 and sz[-1] > 1:
        raise ValueError("%s: channels must be contiguous" % name)
    # the stride of a dimension of one element is never used
    H = sz[-2]
    return sz, _VIEW.pack(t.data_ptr(), st[0] if sz[0] > 1 else 0, st[1] if n == 4 and sz[1] > 1 else 0,
                          st[-2] if H > 1 else 0, H, 0)


def _new_head_view(like, sz):
    """A new dense tensor like ``like`` (of shape ``sz``) and its packed ratp_view."""
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    H, Dh = sz[-2], sz[-1]
    T = sz[1] if len(sz) == 4 else 1
    return t, _VIEW.pack(t.data_ptr(), T * H * Dh, H * Dh, Dh, H, 0)


_NO_VIEW = _VIEW.pack(0, 0, 0, 0, 0, 0)


def _vector(t, name, n, device):
    """Address of a contiguous fp32 [n] tensor (n None: of any length), or None."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.get_device() == device and t.is_contiguous():
        sz = t.shape
        if len(sz) == 1 and (n is None or sz[0] == n):
            return t.data_ptr()
    raise ValueError("%s must be a contiguous fp32 [%s] tensor on cuda:%d" % (name, "rot / 2" if n is None else n, device))


def qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions=None, eps=1e-6, interleaved=False,
                 q_out=None, k_out=None):
    """(q_out, k_out): RMS norm of every head of q and k, times the gain of its
    channel, turned by its token's rotary position, in one pass.

    q, k: [B, T, H, Dh] (or [B, H, Dh], one token per sequence), bf16 or fp32,
    Dh 64 or 128; their head counts may differ, and either may be None.  Any
    strides that keep a head's channels contiguous and its row 16-byte aligned
    do, so both may be views of one fused projection.
    q_weight, k_weight: fp32 [Dh] gains, or None.
    inv_freq: fp32 [rot / 2], rot <= Dh a multiple of 16: the first rot
    channels turn by position * inv_freq (the angle is taken in fp64); None
    leaves the rotation out.  Pair i is channels (i, i + rot/2), or (2i, 2i+1)
    with ``interleaved``.
    positions: None (0 .. T-1), int32 [B] (the position of each sequence's
    first token here, e.g. ``KVCache.lengths()``) or int32 [B, T].
    q_out, k_out: outputs; q and k themselves work in place, otherwise outputs
    share no element with q, k or each other."""
    lib = load_library()
    ref = k if q is None else q
    if not isinstance(ref, torch.Tensor) or not ref.is_cuda:
        raise ValueError("q and k must be CUDA tensors (one of them may be None)")
    dt, dev = ref.dtype, ref.get_device()
    code = _DTYPE.get(dt)
    if code is None:
        raise ValueError("unsupported dtype %s" % dt)
    qv = kv = qo = ko = _NO_VIEW
    if q is not None:
        shape, qv = _head_view(q, "q", dt, dev)
        if q_out is None:
            q_out, qo = _new_head_view(q, shape)
        else:
            qo = _head_view(q_out, "q_out", dt, dev, shape)[1]
    else:
        q_out = q_weight = None
    if k is not None:
        ks, kv = _head_view(k, "k", dt, dev)
        if q is not None and (len(ks) != len(shape) or ks[0] != shape[0] or ks[-1] != shape[-1] or
                              (len(ks) == 4 and ks[1] != shape[1])):
            raise ValueError("q and k must agree in batch, tokens and head size")
        shape = ks
        if k_out is None:
            k_out, ko = _new_head_view(k, ks)
        else:
            ko = _head_view(k_out, "k_out", dt, dev, ks)[1]
    else:
        k_out = k_weight = None
    B, T, Dh = shape[0], shape[1] if len(shape) == 4 else 1, shape[-1]
    qw, kw = _vector(q_weight, "q_weight", Dh, dev), _vector(k_weight, "k_weight", Dh, dev)
    freq, rot = _vector(inv_freq, "inv_freq", None, dev), 0 if inv_freq is None else 2 * inv_freq.shape[0]
    pos, per_token = None, 0
    if positions is not None:
        _need(positions, "positions", torch.int32)
        ps = positions.shape
        if (ps != (B,) and ps != (B, T)) or positions.get_device() != dev:
            raise ValueError("positions must be int32 [B] or [B, T] on cuda:%d" % dev)
        pos, per_token = positions.data_ptr(), len(ps) - 1
    with _on(dev):
        _check("ratp_qk_norm_rope", lib.ratp_qk_norm_rope(
            qv, kv, qo, ko, qw, kw, freq, pos, per_token, B, T, Dh, rot, 1 if interleaved else 0, eps, code, _stream(ref)))
    return q_out, k_out


def _linear_args(q, k, v, log_decay, states, out, dims):
    if not isinstance(q, torch.Tensor) or q.dim() != dims:
        raise ValueError("q must be a CUDA tensor of %d dimensions" % dims)
    sh, dev = q.shape, q.get_device()
    if out is None:
        out = torch.empty_like(q)
    elif isinstance(out, torch.Tensor):
        n, at = 2 * q.numel(), out.data_ptr()
        if n and any(isinstance(t, torch.Tensor) and abs(t.data_ptr() - at) < n for t in (q, k, v)):
            raise ValueError("out must not overlap q, k or v")
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        if not (dev >= 0 and isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16 and t.shape == sh and
                t.get_device() == dev and t.is_contiguous()):
            _need(t, nm, torch.bfloat16)
            raise ValueError("q, k, v and out must have one shape, on one device")
    B, H, Dh = sh[0], sh[-2], sh[-1]
    _need(log_decay, "log_decay", torch.float32)
    if log_decay.shape != (H,) or log_decay.get_device() != dev:
        raise ValueError("log_decay must be [H] on cuda:%d" % dev)
    for s, nm in states:
        if s is not None:
            _need(s, nm, torch.float32)
            if s.shape != (B, H, Dh, Dh) or s.get_device() != dev:
                raise ValueError("%s must be [B, H, Dh, Dh] on cuda:%d" % (nm, dev))
    return out


def linear_attn_prefill(q, k, v, log_decay, initial_state=None, final_state=None, scale=None, out=None,
                        workspace=None):
    """Linear attention with a decay for each head over [B, T, H, Dh] (bf16, Dh
    64 or 128): S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t.

    log_decay: fp32 [H], <= 0.  initial_state: fp32 [B, H, Dh, Dh] before the
    first token (None: zero); final_state: receives the state after the last
    one, and may be initial_state itself, but not overlap it in part.  scale:
    Dh ** -0.5 by default.  out: must not overlap q, k, v or a state.
    workspace: uint8 tensor of ``linear_attn_workspace_bytes`` (default: one
    from the current stream's allocator, so that no two calls or captured
    graphs share one)."""
    lib = load_library()
    out = _linear_args(q, k, v, log_decay, ((initial_state, "initial_state"), (final_state, "final_state")), out, 4)
    B, T, H, Dh = q.shape
    with _on(q.get_device()):
        if workspace is None:
            n = linear_attn_workspace_bytes(B, T, H, Dh)
            workspace = q.new_empty(n, dtype=torch.uint8) if n else None
        else:
            _need(workspace, "workspace", torch.uint8)
            if workspace.get_device() != q.get_device():
                raise ValueError("workspace must be on the device of q")
        _check("ratp_linear_attn_prefill", lib.ratp_linear_attn_prefill(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _addr(initial_state), _addr(final_state),
            out.data_ptr(), B, T, H, Dh, Dh ** -0.5 if scale is None else scale, RATP_BF16, _addr(workspace),
            workspace.numel() if workspace is not None else 0, _stream(q)))
    return out


def linear_attn_workspace_bytes(B, T, H, Dh) -> int:
    """Bytes of device scratch that one ``linear_attn_prefill`` of this shape needs."""
    n = ctypes.c_size_t()
    _check("ratp_linear_attn_workspace_bytes",
           load_library().ratp_linear_attn_workspace_bytes(B, T, H, Dh, ctypes.byref(n)))
    return n.value


def linear_attn_step(q, k, v, log_decay, state, scale=None, out=None):
    """One token per sequence of ``linear_attn_prefill``'s recurrence: q, k, v
    bf16 [B, H, Dh]; state fp32 [B, H, Dh, Dh], updated in place."""
    lib = load_library()
    if state is None:
        raise ValueError("state must be a CUDA tensor")
    out = _linear_args(q, k, v, log_decay, ((state, "state"),), out, 3)
    B, H, Dh = q.shape
    with _on(q.get_device()):
        _check("ratp_linear_attn_step", lib.ratp_linear_attn_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state.data_ptr(), out.data_ptr(), B, H, Dh,
            Dh ** -0.5 if scale is None else scale, RATP_BF16, _stream(q)))
    return out


def last_error(device=None):
    """Synchronise and raise if any kernel recorded a device-side error."""
    lib = load_library()
    dev = torch.device("cuda" if device is None else device)
    s = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
    _check("ratp_last_error", lib.ratp_last_error(s))


FAULT_NONE, FAULT_SPIN_LIMIT, FAULT_SCAN_DROP, FAULT_ATTN_DROP_K, FAULT_FUSED_DROP_CHUNK = 0, 1, 2, 3, 4


def debug_fault(kind: int, arg: int = 0):
    """Plant a failure for tests of the error paths (see ``ratp_debug_fault``)."""
    _check("ratp_debug_fault", load_library().ratp_debug_fault(int(kind), int(arg)))


def sm_count() -> int:
    n = ctypes.c_int()
    _check("ratp_device_sm_count", load_library().ratp_device_sm_count(ctypes.byref(n)))
    return n.value


class KVCache:
    """D-compressed KV cache for decode (one device buffer, see ``ratp.h``)."""

    def __init__(self, B, H, Dh, T_max, D, W=0, head_mask=None, device="cuda", L=0, kv_bits=16):
        """L >= 1: decode continues a chunk-local recurrence of block L.

        kv_bits: 16 holds the dilated rows in bf16; 4 holds them in 4 bits a
        channel with a minimum and a step for every 32 channels (80 bytes a row
        of 128 channels instead of 256); the last W positions and the state
        stay bf16 and fp32.  Every method works on both."""
        lib = load_library()
        if kv_bits not in (4, 16):
            raise ValueError("kv_bits must be 4 or 16, got %r" % (kv_bits,))
        self.kv_bits = int(kv_bits)
        q4 = self.kv_bits == 4
        size, init = ("ratp_cache_bytes_q4", "ratp_cache_init_q4") if q4 else ("ratp_cache_bytes", "ratp_cache_init")
        self.B, self.H, self.Dh, self.T_max, self.D, self.W = B, H, Dh, T_max, D, W
        self.head_mask = [1 if v else 0 for v in head_mask] if head_mask is not None else None
        self._mask_buf, mp = _mask_buf(self.head_mask, H)
        n = ctypes.c_size_t()
        _check(size, getattr(lib, size)(B, H, Dh, T_max, D, W, mp, ctypes.byref(n)))
        self.buffer = torch.empty(n.value, dtype=torch.uint8, device=device)
        if not self.buffer.is_cuda:
            raise ValueError("a cache lives on a CUDA device, got %s" % self.buffer.device)
        self._dev = self.buffer.get_device()
        self.c = CacheStruct()
        with _on(self._dev):
            _check(init, getattr(lib, init)(
                ctypes.byref(self.c), _ptr(self.buffer), n.value, B, H, Dh, T_max, D, W, mp,
                _stream(self.buffer)))
        self._mask_ptr = mp
        self._ref = ctypes.byref(self.c)
        self._len = self._view(self.c.len, B, torch.int32)
        self._rings = {}
        self.L = int(L)
        _check("ratp_cache_set_chunk_local", lib.ratp_cache_set_chunk_local(ctypes.byref(self.c), self.L))

    def _view(self, addr, numel, dtype):
        off = addr - self.buffer.data_ptr()
        esz = torch.empty((), dtype=dtype).element_size()
        return self.buffer[off: off + numel * esz].view(dtype)

    def dil_rows(self, which="k"):
        """Kc or Vc as [B, rows_per_b, Dh]: bf16, a view of the buffer; for a
        4-bit cache the fp32 values that the held rows stand for."""
        if self.kv_bits == 4:
            out = self._len.new_empty((self.B, self.c.rows_per_b, self.Dh), dtype=torch.float32)
            with _on(self._dev):
                _check("ratp_cache_read_q4", load_library().ratp_cache_read_q4(
                    self._ref, out.data_ptr() if which == "k" else None,
                    None if which == "k" else out.data_ptr(), _stream(out)))
            return out
        addr = self.c.Kc if which == "k" else self.c.Vc
        rows = self.B * self.c.rows_per_b
        return self._view(addr, rows * self.Dh, torch.bfloat16).view(self.B, self.c.rows_per_b, self.Dh)

    def ring(self, which="k"):
        """Kw or Vw as [B, H, W, Dh] bf16 (None when W == 0)."""
        if self.W == 0:
            return None
        ring = self._rings.get(which)
        if ring is None:
            addr = self.c.Kw if which == "k" else self.c.Vw
            n = self.B * self.H * self.W * self.Dh
            ring = self._view(addr, n, torch.bfloat16).view(self.B, self.H, self.W, self.Dh)
            self._rings[which] = ring
        return ring

    def lengths(self):
        return self._len

    def head_rows(self, h):
        """(offset, capacity) of head h inside one batch item's dilated rows."""
        off = 0
        for k in range(self.H):
            cap = self.T_max if (self.head_mask and self.head_mask[k]) else self.T_max // self.D
            if k == h:
                return off, cap
            off += cap
        raise IndexError(h)

    def _fit(self, t, name, dtype, numel):
        """``t`` has what a call reads of it: type, elements (its front, if it
        has more), the cache's device."""
        if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.get_device() == self._dev and t.is_contiguous() and
                t.numel() >= numel):
            return
        _need(t, name, dtype)
        raise ValueError("%s: %s on %s does not fit the cache (B %d, H %d, Dh %d) on %s" % (
            name, tuple(t.shape), t.device, self.B, self.H, self.Dh, self.buffer.device))

    def _step_args(self, q, xk, xv, g, state, out):
        n, bf16 = self.B * self.H * self.Dh, torch.bfloat16
        self._fit(q, "q", bf16, n)
        self._fit(xk, "xk", bf16, n)
        self._fit(xv, "xv", bf16, n)
        self._fit(g, "g", bf16, n)
        self._fit(out, "out", bf16, n)
        self._fit(state, "state", torch.float32, 2 * n)
        # a larger buffer whose front is the state is taken; a state of another
        # batch is not, since its value stream does not begin where this one's does
        if state.numel() > 2 * n and state.dim() in (3, 4) and state.shape[0] == 2:
            raise ValueError("state: %s is not the state of a batch of %d" % (tuple(state.shape), self.B))

    def _prompt(self, t, name, T):
        """What a hand-off of T tokens reads of ``t``, dense [B, T, H, Dh].  A
        tensor of more sequences or tokens (its first two dimensions, with H * Dh
        elements in the rest) gives the first T tokens of its first B sequences;
        any other, its first elements."""
        row = self.H * self.Dh
        if isinstance(t, torch.Tensor) and t.dim() > 2:
            n, m = t.shape[:2]
            if n * m * row == t.numel() and n >= self.B and m > T > 0 and t.is_contiguous():
                t = t[:self.B, :T].contiguous()        # no copy where B is 1
        self._fit(t, name, torch.bfloat16, self.B * T * row)
        return t

    def pack(self, hk, hv, T=None):
        """Prefill -> cache hand-off of the first T tokens (default: all) of hk
        and hv, bf16 [B, >= T, H, Dh]; T below their own length copies those
        tokens out first where B > 1."""
        _need(hk, "hk", torch.bfloat16)
        T = int(hk.shape[1] if T is None else T)
        hk, hv = self._prompt(hk, "hk", T), self._prompt(hv, "hv", T)
        with _on(self._dev):
            _check("ratp_cache_pack", load_library().ratp_cache_pack(
                self._ref, _ptr(hk), _ptr(hv), T, _stream(hk)))

    def attach_window(self, L):
        """Continue a fixed look-back recurrence of window L at decode: keeps a
        ring of the last L inputs (x_k, x_v, g) beside the cache."""
        lib = load_library()
        n = ctypes.c_size_t()
        _check("ratp_cache_window_bytes",
               lib.ratp_cache_window_bytes(self.B, self.H, self.Dh, int(L), ctypes.byref(n)))
        self.in_ring = torch.empty(n.value, dtype=torch.uint8, device=self.buffer.device)
        _check("ratp_cache_set_window", lib.ratp_cache_set_window(
            ctypes.byref(self.c), _ptr(self.in_ring), n.value, int(L)))

    def pack_inputs(self, xk, xv, g, T=None):
        """Prefill -> decode hand-off of the look-back inputs (last L positions
        before T); tensors as for ``pack``."""
        _need(xk, "xk", torch.bfloat16)
        T = int(xk.shape[1] if T is None else T)
        xk, xv, g = self._prompt(xk, "xk", T), self._prompt(xv, "xv", T), self._prompt(g, "g", T)
        with _on(self._dev):
            _check("ratp_cache_pack_inputs", load_library().ratp_cache_pack_inputs(
                self._ref, _ptr(xk), _ptr(xv), _ptr(g), T, _stream(xk)))

    def decode_step(self, q, xk, xv, g, state, out=None):
        """One token per sequence: q, xk, xv, g, out bf16 [B, H, Dh]; state: fp32
        [2, B, H, Dh] updated in place.  Of a larger contiguous tensor (a batch
        padded at its end) the front is used; the rest of out is not written."""
        if out is None and isinstance(q, torch.Tensor):
            out = torch.empty_like(q)
        self._step_args(q, xk, xv, g, state, out)
        with _on(q.get_device()):
            _check("ratp_decode_step", load_library().ratp_decode_step(
                q.data_ptr(), xk.data_ptr(), xv.data_ptr(), g.data_ptr(), state.data_ptr(), self._ref, out.data_ptr(),
                self.D, self.W, self._mask_ptr, _stream(q)))
        return out


def decode_step_layers(layers):
    """One decode token through a stack of layers in one call.

    layers: sequence of (cache, q, xk, xv, g, state, out) with ``cache`` a
    ``KVCache`` (its own D, W, head mask and recurrence), q/xk/xv/g/out bf16
    [B, H, Dh] and state fp32 [2, B, H, Dh] (updated in place).  The layers
    run in order on the current stream of the first q.
    """
    n = len(layers)
    arr = (DecodeLayerStruct * max(n, 1))()
    for i, (cache, q, xk, xv, g, state, out) in enumerate(layers):
        cache._step_args(q, xk, xv, g, state, out)
        arr[i] = DecodeLayerStruct(q.data_ptr(), xk.data_ptr(), xv.data_ptr(), g.data_ptr(),
                                   state.data_ptr(), ctypes.pointer(cache.c), out.data_ptr())
        if q.get_device() != layers[0][1].get_device():
            raise ValueError("the layers of one call must be on one device")
    if n == 0:
        _check("ratp_decode_step_layers", load_library().ratp_decode_step_layers(arr, 0, None))
        return
    with _on(layers[0][1].get_device()):
        _check("ratp_decode_step_layers", load_library().ratp_decode_step_layers(arr, n, _stream(layers[0][1])))


def guard_line():
    """(guarded build?, source line of the first refused access or 0); the
    call clears the recorded line."""
    n = ctypes.c_int()
    rc = load_library().ratp_guard_line(ctypes.byref(n))
    if rc == 7:
        return False, 0
    _check("ratp_guard_line", rc)
    return True, n.value
