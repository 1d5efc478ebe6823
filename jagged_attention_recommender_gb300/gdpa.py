"""Python binding of libgdpa (the C ABI in include/gdpa.h).

Argument marshalling only: every step of the forward pass runs in the CUDA
library.  Functions keep the C names.  Device tensors may be torch tensors or
raw integer addresses; host arrays are numpy arrays.  A non-OK status raises
:class:`GdpaError`.  If ``libgdpa.so`` has not been built the import of the
library fails loudly -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdpa.so")

GDPA_ACT_SOFTMAX = 0
GDPA_ACT_GELU_TANH = 1

GDPA_ROUTE_SFU = 0
GDPA_ROUTE_ALU = 1

GDPA_ROPE_HALF = 0
GDPA_ROPE_INTERLEAVED = 1

GDPA_OK = 0
GDPA_ERR_INVALID_ARG = 1
GDPA_ERR_UNSUPPORTED = 2
GDPA_ERR_CUDA = 3
GDPA_ERR_DEVICE_TIMEOUT = 4
GDPA_ERR_NO_MEMORY = 5

# Every symbol include/gdpa.h declares.
EXPORTS = ("gdpa_fwd", "gdpa_fwd_async", "gdpa_fwd_lse", "gdpa_fwd_sliding", "gdpa_fwd_mx", "gdpa_fwd_mxfp8", "gdpa_bwd", "gdpa_bwd_sliding", "gdpa_fwd_noalloc", "gdpa_plan_create", "gdpa_plan_create_sliding", "gdpa_fwd_planned", "gdpa_plan_destroy", "gdpa_plan_num_items",
           "gdpa_plan_num_ctas", "gdpa_fwd_host", "gdpa_plan_enumerate", "gdpa_act_eval", "gdpa_set_act_route",
           "gdpa_get_act_route", "gdpa_device_status", "gdpa_wait_selftest", "gdpa_status_string", "gdpa_version",
           "gdpa_cache_append", "gdpa_cache_fwd", "gdpa_cache_workspace_size")


class GdpaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s" % (where, gdpa_status_string(code)))


class WorkItem(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_int32), ("head", ctypes.c_int32), ("q0", ctypes.c_int32), ("kv0", ctypes.c_int32)]


class _CacheDesc(ctypes.Structure):
    """gdpa_cache_t"""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_sf", ctypes.c_void_p),
                ("v_sf", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("H", ctypes.c_int32), ("D", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
                ("rot_dim", ctypes.c_int32), ("rope_style", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgdpa.so (raises if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libgdpa.so is not built (%s); run jagged_attention_recommender_gb300.build" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    L.gdpa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, P]
    L.gdpa_fwd_async.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, P, P]
    L.gdpa_fwd_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, P]
    L.gdpa_fwd_lse.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P]
    L.gdpa_fwd_sliding.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P]
    L.gdpa_fwd_mx.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, F, P, P, P]
    L.gdpa_fwd_mxfp8.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, F, P, P, P]
    L.gdpa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P, P]
    L.gdpa_bwd_sliding.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P, P]
    L.gdpa_plan_create.argtypes = [P, P, I, I, I, I, I, ctypes.POINTER(P)]
    L.gdpa_plan_create_sliding.argtypes = [P, P, I, I, I, I, I, ctypes.POINTER(P)]
    L.gdpa_fwd_planned.argtypes = [P, P, P, P, P, P, F, P, P]
    L.gdpa_plan_destroy.argtypes = [P]
    L.gdpa_plan_destroy.restype = None
    L.gdpa_plan_num_items.argtypes = [P]
    L.gdpa_plan_num_items.restype = I64
    L.gdpa_plan_num_ctas.argtypes = [P]
    L.gdpa_fwd_host.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, P]
    L.gdpa_plan_enumerate.argtypes = [P, P, I, I, I, I, I, I, P, I64, P, P, ctypes.POINTER(I64),
                                      ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    L.gdpa_act_eval.argtypes = [I, P, P, I64, P]
    L.gdpa_set_act_route.argtypes = [I]
    L.gdpa_get_act_route.argtypes = []
    L.gdpa_get_act_route.restype = I
    L.gdpa_device_status.argtypes = [P]
    L.gdpa_wait_selftest.argtypes = [I, P]
    L.gdpa_cache_append.argtypes = [P, P, I64, P, I64, P, I64, P, P, P, I64, I, I, I, P, P]
    L.gdpa_cache_fwd.argtypes = [P, P, I64, P, P, P, I64, I, I, I, I, I, I, F, P, P, P, I64, P]
    L.gdpa_cache_workspace_size.argtypes = [P, I, I, ctypes.POINTER(I64)]
    L.gdpa_status_string.argtypes = [I]
    L.gdpa_status_string.restype = ctypes.c_char_p
    L.gdpa_version.argtypes = []
    L.gdpa_version.restype = ctypes.c_char_p
    for name in ("gdpa_fwd", "gdpa_fwd_async", "gdpa_fwd_lse", "gdpa_fwd_sliding", "gdpa_fwd_mxfp8", "gdpa_bwd", "gdpa_bwd_sliding", "gdpa_fwd_noalloc", "gdpa_plan_create", "gdpa_plan_create_sliding", "gdpa_fwd_planned", "gdpa_plan_num_ctas", "gdpa_fwd_host",
                 "gdpa_plan_enumerate", "gdpa_act_eval", "gdpa_set_act_route", "gdpa_device_status", "gdpa_wait_selftest",
                 "gdpa_cache_append", "gdpa_cache_fwd", "gdpa_cache_workspace_size"):
        getattr(L, name).restype = I
    _lib = L
    return L


def _addr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _check(code: int, where: str):
    if code != GDPA_OK:
        raise GdpaError(code, where)


def gdpa_status_string(code: int) -> str:
    return lib().gdpa_status_string(int(code)).decode()


def gdpa_version() -> str:
    return lib().gdpa_version().decode()


def gdpa_fwd(q, k, v, q_offsets, kv_offsets, B, H, D, act, window_blocks, scale, out, stream=None):
    _check(lib().gdpa_fwd(_addr(q), _addr(k), _addr(v), _addr(q_offsets), _addr(kv_offsets), int(B), int(H),
                          int(D), int(act), int(window_blocks), float(scale), _addr(out), _stream(stream)),
           "gdpa_fwd")


def gdpa_fwd_noalloc(q, k, v, q_offsets, kv_offsets, B, H, D, act, window_blocks, scale, out, stream=None):
    """gdpa_fwd without any allocation (fixed 4 MiB device work-list array; see include/gdpa.h)."""
    _check(lib().gdpa_fwd_noalloc(_addr(q), _addr(k), _addr(v), _addr(q_offsets), _addr(kv_offsets), int(B), int(H),
                                  int(D), int(act), int(window_blocks), float(scale), _addr(out), _stream(stream)),
           "gdpa_fwd_noalloc")


def gdpa_fwd_async(q, k, v, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act, window_blocks, scale,
                   out, stream=None):
    """Host offsets (numpy int32) plan the work; device offsets feed the kernel.  No sync."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_fwd_async(_addr(q), _addr(k), _addr(v), qo.ctypes.data, ko.ctypes.data, _addr(q_offsets),
                                _addr(kv_offsets), int(B), int(H), int(D), int(act), int(window_blocks),
                                float(scale), _addr(out), _stream(stream)), "gdpa_fwd_async")


def gdpa_fwd_lse(q, k, v, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act, window_blocks, scale,
                 out, lse, stream=None):
    """gdpa_fwd_async that also writes the softmax row logsumexp ``lse`` (device fp32 [Tq, H])."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_fwd_lse(_addr(q), _addr(k), _addr(v), qo.ctypes.data, ko.ctypes.data, _addr(q_offsets),
                              _addr(kv_offsets), int(B), int(H), int(D), int(act), int(window_blocks), float(scale),
                              _addr(out), _addr(lse), _stream(stream)), "gdpa_fwd_lse")


def gdpa_fwd_sliding(q, k, v, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act, window_tokens, scale,
                     out, lse=None, stream=None):
    """The forward with a causal sliding window of ``window_tokens`` tokens (optional ``lse`` output)."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_fwd_sliding(_addr(q), _addr(k), _addr(v), qo.ctypes.data, ko.ctypes.data, _addr(q_offsets),
                                  _addr(kv_offsets), int(B), int(H), int(D), int(act), int(window_tokens),
                                  float(scale), _addr(out), _addr(lse), _stream(stream)), "gdpa_fwd_sliding")


def gdpa_fwd_mx(q8, q_sf, k8, k_sf, v, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act, scale, out,
                lse=None, stream=None):
    """The forward with MXFP8 ``q8``/``k8`` (e4m3 codes) and E8M0 block scales ``q_sf``/``k_sf``."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_fwd_mx(_addr(q8), _addr(q_sf), _addr(k8), _addr(k_sf), _addr(v), qo.ctypes.data,
                             ko.ctypes.data, _addr(q_offsets), _addr(kv_offsets), int(B), int(H), int(D), int(act),
                             float(scale), _addr(out), _addr(lse), _stream(stream)), "gdpa_fwd_mx")


def gdpa_fwd_mxfp8(q8, q_sf, k8, k_sf, vt8, vt_sf, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act,
                   scale, out, lse=None, stream=None):
    """The forward with ``q8``/``k8`` and the key-major ``vt8`` all MXFP8 (e4m3 codes with E8M0 scales)."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_fwd_mxfp8(_addr(q8), _addr(q_sf), _addr(k8), _addr(k_sf), _addr(vt8), _addr(vt_sf),
                                qo.ctypes.data, ko.ctypes.data, _addr(q_offsets), _addr(kv_offsets), int(B), int(H),
                                int(D), int(act), float(scale), _addr(out), _addr(lse), _stream(stream)),
           "gdpa_fwd_mxfp8")


def gdpa_bwd(q, k, v, out, dout, lse, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act, window_blocks,
             scale, dq, dk, dv, stream=None):
    """Gradients dq, dk, dv (device bf16) of the forward for the upstream gradient ``dout``."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_bwd(_addr(q), _addr(k), _addr(v), _addr(out), _addr(dout), _addr(lse), qo.ctypes.data,
                          ko.ctypes.data, _addr(q_offsets), _addr(kv_offsets), int(B), int(H), int(D), int(act),
                          int(window_blocks), float(scale), _addr(dq), _addr(dk), _addr(dv), _stream(stream)),
           "gdpa_bwd")


def gdpa_bwd_sliding(q, k, v, out, dout, lse, h_q_offsets, h_kv_offsets, q_offsets, kv_offsets, B, H, D, act,
                     window_tokens, scale, dq, dk, dv, stream=None):
    """gdpa_bwd for the causal sliding window of ``window_tokens`` tokens."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_bwd_sliding(_addr(q), _addr(k), _addr(v), _addr(out), _addr(dout), _addr(lse), qo.ctypes.data,
                                  ko.ctypes.data, _addr(q_offsets), _addr(kv_offsets), int(B), int(H), int(D),
                                  int(act), int(window_tokens), float(scale), _addr(dq), _addr(dk), _addr(dv),
                                  _stream(stream)), "gdpa_bwd_sliding")


class Plan:
    """Owns a gdpa_plan_t; freed by gdpa_plan_destroy (or when collected)."""

    def __init__(self, handle: int):
        self.handle = handle

    @property
    def num_items(self) -> int:
        return lib().gdpa_plan_num_items(self.handle)

    @property
    def num_ctas(self) -> int:
        return lib().gdpa_plan_num_ctas(self.handle)

    def __del__(self):
        if getattr(self, "handle", None):
            try:
                lib().gdpa_plan_destroy(self.handle)
            except Exception:
                pass
            self.handle = None


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int32)


def gdpa_plan_create(h_q_offsets, h_kv_offsets, B, H, D, act, window_blocks) -> Plan:
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    h = ctypes.c_void_p()
    _check(lib().gdpa_plan_create(qo.ctypes.data, ko.ctypes.data, int(B), int(H), int(D), int(act),
                                  int(window_blocks), ctypes.byref(h)), "gdpa_plan_create")
    return Plan(h.value)


def gdpa_plan_create_sliding(h_q_offsets, h_kv_offsets, B, H, D, act, window_tokens) -> Plan:
    """The plan of gdpa_fwd_sliding (causal window of ``window_tokens`` tokens), for gdpa_fwd_planned."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    h = ctypes.c_void_p()
    _check(lib().gdpa_plan_create_sliding(qo.ctypes.data, ko.ctypes.data, int(B), int(H), int(D), int(act),
                                          int(window_tokens), ctypes.byref(h)), "gdpa_plan_create_sliding")
    return Plan(h.value)


def gdpa_fwd_planned(plan: Plan, q, k, v, q_offsets, kv_offsets, scale, out, stream=None):
    _check(lib().gdpa_fwd_planned(plan.handle, _addr(q), _addr(k), _addr(v), _addr(q_offsets), _addr(kv_offsets),
                                  float(scale), _addr(out), _stream(stream)), "gdpa_fwd_planned")


def gdpa_plan_destroy(plan: Plan):
    if plan.handle:
        lib().gdpa_plan_destroy(plan.handle)
        plan.handle = None


def gdpa_fwd_host(h_q, h_k, h_v, h_q_offsets, h_kv_offsets, B, H, D, act, window_blocks, scale, h_out,
                  stream=None):
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    _check(lib().gdpa_fwd_host(_addr(h_q), _addr(h_k), _addr(h_v), qo.ctypes.data, ko.ctypes.data, int(B),
                               int(H), int(D), int(act), int(window_blocks), float(scale), _addr(h_out),
                               _stream(stream)), "gdpa_fwd_host")


def gdpa_plan_enumerate(h_q_offsets, h_kv_offsets, B, H, D, act, window_blocks, num_ctas, with_rows=False):
    """Host planner only: returns (items [n, 4] int32, cta_begin [num_ctas+1], cost [n])
    (and, when ``with_rows``, the query rows per item and the keys per K/V tile)."""
    qo, ko = _i32(h_q_offsets), _i32(h_kv_offsets)
    n = ctypes.c_int64(0)
    rows = ctypes.c_int32(0)
    kvt = ctypes.c_int32(0)
    cta = np.zeros(num_ctas + 1, dtype=np.int32)
    code = lib().gdpa_plan_enumerate(qo.ctypes.data, ko.ctypes.data, int(B), int(H), int(D), int(act),
                                     int(window_blocks), int(num_ctas), None, 0, cta.ctypes.data, None,
                                     ctypes.byref(n), ctypes.byref(rows), ctypes.byref(kvt))
    if code not in (GDPA_OK, GDPA_ERR_NO_MEMORY):
        raise GdpaError(code, "gdpa_plan_enumerate")
    items = np.zeros((max(n.value, 1), 4), dtype=np.int32)
    cost = np.zeros(max(n.value, 1), dtype=np.int64)
    _check(lib().gdpa_plan_enumerate(qo.ctypes.data, ko.ctypes.data, int(B), int(H), int(D), int(act),
                                     int(window_blocks), int(num_ctas), items.ctypes.data, n.value,
                                     cta.ctypes.data, cost.ctypes.data, ctypes.byref(n), ctypes.byref(rows),
                                     ctypes.byref(kvt)),
           "gdpa_plan_enumerate")
    if with_rows:
        return items[:n.value], cta, cost[:n.value], rows.value, kvt.value
    return items[:n.value], cta, cost[:n.value]


def gdpa_act_eval(act, x, y, *, stream=None):
    """y = act(x) elementwise on the device (``stream`` keyword-only: a stray
    positional argument must not be taken for a stream handle)."""
    _check(lib().gdpa_act_eval(int(act), _addr(x), _addr(y), int(x.numel()), _stream(stream)), "gdpa_act_eval")


def gdpa_set_act_route(route) -> None:
    """Selects the sigma route of the GELU / SiLU activations for later
    launches (GDPA_ROUTE_SFU or GDPA_ROUTE_ALU)."""
    _check(lib().gdpa_set_act_route(int(route)), "gdpa_set_act_route")


def gdpa_get_act_route() -> int:
    return int(lib().gdpa_get_act_route())


def gdpa_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status code."""
    return lib().gdpa_device_status(_stream(stream))


def gdpa_wait_selftest(timeout_ms: int, stream=None):
    _check(lib().gdpa_wait_selftest(int(timeout_ms), _stream(stream)), "gdpa_wait_selftest")


_torch = None
_bf16 = _i32_t = _f32 = _u8 = None  # torch's types
_cuda = False  # whether torch has found a CUDA device
_raw_stream = None  # the address of a device's current stream


def _device() -> int:
    """The current CUDA device (-2: there is none)."""
    global _torch, _bf16, _i32_t, _f32, _u8, _cuda, _raw_stream
    if _torch is None:
        import torch
        _bf16, _i32_t, _f32, _u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
        # (no Stream object is made where torch offers that)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _torch = torch
    _cuda = _cuda or _torch.cuda.is_available()
    return _torch.cuda.current_device() if _cuda else -2


def _at(where, device, dtype, t, least=0):
    """The address of a contiguous tensor of type ``dtype`` on ``device``, of ``least`` elements or more; another one is
    refused (addresses and None pass)."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous() and t.numel() >= least:
        return t.data_ptr()
    _kind(where, device, dtype, t)
    if not t.is_contiguous():
        raise ValueError("%s: a contiguous tensor wanted, got strides %r" % (where, t.stride()))
    raise ValueError("%s: a %s tensor of %d elements or more wanted, got shape %r" % (where, dtype, least, tuple(t.shape)))


def _kind(where, device, dtype, t):
    if t.dtype is not dtype:
        raise TypeError("%s: %s wanted, got %s" % (where, dtype, t.dtype))
    if t.get_device() != device:
        raise ValueError("%s: tensor on %s, not on the current CUDA device" % (where, t.device))


def _table_at(where, device, t, B, max_pages):
    """The address of a page table whose rows are ``max_pages`` entries."""
    at = _at(where, device, _i32_t, t, B * max_pages)
    if B > 1 and t.__class__ is not int and t is not None and t.dim() > 1 and t.shape[-1] != max_pages:
        raise ValueError("%s: a page table of %d entries a row wanted, got shape %r" % (where, max_pages, tuple(t.shape)))
    return at


def _heads_at(where, device, cache, t, rows):
    """The address of ``rows`` or more contiguous heads of D bf16."""
    return t if t is None or t.__class__ is int else _at(where, device, _bf16, t, rows * cache.D)


def _cache_at(where, device, cache):
    """The address of the cache's descriptor; a cache on another device than the current one is refused."""
    if getattr(cache, "device", device) != device:
        raise ValueError("%s: the cache is on cuda:%d, not on the current CUDA device" % (where, cache.device))
    return cache.addr


def _rows_at(where, device, cache, t, stride, T, heads=0):
    """The address of bf16 rows ``stride`` apart, T of them or more, each of ``heads`` heads (0: the cache's) of D
    elements side by side; a tensor laid out in another way is refused."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not _bf16 or t.get_device() != device:
        _kind(where, device, _bf16, t)
    heads, D, st = heads or cache.H, cache.D, t.stride()
    if st == (stride, D, 1):
        n, h, d = t.shape
        if h == heads and d == D and n >= T:
            return t.data_ptr()
    if T <= 0:
        return t.data_ptr()
    shape = t.shape
    dims = [(n, s) for n, s in zip(shape, st) if n != 1]  # the stride of a single element says nothing
    rows = 0
    if dims and dims[-1][1] == 1:
        if dims[-1][0] == D and heads == 1:
            rows, dims = 1, dims[:-1]
        elif dims[-1][0] == D and len(dims) > 1 and dims[-2] == (heads, D):
            rows, dims = 1, dims[:-2]
        elif dims[-1][0] == D and len(dims) == 2 and dims[0][1] == D and stride == heads * D:
            rows, dims = dims[0][0] // heads, []  # all heads of all rows one behind the other
        elif dims[-1][0] >= heads * D:  # rows not cut into heads, or one behind the other
            rows = 1 + ((dims[-1][0] - heads * D) // stride if len(dims) == 1 and stride > 0 else 0)
            dims = dims[:-1]
    step = stride
    for n, s in reversed(dims):
        if s != step:
            rows = 0
        rows, step = rows * n, step * n
    if rows < T:
        raise ValueError("%s: %d rows of %d heads of %d side by side wanted, %d elements apart, got shape %r, strides %r"
                         % (where, T, heads, D, stride, tuple(shape), st))
    return t.data_ptr()


class KvCache:
    """A gdpa_cache_t over the caller's tensors, which it keeps alive: codes uint8 ``[num_pages, H, page_tokens, D]``
    (e4m3), scales uint8 ``[num_pages, H, page_tokens // 16]`` (E8M0), ``inv_freq`` host float64 ``[rot_dim // 2]``
    (radians per position; None: no rotation) and the pairing (GDPA_ROPE_HALF or GDPA_ROPE_INTERLEAVED)."""

    def __init__(self, k_codes, v_codes, k_sf, v_sf, inv_freq=None, rope_style=GDPA_ROPE_HALF):
        pages, H, tokens, D = (int(n) for n in k_codes.shape)
        for name, t, shape in (("k_codes", k_codes, (pages, H, tokens, D)), ("v_codes", v_codes, (pages, H, tokens, D)),
                               ("k_sf", k_sf, (pages, H, tokens // 16)), ("v_sf", v_sf, (pages, H, tokens // 16))):
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError("KvCache: %s must be contiguous %r, got %r" % (name, shape, tuple(t.shape)))
        device = _device()
        at = [_at("KvCache", device, _u8, t) for t in (k_codes, v_codes, k_sf, v_sf)]
        self.tensors = (k_codes, v_codes, k_sf, v_sf)
        self.H, self.D, self.device = H, D, device
        self.inv_freq = None if inv_freq is None else np.ascontiguousarray(inv_freq, dtype=np.float64)
        n = 0 if self.inv_freq is None else self.inv_freq.size
        self.desc = _CacheDesc(*at, pages, tokens, H, D,
                               self.inv_freq.ctypes.data if n else None, 2 * n, int(rope_style))
        self.addr = ctypes.addressof(self.desc)


def gdpa_cache_append(cache: KvCache, q, q_stride, k, k_stride, v, v_stride, offsets, kv_lens, page_table, T, B, Hq,
                      max_pages, q_out, stream=None):
    """Stores the new tokens' ``k`` and ``v`` in the cache (``k`` rotated by position) and the rotated ``q`` in
    ``q_out``.  ``kv_lens``: tokens of each sequence after this call.  Strides of rows in elements."""
    d, where = _device(), "gdpa_cache_append"
    n, b = (T, B) if T > 0 and B > 0 else (0, -1)  # a call with nothing to do wants nothing of its tensors
    _check(lib().gdpa_cache_append(
        _cache_at(where, d, cache), _rows_at(where, d, cache, q, q_stride, n, Hq), q_stride,
        _rows_at(where, d, cache, k, k_stride, n), k_stride, _rows_at(where, d, cache, v, v_stride, n), v_stride,
        _at(where, d, _i32_t, offsets, b + 1), _at(where, d, _i32_t, kv_lens, b),
        _table_at(where, d, page_table, b, max_pages), T, B, Hq, max_pages,
        _heads_at(where, d, cache, q_out, 0 if q is None else n * Hq),
        (_raw_stream(d) or None) if stream is None else _stream(stream)), where)


def gdpa_cache_fwd(cache: KvCache, q, q_stride, offsets, kv_lens, page_table, T, B, Hq, max_pages, max_q, causal,
                   window_tokens, scale, out, lse, workspace, workspace_bytes=None, stream=None):
    """Attention of the new tokens' ``q`` over the cache.  ``workspace``: a device tensor of at least
    gdpa_cache_workspace_size() bytes (or an address, with its ``workspace_bytes``); calls that may overlap need one
    each."""
    d, where = _device(), "gdpa_cache_fwd"
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else workspace.numel()
    n, b = (T, B) if T > 0 and B > 0 else (0, -1)  # a call with nothing to do wants nothing of its tensors
    _check(lib().gdpa_cache_fwd(
        _cache_at(where, d, cache), _rows_at(where, d, cache, q, q_stride, n, Hq), q_stride,
        _at(where, d, _i32_t, offsets, b + 1), _at(where, d, _i32_t, kv_lens, b),
        _table_at(where, d, page_table, b, max_pages), T, B, Hq, max_pages, max_q, causal, window_tokens, scale,
        _heads_at(where, d, cache, out, n * Hq),
        _at(where, d, _f32, lse, n * Hq), _at(where, d, _u8, workspace, workspace_bytes), workspace_bytes,
        (_raw_stream(d) or None) if stream is None else _stream(stream)), where)


def gdpa_cache_workspace_size(cache: KvCache, Hq, max_q) -> int:
    """Bytes of workspace gdpa_cache_fwd needs on the current device."""
    n = ctypes.c_int64(0)
    _check(lib().gdpa_cache_workspace_size(cache.addr, int(Hq), int(max_q), ctypes.byref(n)),
           "gdpa_cache_workspace_size")
    return n.value
