"""Thin ctypes binding of libw12.so (include/w12.h), same names as the C calls.

Argument marshalling only: host arrays are numpy, device buffers are torch
CUDA tensors (used for their memory and streams); every computation runs in
the library's kernels or its host encoder.  The library is loaded on first
use from ``lossless_bit_weight_w12_gb300/_build/libw12.so``; if it is missing
this raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libw12.so")

OK = 0
ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_BLOB = 1, 2, 3, 4, 5
ERR_TOO_MANY_ESCAPES, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE = 6, 7, 8, 9
LAYOUT_KN, LAYOUT_NK = 0, 1
F32, BF16 = 0, 1
PATH_AUTO, PATH_GEMV, PATH_MMA, PATH_TC = 0, 1, 2, 3
OPT_EARLY_WEIGHTS = 0x100  # OR into a path: weight copies start under the previous kernel's tail
MAX_M = 128
ATTEND_MAX_R = 512
SAMPLE_MAX_V = 524288
KV_BF16, KV_E4M3 = 0, 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BASE, ROPE_SCALE_BANDS, ROPE_SCALE_YARN = 0, 1, 2, 3, 4

# every symbol include/w12.h declares
EXPORTS = (
    "w12_status_string", "w12_version", "w12_encode_plan", "w12_encode", "w12_validate",
    "w12_decode", "w12_gemm_workspace_size", "w12_gemm", "w12_gemm_ex",
    "w12_verify_workspace_size", "w12_verify_greedy", "w12_verify_lmhead_workspace_size",
    "w12_verify_greedy_lmhead", "w12_get_device_error", "w12_verify_greedy_noalloc",
    "w12_gemm_batched_workspace_size", "w12_gemm_batched", "w12_gemm_batched_ex",
    "w12_encode_device_workspace_size", "w12_encode_plan_device", "w12_encode_device",
    "w12_gemm_batched_debug", "w12_rope_table", "w12_kv_append", "w12_kv_read",
    "w12_attend_workspace_size", "w12_attend", "w12_sample_workspace_size", "w12_sample",
)


class W12Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


class _CDesc(ctypes.Structure):
    _fields_ = [("version", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("G", ctypes.c_int64),
                ("tiles", ctypes.c_uint64), ("unit_bytes", ctypes.c_uint64),
                ("n_units", ctypes.c_uint64), ("off_units", ctypes.c_uint64),
                ("off_esc", ctypes.c_uint64), ("n_esc", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64)]


class _CDebug(ctypes.Structure):
    _fields_ = [("withhold_unit", ctypes.c_int32), ("wait_limit_us", ctypes.c_uint32)]


class _CKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _CRopeScaling(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("reserved", ctypes.c_int32), ("factor", ctypes.c_double),
                ("original", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("attention", ctypes.c_double)]


@dataclass(frozen=True)
class Desc:
    """w12_desc of one encoded K x N matrix."""
    version: int
    K: int
    N: int
    G: int
    tiles: int
    unit_bytes: int
    n_units: int
    off_units: int
    off_esc: int
    n_esc: int
    total_bytes: int

    def c(self) -> _CDesc:
        return _CDesc(self.version, 0, self.K, self.N, self.G, self.tiles, self.unit_bytes,
                      self.n_units, self.off_units, self.off_esc, self.n_esc, self.total_bytes)

    @staticmethod
    def from_c(c: _CDesc) -> "Desc":
        return Desc(c.version, c.K, c.N, c.G, c.tiles, c.unit_bytes, c.n_units, c.off_units,
                    c.off_esc, c.n_esc, c.total_bytes)


_lib = None


def lib():
    """Load libw12.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libw12.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        D = ctypes.POINTER(_CDesc)
        L.w12_status_string.restype = ctypes.c_char_p
        L.w12_status_string.argtypes = [I]
        L.w12_version.argtypes = []
        L.w12_encode_plan.argtypes = [P, I64, I64, I, D]
        L.w12_encode.argtypes = [P, I64, I64, I, D, P]
        L.w12_validate.argtypes = [D, P]
        L.w12_decode.argtypes = [D, P, P, I, P, P]
        L.w12_gemm_workspace_size.restype = SZ
        L.w12_gemm_workspace_size.argtypes = [D, I64]
        L.w12_gemm.argtypes = [D, P, P, I64, P, I, P, SZ, P]
        L.w12_gemm_ex.argtypes = [D, P, P, I64, P, I, P, SZ, I, P]
        L.w12_verify_workspace_size.restype = SZ
        L.w12_verify_workspace_size.argtypes = [I64, I64, I64]
        L.w12_verify_greedy.argtypes = [P, I, I64, I64, I64, P, P, P, P, SZ, P]
        L.w12_verify_lmhead_workspace_size.restype = SZ
        L.w12_verify_lmhead_workspace_size.argtypes = [D, I64, I64]
        L.w12_verify_greedy_lmhead.argtypes = [P, D, P, I64, I64, P, P, P, P, P, SZ, P]
        L.w12_get_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_int), P]
        L.w12_verify_greedy_noalloc.argtypes = [P, I, I64, I64, I64, P, P, P, P]
        L.w12_gemm_batched_workspace_size.restype = SZ
        L.w12_gemm_batched_workspace_size.argtypes = [D, I, I64]
        L.w12_gemm_batched.argtypes = [D, P, P, I64, P, I, I, P, SZ, P]
        L.w12_gemm_batched_ex.argtypes = [D, P, P, I64, P, I, I, P, SZ, I, P]
        L.w12_encode_device_workspace_size.restype = SZ
        L.w12_encode_device_workspace_size.argtypes = [I64, I64]
        L.w12_encode_plan_device.argtypes = [P, I64, I64, I, D, P, SZ, P]
        L.w12_encode_device.argtypes = [P, I64, I64, I, D, P, P, SZ, P]
        L.w12_gemm_batched_debug.argtypes = [D, P, P, I64, P, I, I, P, SZ, I, ctypes.POINTER(_CDebug), P]
        KV = ctypes.POINTER(_CKV)
        L.w12_rope_table.argtypes = [I64, I, ctypes.c_double, ctypes.POINTER(_CRopeScaling), P]
        L.w12_kv_append.argtypes = [KV, P, I64, P, I64, P, I64, I, I64, I64, I, P, I64, P, P, I64, I, I, P, I64,
                                    P, P]
        L.w12_kv_read.argtypes = [KV, P, I64, P, I64, I64, P, P, P, P]
        L.w12_attend_workspace_size.restype = SZ
        L.w12_attend_workspace_size.argtypes = [KV, I64, I64, I, I64, I64]
        L.w12_attend.argtypes = [KV, P, I64, I64, I64, I, P, I64, P, I64, I64, ctypes.c_float, P, I64, P, P, SZ, P]
        L.w12_sample_workspace_size.restype = SZ
        L.w12_sample_workspace_size.argtypes = [I64, I64, I64]
        L.w12_sample.argtypes = [P, I, I64, I64, I64, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().w12_status_string(status).decode()


def version() -> int:
    return lib().w12_version()


def _check(st: int, what: str):
    if st != OK:
        raise W12Error(st, what)


def _np_ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dptr(t):
    """Device pointer of a torch CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_raw_stream = None


def _stream_of(t, stream):
    """The stream handle for a call on tensor t's device (the decode-step
    calls take microseconds: the current stream is asked for without a
    torch.cuda.Stream object where torch can)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(t.get_device())


def _kn(w, layout):
    return (w.shape[0], w.shape[1]) if layout == LAYOUT_KN else (w.shape[1], w.shape[0])


# --------------------------------------------------------------------- host

def encode_plan(w: np.ndarray, layout: int = LAYOUT_NK) -> Desc:
    w = np.ascontiguousarray(w, dtype=np.uint16)
    K, N = _kn(w, layout)
    c = _CDesc()
    _check(lib().w12_encode_plan(_np_ptr(w), K, N, layout, ctypes.byref(c)), "w12_encode_plan")
    return Desc.from_c(c)


def encode(w: np.ndarray, layout: int = LAYOUT_NK, desc: Desc | None = None):
    """Encode bf16 bit patterns w on the host; returns (Desc, blob uint8 array)."""
    w = np.ascontiguousarray(w, dtype=np.uint16)
    K, N = _kn(w, layout)
    d = desc if desc is not None else encode_plan(w, layout)
    blob = np.empty(d.total_bytes, dtype=np.uint8)
    c = d.c()
    _check(lib().w12_encode(_np_ptr(w), K, N, layout, ctypes.byref(c), _np_ptr(blob)),
           "w12_encode")
    return d, blob


def validate(d: Desc, blob: np.ndarray) -> int:
    """Returns the status (OK or ERR_BLOB / ERR_ARG) without raising."""
    blob = np.ascontiguousarray(blob, dtype=np.uint8)
    c = d.c()
    return lib().w12_validate(ctypes.byref(c), _np_ptr(blob))


# ------------------------------------------------------------------- device

def decode(d: Desc, blob_dev, w_dev, layout: int = LAYOUT_NK, err_dev=None, stream=None):
    c = d.c()
    _check(lib().w12_decode(ctypes.byref(c), _dptr(blob_dev), _dptr(w_dev), layout,
                            _dptr(err_dev), _stream(stream)), "w12_decode")


def encode_device(w_dev, layout: int = LAYOUT_NK, stream=None):
    """Encode bf16 bit patterns already on the device (a torch int16/uint16
    CUDA tensor, [N, K] for LAYOUT_NK or [K, N] for LAYOUT_KN) on the GPU;
    returns (Desc, blob device tensor, 256-byte aligned)."""
    import torch
    K, N = _kn(w_dev, layout)
    ws = workspace(lib().w12_encode_device_workspace_size(K, N), w_dev.device)
    c = _CDesc()
    _check(lib().w12_encode_plan_device(_dptr(w_dev), K, N, layout, ctypes.byref(c), _dptr(ws), ws.numel(),
                                        _stream(stream)), "w12_encode_plan_device")
    d = Desc.from_c(c)
    t = torch.empty(d.total_bytes + 256, dtype=torch.uint8, device=w_dev.device)
    off = (-t.data_ptr()) % 256
    blob = t[off:off + d.total_bytes]
    if d.total_bytes:
        c = d.c()
        _check(lib().w12_encode_device(_dptr(w_dev), K, N, layout, ctypes.byref(c), _dptr(blob), _dptr(ws),
                                       ws.numel(), _stream(stream)), "w12_encode_device")
    return d, blob


def gemm_workspace_size(d: Desc, M: int) -> int:
    c = d.c()
    return int(lib().w12_gemm_workspace_size(ctypes.byref(c), M))


def gemm(d: Desc, blob_dev, x_dev, y_dev, ws_dev, path: int = PATH_AUTO, stream=None):
    """y_dev[M, N] (float32 or bfloat16) = x_dev[M, K] (bfloat16) @ W."""
    import torch
    M = x_dev.shape[0]
    y_dtype = F32 if y_dev.dtype == torch.float32 else BF16
    c = d.c()
    _check(lib().w12_gemm_ex(ctypes.byref(c), _dptr(blob_dev), _dptr(x_dev), M, _dptr(y_dev),
                             y_dtype, _dptr(ws_dev), ws_dev.numel() * ws_dev.element_size(),
                             path, _stream(stream)), "w12_gemm")


def _desc_array(descs):
    arr = (_CDesc * len(descs))()
    for i, d in enumerate(descs):
        arr[i] = d.c()
    return arr


def gemm_batched_workspace_size(descs, M: int) -> int:
    return int(lib().w12_gemm_batched_workspace_size(_desc_array(descs), len(descs), M))


class GemmBatch:
    """Marshalled arguments of one w12_gemm_batched call (built once, reused:
    the pointer arrays stay valid while the tensors live)."""

    def __init__(self, descs, blobs, xs, ys, ws, path: int = PATH_AUTO):
        import torch
        n = len(descs)
        self.path = path
        self.descs = _desc_array(descs)
        self.blobs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in blobs])
        self.xs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in xs])
        self.ys = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ys])
        self.M = xs[0].shape[0]
        self.y_dtype = F32 if ys[0].dtype == torch.float32 else BF16
        self.count = n
        self.ws = ws
        self._keep = (blobs, xs, ys, ws)

    def __call__(self, stream=None):
        _check(lib().w12_gemm_batched_ex(self.descs, self.blobs, self.xs, self.M, self.ys,
                                         self.y_dtype, self.count, _dptr(self.ws),
                                         self.ws.numel() * self.ws.element_size(), self.path,
                                         _stream(stream)),
               "w12_gemm_batched_ex")


def gemm_batched(descs, blobs, xs, ys, ws, path: int = PATH_AUTO, stream=None):
    """ys[i] = xs[i] @ W_i for every i, in one launch."""
    GemmBatch(descs, blobs, xs, ys, ws, path)(stream)


def gemm_batched_debug(descs, blobs, xs, ys, ws, withhold_unit: int = -1, wait_limit_us: int = 0,
                       path: int = PATH_AUTO, stream=None):
    """w12_gemm_batched_debug: the batched GEMM with the test hooks (a
    withheld weight copy, a short wait limit)."""
    b = GemmBatch(descs, blobs, xs, ys, ws, path)
    dbg = _CDebug(withhold_unit, wait_limit_us)
    _check(lib().w12_gemm_batched_debug(b.descs, b.blobs, b.xs, b.M, b.ys, b.y_dtype, b.count, _dptr(ws),
                                        ws.numel() * ws.element_size(), path, ctypes.byref(dbg),
                                        _stream(stream)),
           "w12_gemm_batched_debug")


def verify_workspace_size(R: int, T: int, V: int) -> int:
    return int(lib().w12_verify_workspace_size(R, T, V))


def verify_greedy(logits_dev, R: int, T: int, draft_dev, accept_dev, next_dev, ws_dev,
                  stream=None):
    import torch
    dtype = F32 if logits_dev.dtype == torch.float32 else BF16
    V = logits_dev.shape[-1]
    _check(lib().w12_verify_greedy(_dptr(logits_dev), dtype, R, T, V, _dptr(draft_dev),
                                   _dptr(accept_dev), _dptr(next_dev), _dptr(ws_dev),
                                   ws_dev.numel() * ws_dev.element_size(), _stream(stream)),
           "w12_verify_greedy")


def verify_lmhead_workspace_size(d: Desc, R: int, T: int) -> int:
    c = d.c()
    return int(lib().w12_verify_lmhead_workspace_size(ctypes.byref(c), R, T))


def verify_greedy_lmhead(hidden_dev, d: Desc, blob_dev, R: int, T: int, draft_dev, accept_dev,
                         next_dev, ws_dev, logits_out_dev=None, stream=None):
    c = d.c()
    _check(lib().w12_verify_greedy_lmhead(_dptr(hidden_dev), ctypes.byref(c), _dptr(blob_dev),
                                          R, T, _dptr(draft_dev), _dptr(accept_dev),
                                          _dptr(next_dev), _dptr(logits_out_dev), _dptr(ws_dev),
                                          ws_dev.numel() * ws_dev.element_size(),
                                          _stream(stream)), "w12_verify_greedy_lmhead")


def verify_greedy_noalloc(logits_dev, R: int, T: int, draft_dev, accept_dev, next_dev,
                          stream=None):
    """verify_greedy() on the library's own fixed scratch array: for callers
    that cannot allocate device memory (see include/w12.h)."""
    import torch
    dtype = F32 if logits_dev.dtype == torch.float32 else BF16
    V = logits_dev.shape[-1]
    _check(lib().w12_verify_greedy_noalloc(_dptr(logits_dev), dtype, R, T, V, _dptr(draft_dev),
                                           _dptr(accept_dev), _dptr(next_dev), _stream(stream)),
           "w12_verify_greedy_noalloc")


def get_device_error(ws_dev, stream=None) -> int:
    v = ctypes.c_int(0)
    _check(lib().w12_get_device_error(_dptr(ws_dev), ctypes.byref(v), _stream(stream)),
           "w12_get_device_error")
    return v.value


# ------------------------------------------------- decode step: paged cache

class KVCache:
    """A paged cache over device tensors (w12_kv): k, v [n_pages, heads, page,
    head_dim] bfloat16 or float8_e4m3fn; for e4m3 the scales [n_pages, heads,
    page] float32.  Holds the tensors and the marshalled descriptor."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        kinds = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3}
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in kinds:
            raise ValueError("k and v: bfloat16 or float8_e4m3fn tensors [n_pages, heads, page, head_dim]")
        self.dtype = kinds[k.dtype]
        for t in (k_scale, v_scale):
            if (t is None) != (self.dtype == KV_BF16):
                raise ValueError("e4m3 caches have scales, bf16 caches have none")
            if t is not None and (t.shape != k.shape[:3] or t.dtype != torch.float32):
                raise ValueError("scales: float32 tensors [n_pages, heads, page]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.heads, self.page, self.head_dim = k.shape
        self.c = _CKV(_dptr(k), _dptr(v), _dptr(k_scale), _dptr(v_scale), self.n_pages, self.heads,
                      self.head_dim, self.page, self.dtype)
        self.ref = ctypes.byref(self.c)

    @staticmethod
    def alloc(n_pages: int, heads: int, head_dim: int, page: int = 64, dtype: int = KV_BF16, device="cuda"):
        """An empty cache of n_pages pages."""
        import torch
        shape = (n_pages, heads, page, head_dim)
        if dtype == KV_BF16:
            return KVCache(*(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        kv = [torch.empty(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        return KVCache(*kv, *(torch.empty(shape[:3], device=device) for _ in range(2)))


def _ptr(t):
    """Address of a contiguous CUDA tensor (None: NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _heads_ptr(t, n: int, heads: int, dim: int, dtype):
    """(address, token stride) of [n, heads, dim] rows of a type with contiguous heads."""
    if t.shape != (n, heads, dim) or t.dtype is not dtype:
        raise ValueError(f"expected {dtype} [{n}, {heads}, {dim}], got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    token, head, one = t.stride()
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError("expected contiguous heads")
    return t.data_ptr(), token


def _typed_ptr(t, dtype, n: int, what: str):
    """Address of a contiguous CUDA tensor of n elements of a type (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n:
        raise ValueError(f"{what}: expected {n} elements of {dtype}")
    return _ptr(t)


def _err_ptr(t):
    """Address of an error word, the first element of an int32 CUDA tensor (None: NULL)."""
    if t is None:
        return None
    import torch
    if t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError("err_dev: expected an int32 tensor")
    return _ptr(t)


def rope_table(positions: int, rot: int, base: float = 10000.0, mode: int = ROPE_SCALE_NONE, factor: float = 1.0,
               original: float = 0.0, low: float = 1.0, high: float = 32.0, attention: float = 0.0) -> np.ndarray:
    """w12_rope_table: float32 [positions, rot], cosines then sines (host)."""
    table = np.empty((positions, rot), dtype=np.float32)
    sc = _CRopeScaling(mode, 0, factor, original, low, high, attention)
    _check(lib().w12_rope_table(positions, rot, base, ctypes.byref(sc), _np_ptr(table)), "w12_rope_table")
    return table


def kv_append(kv: KVCache, q, k, v, block_table, kv_len, T: int, q_out, table=None, layout: int = ROPE_HALF,
              err_dev=None, stream=None):
    """Rotate the new tokens' queries (into q_out, bfloat16) and keys and write
    keys and values into the cache.  q [R*T, q_heads, head_dim], k and v
    [R*T, heads, head_dim]: float32 or bfloat16, any token stride (parts of
    one projection output); block_table [R, blocks] and kv_len [R] int32;
    table: the rotary table on the device (None: no rotation)."""
    import torch
    n, hq, dim = q.shape
    R, blocks = block_table.shape
    x = q.dtype
    if n != R * T or dim != kv.head_dim or (x is not torch.float32 and x is not torch.bfloat16):
        raise ValueError("q: R * T tokens of head_dim channels, float32 or bfloat16")
    qp, qs = _heads_ptr(q, n, hq, dim, x)
    kp, ks = _heads_ptr(k, n, kv.heads, dim, x)
    vp, vs = _heads_ptr(v, n, kv.heads, dim, x)
    op, os_ = _heads_ptr(q_out, n, hq, dim, torch.bfloat16)
    positions, rot = (0, 0) if table is None else table.shape
    st = lib().w12_kv_append(kv.ref, qp, qs, kp, ks, vp, vs, F32 if x is torch.float32 else BF16, R, T, hq,
                             _typed_ptr(block_table, torch.int32, R * blocks, "block_table"), blocks,
                             _typed_ptr(kv_len, torch.int32, R, "kv_len"),
                             _typed_ptr(table, torch.float32, positions * rot, "table"), positions, rot, layout, op,
                             os_, _err_ptr(err_dev), _stream_of(q, stream))
    if st:
        raise W12Error(st, "w12_kv_append")


def kv_read(kv: KVCache, block_table, cu_len, k_out, v_out, err_dev=None, stream=None):
    """Read rows 0 .. cu_len[r+1] - cu_len[r] - 1 of every request back, packed
    into k_out and v_out [tokens, heads, head_dim] bfloat16."""
    import torch
    R, blocks = block_table.shape
    n = k_out.shape[0]
    kp, _ = _heads_ptr(k_out, n, kv.heads, kv.head_dim, torch.bfloat16)
    vp, _ = _heads_ptr(v_out, n, kv.heads, kv.head_dim, torch.bfloat16)
    if not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError("outputs: contiguous")
    st = lib().w12_kv_read(kv.ref, _typed_ptr(block_table, torch.int32, R * blocks, "block_table"), blocks,
                           _typed_ptr(cu_len, torch.int32, R + 1, "cu_len"), R, n, kp, vp, _err_ptr(err_dev),
                           _stream_of(k_out, stream))
    if st:
        raise W12Error(st, "w12_kv_read")


def attend_workspace_size(kv: KVCache, R: int, T: int, q_heads: int, max_len: int, prefix_len: int = 0) -> int:
    return int(lib().w12_attend_workspace_size(kv.ref, R, T, q_heads, max_len, prefix_len))


def attend(kv: KVCache, q, block_table, kv_len, T: int, max_len: int, out, ws_dev, scale: float | None = None,
           prefix_len: int = 0, lse_dev=None, stream=None):
    """Causal attention of the R * T newest tokens over the cache.  q and out
    [R*T, q_heads, head_dim] bfloat16 (any token stride); scale: 1 /
    sqrt(head_dim) by default; the first prefix_len keys are shared by all
    requests; lse_dev: float32 [R*T, q_heads] or None."""
    import torch
    n, hq, dim = q.shape
    R, blocks = block_table.shape
    if n != R * T or dim != kv.head_dim:
        raise ValueError("q: R * T tokens of head_dim channels")
    qp, qs = _heads_ptr(q, n, hq, dim, torch.bfloat16)
    op, os_ = _heads_ptr(out, n, hq, dim, torch.bfloat16)
    st = lib().w12_attend(kv.ref, qp, qs, R, T, hq, _typed_ptr(block_table, torch.int32, R * blocks, "block_table"),
                          blocks, _typed_ptr(kv_len, torch.int32, R, "kv_len"), max_len, prefix_len,
                          dim ** -0.5 if scale is None else scale, op, os_,
                          _typed_ptr(lse_dev, torch.float32, n * hq, "lse"), _ptr(ws_dev), ws_dev.nbytes,
                          _stream_of(q, stream))
    if st:
        raise W12Error(st, "w12_attend")


# ---------------------------------------------------- decode step: sampling

def sample_workspace_size(R: int, T: int, V: int) -> int:
    return int(lib().w12_sample_workspace_size(R, T, V))


def sample(logits, R: int, T: int, u, tokens_dev, ws_dev, temperature=None, top_k=None, top_p=None, min_p=None,
           prob_dev=None, draft_dev=None, accept_dev=None, next_dev=None, stream=None):
    """One token for each of R * T rows of logits [R*T, V] (float32 or
    bfloat16) from the random numbers u [R*T]; temperature, top_p, min_p
    (float32) and top_k (int32): [R] or None; with accept_dev and next_dev the
    drafts are accepted against the sampled tokens."""
    import torch
    x, f32, i32 = logits.dtype, torch.float32, torch.int32
    V = logits.shape[-1]
    n = R * T
    if x is not f32 and x is not torch.bfloat16:
        raise ValueError("logits: float32 or bfloat16")
    st = lib().w12_sample(_typed_ptr(logits, x, n * V, "logits"), F32 if x is f32 else BF16, R, T, V,
                          _typed_ptr(temperature, f32, R, "temperature"), _typed_ptr(top_k, i32, R, "top_k"),
                          _typed_ptr(top_p, f32, R, "top_p"), _typed_ptr(min_p, f32, R, "min_p"),
                          _typed_ptr(u, f32, n, "u"), _typed_ptr(tokens_dev, i32, n, "tokens"),
                          _typed_ptr(prob_dev, f32, n, "prob"), _typed_ptr(draft_dev, i32, R * (T - 1), "draft"),
                          _typed_ptr(accept_dev, i32, R, "accept"), _typed_ptr(next_dev, i32, R, "next"),
                          _ptr(ws_dev), ws_dev.nbytes, _stream_of(logits, stream))
    if st:
        raise W12Error(st, "w12_sample")


# --------------------------------------------------------------- helpers

def workspace(nbytes: int, device="cuda"):
    """A zero-filled, 256-byte aligned device workspace of nbytes (torch uint8)."""
    import torch
    t = torch.zeros(max(int(nbytes), 256) + 256, dtype=torch.uint8, device=device)
    off = (-t.data_ptr()) % 256
    return t[off:off + max(int(nbytes), 256)]


def upload(blob: np.ndarray, device="cuda"):
    """Copy a host blob to a 256-byte aligned device buffer."""
    import torch
    n = blob.size
    t = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-t.data_ptr()) % 256
    t = t[off:off + n]
    t.copy_(torch.from_numpy(np.ascontiguousarray(blob)))
    return t


class Weight:
    """An encoded matrix resident on the device: desc + 256-byte aligned blob."""

    def __init__(self, w: np.ndarray, layout: int = LAYOUT_NK, device="cuda"):
        self.desc, blob = encode(w, layout)
        self.blob = upload(blob, device)

    @property
    def K(self):
        return self.desc.K

    @property
    def N(self):
        return self.desc.N
