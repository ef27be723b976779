"""Python binding of attention over the int8 K/V cache (include/kv8.h), same
names as the C ABI; the functions live in the same libi2s.so.

Argument marshalling only: every step runs in the library's HIP kernels.  No
fallback: a missing library or a failed call raises.  A KV8Cache names the
four tensors of a cache, a KV8Batch the sequences of a call; both only hold
tensors and may be kept as long as those are in place (their contents may
change from call to call).

Every call runs on the device of its tensors.  `stream` (a torch stream or a
raw handle; default: that device's current stream) is where the kernels are
enqueued: outputs and workspaces that a call allocates are recorded on it.
"""

from __future__ import annotations

import ctypes
import os
import re

import torch

from . import i2s
from .i2s import I2SError

HEADER_PATH = os.path.join(os.path.dirname(i2s._PKG), "include", "kv8.h")

KV8_F32, KV8_F16, KV8_BF16 = 0, 1, 2
KV8_MAX_DIM, KV8_MAX_PAGE = 256, 256
_TYPES = {torch.float32: KV8_F32, torch.float16: KV8_F16, torch.bfloat16: KV8_BF16}

_lib = None


class _Cache(ctypes.Structure):
    """struct kv8_cache of include/kv8.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    """struct kv8_batch of include/kv8.h."""
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("blocks", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("seqs", ctypes.c_int64),
                ("max_len", ctypes.c_int64)]


def declared_symbols() -> list[str]:
    """Names of the functions include/kv8.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^[A-Za-z_][\w \*]*?\b(kv8_\w+)\s*\(", text, flags=re.M)


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = i2s.lib()
        i64, p, sz, ci, f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
        L.kv8_append.restype = ci
        L.kv8_append.argtypes = [p, p, ci, p, i64, p, i64, i64, p]
        L.kv8_read.restype = ci
        L.kv8_read.argtypes = [p, p, ci, p, i64, p, i64, i64, p]
        L.kv8_attention_workspace_bytes.restype = sz
        L.kv8_attention_workspace_bytes.argtypes = [p, p, i64, i64]
        L.kv8_attention.restype = ci
        L.kv8_attention.argtypes = [p, p, ci, p, i64, i64, i64, f, ci, i64, p, i64, p, p, sz, p]
        L.kv8_qk_norm_rope.restype = ci
        L.kv8_qk_norm_rope.argtypes = [ci, i64, i64, p, i64, i64, p, i64, i64, p, p, i64, ci, p, p, f, p, i64, p, i64, p]
        _lib = L
    return _lib


def _need(t, dtype, dim: int, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {tuple(t.shape)}")
    return t


class KV8Cache:
    """A cache's tensors: k int8 [pages][heads][P][dim], v int8
    [pages][heads][dim][P], k_scale and v_scale F32 [pages][heads]."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "heads", "dim", "page_tokens", "device", "_c", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _need(k, torch.int8, 4, "k")
        _need(v, torch.int8, 4, "v")
        pages, heads, page_tokens, dim = k.shape
        if tuple(v.shape) != (pages, heads, dim, page_tokens):
            raise ValueError(f"v must be [pages][heads][dim][page_tokens] to k's {tuple(k.shape)}, got {tuple(v.shape)}")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if tuple(_need(s, torch.float32, 2, name).shape) != (pages, heads):
                raise ValueError(f"{name} must be [{pages}][{heads}], got {tuple(s.shape)}")
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.device != k.device:
                raise ValueError(f"{name} is on another device than k")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.dim, self.page_tokens = pages, heads, dim, page_tokens
        self.device = k.device
        self._c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads, dim, page_tokens)
        self._ref = ctypes.addressof(self._c)


def new_cache(pages: int, heads: int, dim: int, page_tokens: int = 64, device="cuda") -> KV8Cache:
    """An empty cache (codes and scales zero)."""
    return KV8Cache(torch.zeros((pages, heads, page_tokens, dim), dtype=torch.int8, device=device),
                    torch.zeros((pages, heads, dim, page_tokens), dtype=torch.int8, device=device),
                    torch.zeros((pages, heads), dtype=torch.float32, device=device),
                    torch.zeros((pages, heads), dtype=torch.float32, device=device))


class KV8Batch:
    """The sequences of a call: table int32 [seqs][blocks], lens int32 [seqs],
    starts None (every sequence has as many rows) or int32 [seqs + 1].
    max_len: 0, or a bound of the lengths; it steers the attention's split."""

    __slots__ = ("table", "lens", "starts", "max_len", "seqs", "device", "_c", "_ref")

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor | None = None, max_len: int = 0):
        _need(table, torch.int32, 2, "table")
        _need(lens, torch.int32, 1, "lens")
        seqs, blocks = table.shape
        if blocks > 1 and table.stride(1) != 1:
            raise ValueError("table must have unit innermost stride")
        if lens.shape[0] != seqs or not lens.is_contiguous():
            raise ValueError(f"lens must be a contiguous [{seqs}], got {tuple(lens.shape)}")
        if starts is not None:
            _need(starts, torch.int32, 1, "starts")
            if starts.shape[0] != seqs + 1 or not starts.is_contiguous():
                raise ValueError(f"starts must be a contiguous [{seqs + 1}], got {tuple(starts.shape)}")
        if lens.device != table.device or (starts is not None and starts.device != table.device):
            raise ValueError("table, lens and starts are on different devices")
        self.table, self.lens, self.starts, self.max_len, self.seqs = table, lens, starts, max_len, seqs
        self.device = table.device
        self._c = _Batch(table.data_ptr(), max(table.stride(0), blocks), blocks, lens.data_ptr(),
                         None if starts is None else starts.data_ptr(), seqs, max_len)
        self._ref = ctypes.addressof(self._c)


_raw_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """The device a call runs on made current, if it is not, and its stream."""

    __slots__ = ("stream", "apart", "_guard")

    def __init__(self, device: torch.device, stream):
        index = device.index
        current = torch.cuda.current_device()
        self._guard = None if index == current else torch.cuda.device(index)
        own = _raw_stream(index)
        if stream is None:
            self.stream, self.apart = own, None
            return
        if hasattr(stream, "cuda_stream"):
            if stream.device.index != index:
                raise ValueError("stream is on another device than the tensors")
            self.stream = stream.cuda_stream
        else:
            self.stream = int(stream)
        self.apart = None
        if self.stream != own:
            self.apart = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(self.stream, device=device)

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        return self

    def __exit__(self, *a):
        if self._guard is not None:
            self._guard.__exit__(*a)

    def made(self, t: torch.Tensor) -> torch.Tensor:
        """A tensor that the call allocated (on the current stream) for use on its stream."""
        if self.apart is not None:
            t.record_stream(self.apart)
        return t


def _heads(t, heads, dim: int, dtype, device, name: str):
    """(pointer, row stride, heads) of rows [rows][heads][dim] with dense heads."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [rows][heads][{dim}] tensor")
    shape, stride = t.shape, t.stride()
    if (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must be [rows][{'heads' if heads is None else heads}][{dim}], got {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if shape[0] and shape[1] and (stride[2] != 1 or (shape[1] > 1 and stride[1] != dim)):
        raise ValueError(f"{name} must have dense heads (strides [*, {dim}, 1]), got {stride}")
    width = shape[1] * dim
    return t.data_ptr(), (stride[0] if shape[0] > 1 else width), shape[1]


def _type(dtype) -> int:
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError(f"rows must be float32, float16 or bfloat16, got {dtype}")
    return code


def _same_device(cache: KV8Cache, batch: KV8Batch) -> torch.device:
    if cache.device != batch.device:
        raise ValueError("cache and batch are on different devices")
    return cache.device


def _fail(fn: str, status: int):
    raise I2SError(fn, status)


def kv8_append(cache: KV8Cache, batch: KV8Batch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Quantize rows k, v [rows][heads][dim] into the cache's pages."""
    device = _same_device(cache, batch)
    code = _type(k.dtype)
    kp, ks, _ = _heads(k, cache.heads, cache.dim, k.dtype, device, "k")
    vp, vs, _ = _heads(v, cache.heads, cache.dim, k.dtype, device, "v")
    rows = k.shape[0]
    if v.shape[0] != rows:
        raise ValueError("k and v have different numbers of rows")
    with _On(device, stream) as on:
        st = lib().kv8_append(cache._ref, batch._ref, code, kp, ks, vp, vs, rows, on.stream)
    if st:
        _fail("kv8_append", st)


def kv8_read(cache: KV8Cache, batch: KV8Batch, rows: int, dtype=torch.float32, k=None, v=None, stream=None):
    """(k, v), each [rows][heads][dim] of `dtype`: the batch's tokens as values.
    Rows outside the batch's are left as they were in a given k or v, and are
    undefined in one allocated here."""
    device = _same_device(cache, batch)
    with _On(device, stream) as on:
        shape = (rows, cache.heads, cache.dim)
        k = on.made(torch.empty(shape, dtype=dtype, device=device)) if k is None else k
        v = on.made(torch.empty(shape, dtype=dtype, device=device)) if v is None else v
        if k.shape[0] != rows or v.shape[0] != rows:
            raise ValueError(f"k and v must have {rows} rows")
        code = _type(k.dtype)
        kp, ks, _ = _heads(k, cache.heads, cache.dim, k.dtype, device, "k")
        vp, vs, _ = _heads(v, cache.heads, cache.dim, k.dtype, device, "v")
        st = lib().kv8_read(cache._ref, batch._ref, code, kp, ks, vp, vs, rows, on.stream)
    if st:
        _fail("kv8_read", st)
    return k, v


def kv8_attention_workspace_bytes(cache: KV8Cache, batch: KV8Batch, q_heads: int, rows: int) -> int:
    return int(lib().kv8_attention_workspace_bytes(cache._ref, batch._ref, q_heads, rows))


def kv8_attention(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, scale: float | None = None, causal: bool = True,
                  window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [rows][q_heads][dim] over the batch's cached tokens: out,
    of q's shape and type (and lse F32 [rows][q_heads] if lse is a tensor or
    True).  scale: default dim ** -0.5.  Rows outside the batch's are left as
    they were in a given out or lse, and are undefined in one allocated here."""
    device = _same_device(cache, batch)
    code = _type(q.dtype)
    dim = cache.dim
    qp, qs, q_heads = _heads(q, None, dim, q.dtype, device, "q")
    rows = q.shape[0]
    L = lib()
    with _On(device, stream) as on:
        if out is None:
            out = on.made(torch.empty((rows, q_heads, dim), dtype=q.dtype, device=device))
        elif out.shape[0] != rows:
            raise ValueError(f"out must have {rows} rows")
        op, os_, _ = _heads(out, q_heads, dim, q.dtype, device, "out")
        lp = None
        if lse is not None and lse is not False:
            if lse is True:
                lse = on.made(torch.empty((rows, q_heads), dtype=torch.float32, device=device))
            if tuple(_need(lse, torch.float32, 2, "lse").shape) != (rows, q_heads) or not lse.is_contiguous() or lse.device != device:
                raise ValueError(f"lse must be a contiguous [{rows}][{q_heads}] on {device}")
            lp = lse.data_ptr()
        if workspace is None:
            n = L.kv8_attention_workspace_bytes(cache._ref, batch._ref, q_heads, rows)
            if n:
                workspace = on.made(torch.empty(n, dtype=torch.uint8, device=device))
        elif workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
        wp, wn = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
        st = L.kv8_attention(cache._ref, batch._ref, code, qp, qs, q_heads, rows, dim ** -0.5 if scale is None else scale,
                             1 if causal else 0, window, op, os_, lp, wp, wn, on.stream)
    if st:
        _fail("kv8_attention", st)
    return out if lp is None else (out, lse)


def kv8_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor, inv_freq: torch.Tensor, q_weight=None,
                     k_weight=None, eps: float = 1e-6, neighbours: bool = False, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): queries q [rows][q_heads][dim] and keys k
    [rows][k_heads][dim], RMS-normed per head where a weight F32 [dim] is
    given, then rotated by pos int32 [rows] times inv_freq F32 [pairs].  q_out
    may be q and k_out k."""
    device, dtype = q.device, q.dtype
    if not q.is_cuda:
        raise TypeError("q must be a CUDA (HIP) tensor")
    code = _type(dtype)
    rows, dim = q.shape[0], q.shape[-1]
    qp, qs, q_heads = _heads(q, None, dim, dtype, device, "q")
    kp, ks, k_heads = _heads(k, None, dim, dtype, device, "k")
    if k.shape[0] != rows:
        raise ValueError("q and k have different numbers of rows")
    if pos.dtype != torch.int32 or pos.dim() != 1 or pos.shape[0] != rows or not pos.is_contiguous() or pos.device != device:
        raise ValueError(f"pos must be a contiguous int32 [{rows}] on {device}")
    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous() or inv_freq.device != device:
        raise ValueError(f"inv_freq must be a contiguous float32 [pairs] on {device}")
    weights = []
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (dim,) or not w.is_contiguous() or w.device != device):
            raise ValueError(f"{name} must be a contiguous float32 [{dim}] on {device}")
        weights.append(None if w is None else w.data_ptr())
    with _On(device, stream) as on:
        if q_out is None:
            q_out = on.made(torch.empty(q.shape, dtype=dtype, device=device))
        if k_out is None:
            k_out = on.made(torch.empty(k.shape, dtype=dtype, device=device))
        if q_out.shape[0] != rows or k_out.shape[0] != rows:
            raise ValueError(f"q_out and k_out must have {rows} rows")
        qop, qos, _ = _heads(q_out, q_heads, dim, dtype, device, "q_out")
        kop, kos, _ = _heads(k_out, k_heads, dim, dtype, device, "k_out")
        st = lib().kv8_qk_norm_rope(code, rows, dim, qp, qs, q_heads, kp, ks, k_heads, pos.data_ptr(), inv_freq.data_ptr(),
                                    inv_freq.shape[0], 1 if neighbours else 0, weights[0], weights[1], eps, qop, qos, kop, kos,
                                    on.stream)
    if st:
        _fail("kv8_qk_norm_rope", st)
    return q_out, k_out


__all__ = ["KV8Cache", "KV8Batch", "new_cache", "I2SError", "kv8_append", "kv8_read", "kv8_attention",
           "kv8_attention_workspace_bytes", "kv8_qk_norm_rope"]
