"""Python binding of attention over the int8 K/V cache (include/kv8.h), same
names as the C ABI; the functions live in the same libi2s.so.

Argument marshalling only: every step runs in the library's HIP kernels.  No
fallback: a missing library or a failed call raises.  A KV8Cache names the
four tensors of a cache, a KV8Batch the sequences of a call; both only hold
tensors and may be kept as long as those are in place (their contents may
change from call to call).

Every call runs on the device of its tensors.  `stream` (a torch stream or a
raw handle; default: that device's current stream) is where the kernels are
enqueued, and of whose memory outputs and workspaces that a call allocates are
taken: work still queued on the current stream cannot be using it.  Outputs are
recorded on the current stream too, where their user is taken to read them
(after a wait of its own).
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

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "heads", "dim", "page_tokens", "device", "index", "scale",
                 "_c", "_ref")

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
        self.device, self.index, self.scale = k.device, k.get_device(), dim ** -0.5
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

    __slots__ = ("table", "lens", "starts", "max_len", "seqs", "index", "_c", "_ref")

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, starts: torch.Tensor | None = None, max_len: int = 0):
        _need(table, torch.int32, 2, "table")
        _need(lens, torch.int32, 1, "lens")
        seqs, blocks = table.shape
        if blocks > 1 and table.stride(1) != 1:
            raise ValueError("table must have unit innermost stride")
        if seqs > 1 and table.stride(0) < blocks:
            raise ValueError(f"table's rows must not overlap, got strides {table.stride()}")
        if lens.shape[0] != seqs or not lens.is_contiguous():
            raise ValueError(f"lens must be a contiguous [{seqs}], got {tuple(lens.shape)}")
        if starts is not None:
            _need(starts, torch.int32, 1, "starts")
            if starts.shape[0] != seqs + 1 or not starts.is_contiguous():
                raise ValueError(f"starts must be a contiguous [{seqs + 1}], got {tuple(starts.shape)}")
        if lens.device != table.device or (starts is not None and starts.device != table.device):
            raise ValueError("table, lens and starts are on different devices")
        self.table, self.lens, self.starts, self.max_len, self.seqs = table, lens, starts, max_len, seqs
        self.index = table.get_device()
        self._c = _Batch(table.data_ptr(), max(table.stride(0), blocks), blocks, lens.data_ptr(),
                         None if starts is None else starts.data_ptr(), seqs, max_len)
        self._ref = ctypes.addressof(self._c)


_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice


class _Apart:
    """A call on another stream than the tensors' device's current one, or on
    a device that is not current."""

    def __init__(self, index: int, stream):
        self.index, self.other = index, None
        if stream is None:
            self.raw = _raw_stream(index)
        elif hasattr(stream, "cuda_stream"):
            if stream.device.index != index:
                raise ValueError("stream is on another device than the tensors")
            self.raw = stream.cuda_stream
        else:
            self.raw = int(stream)
        if self.raw != _raw_stream(index):
            if hasattr(stream, "cuda_stream"):
                self.other = stream
            elif self.raw:
                self.other = torch.cuda.ExternalStream(self.raw, device=index)
            else:
                self.other = torch.cuda.default_stream(index)

    def new(self, kept: bool, shape, dtype, device) -> torch.Tensor:
        """A new tensor of the memory of the call's stream, recorded on the
        current one if the caller gets it (kept)."""
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(self.other):
            t = torch.empty(shape, dtype=dtype, device=device)
        if kept:
            t.record_stream(torch.cuda.current_stream(self.index))
        return t

    def run(self, fn, args) -> int:
        with torch.cuda.device(self.index):
            return fn(*args, self.raw)


def _place(index: int, stream):
    """Where a call runs: None for the current stream of the current device."""
    return None if stream is None and index == _current() else _Apart(index, stream)


def _call(name: str, fn, args, index: int, at):
    status = fn(*args, _raw_stream(index)) if at is None else at.run(fn, args)
    if status:
        raise I2SError(name, status)


def _heads(t, heads, dim: int, dtype, index: int, name: str):
    """(pointer, row stride, heads, rows) of t [rows][heads][dim] with dense
    heads; heads: their number, or None for any."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be a [rows][heads][{dim}] tensor")
    rows, h, d = t.shape
    if d != dim or (heads is not None and h != heads):
        raise ValueError(f"{name} must be [rows][{'heads' if heads is None else heads}][{dim}], got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), h * d, h, rows
    stride = t.stride()
    if stride[2] != 1 or (h > 1 and stride[1] != dim):
        raise ValueError(f"{name} must have dense heads (strides [*, {dim}, 1]), got {stride}")
    return t.data_ptr(), (stride[0] if rows > 1 else h * d), h, rows


def _dense(at, shape, dtype, device, kept: bool = True) -> torch.Tensor:
    """A new tensor for a call that runs at `at`."""
    return torch.empty(shape, dtype=dtype, device=device) if at is None else at.new(kept, shape, dtype, device)


def _like(t, rows: int, heads: int, dim: int, at) -> torch.Tensor:
    """A dense tensor of t's shape, type and device."""
    return torch.empty_like(t) if at is None and t.is_contiguous() else _dense(at, (rows, heads, dim), t.dtype, t.device)


def _type(t, name: str) -> int:
    code = _TYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or t.get_device() < 0:
        raise TypeError(f"{name} must be a float32, float16 or bfloat16 CUDA (HIP) tensor")
    return code


def _index(cache: KV8Cache, batch: KV8Batch) -> int:
    if cache.index != batch.index:
        raise ValueError("cache and batch are on different devices")
    return cache.index


def kv8_append(cache: KV8Cache, batch: KV8Batch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Quantize rows k, v [rows][heads][dim] into the cache's pages."""
    index = _index(cache, batch)
    code = _type(k, "k")
    kp, ks, _, rows = _heads(k, cache.heads, cache.dim, k.dtype, index, "k")
    vp, vs, _, v_rows = _heads(v, cache.heads, cache.dim, k.dtype, index, "v")
    if v_rows != rows:
        raise ValueError("k and v have different numbers of rows")
    _call("kv8_append", lib().kv8_append, (cache._ref, batch._ref, code, kp, ks, vp, vs, rows), index, _place(index, stream))


def kv8_read(cache: KV8Cache, batch: KV8Batch, rows: int, dtype=torch.float32, k=None, v=None, stream=None):
    """(k, v), each [rows][heads][dim] of `dtype` (or k's or v's own): the
    batch's tokens as values.  Rows outside the batch's are left as they were
    in a given k or v, and are undefined in one allocated here."""
    index = _index(cache, batch)
    heads, dim = cache.heads, cache.dim
    given = k if k is not None else v
    dtype = dtype if given is None else given.dtype
    at, made = _place(index, stream), False
    if k is None:
        k = _dense(at, (rows, heads, dim), dtype, cache.device)
        kp, ks, made = k.data_ptr(), heads * dim, True
    else:
        kp, ks, _, n = _heads(k, heads, dim, dtype, index, "k")
        if n != rows:
            raise ValueError(f"k must have {rows} rows")
    if v is None:
        v = torch.empty_like(k) if made and at is None else _dense(at, (rows, heads, dim), dtype, cache.device)
        vp, vs = v.data_ptr(), heads * dim
    else:
        vp, vs, _, n = _heads(v, heads, dim, dtype, index, "v")
        if n != rows:
            raise ValueError(f"v must have {rows} rows")
    code = _type(k, "k")
    _call("kv8_read", lib().kv8_read, (cache._ref, batch._ref, code, kp, ks, vp, vs, rows), index, at)
    return k, v


def kv8_attention_workspace_bytes(cache: KV8Cache, batch: KV8Batch, q_heads: int, rows: int) -> int:
    return int(lib().kv8_attention_workspace_bytes(cache._ref, batch._ref, q_heads, rows))


def kv8_attention(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, scale: float | None = None, causal: bool = True,
                  window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [rows][q_heads][dim] over the batch's cached tokens: out,
    of q's shape and type (and lse F32 [rows][q_heads] if lse is a tensor or
    True).  scale: default dim ** -0.5.  Rows outside the batch's are left as
    they were in a given out or lse, and are undefined in one allocated here."""
    index = _index(cache, batch)
    code, dim = _type(q, "q"), cache.dim
    qp, qs, q_heads, rows = _heads(q, None, dim, q.dtype, index, "q")
    L, at = lib(), _place(index, stream)
    if out is None:
        out = _like(q, rows, q_heads, dim, at)
        op, os_ = out.data_ptr(), q_heads * dim
    else:
        op, os_, _, n = _heads(out, q_heads, dim, q.dtype, index, "out")
        if n != rows:
            raise ValueError(f"out must have {rows} rows")
    lp = None
    if lse is not None and lse is not False:
        if lse is True:
            lse = _dense(at, (rows, q_heads), torch.float32, cache.device)
        if tuple(_need(lse, torch.float32, 2, "lse").shape) != (rows, q_heads) or not lse.is_contiguous() or lse.get_device() != index:
            raise ValueError(f"lse must be a contiguous [{rows}][{q_heads}] on cuda:{index}")
        lp = lse.data_ptr()
    wp, wn = None, 0
    if workspace is None:
        wn = L.kv8_attention_workspace_bytes(cache._ref, batch._ref, q_heads, rows)
        if wn:
            workspace = _dense(at, wn, torch.uint8, cache.device, kept=False)
            wp = workspace.data_ptr()
    elif workspace.dtype != torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    else:
        wp, wn = workspace.data_ptr(), workspace.numel()
    _call("kv8_attention", L.kv8_attention,
          (cache._ref, batch._ref, code, qp, qs, q_heads, rows, cache.scale if scale is None else scale, 1 if causal else 0, window,
           op, os_, lp, wp, wn), index, at)
    return out if lp is None else (out, lse)


def _vector(t, n: int, dtype, index: int, name: str):
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 1 or (n >= 0 and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{n if n >= 0 else 'pairs'}] on cuda:{index}")
    return t.data_ptr()


def kv8_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor, inv_freq: torch.Tensor, q_weight=None,
                     k_weight=None, eps: float = 1e-6, neighbours: bool = False, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): queries q [rows][q_heads][dim] and keys k
    [rows][k_heads][dim], RMS-normed per head where a weight F32 [dim] is
    given, then rotated by pos int32 [rows] times inv_freq F32 [pairs].  q_out
    may be q and k_out k."""
    code, dtype, index = _type(q, "q"), q.dtype, q.get_device()
    dim = q.shape[-1]
    qp, qs, q_heads, rows = _heads(q, None, dim, dtype, index, "q")
    kp, ks, k_heads, k_rows = _heads(k, None, dim, dtype, index, "k")
    if k_rows != rows:
        raise ValueError("q and k have different numbers of rows")
    pp, fp = _vector(pos, rows, torch.int32, index, "pos"), _vector(inv_freq, -1, torch.float32, index, "inv_freq")
    qw, kw = _vector(q_weight, dim, torch.float32, index, "q_weight"), _vector(k_weight, dim, torch.float32, index, "k_weight")
    at = _place(index, stream)
    if q_out is None:
        q_out = _like(q, rows, q_heads, dim, at)
        qop, qos = q_out.data_ptr(), q_heads * dim
    else:
        qop, qos, _, n = _heads(q_out, q_heads, dim, dtype, index, "q_out")
        if n != rows:
            raise ValueError(f"q_out must have {rows} rows")
    if k_out is None:
        k_out = _like(k, rows, k_heads, dim, at)
        kop, kos = k_out.data_ptr(), k_heads * dim
    else:
        kop, kos, _, n = _heads(k_out, k_heads, dim, dtype, index, "k_out")
        if n != rows:
            raise ValueError(f"k_out must have {rows} rows")
    _call("kv8_qk_norm_rope", lib().kv8_qk_norm_rope,
          (code, rows, dim, qp, qs, q_heads, kp, ks, k_heads, pp, fp, 0 if fp is None else inv_freq.shape[0], 1 if neighbours else 0,
           qw, kw, eps, qop, qos, kop, kos), index, at)
    return q_out, k_out


__all__ = ["KV8Cache", "KV8Batch", "new_cache", "I2SError", "kv8_append", "kv8_read", "kv8_attention",
           "kv8_attention_workspace_bytes", "kv8_qk_norm_rope"]
