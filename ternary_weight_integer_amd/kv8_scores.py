"""Python binding of scores, weights and eviction over the int8 K/V cache
(include/kv8_scores.h), same names as the C ABI; the functions live in the same
libi2s.so.

Argument marshalling only: every step runs in the library's HIP kernels.  No
fallback: a missing library or a failed call raises.  Caches, batches and
streams are those of kv8.
"""

from __future__ import annotations

import ctypes
import os
import re

import torch

from . import i2s, kv8
from .i2s import I2SError
from .kv8 import KV8Batch, KV8Cache, _call, _dense, _heads, _index, _like, _need, _place, _type

HEADER_PATH = os.path.join(os.path.dirname(i2s._PKG), "include", "kv8_scores.h")

_lib = None


def declared_symbols() -> list[str]:
    """Names of the functions include/kv8_scores.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^[A-Za-z_][\w \*]*?\b(kv8_\w+)\s*\(", text, flags=re.M)


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = kv8.lib()
        i64, p, sz, ci, f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
        L.kv8_attention_scored.restype = ci
        L.kv8_attention_scored.argtypes = [p, p, ci, p, i64, i64, i64, f, ci, i64, f, p, p, p, i64, p, p, sz, p]
        L.kv8_weigh_workspace_bytes.restype = sz
        L.kv8_weigh_workspace_bytes.argtypes = [p, p, i64, i64]
        L.kv8_weigh.restype = ci
        L.kv8_weigh.argtypes = [p, p, ci, p, i64, i64, i64, f, ci, i64, f, p, p, p, p, p, sz, p]
        L.kv8_choose.restype = ci
        L.kv8_choose.argtypes = [p, p, p, i64, i64, i64, p, p, p]
        L.kv8_move.restype = ci
        L.kv8_move.argtypes = [p, p, p, p, i64, p, i64, i64, p, p]
        _lib = L
    return _lib


def _on(t, dtype, shape, index: int, name: str) -> int:
    """The pointer of a contiguous tensor of that type and shape on the device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} on cuda:{index}")
    return t.data_ptr()


def _workspace(workspace, need: int, index: int, at, device):
    """(tensor that holds it, pointer, bytes) of a call's workspace."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _dense(at, need, torch.uint8, device, kept=False)
        return workspace, workspace.data_ptr(), need
    if workspace.dtype != torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    return workspace, workspace.data_ptr(), workspace.numel()


def _cap(fn: str, cap: float) -> float:
    """A cap that F32 rounds to 0 is refused as the library refuses all below 2^-60: 0 is none."""
    if cap and not ctypes.c_float(cap).value:
        raise I2SError(fn, i2s.I2S_EINVAL)
    return cap


def _shape(batch: KV8Batch, q_heads: int, slopes, prefix, index: int):
    """Pointers of the scores' slopes and prefix."""
    return (None if slopes is None else _on(slopes, torch.float32, (q_heads,), index, "slopes"),
            None if prefix is None else _on(prefix, torch.int32, (batch.seqs,), index, "prefix"))


def kv8_attention_scored(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, scale: float | None = None, causal: bool = True,
                         window: int = 0, cap: float = 0.0, slopes=None, prefix=None, out=None, lse=None, workspace=None,
                         stream=None):
    """kv8_attention with shaped scores: capped at cap (0: not), less slopes F32
    [q_heads] times the distance, with tokens in front of prefix int32 [seqs]
    seen by every row.  Outputs and other arguments as kv8_attention's."""
    index = _index(cache, batch)
    code, dim = _type(q, "q"), cache.dim
    qp, qs, q_heads, rows = _heads(q, None, dim, q.dtype, index, "q")
    sp, fp = _shape(batch, q_heads, slopes, prefix, index)
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
        lp = _on(lse, torch.float32, (rows, q_heads), index, "lse")
    need = 0 if workspace is not None else L.kv8_attention_workspace_bytes(cache._ref, batch._ref, q_heads, rows)
    held, wp, wn = _workspace(workspace, need, index, at, cache.device)
    _call("kv8_attention_scored", L.kv8_attention_scored,
          (cache._ref, batch._ref, code, qp, qs, q_heads, rows, cache.scale if scale is None else scale, 1 if causal else 0, window,
           _cap("kv8_attention_scored", cap), sp, fp, op, os_, lp, wp, wn), index, at)
    return out if lp is None else (out, lse)


def new_mass(cache: KV8Cache) -> torch.Tensor:
    """Masses for a cache's pages, F32 [pages][heads][page_tokens], zero."""
    return torch.zeros((cache.pages, cache.heads, cache.page_tokens), dtype=torch.float32, device=cache.device)


def _mass(cache: KV8Cache, mass, index: int) -> int:
    return _on(mass, torch.float32, (cache.pages, cache.heads, cache.page_tokens), index, "mass")


def kv8_weigh_workspace_bytes(cache: KV8Cache, batch: KV8Batch, q_heads: int, rows: int) -> int:
    return int(lib().kv8_weigh_workspace_bytes(cache._ref, batch._ref, q_heads, rows))


def kv8_weigh(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, lse: torch.Tensor, mass: torch.Tensor, scale: float | None = None,
              causal: bool = True, window: int = 0, cap: float = 0.0, slopes=None, prefix=None, workspace=None, stream=None) -> None:
    """Add the attention weight that rows q [rows][q_heads][dim], with the lse
    F32 [rows][q_heads] of the attention with the same scores, give each cached
    token to mass F32 [pages][heads][page_tokens]; masses of the call's own
    tokens are set to it.  Tokens that no call has as rows (a prompt's before
    its last ones) are added to what their pages' masses hold: mass[pages] = 0
    where such a page is begun."""
    index = _index(cache, batch)
    code = _type(q, "q")
    qp, qs, q_heads, rows = _heads(q, None, cache.dim, q.dtype, index, "q")
    sp, fp = _shape(batch, q_heads, slopes, prefix, index)
    lp, mp = _on(lse, torch.float32, (rows, q_heads), index, "lse"), _mass(cache, mass, index)
    L, at = lib(), _place(index, stream)
    need = 0 if workspace is not None else L.kv8_weigh_workspace_bytes(cache._ref, batch._ref, q_heads, rows)
    held, wp, wn = _workspace(workspace, need, index, at, cache.device)
    _call("kv8_weigh", L.kv8_weigh,
          (cache._ref, batch._ref, code, qp, qs, q_heads, rows, cache.scale if scale is None else scale, 1 if causal else 0, window,
           _cap("kv8_weigh", cap), sp, fp, lp, mp, wp, wn), index, at)


def kv8_choose(cache: KV8Cache, batch: KV8Batch, mass: torch.Tensor, keep: int, first: int = 0, recent: int = 0, index=None,
               kept=None, stream=None):
    """(index int32 [seqs][heads][keep], kept int32 [seqs]): the tokens of each
    sequence and head that stay, rising, then -1: the first, the newest
    `recent`, then those of the largest mass."""
    on = _index(cache, batch)
    mp, at = _mass(cache, mass, on), _place(on, stream)
    if keep < 0:
        raise I2SError("kv8_choose", i2s.I2S_EINVAL)
    index = _dense(at, (batch.seqs, cache.heads, keep), torch.int32, cache.device) if index is None else index
    kept = _dense(at, (batch.seqs,), torch.int32, cache.device) if kept is None else kept
    ip, kp = _on(index, torch.int32, (batch.seqs, cache.heads, keep), on, "index"), _on(kept, torch.int32, (batch.seqs,), on, "kept")
    _call("kv8_choose", lib().kv8_choose, (cache._ref, batch._ref, mp, keep, first, recent, ip, kp), on, at)
    return index, kept


def kv8_move(cache: KV8Cache, batch: KV8Batch, index: torch.Tensor, kept: torch.Tensor, to_table: torch.Tensor, mass=None,
             stream=None) -> None:
    """Gather the chosen tokens of each sequence and head (index int32
    [seqs][heads][keep], kept int32 [seqs]) into the pages of to_table int32
    [seqs][blocks], and their masses, if given, into those pages'."""
    on = _index(cache, batch)
    _need(index, torch.int32, 3, "index")
    _need(to_table, torch.int32, 2, "to_table")
    keep, (seqs, blocks) = index.shape[2], to_table.shape
    if seqs != batch.seqs or to_table.get_device() != on:
        raise ValueError(f"to_table must be [{batch.seqs}][blocks] on cuda:{on}")
    if blocks > 1 and to_table.stride(1) != 1:
        raise ValueError("to_table must have unit innermost stride")
    if seqs > 1 and to_table.stride(0) < blocks:
        raise ValueError(f"to_table's rows must not overlap, got strides {to_table.stride()}")
    ip, kp = _on(index, torch.int32, (seqs, cache.heads, keep), on, "index"), _on(kept, torch.int32, (seqs,), on, "kept")
    mp = None if mass is None else _mass(cache, mass, on)
    _call("kv8_move", lib().kv8_move,
          (cache._ref, batch._ref, ip, kp, keep, to_table.data_ptr(), max(to_table.stride(0), blocks), blocks, mp), on,
          _place(on, stream))


__all__ = ["I2SError", "kv8_attention_scored", "new_mass", "kv8_weigh_workspace_bytes", "kv8_weigh", "kv8_choose", "kv8_move"]
