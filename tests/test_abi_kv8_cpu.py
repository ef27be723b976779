"""CPU-side checks of the K/V cache part of the C ABI (include/kv8.h): every
declared symbol is exported, host-side argument checks (these calls return
before any launch), and the arithmetic by which grids of page slots and of row
tiles cover ragged batches."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import i2s, kv8

FAKE = 1 << 20


def test_every_declared_symbol_is_exported():
    names = kv8.declared_symbols()
    assert set(names) == {"kv8_append", "kv8_read", "kv8_attention_workspace_bytes", "kv8_attention", "kv8_qk_norm_rope"}
    raw = ctypes.CDLL(i2s.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


def _cache(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=8, heads=2, dim=128, page_tokens=64):
    return kv8._Cache(k, v, k_scale, v_scale, pages, heads, dim, page_tokens)


def _batch(table=FAKE, table_stride=4, blocks=4, lens=FAKE, starts=FAKE, seqs=2, max_len=0):
    return kv8._Batch(table, table_stride, blocks, lens, starts, seqs, max_len)


def _call(fn, cache, batch, type=kv8.KV8_F32, rows=6, a=FAKE, a_stride=256, b=FAKE, b_stride=256):
    c, s = ctypes.addressof(cache) if cache else None, ctypes.addressof(batch) if batch else None
    return getattr(kv8.lib(), fn)(c, s, type, a, a_stride, b, b_stride, rows, None)


SHARED = [
    (dict(cache=None), i2s.I2S_EINVAL),
    (dict(batch=None), i2s.I2S_EINVAL),
    (dict(cache=dict(k=None)), i2s.I2S_EINVAL),
    (dict(cache=dict(v=FAKE + 8)), i2s.I2S_EINVAL),
    (dict(cache=dict(k_scale=FAKE + 2)), i2s.I2S_EINVAL),
    (dict(cache=dict(v_scale=None)), i2s.I2S_EINVAL),
    (dict(cache=dict(pages=0)), i2s.I2S_EINVAL),
    (dict(cache=dict(pages=1 << 31)), i2s.I2S_ERANGE),
    (dict(cache=dict(heads=0)), i2s.I2S_EINVAL),
    (dict(cache=dict(heads=1025)), i2s.I2S_ERANGE),
    (dict(cache=dict(dim=0)), i2s.I2S_EALIGN),
    (dict(cache=dict(dim=120)), i2s.I2S_EALIGN),
    (dict(cache=dict(dim=272)), i2s.I2S_EALIGN),
    (dict(cache=dict(page_tokens=8)), i2s.I2S_EALIGN),
    (dict(cache=dict(page_tokens=48)), i2s.I2S_EALIGN),
    (dict(cache=dict(page_tokens=512)), i2s.I2S_EALIGN),
    (dict(batch=dict(seqs=-1)), i2s.I2S_EINVAL),
    (dict(batch=dict(seqs=(1 << 20) + 1)), i2s.I2S_ERANGE),
    (dict(batch=dict(blocks=-1)), i2s.I2S_EINVAL),
    (dict(batch=dict(table_stride=3)), i2s.I2S_EINVAL),
    (dict(batch=dict(table=None)), i2s.I2S_EINVAL),
    (dict(batch=dict(lens=None)), i2s.I2S_EINVAL),
    (dict(batch=dict(lens=FAKE + 1)), i2s.I2S_EINVAL),
    (dict(batch=dict(starts=FAKE + 2)), i2s.I2S_EINVAL),
    (dict(batch=dict(max_len=-1)), i2s.I2S_EINVAL),
    (dict(batch=dict(starts=None), rows=5), i2s.I2S_EINVAL),  # 5 rows of 2 sequences
    (dict(type=3), i2s.I2S_EINVAL),
    (dict(rows=-1), i2s.I2S_EINVAL),
    (dict(rows=1 << 31), i2s.I2S_ERANGE),
]


def _objects(kw):
    kw = dict(kw)
    kw["cache"] = None if kw.get("cache", 0) is None else _cache(**kw.get("cache", {}))
    kw["batch"] = None if kw.get("batch", 0) is None else _batch(**kw.get("batch", {}))
    return kw


@pytest.mark.parametrize("fn", ["kv8_append", "kv8_read"])
@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(a=None), i2s.I2S_EINVAL),
    (dict(b=None), i2s.I2S_EINVAL),
    (dict(a=FAKE + 8), i2s.I2S_EINVAL),
    (dict(a_stride=255), i2s.I2S_EINVAL),
    (dict(b_stride=258), i2s.I2S_EINVAL),
    (dict(type=kv8.KV8_BF16, b_stride=260), i2s.I2S_EINVAL),
])
def test_append_and_read_reject_on_host(fn, kw, expect):
    assert _call(fn, **_objects(kw)) == expect


def _attend(cache, batch, type=kv8.KV8_F32, q=FAKE, q_stride=1536, q_heads=12, rows=6, scale=0.1, causal=1, window=0, out=FAKE,
            out_stride=1536, lse=None, ws=FAKE, ws_bytes=1 << 40):
    c, s = ctypes.addressof(cache) if cache else None, ctypes.addressof(batch) if batch else None
    return kv8.lib().kv8_attention(c, s, type, q, q_stride, q_heads, rows, scale, causal, window, out, out_stride, lse, ws, ws_bytes,
                                   None)


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(q=None), i2s.I2S_EINVAL),
    (dict(q=FAKE + 4), i2s.I2S_EINVAL),
    (dict(q_stride=1535), i2s.I2S_EINVAL),
    (dict(q_stride=1538), i2s.I2S_EINVAL),
    (dict(out=None), i2s.I2S_EINVAL),
    (dict(out_stride=1528), i2s.I2S_EINVAL),
    (dict(q_heads=0), i2s.I2S_EINVAL),
    (dict(q_heads=13), i2s.I2S_EINVAL),
    (dict(q_heads=1 << 17), i2s.I2S_ERANGE),
    (dict(scale=float("nan")), i2s.I2S_EINVAL),
    (dict(scale=float("inf")), i2s.I2S_EINVAL),
    (dict(window=-1), i2s.I2S_EINVAL),
    (dict(lse=FAKE + 2), i2s.I2S_EINVAL),
])
def test_attention_rejects_on_host(kw, expect):
    assert _attend(**_objects(kw)) == expect


def _rope(type=kv8.KV8_F32, rows=3, dim=128, q=FAKE, q_stride=1536, q_heads=12, k=FAKE, k_stride=256, k_heads=2, pos=FAKE,
          freq=FAKE, pairs=64, neighbours=0, qw=None, kw=None, eps=1e-6, qo=FAKE, qo_stride=1536, ko=FAKE, ko_stride=256):
    return kv8.lib().kv8_qk_norm_rope(type, rows, dim, q, q_stride, q_heads, k, k_stride, k_heads, pos, freq, pairs, neighbours, qw,
                                      kw, eps, qo, qo_stride, ko, ko_stride, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(type=-1), i2s.I2S_EINVAL),
    (dict(rows=-1), i2s.I2S_EINVAL),
    (dict(rows=1 << 31), i2s.I2S_ERANGE),
    (dict(dim=8), i2s.I2S_EALIGN),
    (dict(dim=136), i2s.I2S_EALIGN),
    (dict(dim=512), i2s.I2S_EALIGN),
    (dict(pairs=12), i2s.I2S_EALIGN),
    (dict(pairs=72), i2s.I2S_EALIGN),
    (dict(pairs=-8), i2s.I2S_EINVAL),
    (dict(q=None), i2s.I2S_EINVAL),
    (dict(q=FAKE + 4), i2s.I2S_EINVAL),
    (dict(q_stride=1532), i2s.I2S_EINVAL),
    (dict(k_stride=258), i2s.I2S_EINVAL),
    (dict(qo=None), i2s.I2S_EINVAL),
    (dict(ko=FAKE + 8), i2s.I2S_EINVAL),
    (dict(q_heads=-1), i2s.I2S_EINVAL),
    (dict(k_heads=1 << 16), i2s.I2S_ERANGE),
    (dict(pos=None), i2s.I2S_EINVAL),
    (dict(pos=FAKE + 2), i2s.I2S_EINVAL),
    (dict(freq=None), i2s.I2S_EINVAL),
    (dict(qw=FAKE + 1), i2s.I2S_EINVAL),
    (dict(kw=FAKE + 2), i2s.I2S_EINVAL),
    (dict(eps=-1.0), i2s.I2S_EINVAL),
    (dict(eps=float("nan")), i2s.I2S_EINVAL),
])
def test_rope_rejects_on_host(kw, expect):
    assert _rope(**kw) == expect


def test_empty_calls_are_no_ops():
    assert _call("kv8_append", _cache(), _batch(), rows=0, a=None, b=None) == i2s.I2S_OK
    assert _call("kv8_read", _cache(), _batch(seqs=0, lens=None, table=None, starts=None), rows=3) == i2s.I2S_OK
    assert _attend(_cache(), _batch(seqs=0)) == i2s.I2S_OK
    assert _attend(_cache(), _batch(), rows=0, q=None, out=None) == i2s.I2S_OK
    assert _rope(rows=0) == i2s.I2S_OK
    assert _rope(q_heads=0, k_heads=0) == i2s.I2S_OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z = torch.zeros
    with pytest.raises(TypeError):
        kv8.KV8Cache(z((1, 1, 16, 16), dtype=torch.int8), z((1, 1, 16, 16), dtype=torch.int8), z((1, 1)), z((1, 1)))
    with pytest.raises(TypeError):
        kv8.KV8Batch(z((1, 1), dtype=torch.int32), z(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        kv8.kv8_qk_norm_rope(z((1, 1, 16)), z((1, 1, 16)), z(1, dtype=torch.int32), z(8))


def test_binding_refuses_a_table_whose_rows_overlap(monkeypatch):
    """A broadcast table has a row stride of 0: taken as dense, its rows would
    be looked for behind its memory."""
    monkeypatch.setattr(kv8, "_need", lambda t, dtype, dim, name: t)  # the checks of strides, on host tensors
    lens = torch.zeros(4, dtype=torch.int32)
    wide = torch.zeros((4, 10), dtype=torch.int32)
    for table in (wide[:1].expand(4, 10), wide[:1, :1].expand(4, 1), torch.as_strided(wide, (4, 5), (3, 1))):
        with pytest.raises(ValueError, match="overlap"):
            kv8.KV8Batch(table, lens)
    assert kv8.KV8Batch(wide[:, :6], lens)._c.table_stride == 10
    assert kv8.KV8Batch(wide[:1].expand(1, 10), lens[:1])._c.table_stride == 10
    assert kv8.KV8Batch(wide[:, :0], lens)._c.blocks == 0


def test_page_slots_cover_every_touched_page_once():
    """The kernels' slot arithmetic (key(b) = start(b) / P + 2 b, rows / P + 2
    seqs slots), modelled here: every page that receives rows has one slot of
    its own, inside the grid, also with empty sequences and leading rows."""
    rng = np.random.default_rng(5)
    for _ in range(200):
        P = int(rng.choice([16, 32, 64]))
        seqs = int(rng.integers(1, 12))
        news = rng.integers(0, 4 * P, size=seqs) * (rng.random(seqs) < 0.8)
        lens = news + rng.integers(-10, 3 * P, size=seqs)
        starts = np.concatenate([[int(rng.integers(0, 50))], np.zeros(seqs, np.int64)])
        starts[1:] = starts[0] + np.cumsum(news)
        rows = int(starts[-1] + rng.integers(0, 40))
        grid = rows // P + 2 * seqs
        key = starts[:-1] // P + 2 * np.arange(seqs)
        hit = []
        for x in range(grid):
            below = np.nonzero(key <= x)[0]
            if len(below) == 0:
                continue
            b = int(below[-1])
            ln = max(int(lens[b]), 0)
            done = ln - int(news[b])
            j = max(done, 0) // P + x - int(key[b])
            if max(done, j * P, 0) < min(ln, (j + 1) * P):
                hit.append((b, j))
        want = [(b, j) for b in range(seqs) for j in range(200)
                if max(max(int(lens[b]), 0) - int(news[b]), j * P, 0) < min(max(int(lens[b]), 0), (j + 1) * P)]
        assert sorted(hit) == sorted(want) and len(set(hit)) == len(hit)
