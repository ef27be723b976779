"""CPU-side checks of the scores' part of the C ABI (include/kv8_scores.h):
every declared symbol is exported, and the host's checks of arguments (these
calls return before any launch)."""

from __future__ import annotations

import ctypes
import math

import pytest
import torch

from ternary_weight_integer_amd import i2s, kv8, kv8_scores

FAKE = 1 << 20


def test_every_declared_symbol_is_exported():
    names = kv8_scores.declared_symbols()
    assert set(names) == {"kv8_attention_scored", "kv8_weigh_workspace_bytes", "kv8_weigh", "kv8_choose", "kv8_move"}
    raw = ctypes.CDLL(i2s.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


def _cache(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=8, heads=2, dim=128, page_tokens=64):
    return kv8._Cache(k, v, k_scale, v_scale, pages, heads, dim, page_tokens)


def _batch(table=FAKE, table_stride=4, blocks=4, lens=FAKE, starts=FAKE, seqs=2, max_len=0):
    return kv8._Batch(table, table_stride, blocks, lens, starts, seqs, max_len)


def _ref(x):
    return None if x is None else ctypes.addressof(x)


def scored(cache=0, batch=0, type=kv8.KV8_F32, q=FAKE, q_stride=1536, q_heads=12, rows=6, scale=0.1, causal=1, window=0, cap=0.0,
           slopes=None, prefix=None, out=FAKE, out_stride=1536, lse=None, workspace=FAKE, workspace_bytes=1 << 40):
    c, b = _cache() if cache == 0 else cache, _batch() if batch == 0 else batch
    return kv8_scores.lib().kv8_attention_scored(_ref(c), _ref(b), type, q, q_stride, q_heads, rows, scale, causal, window, cap, slopes,
                                                 prefix, out, out_stride, lse, workspace, workspace_bytes, None)


def weigh(cache=0, batch=0, type=kv8.KV8_F32, q=FAKE, q_stride=1536, q_heads=12, rows=6, scale=0.1, causal=1, window=0, cap=0.0,
          slopes=None, prefix=None, lse=FAKE, mass=FAKE, workspace=FAKE, workspace_bytes=1 << 40):
    c, b = _cache() if cache == 0 else cache, _batch() if batch == 0 else batch
    return kv8_scores.lib().kv8_weigh(_ref(c), _ref(b), type, q, q_stride, q_heads, rows, scale, causal, window, cap, slopes, prefix, lse,
                                      mass, workspace, workspace_bytes, None)


def choose(cache=0, batch=0, mass=FAKE, keep=100, first=4, recent=20, index=FAKE, kept=FAKE):
    c, b = _cache() if cache == 0 else cache, _batch() if batch == 0 else batch
    return kv8_scores.lib().kv8_choose(_ref(c), _ref(b), mass, keep, first, recent, index, kept, None)


def move(cache=0, batch=0, index=FAKE, kept=FAKE, keep=100, to_table=FAKE, to_stride=2, to_blocks=2, mass=None):
    c, b = _cache() if cache == 0 else cache, _batch() if batch == 0 else batch
    return kv8_scores.lib().kv8_move(_ref(c), _ref(b), index, kept, keep, to_table, to_stride, to_blocks, mass, None)


SHARED = [
    (dict(cache=None), i2s.I2S_EINVAL),
    (dict(batch=None), i2s.I2S_EINVAL),
    (dict(cache=_cache(k=None)), i2s.I2S_EINVAL),
    (dict(cache=_cache(v=FAKE + 8)), i2s.I2S_EINVAL),
    (dict(cache=_cache(pages=0)), i2s.I2S_EINVAL),
    (dict(cache=_cache(pages=1 << 31)), i2s.I2S_ERANGE),
    (dict(cache=_cache(heads=1025)), i2s.I2S_ERANGE),
    (dict(cache=_cache(dim=120)), i2s.I2S_EALIGN),
    (dict(cache=_cache(page_tokens=48)), i2s.I2S_EALIGN),
    (dict(batch=_batch(seqs=-1)), i2s.I2S_EINVAL),
    (dict(batch=_batch(seqs=(1 << 20) + 1)), i2s.I2S_ERANGE),
    (dict(batch=_batch(table_stride=3)), i2s.I2S_EINVAL),
    (dict(batch=_batch(table=None)), i2s.I2S_EINVAL),
    (dict(batch=_batch(lens=FAKE + 1)), i2s.I2S_EINVAL),
    (dict(batch=_batch(starts=FAKE + 2)), i2s.I2S_EINVAL),
    (dict(batch=_batch(max_len=-1)), i2s.I2S_EINVAL),
    (dict(batch=_batch(table_stride=1 << 26, blocks=1 << 26)), i2s.I2S_ERANGE),  # 2^32 tokens
]


@pytest.mark.parametrize("fn", [scored, weigh, choose])
@pytest.mark.parametrize("kw,status", SHARED)
def test_caches_and_batches(fn, kw, status):
    assert fn(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED[:-1])
def test_caches_and_batches_of_a_move(kw, status):
    assert move(**kw) == status


SHAPES = [
    (dict(scale=math.nan), i2s.I2S_EINVAL),
    (dict(scale=math.inf), i2s.I2S_EINVAL),
    (dict(window=-1), i2s.I2S_EINVAL),
    (dict(cap=-1.0), i2s.I2S_EINVAL),
    (dict(cap=math.nan), i2s.I2S_EINVAL),
    (dict(cap=math.inf), i2s.I2S_EINVAL),
    (dict(cap=2.0 ** -61), i2s.I2S_EINVAL),
    (dict(cap=2.0 ** 61), i2s.I2S_EINVAL),
    (dict(slopes=FAKE + 2), i2s.I2S_EINVAL),
    (dict(prefix=FAKE + 1), i2s.I2S_EINVAL),
    (dict(q_heads=13), i2s.I2S_EINVAL),
    (dict(q_heads=0), i2s.I2S_EINVAL),
    (dict(q_heads=65536), i2s.I2S_ERANGE),
    (dict(type=3), i2s.I2S_EINVAL),
    (dict(rows=-1), i2s.I2S_EINVAL),
    (dict(rows=1 << 31), i2s.I2S_ERANGE),
    (dict(q=None), i2s.I2S_EINVAL),
    (dict(q=FAKE + 8), i2s.I2S_EINVAL),
    (dict(q_stride=1535), i2s.I2S_EINVAL),
    (dict(q_stride=1538), i2s.I2S_EINVAL),
    (dict(q_stride=(1 << 40) + 8), i2s.I2S_ERANGE),
    (dict(batch=_batch(starts=None), rows=5), i2s.I2S_EINVAL),
]


@pytest.mark.parametrize("fn", [scored, weigh])
@pytest.mark.parametrize("kw,status", SHAPES)
def test_shapes_and_queries(fn, kw, status):
    assert fn(**kw) == status


def test_outputs():
    assert scored(out=None) == scored(out=FAKE + 4) == scored(out_stride=1500) == scored(lse=FAKE + 2) == i2s.I2S_EINVAL
    assert weigh(lse=None) == weigh(lse=FAKE + 2) == weigh(mass=None) == weigh(mass=FAKE + 3) == i2s.I2S_EINVAL
    long = _batch(table_stride=1024, blocks=1024, starts=None, seqs=1, max_len=65536)
    assert scored(batch=long, rows=1, workspace=None) == scored(batch=long, rows=1, workspace=FAKE + 64) \
        == scored(batch=long, rows=1, workspace_bytes=16) == i2s.I2S_EWORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(mass=None), i2s.I2S_EINVAL),
    (dict(mass=FAKE + 2), i2s.I2S_EINVAL),
    (dict(index=None), i2s.I2S_EINVAL),
    (dict(index=FAKE + 2), i2s.I2S_EINVAL),
    (dict(kept=None), i2s.I2S_EINVAL),
    (dict(kept=FAKE + 1), i2s.I2S_EINVAL),
    (dict(keep=-1), i2s.I2S_EINVAL),
    (dict(first=-1), i2s.I2S_EINVAL),
    (dict(recent=-1), i2s.I2S_EINVAL),
    (dict(first=81), i2s.I2S_EINVAL),
    (dict(first=1 << 62, recent=1 << 62, keep=1 << 30), i2s.I2S_EINVAL),
    (dict(keep=(1 << 31) - 1024), i2s.I2S_ERANGE),
])
def test_choices(kw, status):
    assert choose(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(index=None), i2s.I2S_EINVAL),
    (dict(index=FAKE + 2), i2s.I2S_EINVAL),
    (dict(kept=None), i2s.I2S_EINVAL),
    (dict(to_table=None), i2s.I2S_EINVAL),
    (dict(to_table=FAKE + 1), i2s.I2S_EINVAL),
    (dict(mass=FAKE + 1), i2s.I2S_EINVAL),
    (dict(keep=-1), i2s.I2S_EINVAL),
    (dict(to_blocks=-1), i2s.I2S_EINVAL),
    (dict(to_stride=1), i2s.I2S_EINVAL),
    (dict(keep=(1 << 31) - 1024), i2s.I2S_ERANGE),
    (dict(to_stride=(1 << 40) + 1), i2s.I2S_ERANGE),
    (dict(to_blocks=1 << 31, to_stride=1 << 31), i2s.I2S_ERANGE),
])
def test_moves(kw, status):
    assert move(**kw) == status


def test_nothing_to_do():
    """No rows, no sequences, nothing kept: done before a launch."""
    none = _batch(seqs=0, table=None, lens=None, starts=None)
    assert scored(rows=0) == weigh(rows=0) == scored(batch=none) == weigh(batch=none) == i2s.I2S_OK
    assert choose(batch=none, mass=None, index=None, kept=None) == i2s.I2S_OK
    assert move(batch=none) == move(keep=0, index=None) == move(to_blocks=0, to_table=None) == i2s.I2S_OK
    lib = kv8_scores.lib()
    c = _cache()
    assert lib.kv8_weigh_workspace_bytes(_ref(c), _ref(none), 12, 6) == 0
    assert lib.kv8_weigh_workspace_bytes(_ref(c), _ref(_batch()), 13, 6) == 0
    assert lib.kv8_weigh_workspace_bytes(None, _ref(_batch()), 12, 6) == 0


def test_tensors_that_are_not_on_a_gpu():
    """The binding refuses what is no device tensor (no GPU is needed to find out)."""
    with pytest.raises(TypeError):
        kv8.KV8Cache(*(torch.zeros(1) for _ in range(4)))
    with pytest.raises(TypeError):
        kv8_scores._need(torch.zeros((1, 1), dtype=torch.int32), torch.int32, 2, "to_table")
