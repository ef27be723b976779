"""Limits of the K/V cache part of the C ABI (include/kv8.h) that the host
decides: calls that return before any launch, and the choice of the attention's
kernel and split, which sees sizes alone."""

from __future__ import annotations

import ctypes

import pytest

from ternary_weight_integer_amd import i2s, kv8

FAKE = 1 << 20


def choice(q_heads, rows, causal, window, *, seqs=1, blocks=1024, max_len=65536):
    """(row tiles, parts) of a call over 2 K/V heads of 128, pages of 64."""
    cache = kv8._Cache(FAKE, FAKE, FAKE, FAKE, seqs * blocks, 2, 128, 64)
    batch = kv8._Batch(FAKE, blocks, blocks, FAKE, None, seqs, max_len)
    row_tiles, parts = ctypes.c_int(), ctypes.c_int()
    status = kv8.lib().kv8_attention_choice(ctypes.byref(cache), ctypes.byref(batch), ctypes.c_int64(q_heads), ctypes.c_int64(rows),
                                            int(causal), ctypes.c_int64(window), ctypes.byref(row_tiles), ctypes.byref(parts))
    assert status == 0
    return row_tiles.value, parts.value


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_heads,rows,seqs", [(12, 1, 1), (12, 5, 1), (32, 4, 4), (12, 2000, 1)])
def test_a_window_past_every_position_is_none(q_heads, rows, seqs, causal):
    whole = choice(q_heads, rows, causal, 0, seqs=seqs)
    assert whole[1] > 1
    for window in (1 << 20, (1 << 31) - 1, 1 << 31, 1 << 62, (1 << 63) - 70, (1 << 63) - 1):
        assert choice(q_heads, rows, causal, window, seqs=seqs) == whole
    assert choice(q_heads, rows, causal, 100, seqs=seqs)[1] <= whole[1]


FAR = [(1 << 40) + 8, 1 << 61, 1 << 62, (1 << 63) - 8]


@pytest.mark.parametrize("stride", FAR)
@pytest.mark.parametrize("type", [kv8.KV8_F32, kv8.KV8_BF16])
def test_far_strides_are_out_of_range(stride, type):
    """In bytes or times a row number they leave 64 bits: 2^62 F32 elements
    are 0 bytes there."""
    lib = kv8.lib()
    cache = kv8._Cache(FAKE, FAKE, FAKE, FAKE, 8, 2, 128, 64)
    batch = kv8._Batch(FAKE, 4, 4, FAKE, FAKE, 2, 0)
    c, b = ctypes.addressof(cache), ctypes.addressof(batch)
    for strides in ((stride, 256), (256, stride)):
        for fn in (lib.kv8_append, lib.kv8_read):
            assert fn(c, b, type, FAKE, strides[0], FAKE, strides[1], 6, None) == i2s.I2S_ERANGE
    for strides in ((stride, 1536), (1536, stride)):
        assert lib.kv8_attention(c, b, type, FAKE, strides[0], 12, 6, 0.1, 1, 0, FAKE, strides[1], None, FAKE, 1 << 40,
                                 None) == i2s.I2S_ERANGE
    near = [1536, 256, 1536, 256]
    for i in range(4):
        q, k, q_out, k_out = near[:i] + [stride] + near[i + 1:]
        assert lib.kv8_qk_norm_rope(type, 3, 128, FAKE, q, 12, FAKE, k, 2, FAKE, FAKE, 64, 0, None, None, 1e-6, FAKE, q_out, FAKE,
                                    k_out, None) == i2s.I2S_ERANGE
