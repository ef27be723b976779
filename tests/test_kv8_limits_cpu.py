"""Limits of the K/V cache part of the C ABI (include/kv8.h) that the host
decides: calls that return before any launch, and the choice of the attention's
kernel and split, which sees sizes alone."""

from __future__ import annotations

import ctypes

import pytest

from ternary_weight_integer_amd import kv8

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
