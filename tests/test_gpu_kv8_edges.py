"""Attention over the int8 K/V cache where its kernels and its binding meet
their edges, against the CPU oracle; tolerances as derived in test_gpu_kv8,
whose worlds are used."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import kv8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from test_gpu_kv8 import F32, World, check_attention  # noqa: E402


def parts_of(w, q_heads, rows):
    """Parts that the workspace has room for (0: the call is not split)."""
    return kv8.kv8_attention_workspace_bytes(w.cache, w.batch, q_heads, rows) // (4 * rows * q_heads * (w.ref.D + 2))


# ---------------------------------------------------------------------------
# Joining the parts of split rows

@pytest.mark.parametrize("lead", [1, 2, 3])
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 7), (3, 1), (1, 2)])
@pytest.mark.parametrize("lens,news", [
    ([2000], [1]),
    ([4000], [1]),
    ([1500, 1100, 3000], [1, 2, 1]),
    ([5, 1300, 9, 2100, 1400], [0, 1, 0, 0, 3]),          # sequences without rows, at the front and between
    ([1200] * 3 + [2400] * 62, [0] * 3 + [1] * 62),       # more than one load of starts
    ([1200] * 70 + [2500, 1300], [0] * 69 + [1, 0, 1]),
])
def test_few_parts_join_the_first_rows_of_a_batch(lens, news, heads, group, lead):
    """Rows in front of the batch's first share a wave of the join with it
    (an odd number of heads), or do not (an even one)."""
    w = World(lead + len(lens), heads, 128, 64, lens, news, lead=lead)
    rows = w.rows + 2
    assert 2 <= parts_of(w, heads * group, rows) <= 8
    check_attention(w, group, F32, rows=rows, tag="few parts")


def test_many_parts_join_the_first_rows_of_a_batch():
    for lens, news in (([30000], [1]), ([200, 20000], [0, 2])):
        w = World(5, 1, 64, 64, lens, news, lead=1)
        assert parts_of(w, 3, w.rows + 2) > 8
        check_attention(w, 3, F32, tag="many parts")
