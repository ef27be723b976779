"""CPU-side checks of the limits of include/kv8_scores.h (these calls return
before any launch)."""

from __future__ import annotations

import pytest

from ternary_weight_integer_amd import i2s, kv8_scores
from ternary_weight_integer_amd.i2s import I2SError
from test_abi_kv8_scores_cpu import FAKE, _batch, _cache, _ref, scored, weigh


def weigh_workspace_bytes(cache, batch, rows):
    return kv8_scores.lib().kv8_weigh_workspace_bytes(_ref(cache), _ref(batch), 12, rows)


@pytest.mark.parametrize("fn", [scored, weigh])
def test_scales(fn):
    """Up to 2^126, which log2 e leaves in F32's range."""
    for scale in (2.0 ** 126, -2.0 ** 126, 0.0):
        assert fn(scale=scale, rows=0) == i2s.I2S_OK
    for scale in (2.4e38, -3.4e38):
        assert fn(scale=scale) == i2s.I2S_EINVAL


@pytest.mark.parametrize("seqs,blocks,rows", [(1, 64, 4096), (3, 20, 3 * 200)])
def test_weigh_workspace(seqs, blocks, rows):
    """Rows that several workgroups share: a workspace of the size asked for, aligned, or none of the call runs."""
    batch = _batch(table_stride=blocks, blocks=blocks, starts=None, seqs=seqs, max_len=64 * blocks)
    need = weigh_workspace_bytes(_cache(), batch, rows)
    assert need > 0 and need % 1024 == 0
    for kw in (dict(workspace=None), dict(workspace=FAKE + 128), dict(workspace_bytes=need - 1), dict(workspace_bytes=0)):
        assert weigh(batch=batch, rows=rows, **kw) == i2s.I2S_EWORKSPACE


def test_weigh_without_a_workspace():
    """None where a sequence's rows are a stage or two, and for arguments that are refused."""
    for seqs, rows in ((1, 1), (64, 64), (4, 80)):
        assert weigh_workspace_bytes(_cache(), _batch(starts=None, seqs=seqs), rows) == 0
    assert weigh_workspace_bytes(_cache(dim=120), _batch(), 4096) == weigh_workspace_bytes(_cache(), _batch(), -1) == 0


def test_caps_that_round_to_none():
    """A cap under F32's least number is no cap of 0."""
    for cap in (1e-50, -1e-50, 2.0 ** -151):
        with pytest.raises(I2SError) as refused:
            kv8_scores._cap("kv8_weigh", cap)
        assert refused.value.status == i2s.I2S_EINVAL
    assert kv8_scores._cap("kv8_weigh", 0.0) == 0 and kv8_scores._cap("kv8_weigh", 30.0) == 30
