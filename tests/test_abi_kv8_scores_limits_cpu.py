"""CPU-side checks of the limits of include/kv8_scores.h (these calls return
before any launch)."""

from __future__ import annotations

import pytest

from ternary_weight_integer_amd import i2s
from test_abi_kv8_scores_cpu import scored, weigh


@pytest.mark.parametrize("fn", [scored, weigh])
def test_scales(fn):
    """Up to 2^126, which log2 e leaves in F32's range."""
    for scale in (2.0 ** 126, -2.0 ** 126, 0.0):
        assert fn(scale=scale, rows=0) == i2s.I2S_OK
    for scale in (2.4e38, -3.4e38):
        assert fn(scale=scale) == i2s.I2S_EINVAL
