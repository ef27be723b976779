"""Scores, weights and eviction over the int8 K/V cache at the limits of what
include/kv8_scores.h promises: roundings, numbers at the ends of their range,
masses of pages taken anew, workspaces of the size asked for.  Tolerances as
derived in test_gpu_kv8_scores."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import kv8, kv8_scores

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import kv8_plain as plain  # noqa: E402
from test_gpu_kv8 import BF16, F16, F32, U, World, dev, host, rounded, say  # noqa: E402
from test_gpu_kv8_scores import noise, shape_of  # noqa: E402


@pytest.mark.parametrize("lens,heads,group", [([300, 129], 2, 4), (list(range(30, 90)), 8, 4)])
@pytest.mark.parametrize("kw", [dict(cap=4.0), dict(slopes=True), dict(prefix=True), dict(cap=4.0, slopes=True, prefix=True)])
def test_bf16_prompts_are_rounded_once(lens, heads, group, kw):
    """A BF16 result is what rounds a number that F32 sums and weights of 22 bits allow: of at most 4 tokens (a window), whose
    sums take 4 roundings, and one more for each of the 64-token tiles that they may lie in."""
    D, window = 64, 4
    w = World(D + heads, heads, D, 64, lens, lens)
    kw = dict(kw, prefix=[n // 3 for n in lens]) if "prefix" in kw else kw
    theirs, ours = shape_of(w, group, **kw)
    q = rounded(0.2 * w.rng.normal(size=(w.rows, heads * group, D)), BF16)
    say(f"roundings lens={lens[:4]} heads={heads} {kw.keys()}")
    ref = plain.attention(w.ref, q, float(np.float32(D ** -0.5)), window=window, **theirs)
    got = host(kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q, BF16), window=window, **ours))
    e = noise(D, BF16)(ref["parts"], ref["spread"]) + 8 * U * (2 * ref["top"] + 25) + 4 * U
    vs = w.ref.vs[np.isfinite(w.ref.vs)].max()
    tol = ref["mag"] * (2 * e + 2 * (window + 2) * U + 2.0 ** -22)[..., None] + 127 * vs * window * 2.0 ** -40 + U * np.abs(ref["out"])
    low, high = rounded(ref["out"] - tol, BF16), rounded(ref["out"] + tol, BF16)
    off = (got < low) | (got > high)
    assert not off.any(), f"{off.sum()} of {off.size} results are no rounding of the sum"
