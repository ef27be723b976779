"""Pins of the oracle's K/V cache functions: hand-worked codes and scales, the
two layouts, an independent numpy attention, rotation identities."""

from __future__ import annotations

import numpy as np
import pytest

import oracle


def empty(pages, heads, P, D, table, lens, starts):
    return oracle.KV8(np.zeros((pages, heads, P, D), np.int8), np.zeros((pages, heads, D, P), np.int8),
                      np.zeros((pages, heads), np.float32), np.zeros((pages, heads), np.float32), table, lens, starts)


def test_hand_worked_append():
    """One page of 16 tokens, one head.  Token 0 has the largest magnitude 127
    (scale 1 exactly): codes are its values, halves rounded away from zero.
    Token 1 brings 254 (scale 2): the ratio is 0.5, so 127 -> 63.5 -> 64,
    3 -> 1.5 -> 2, -5 -> -2.5 -> -3, and its own 5 -> 2.5 -> 3.  Token 2 is
    smaller: the scale stays."""
    D = 16
    c = empty(3, 1, 16, D, [[2]], [1], [0, 1])
    x = np.zeros((1, 1, D), np.float32)
    x[0, 0, :5] = [127, 2.5, -5, 0.49999997, -0.5]
    c.append(x, -x)
    assert c.ks[2, 0] == 1.0 and c.vs[2, 0] == 1.0
    assert list(c.k[2, 0, 0, :5]) == [127, 3, -5, 0, -1]
    assert list(c.v[2, 0, :5, 0]) == [-127, -3, 5, 0, 1]
    c.lens[0] = 2
    y = np.zeros((1, 1, D), np.float32)
    y[0, 0, :2] = [-254, 5]
    c.append(y, x)
    assert c.ks[2, 0] == 2.0 and c.vs[2, 0] == 1.0
    assert list(c.k[2, 0, 0, :5]) == [64, 2, -3, 0, -1]  # -1 * 0.5 = -0.5 -> -1
    assert list(c.k[2, 0, 1, :2]) == [-127, 3]
    assert list(c.v[2, 0, :5, 1]) == [127, 3, -5, 0, -1]
    c.lens[0] = 3
    c.append(np.ones((1, 1, D), np.float32), np.zeros((1, 1, D), np.float32))
    assert c.ks[2, 0] == 2.0 and list(c.k[2, 0, 2, :2]) == [1, 1]
    k, v = c.read(1)
    assert k[0, 0, 0] == 2.0 and v[0, 0, 0] == 0.0
    assert not c.k[:2].any() and not c.v[:2].any() and not c.k[2, 0, 3:].any() and not c.v[2, 0, :, 3:].any()


def test_floor_and_fresh_page():
    """An all-zero page has the scale 1e-5 / 127 (0x33A917DC); a page begun by
    the call forgets whatever scale it had."""
    c = empty(2, 1, 16, 16, [[0]], [2], [0, 2])
    c.ks[0, 0] = 1e9
    c.append(np.zeros((2, 1, 16), np.float32), np.zeros((2, 1, 16), np.float32))
    assert c.ks[0, 0].view(np.uint32) == 0x33A917DC and c.vs[0, 0].view(np.uint32) == 0x33A917DC


def test_round_trip_is_within_half_a_step():
    rng = np.random.default_rng(0)
    lens, P, heads, D = [37, 5, 64], 16, 2, 32
    starts = np.concatenate([[0], np.cumsum(lens)])
    table = np.full((3, 4), -1)
    pages = rng.permutation(12)
    table[0, :3], table[1, :1], table[2, :4] = pages[:3], pages[3:4], pages[4:8]
    c = empty(12, heads, P, D, table, lens, starts)
    x, y = (rng.normal(0, 2, size=(starts[-1], heads, D)).astype(np.float32) for _ in range(2))
    c.append(x, y)
    k, v = c.read(starts[-1])
    assert np.abs(k - x).max() <= c.ks.max() * 0.5001 and np.abs(v - y).max() <= c.vs.max() * 0.5001


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 7), (False, 9)])
def test_attention_against_numpy(causal, window):
    rng = np.random.default_rng(3)
    P, heads, D, group = 16, 2, 16, 3
    lens, news = [33, 0, 1, 20], [5, 0, 1, 20]
    starts = np.concatenate([[0], np.cumsum(news)])
    table = np.full((4, 3), -1)
    table[0], table[2, 0], table[3, :2] = [4, 1, 6], 0, [2, 5]
    c = oracle.KV8(rng.integers(-127, 128, size=(7, heads, P, D)), rng.integers(-127, 128, size=(7, heads, D, P)),
                   rng.uniform(0.01, 0.03, size=(7, heads)), rng.uniform(0.01, 0.03, size=(7, heads)), table, lens, starts)
    q = rng.normal(0, 1, size=(starts[-1], heads * group, D)).astype(np.float32)
    got = c.attention(q, 0.25, causal, window)
    for b in range(4):
        if not news[b]:
            continue
        at = table[b, :-(-lens[b] // P)]
        K = (c.k[at].astype(float) * c.ks[at][..., None, None]).transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :lens[b]]
        V = (c.v[at].astype(float) * c.vs[at][..., None, None]).transpose(1, 0, 3, 2).reshape(heads, -1, D)[:, :lens[b]]
        pos = lens[b] - news[b] + np.arange(news[b])[:, None]
        t = np.arange(lens[b])[None, :]
        seen = (t <= pos) | (not causal)
        if window:
            seen = seen & (t > pos - window)
        for hq in range(heads * group):
            e = 0.25 * q[starts[b]:starts[b + 1], hq].astype(float) @ K[hq // group].T
            p = np.exp(e) * seen
            np.testing.assert_allclose(got["out"][starts[b]:starts[b + 1], hq], p @ V[hq // group] / p.sum(1, keepdims=True), rtol=1e-10)
            np.testing.assert_allclose(got["lse"][starts[b]:starts[b + 1], hq], np.log(p.sum(1)), rtol=1e-10)


def test_rows_that_see_nothing():
    c = empty(2, 1, 16, 16, [[0], [-1]], [1, 16], [0, 3, 4])
    r = c.attention(np.ones((4, 1, 16), np.float32), 1.0)
    assert not r["out"].any()
    assert list(np.isneginf(r["lse"][:, 0])) == [True, True, False, True]  # positions -2, -1, 0; a hole


@pytest.mark.parametrize("neighbours", [False, True])
def test_rotation(neighbours):
    """A quarter turn, a norm that keeps lengths, and inner products that rest
    on the difference of positions alone."""
    freq = np.array([np.pi / 2] * 8, np.float32)
    x = np.arange(1, 17, dtype=np.float32).reshape(1, 1, 16)
    y = oracle.kv8_norm_rope(x, [1], freq, neighbours)
    iu, iv = (np.arange(0, 16, 2), np.arange(1, 16, 2)) if neighbours else (np.arange(8), np.arange(8, 16))
    np.testing.assert_allclose(y[0, 0, iu], -x[0, 0, iv], atol=1e-6)
    np.testing.assert_allclose(y[0, 0, iv], x[0, 0, iu], atol=1e-6)
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 32)).astype(np.float32)
    freq = (1e4 ** (-np.arange(12) / 12)).astype(np.float32)[:8]
    dots = [float((oracle.kv8_norm_rope(q, [p + 5], freq, neighbours) * oracle.kv8_norm_rope(k, [p], freq, neighbours)).sum())
            for p in (0, 17, 60000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-8)
    w = np.ones(32, np.float32)
    n = oracle.kv8_norm_rope(100 * q, [3], freq, neighbours, w, 0.0)
    np.testing.assert_allclose(np.square(n).mean(), 1.0, rtol=1e-10)
