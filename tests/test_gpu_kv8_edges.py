"""Attention over the int8 K/V cache where its kernels and its binding meet
their edges, against the CPU oracle; tolerances as derived in test_gpu_kv8,
whose worlds are used."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import kv8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import test_gpu_kv8 as base  # noqa: E402
from test_gpu_kv8 import BF16, F16, F32, World, check_attention  # noqa: E402


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


# ---------------------------------------------------------------------------
# Streams: what a call allocates

def split_world(seed):
    w = World(seed, 2, 128, 64, [3000, 900], [1, 1])
    assert parts_of(w, 12, 2) > 1
    return w, base.dev(w.values(2, F32, heads=12))


def test_allocations_are_of_the_calls_stream(monkeypatch):
    """A block of the current stream's memory may still be in use by work that
    is queued there: another stream must not be given it."""
    w, q = split_world(1)
    k = base.dev(w.values(2, F32))
    pos, freq = torch.arange(2, dtype=torch.int32, device=base.DEV), torch.ones(64, device=base.DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = []
    for name in ("empty", "empty_like"):
        def new(*args, fn=getattr(torch, name), **kw):
            made.append(torch.cuda.current_stream().cuda_stream)
            return fn(*args, **kw)
        monkeypatch.setattr(torch, name, new)

    def calls(stream):
        del made[:]
        out = kv8.kv8_attention(w.cache, w.batch, q, lse=True, stream=stream)
        assert len(made) == 3  # out, lse, workspace
        out += kv8.kv8_read(w.cache, w.batch, 2, stream=stream) + kv8.kv8_qk_norm_rope(q, k, pos, freq, stream=stream)
        assert len(made) == 7
        torch.cuda.synchronize()
        return out

    here = torch.cuda.current_stream().cuda_stream
    want = calls(None)
    assert set(made) == {here}
    for stream in (side, side.cuda_stream):
        got = calls(stream)
        assert set(made) == {side.cuda_stream}
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = calls(torch.cuda.default_stream().cuda_stream)  # 0
        assert set(made) == {torch.cuda.default_stream().cuda_stream}
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_split_calls_on_two_streams_without_a_wait():
    w, q = split_world(2)
    x, p = split_world(3)
    want = kv8.kv8_attention(w.cache, w.batch, q), kv8.kv8_attention(x.cache, x.batch, p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        got.append((kv8.kv8_attention(w.cache, w.batch, q), kv8.kv8_attention(x.cache, x.batch, p, stream=side)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


# ---------------------------------------------------------------------------
# Each form of the kernels

def choice(w, q_heads, rows, causal=True, window=0):
    """(row tiles of a wave, 0 where four waves share one; parts) of a call."""
    row_tiles, parts = ctypes.c_int(), ctypes.c_int()
    status = kv8.lib().kv8_attention_choice(ctypes.c_void_p(w.cache._ref), ctypes.c_void_p(w.batch._ref), ctypes.c_int64(q_heads),
                                            ctypes.c_int64(rows), int(causal), ctypes.c_int64(window), ctypes.byref(row_tiles),
                                            ctypes.byref(parts))
    assert status == 0
    return row_tiles.value, parts.value


# (heads, D, P, group, lens, news, bound of the lengths, row tiles, split)
LONG, SHORT = [330] + [70] * 12, [50] * 13
FORMS = [
    (2, 128, 64, 16, LONG, SHORT, 330, 1, False),
    (2, 128, 64, 16, LONG, SHORT, 6000, 1, True),
    (2, 128, 16, 16, LONG, SHORT, 330, 1, False),
    (2, 128, 16, 16, LONG, SHORT, 6000, 1, True),
    (1, 128, 256, 33, LONG, SHORT, 6000, 1, True),
    (2, 96, 32, 20, LONG, SHORT, 6000, 1, True),
    (1, 256, 64, 24, LONG, SHORT, 330, 1, False),
    (1, 256, 16, 24, LONG, SHORT, 6000, 1, True),
    (1, 160, 32, 28, LONG, SHORT, 330, 1, False),
    (1, 208, 128, 28, LONG, SHORT, 6000, 1, True),
    (2, 64, 64, 25, LONG, SHORT, 330, 1, False),
    (2, 48, 16, 20, LONG, SHORT, 6000, 1, True),
    (1, 16, 16, 5, [1200], [1000], 60000, 1, True),        # more parts than eight
    (16, 64, 64, 4, [60, 40] * 30, [20, 37] * 30, 60, 2, False),
    (16, 128, 128, 4, [130, 40] * 17, [20, 37] * 17, 130, 2, False),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,P,group,lens,news,bound,row_tiles,split", FORMS)
def test_every_form_of_the_kernel_for_many_rows(heads, D, P, group, lens, news, bound, row_tiles, split, dtype):
    for causal, window, holes in ((True, 0, 0.0), (True, 150, 0.0), (False, 0, 0.1)):
        w = World(D + P, heads, D, P, lens, news, holes=holes, lead=1, blocks=-(-max(lens) // P) + 2 if bound < 1000 else -(-bound // P))
        w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=bound)
        rows = w.rows + 2
        chosen = choice(w, heads * group, rows, causal, window)
        assert chosen[0] == row_tiles and (window or (chosen[1] > 1) == split), chosen
        check_attention(w, group, dtype, causal=causal, window=window, tag=f"{chosen[0]} tiles, {chosen[1]} parts")


# ---------------------------------------------------------------------------
# As exact as the plain form

def plain_attention(w, q, scale):
    """Causal attention in F32 products, exponents and sums."""
    ref, out = w.ref, np.zeros(q.shape, np.float32)
    group = q.shape[1] // ref.heads
    for b, n in enumerate(ref.lens):
        lo, hi = ref.starts[b], ref.starts[b + 1]
        at, pos = ref.table[b, :-(-n // ref.P)], n - (hi - lo) + np.arange(hi - lo)
        for h in range(ref.heads):
            k = (ref.k[at, h].astype(np.float32) * ref.ks[at, h][:, None, None]).reshape(-1, ref.D)[:n]
            v = (ref.v[at, h].astype(np.float32) * ref.vs[at, h][:, None, None]).swapaxes(1, 2).reshape(-1, ref.D)[:n]
            for hq in range(h * group, (h + 1) * group):
                e = np.float32(scale) * (q[lo:hi, hq] @ k.T)
                e[np.arange(n)[None, :] > pos[:, None]] = -np.inf
                p = np.exp(e - e.max(1, keepdims=True))
                out[lo:hi, hq] = (p @ v) / p.sum(1, keepdims=True)
    return out


# (heads, D, P, group, lens, news, row tiles)
EXACT = [
    (2, 128, 64, 6, [2048], [1], 0),
    (2, 64, 16, 3, [700, 300], [3, 40], 0),
    (2, 128, 64, 16, LONG, SHORT, 1),
    (16, 64, 64, 4, [60, 40] * 30, [20, 37] * 30, 2),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,P,group,lens,news,row_tiles", EXACT)
def test_wide_query_channels(heads, D, P, group, lens, news, row_tiles, dtype):
    """One component of a query `wide` times the others, as the biases of
    projections leave them, where keys are small: what is kept of the others
    may not rest on it.  Root mean square errors against 64 bits: in 16-bit rows
    the result's own rounding (2^-11, 2^-8 at most), besides which F32 sums and
    22-bit weights (F16) are nothing and 11-bit weights (BF16) are 2^-11 to its
    2^-8, 1 + 2^-7 times the whole; in F32 rows no more than three times the
    plain form's, whose products and sums have 24 bits: a query's 22 bits (2^-23
    on average at most, in each component) are twice its 2^-24, its sums and
    exponents add as much as the plain form's own."""
    for wide in (1.0, 30.0, 1000.0):
        w = World(D + P, heads, D, P, lens, news)
        q = w.rng.normal(0, 1, size=(w.rows, heads * group, D))
        q[:, :, 5] *= wide
        q = base.rounded(q, dtype)
        w.ref.k[:, :, :, 5] = w.rng.integers(-1, 2, size=w.ref.k.shape[:3])
        w.ref.ks[np.isfinite(w.ref.ks)] /= 4  # logits of a few units
        w.cache = kv8.KV8Cache(base.dev(w.ref.k), base.dev(w.ref.v), base.dev(w.ref.ks), base.dev(w.ref.vs))
        assert choice(w, heads * group, w.rows)[0] == row_tiles
        scale = float(np.float32(D ** -0.5))
        base.say(f"kv8 wide channel {wide} D={D} tiles={row_tiles} {dtype}")
        exact = w.ref.attention(q, scale)["out"]
        got = base.host(kv8.kv8_attention(w.cache, w.batch, base.dev(q, dtype), scale=scale))
        rms = lambda a: float(np.sqrt(np.mean(np.square(a - exact))))  # noqa: E731
        if dtype == F32:
            own, allowed = rms(plain_attention(w, q, scale)), 3.0
        else:
            own, allowed = rms(base.rounded(exact, dtype)), 1.0 + 2.0 ** -7
        base.say(f"  error {rms(got):.3g}, {rms(got) / own:.3f} of {own:.3g}")
        assert rms(got) <= allowed * own


@pytest.mark.parametrize("heads,D,P,group,lens,news,row_tiles", EXACT)
def test_f16_rows_are_held_to_f32_weights(heads, D, P, group, lens, news, row_tiles):
    """F16 queries are held exactly and weights in 22 bits: the bound that
    test_gpu_kv8 derives for F32 rows, and half a step of the result."""
    w = World(3 * D + P, heads, D, P, lens, news)
    q = w.values(w.rows, F16, heads=heads * group, spread=0.4)
    scale = float(np.float32(D ** -0.5))
    assert choice(w, heads * group, w.rows)[0] == row_tiles
    ref = w.ref.attention(q, scale)
    out, lse = kv8.kv8_attention(w.cache, w.batch, base.dev(q, F16), scale=scale, lse=True)
    tol, tol_lse = base.attention_bound(ref, w, F32, max(lens))
    tol = tol + torch.finfo(F16).eps / 2 * np.abs(ref["out"]) + 2.0 ** -25
    assert (np.abs(base.host(out) - ref["out"]) <= tol).all() and (np.abs(base.host(lse) - ref["lse"]) <= tol_lse).all()


# ---------------------------------------------------------------------------
# Scales of zero

def zero_bound(ref, w, n):
    """That of test_gpu_kv8 for F32 rows, with exponents that hold a value
    scale's logarithm of up to 67 (a scale of zero counts as 1e-20 in them)."""
    out, lse = base.attention_bound(ref, w, F32, n)
    more = 8 * base.U * 42
    return out + 2 * more * ref["mag"], lse + more


@pytest.mark.parametrize("heads,D,P,group,lens,news,bound", [
    (1, 64, 64, 4, [20000, 300], [1, 1], 20000),       # few rows, split
    (1, 64, 64, 4, [700], [1], 700),
    (2, 128, 64, 16, LONG, SHORT, 330),                # many rows, one row tile
    (2, 64, 32, 25, LONG, SHORT, 330),
    (16, 64, 64, 4, [60, 40] * 30, [20, 37] * 30, 60),  # two
])
def test_value_scales_of_zero(heads, D, P, group, lens, news, bound):
    """Pages of zeros (whatever their codes) add to the denominator alone."""
    for which, by in (("all", 0.0), ("some", 0.0), ("some", 0.9e-20)):
        w = World(D, heads, D, P, lens, news)
        named = np.unique(w.ref.table[(w.ref.table >= 0) & (w.ref.table < w.ref.pages)])
        hit = named if which == "all" else named[::2]
        w.ref.vs[hit] = by
        w.cache.v_scale.copy_(base.dev(w.ref.vs))
        w.ref.vs[hit] = 0.0
        q = w.values(w.rows, F32, heads=heads * group, spread=0.4)
        scale = float(np.float32(D ** -0.5))
        base.say(f"kv8 value scales of {by}: {which} D={D} lens={lens[:3]}")
        ref = w.ref.attention(q, scale)
        out, lse = (base.host(t) for t in kv8.kv8_attention(w.cache, w.batch, base.dev(q), scale=scale, lse=True))
        if which == "all":
            assert not out.any()
        tol, tol_lse = zero_bound(ref, w, max(lens))
        assert (np.abs(out - ref["out"]) <= tol).all() and (np.abs(lse - ref["lse"]) <= tol_lse).all()


def test_a_new_cache_reads_as_zeros():
    """Equal weights: a lane adds 16 of each of at most 100 tiles (116 u), log2
    of the sum and the maximum less headroom are below 100 (a few u of that)."""
    cache = kv8.new_cache(400, 1, 64, 64, device=base.DEV)
    batch = kv8.KV8Batch(torch.arange(400, dtype=torch.int32, device=base.DEV)[None, :],
                         torch.tensor([25600], dtype=torch.int32, device=base.DEV))
    q = torch.ones((1, 3, 64), device=base.DEV)
    out, lse = kv8.kv8_attention(cache, batch, q, lse=True)
    assert not out.any()
    assert (lse - np.log(25600)).abs().max() <= 1e-4


# ---------------------------------------------------------------------------
# Large exponents

@pytest.mark.parametrize("dtype,sizes", [(F32, (1e4, 1e6, 1e7, 1e9, 3e20, 1e30, 3e34)), (F16, (400,)), (BF16, (1e9, 3e34))])
@pytest.mark.parametrize("heads,D,P,group,lens,news,row_tiles", EXACT)
def test_large_exponents(heads, D, P, group, lens, news, row_tiles, dtype, sizes):
    """Exponents that rise with the token by 2^-6 |q| scale, at least 100, to as
    much as 1e36, of either sign: the largest (a row's last token, or the first)
    takes all.  Its weight is rounded like its share of the sum, then the
    reciprocals, the product and the result: 16 u, and half a step of the type.
    Where all keys are equal, means of the values, whatever the weights."""
    scale = 1e5 if dtype == F16 else 1.0
    for size in sizes:
        for equal in (False, True):
            w = World(D + P, heads, D, P, lens, news)
            w.ref.ks[:], w.ref.vs[:] = 2.0 ** -6, np.nan_to_num(w.ref.vs, nan=0.1)
            w.ref.k[:, :, :, :2] = 50
            for b, n in enumerate(lens):
                for t in range(0 if equal else n):  # 128 (t / 100) + t % 100 in all
                    w.ref.k[w.ref.table[b, t // P], :, t % P, :2] = t // 100, t % 100
            w.cache = kv8.KV8Cache(*(base.dev(a) for a in (w.ref.k, w.ref.v, w.ref.ks, w.ref.vs)))
            q = np.zeros((w.rows, heads * group, D))
            q[:, :, 1] = size * w.rng.choice([-1.0, 1.0], size=q.shape[:2])
            q = base.rounded(q, dtype)
            q[:, :, 0] = 128 * q[:, :, 1]
            assert choice(w, heads * group, w.rows)[0] == row_tiles
            base.say(f"kv8 large exponents {size} equal={equal} D={D} tiles={row_tiles} {dtype}")
            out, lse = (base.host(t) for t in kv8.kv8_attention(w.cache, w.batch, base.dev(q, dtype), scale=scale, lse=True))
            ref = w.ref.attention(q, scale)
            assert np.isfinite(out).all()
            assert (np.abs(lse - ref["lse"]) <= 8 * base.U * np.abs(ref["lse"]) + 1e-3).all()
            if equal:
                assert (np.abs(out) <= 127.5 * w.ref.vs.max()).all()
            else:
                tol = 16 * base.U * ref["mag"] + torch.finfo(dtype).eps / 2 * np.abs(ref["out"]) + 2.0 ** -25
                assert (np.abs(out - ref["out"]) <= tol).all()


# ---------------------------------------------------------------------------
# Rows in front of position 0

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_in_front_of_position_0(dtype):
    """They see nothing where causal.  Else they see as any row does: with the
    query of a row at position 0 or later, and no window, the same."""
    w = World(70, 2, 64, 16, [3, 40], [9, 4])  # positions -6 .. 2 and 36 .. 39
    q = w.values(13, dtype, heads=6)
    q[0] = q[5] = q[8]
    for window in (0, 7):
        check_attention(w, 3, dtype, causal=True, window=window, rows=13, q=q, tag="in front")
        check_attention(w, 3, dtype, causal=False, window=window, rows=13, q=q, tag="in front")
    out, lse = kv8.kv8_attention(w.cache, w.batch, base.dev(q, dtype), lse=True)
    assert not out[:6].any() and torch.isneginf(lse[:6]).all()
    out, lse = kv8.kv8_attention(w.cache, w.batch, base.dev(q, dtype), causal=False, lse=True)
    for row in (0, 5):
        assert torch.equal(out[row], out[8]) and torch.equal(lse[row], lse[8])


@pytest.mark.parametrize("heads,D,P,group,lens,news", [(2, 128, 64, 6, [2048], [1]), (2, 64, 16, 3, [700, 300], [3, 12]),
                                                       (1, 256, 64, 4, [900], [2])])
def test_few_bf16_rows_are_held_to_the_bound_of_f32(heads, D, P, group, lens, news):
    """Queries in 30 bits and weights in 22, whatever the rows' type: the bound
    of F32 rows, and half a step of the result."""
    w = World(5 * D + P, heads, D, P, lens, news)
    q = w.values(w.rows, BF16, heads=heads * group, spread=0.4)
    scale = float(np.float32(D ** -0.5))
    assert choice(w, heads * group, w.rows)[0] == 0
    ref = w.ref.attention(q, scale)
    out, lse = kv8.kv8_attention(w.cache, w.batch, base.dev(q, BF16), scale=scale, lse=True)
    tol, tol_lse = base.attention_bound(ref, w, F32, max(lens))
    tol = tol + torch.finfo(BF16).eps / 2 * np.abs(ref["out"])
    assert (np.abs(base.host(out) - ref["out"]) <= tol).all() and (np.abs(base.host(lse) - ref["lse"]) <= tol_lse).all()


@pytest.mark.parametrize("D,P,lens,news", [(128, 64, [100], [1]), (64, 16, [90, 120], [1, 1]), (256, 64, [60], [1])])
def test_few_bf16_rows_whose_values_cancel(D, P, lens, news):
    """Tokens of two kinds in turn, values +100 and -100, exponents that differ
    by less than 0.01: results are a hundredth of what they are made of, and half
    a step of theirs is nothing beside a rounding of the weights to 11 bits, up
    to 2^-13 of the values (the smaller kind's 2^-12, halved)."""
    w = World(D, 2, D, P, lens, news)
    w.ref.k[:, :, :, 0] = 100 - np.arange(P) % 2
    w.ref.v[:] = np.where(np.arange(P) % 2, -100, 100)
    w.ref.ks[:] = w.ref.vs[:] = 2.0 ** -6
    w.cache = kv8.KV8Cache(*(base.dev(a) for a in (w.ref.k, w.ref.v, w.ref.ks, w.ref.vs)))
    q = np.zeros((w.rows, 2 * 33, D))
    q[:, :, 0] = w.rng.uniform(0.5, 2.0, size=q.shape[:2])
    q = base.rounded(q, BF16)
    assert choice(w, 66, w.rows)[0] == 0
    ref = w.ref.attention(q, 0.2)
    out = base.host(kv8.kv8_attention(w.cache, w.batch, base.dev(q, BF16), scale=0.2))
    # As in test_gpu_kv8, but that a query's one component is held exactly.
    n, weight = max(lens), 8 * base.U * (2 * ref["top"] + 25) + 4 * base.U
    tol = ref["mag"] * (2 * weight + 2 * n * base.U + 2.0 ** -22)[..., None] + torch.finfo(BF16).eps / 2 * np.abs(ref["out"])
    assert tol.max() < 2.0 ** -14 * ref["mag"].max()
    assert (np.abs(out - ref["out"]) <= tol).all()


# ---------------------------------------------------------------------------
# Many rows beside bad ones, and captured

@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,P,group,lens,news,row_tiles", EXACT[2:] + [(1, 256, 64, 24, LONG, SHORT, 1)])
def test_bad_queries_stay_in_their_rows_of_many(heads, D, P, group, lens, news, row_tiles, dtype):
    w = World(80 + D, heads, D, P, lens, news)
    q = w.values(w.rows, dtype, heads=heads * group, spread=0.0)
    assert choice(w, heads * group, w.rows)[0] == row_tiles
    clean = kv8.kv8_attention(w.cache, w.batch, base.dev(q, dtype))
    hit = w.rng.random(q.shape[:2]) < 0.05
    for row, head in zip(*np.nonzero(hit)):
        q[row, head, w.rng.integers(D)] = w.rng.choice([np.nan, np.inf, -np.inf])
    got, lse = kv8.kv8_attention(w.cache, w.batch, base.dev(q, dtype), lse=True)
    a, b, s = base.host(clean), base.host(got), base.host(lse)
    assert np.isnan(b[hit]).all() and np.isnan(s[hit]).all()
    assert np.array_equal(a[~hit], b[~hit]) and np.isfinite(s[~hit]).all()


def test_captured_calls_of_many_rows_and_on_a_forked_stream():
    """Prompts split over the tokens, captured with the workspace of the
    graph's own memory, and beside them a decode call on a stream that the
    capture forks; replayed with other lengths and queries, eager calls between.
    Every replay equals the eager calls bit for bit."""
    w = World(91, 2, 128, 64, LONG, SHORT, blocks=-(-6000 // 64))
    w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=6000)
    assert choice(w, 32, w.rows) == (1, 2)
    x, p = split_world(92)
    lens = x.batch.lens
    q = base.dev(w.values(w.rows, F16, heads=32), F16)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    kv8.kv8_attention(w.cache, w.batch, q), kv8.kv8_attention(x.cache, x.batch, p, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        two = kv8.kv8_attention(x.cache, x.batch, p, lse=True, stream=side)
        one = kv8.kv8_attention(w.cache, w.batch, q, lse=True)
        torch.cuda.current_stream().wait_stream(side)
    for turn in range(5):
        lens.sub_(torch.tensor([100, 7], dtype=torch.int32, device=base.DEV))
        w.batch.lens.sub_(1)
        q.mul_(-0.9), p.mul_(-1.1)
        graph.replay()
        want = kv8.kv8_attention(w.cache, w.batch, q, lse=True) + kv8.kv8_attention(x.cache, x.batch, p, lse=True)
        torch.cuda.synchronize()
        for a, b in zip(one + two, want):
            assert torch.equal(a, b)
