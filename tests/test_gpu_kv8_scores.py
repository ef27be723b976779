"""GPU parity of scores, weights and eviction over the int8 K/V cache against
plain 64-bit implementations (kv8_plain), on the worlds of test_gpu_kv8.

u = 2^-24 below: half a step of F32, relative; n tokens, D components.
Attention with shaped scores:
  - queries: F32 ones are held in 22 bits or more of each component, or as a
    fixed-point number of 23 bits and more of the row's largest: 3 u spread
    (spread = |scale| k_scale sum|code| max|q|); 16-bit ones are exact;
  - the dot's partial sums: at most D / 16 + 8 roundings of u spread, products
    with the scales among them;
  - the cap keeps an error or shrinks it (|tanh'| <= 1) and adds at most 10 u of
    its result (quotient and polynomial 4 u; exponential, sum, difference,
    reciprocal and products 8 u; the cap's own factor log2 e 2 u);
  - the bias: slope times log2 e, one fused product and sum: 2 u of |bias| and
    u of the result.  Both within 12 u (|bias| + |score|);
  - the rest as for plain scores: 8 u (2 max|e| + 25) for exponents in base 2
    with the value scale's logarithm and the maximum, 4 u the exponential, n u
    each for the numerator's and the denominator's sums, weights of 2^-22 (one
    f16, 2^-11, for many BF16 rows) and 2^-40 of the largest.
Weights: a weight's exponent less lse log2 e (4 u |lse|), summed over rows in F32
(as many u as terms), added to the mass (2 u of the result)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import i2s, kv8, kv8_scores

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import kv8_plain as plain  # noqa: E402
from test_gpu_kv8 import BF16, DEV, F16, F32, U, World, bits, dev, host, rounded, say  # noqa: E402

EPS = {F32: 0.0, F16: 2.0 ** -11, BF16: 2.0 ** -8}


def shape_of(w, group, cap=0.0, slopes=False, prefix=None):
    """The scores' shape as keywords: of the plain forms, and of the calls."""
    heads = w.ref.heads * group
    s = None
    if slopes:
        s = (2.0 ** -w.rng.uniform(0.5, 6, heads)).astype(np.float32)
        s[0] = 0.0 if heads > 1 else s[0]
    p = None if prefix is None else np.asarray(prefix, np.int32)
    ours = {"cap": cap, "slopes": None if s is None else dev(s), "prefix": None if p is None else dev(p)}
    return {"cap": cap, "slopes": s, "prefix": p}, ours


def noise(D, dtype):
    fixed = 3 * U if dtype == F32 else 2.0 ** -40
    return lambda parts, spread: (fixed + (D / 16 + 8) * U) * spread + 12 * U * parts


def check_scored(w, group, dtype, *, causal=True, window=0, scale=None, q=None, tag="", rows=None, **kw):
    heads, D = w.ref.heads * group, w.ref.D
    theirs, ours = shape_of(w, group, **kw)
    rows = w.rows + 2 if rows is None else rows
    q = w.values(rows, dtype, heads=heads, spread=0.4) if q is None else q
    q[w.rows:] = np.nan
    scale = float(np.float32(D ** -0.5)) if scale is None else scale
    say(f"scored {tag} heads={heads}/{w.ref.heads} D={D} P={w.ref.P} lens={list(w.ref.lens)[:6]} {dtype} causal={causal} "
        f"window={window} {kw}")
    ref = plain.attention(w.ref, q, scale, causal, window, **theirs)
    out = torch.full((rows, heads, D), 5.0, dtype=dtype, device=DEV)
    lse = torch.full((rows, heads), 5.0, dtype=F32, device=DEV)
    kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q, dtype), scale=scale, causal=causal, window=window, out=out, lse=lse, **ours)
    o, s = host(out), host(lse)
    outside = np.ones(rows, bool)
    outside[w.ref.starts[0]:w.ref.starts[-1]] = False
    assert (o[outside] == 5.0).all() and (s[outside] == 5.0).all()
    none = np.isneginf(ref["lse"])
    assert not o[none].any() and np.isneginf(s[none]).all()
    live = ~outside[:, None] & ~none
    n = max(1, int(w.ref.lens.max()))
    e = noise(D, dtype)(ref["parts"], ref["spread"]) + 8 * U * (2 * ref["top"] + 25) + 4 * U
    weight = 2.0 ** -11 if dtype == BF16 else 2.0 ** -22
    vs = w.ref.vs[np.isfinite(w.ref.vs)].max()
    tol = ref["mag"] * (2 * e + 2 * n * U + weight)[..., None] + 127 * vs * n * 2.0 ** -40
    tol = tol + EPS[dtype] * np.abs(ref["out"]) + (2.0 ** -25 if dtype == F16 else 0.0)
    tol_lse = e + 2 * n * U + 4 * U * np.abs(np.where(none, 0, ref["lse"]))
    err, err_lse = np.abs(o[live] - ref["out"][live]), np.abs(s[live] - ref["lse"][live])
    assert (err <= tol[live]).all(), f"out: worst {np.max(err / tol[live]):.3g} of the bound"
    assert (err_lse <= tol_lse[live]).all(), f"lse: worst {np.max(err_lse / tol_lse[live]):.3g} of the bound"
    return q, ours, theirs, scale, lse, ref


# (heads, D, P, group, lens, news)
SIZES = [
    (1, 16, 16, 1, [1], [1]),
    (2, 128, 64, 6, [777], [1]),
    (2, 128, 64, 6, [64, 65, 1, 0, 63, 200], [1, 1, 1, 0, 1, 1]),
    (1, 64, 16, 1, [15, 16, 17, 100], [1, 1, 1, 1]),
    (2, 80, 32, 3, [70, 33, 5], [4, 2, 5]),
    (2, 256, 64, 2, [300, 20], [3, 20]),
    (1, 112, 128, 16, [260, 128], [2, 1]),
    (1, 128, 16, 33, [90, 40], [1, 2]),
    (2, 128, 64, 6, [130, 64, 200], [130, 64, 70]),
    (3, 48, 16, 7, [100, 37], [100, 37]),
    (2, 96, 256, 4, [300, 257], [290, 30]),
    (2, 64, 32, 8, [150, 0, 40], [150, 0, 3]),
    (1, 128, 64, 4, [3, 0, 70], [9, 4, 3]),        # rows in front of position 0
    (1, 64, 64, 5, [600, 520], [600, 300]),
]

SHAPES = [
    dict(cap=20.0),
    dict(slopes=True, window=37),
    dict(prefix=[50, 7, 0, 2000, -3, 1]),
    dict(cap=3.0, slopes=True, prefix=[20, 300, 33, 0, 5, 61], window=90, holes=0.2),
    dict(cap=0.7, slopes=True, causal=False, holes=0.2),
]


def world(i, size, shape):
    heads, D, P, group, lens, news = size
    kw = dict(shape)
    w = World(100 * i + D + P + group, heads, D, P, lens, news, holes=kw.pop("holes", 0.0), lead=i % 3)
    if "prefix" in kw:
        kw["prefix"] = kw["prefix"][:len(lens)]
    return w, group, kw


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s[:4])))
def test_attention_scored(size, dtype):
    for i, shape in enumerate(SHAPES):
        w, group, kw = world(i, size, shape)
        check_scored(w, group, dtype, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_scored_long_and_split(dtype):
    for lens, news, kw in (([5000], [1], dict(cap=30.0)), ([3, 4100, 0, 1200], [1, 1, 0, 1], dict(slopes=True)),
                           ([2500, 700], [40, 3], dict(window=600, cap=5.0, prefix=[2400, 100])), ([1500], [1500], dict(prefix=[700]))):
        check_scored(World(7, 2, 128, 64, lens, news), 6, dtype, tag="long", **kw)


def test_a_cap_holds_scores_of_any_size():
    """Scores around the branch at 5/8 of the cap, far past it, and past F32's range before it."""
    for scale, cap in ((0.02, 2.0), (0.3, 2.0), (40.0, 2.0), (1e36, 50.0), (0.1, 1e-3), (0.1, 1e9)):
        check_scored(World(12, 2, 128, 32, [513, 100], [2, 1]), 4, F32, scale=scale, cap=cap, tag=f"scale={scale}") \
            if scale < 1e30 else check_saturated(scale, cap)


def check_saturated(scale, cap):
    """Every score is the cap or less the cap."""
    w = World(13, 1, 64, 16, [40], [1])
    q = w.values(1, F32, heads=2)
    ref = plain.attention(w.ref, q, scale, cap=cap)
    out, lse = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q), scale=scale, cap=cap, lse=True)
    assert np.allclose(host(out), ref["out"], rtol=0, atol=1e-4 * np.abs(ref["mag"]).max())
    assert np.allclose(host(lse), ref["lse"], rtol=1e-5)


def test_attention_scored_bad_queries_stay_in_their_rows():
    w = World(15, 2, 128, 64, [200, 90], [2, 20])
    q = w.values(w.rows, F32, heads=12, spread=0.0)
    _, ours = shape_of(w, 6, cap=10.0, slopes=True, prefix=[30, 80])
    clean = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q), **ours)
    bad = q.copy()
    bad[1, 3, 5], bad[4, 0, 127], bad[20, 11, 0] = np.nan, np.inf, -np.inf
    got = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(bad), **ours)
    a, b = host(clean), host(got)
    hit = np.zeros(a.shape[:2], bool)
    hit[1, 3] = hit[4, 0] = hit[20, 11] = True
    assert np.isnan(b[hit]).all() and np.array_equal(a[~hit], b[~hit])


# ---------------------------------------------------------------------------
# Weights

def masses(w):
    """Masses of every slot, NaN in those that no call should look at."""
    m = w.rng.exponential(size=(w.ref.pages, w.ref.heads, w.ref.P)).astype(np.float32)
    used = np.zeros(m.shape[::2], bool)
    for b in range(len(w.ref.lens)):
        n = plain.length(w.ref, b)
        page, slot, there = plain.pages_of(w.ref, b, n)
        earlier = np.arange(n) < n - int(w.ref.starts[b + 1] - w.ref.starts[b])
        used[page[there & earlier], slot[there & earlier]] = True
    m[~np.broadcast_to(used[:, None], m.shape)] = np.nan
    return m


def check_weigh(w, group, dtype, *, causal=True, window=0, scale=None, q=None, lse=None, tag="", rows=None, **kw):
    heads, D = w.ref.heads * group, w.ref.D
    theirs, ours = shape_of(w, group, **kw)
    rows = w.rows + 2 if rows is None else rows
    q = w.values(rows, dtype, heads=heads, spread=0.4) if q is None else q
    scale = float(np.float32(D ** -0.5)) if scale is None else scale
    say(f"weigh {tag} heads={heads}/{w.ref.heads} D={D} P={w.ref.P} lens={list(w.ref.lens)[:6]} {dtype} causal={causal} window={window} {kw}")
    if lse is None:
        lse = plain.attention(w.ref, q, scale, causal, window, **theirs)["lse"].astype(np.float32)
    q[w.rows:], lse[w.rows:] = np.nan, np.nan
    mass = masses(w)
    add = noise(D, dtype)
    want, off = plain.weigh(w.ref, q, lse, mass, scale, causal, window, **theirs,
                            noise=lambda parts, spread, s: add(parts, spread) + 8 * U * parts + 4 * U * np.abs(s) + 8 * U)
    got = dev(mass)
    kv8_scores.kv8_weigh(w.cache, w.batch, dev(q, dtype), dev(lse), got, scale=scale, causal=causal, window=window, **ours)
    m = host(got)
    assert np.array_equal(np.isnan(m), np.isnan(want))
    some = ~np.isnan(want)
    err, tol = np.abs(m - want)[some], off[some] + 1e-37
    assert (err <= tol).all(), f"mass: worst {np.max(err / tol):.3g} of the bound"
    return got


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s[:4])))
def test_weigh(size, dtype):
    for i, shape in enumerate(SHAPES + [{}]):
        w, group, kw = world(i, size, shape)
        check_weigh(w, group, dtype, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weigh_long(dtype):
    for lens, news, kw in (([5000], [1], {}), ([3, 4100, 0, 1200], [1, 1, 0, 1], dict(slopes=True)),
                           ([2500, 700], [40, 3], dict(window=600, cap=5.0, prefix=[2400, 100])), ([1500], [1500], {})):
        check_weigh(World(7, 2, 128, 64, lens, news), 6, dtype, tag="long", **kw)


def test_weigh_rows_that_add_nothing():
    """Rows and heads whose lse is not finite, whatever their queries hold."""
    w = World(21, 2, 64, 16, [90, 33], [20, 5])
    q = w.values(w.rows, F32, heads=8)
    lse = plain.attention(w.ref, q, 0.125)["lse"].astype(np.float32)
    lse[3, 2], lse[9, :], lse[22, 7] = np.nan, -np.inf, np.inf
    q[3, 2, 5], q[9, 1], q[22, 7, 0] = np.nan, np.inf, -np.inf
    with np.errstate(invalid="ignore"):
        check_weigh(w, 4, F32, scale=0.125, q=q, lse=lse, rows=w.rows)


def test_weigh_sums_to_the_rows():
    """A row's weights sum to 1 for each head: a prompt's masses sum to its rows times the group."""
    for dtype in (F32, F16, BF16):
        w = World(22, 2, 128, 64, [700], [700])
        q = dev(w.values(700, dtype, heads=12), dtype)
        _, lse = kv8.kv8_attention(w.cache, w.batch, q, lse=True)
        mass = kv8_scores.new_mass(w.cache)
        kv8_scores.kv8_weigh(w.cache, w.batch, q, lse, mass)
        assert np.allclose(host(mass).astype(np.float64).sum((0, 2)), 700 * 6, rtol=1e-5)


def test_weigh_a_shared_prompt():
    """Two sequences read the same pages: their masses get both's weights."""
    w = World(23, 2, 64, 16, [100, 90], [1, 1])
    w.ref.table[1, :4] = w.ref.table[0, :4]
    w.batch.table.copy_(dev(w.ref.table))
    check_weigh(w, 4, F32, rows=w.rows)


# ---------------------------------------------------------------------------
# Choice

@pytest.mark.parametrize("heads,P,lens,keep,first,recent", [
    (1, 16, [1], 1, 0, 0),
    (2, 64, [777, 100, 0, 300], 300, 4, 50),
    (3, 16, [65, 64, 63, 1], 64, 0, 64),
    (2, 32, [2000, 1025, 1024, 1023], 1024, 1000, 0),
    (1, 128, [5000, 70, -4], 0, 0, 0),
    (1, 256, [5000, 70], 4999, 10, 3),
    (2, 16, [3000, 31], 17, 3, 14),
    (8, 64, [9000], 100, 4, 32),
])
def test_choose(heads, P, lens, keep, first, recent):
    for holes in (0.0, 0.3):
        w = World(P + keep, heads, 16, P, lens, [0] * len(lens), holes=holes)
        m = w.rng.exponential(size=(w.ref.pages, heads, P)).astype(np.float32)
        m[w.rng.random(m.shape) < 0.4] = 0.0
        m[w.rng.random(m.shape) < 0.1] = -0.0
        some = w.rng.random(m.shape) < 0.1
        m[some] = w.rng.choice(np.float32([0.5, 0.25, -1.0, np.inf, -np.inf, np.nan, 1e-40]), size=int(some.sum()))
        say(f"choose heads={heads} P={P} lens={lens} keep={keep} first={first} recent={recent} holes={holes}")
        want = plain.choose(w.ref, m, keep, first, recent)
        got = kv8_scores.kv8_choose(w.cache, w.batch, dev(m), keep, first=first, recent=recent)
        for a, b in zip(got, want):
            assert a.dtype == torch.int32 and np.array_equal(host(a), b)


def test_choose_of_equal_masses_takes_the_lowest():
    w = World(31, 2, 16, 64, [3000, 100], [0, 0])
    for value in (0.0, 1.0, np.nan, np.inf):
        m = np.full((w.ref.pages, 2, 64), value, np.float32)
        index, kept = kv8_scores.kv8_choose(w.cache, w.batch, dev(m), 128, first=2, recent=20)
        want = np.concatenate([np.arange(108), np.arange(2980, 3000)])
        assert (host(index)[0] == want).all() and host(kept).tolist() == [128, 100]


# ---------------------------------------------------------------------------
# Move

MOVES = [
    (1, 16, 16, [1], 1),
    (2, 128, 64, [777, 100, 0, 300], 200),
    (3, 80, 32, [100, 31, 64], 33),
    (1, 256, 16, [50, 17], 40),
    (2, 48, 256, [600, 256, 3], 300),
    (1, 64, 128, [2000], 515),
    (1, 256, 256, [511], 511),
]


def movable(seed, heads, D, P, lens, keep, holes=0.0):
    """A world, a choice in it, and fresh pages for it."""
    need = sum(-(-min(keep, max(0, n)) // P) for n in lens) + 2
    w = World(seed, heads, D, P, lens, [0] * len(lens), holes=holes, spare=need)
    fresh = np.setdiff1d(np.arange(w.ref.pages), w.ref.table)
    to = np.full((len(lens), -(-keep // P) + 1), -1, np.int32)
    kept, at = np.array([min(keep, max(0, n)) for n in lens], np.int32), 0
    for b, n in enumerate(kept):
        to[b, :-(-n // P)] = fresh[at:at + -(-n // P)]
        at += -(-n // P)
    index = np.full((len(lens), heads, keep), -1, np.int32)
    for b, n in enumerate(kept):
        for h in range(heads):
            index[b, h, :n] = np.sort(w.rng.permutation(max(0, lens[b]))[:n])
    return w, index, kept, to


def check_move(w, index, kept, to):
    m = w.rng.exponential(size=(w.ref.pages, w.ref.heads, w.ref.P)).astype(np.float32)
    mass = dev(m)
    plain.move(w.ref, index, kept, to, m)
    kv8_scores.kv8_move(w.cache, w.batch, dev(index), dev(kept), dev(to), mass=mass)
    w.same_cache()
    assert np.array_equal(bits(host(mass)), bits(m))


@pytest.mark.parametrize("heads,D,P,lens,keep", MOVES)
def test_move(heads, D, P, lens, keep):
    for holes in (0.0, 0.3):
        say(f"move heads={heads} D={D} P={P} lens={lens} keep={keep} holes={holes}")
        check_move(*movable(D + P, heads, D, P, lens, keep, holes))


def test_move_odd_choices():
    """Tokens chosen twice, out of order, outside the sequence; counts below 0 and over keep; destinations that are none."""
    w, index, kept, to = movable(41, 2, 64, 32, [300, 200, 100], 120)
    index[0, 0, :7] = [5, 5, 3, 299, 300, -1, 2 ** 31 - 1]
    index[1, 1, 40:80] = -2 ** 31
    index[2, :, :] = index[2, :, ::-1]
    kept[:] = [130, 120, -5]
    to[1, 1] = -1
    to[1, 2] = w.ref.pages
    check_move(w, index, kept, to)


def test_move_equals_read_and_append():
    """What the header says: values read back in F32 and appended to pages begun now."""
    w, index, kept, to = movable(42, 2, 128, 64, [500], 150)
    k, _ = kv8.kv8_read(w.cache, kv8.KV8Batch(w.batch.table, w.batch.lens), 500)
    v = kv8.kv8_read(w.cache, kv8.KV8Batch(w.batch.table, w.batch.lens), 500)[1]
    twin = kv8.KV8Cache(*(t.clone() for t in (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)))
    at = dev(index.astype(np.int64))[0].t()[:, :, None].expand(-1, -1, 128)
    rows = kv8.KV8Batch(dev(to), dev(kept))
    kv8.kv8_append(twin, rows, torch.gather(k, 0, at), torch.gather(v, 0, at))
    kv8_scores.kv8_move(w.cache, w.batch, dev(index), dev(kept), dev(to))
    for a, b in zip((w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale), (twin.k, twin.v, twin.k_scale, twin.v_scale)):
        assert np.array_equal(host(a).view(np.uint8), host(b).view(np.uint8))


# ---------------------------------------------------------------------------
# Together

def test_a_run_that_weighs_evicts_and_goes_on():
    """Prompts, decode steps, an eviction, decode steps over what stayed: each step against the plain forms over the same cache."""
    D, P, heads, group = 64, 16, 2, 3
    lens = [70, 45]
    w = World(51, heads, D, P, lens, lens, spare=20, blocks=8)
    fresh = [int(p) for p in np.setdiff1d(np.arange(w.ref.pages), w.ref.table)]
    w.ref.table[(w.ref.table < 0) | (w.ref.table >= w.ref.pages)] = -1
    mass = kv8_scores.new_mass(w.cache)
    pmass = host(mass)
    _, ours = shape_of(w, group, cap=8.0, slopes=True)
    theirs = {"cap": 8.0, "slopes": host(ours["slopes"]), "prefix": None}
    scale = float(np.float32(D ** -0.5))

    def step(news):
        nonlocal pmass
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        for b, n in enumerate(w.ref.lens):
            for j in range(-(-int(n) // P)):
                if w.ref.table[b, j] < 0:
                    w.ref.table[b, j] = fresh.pop()
        w.ref.starts = starts
        w.batch = kv8.KV8Batch(dev(w.ref.table), dev(w.ref.lens), dev(starts), max_len=int(w.ref.lens.max()))
        rows = int(starts[-1])
        k, v, q = w.values(rows, F32), w.values(rows, F32), w.values(rows, F32, heads=heads * group)
        w.ref.append(k, v)
        kv8.kv8_append(w.cache, w.batch, dev(k), dev(v))
        w.same_cache()
        out, lse = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q), lse=True, **ours)
        kv8_scores.kv8_weigh(w.cache, w.batch, dev(q), lse, mass, **ours)
        ref = plain.attention(w.ref, q, scale, **theirs)
        assert np.allclose(host(out), ref["out"], rtol=1e-4, atol=1e-4 * np.abs(ref["out"]).max())
        pmass, _ = plain.weigh(w.ref, q, host(lse), pmass, scale, **theirs)
        assert np.allclose(host(mass), pmass, rtol=1e-4, atol=1e-6)

    step(lens)
    for _ in range(5):
        w.ref.lens = w.ref.lens + 1
        step([1, 1])
    index, kept = kv8_scores.kv8_choose(w.cache, w.batch, mass, 40, first=2, recent=8)
    want = plain.choose(w.ref, host(mass), 40, 2, 8)
    assert np.array_equal(host(index), want[0]) and np.array_equal(host(kept), want[1])
    to = np.full((2, 8), -1, np.int32)
    for b in range(2):
        for j in range(-(-int(want[1][b]) // P)):
            to[b, j] = fresh.pop()
    m = host(mass).copy()
    plain.move(w.ref, *want, to, m)
    kv8_scores.kv8_move(w.cache, w.batch, index, kept, dev(to), mass=mass)
    w.same_cache()
    assert np.array_equal(bits(host(mass)), bits(m))
    pmass = m.astype(np.float64)
    fresh.extend(int(p) for p in w.ref.table[w.ref.table >= 0])
    w.ref.table, w.ref.lens = to, want[1].astype(np.int32)
    for _ in range(6):
        w.ref.lens = w.ref.lens + 1
        step([1, 1])


@pytest.mark.parametrize("lens,keep", [
    ([4096, 4097, 3000], 1000),            # 16 tokens a lane, 256 or 512 lanes
    ([8192, 8193], 8000),
    ([16384, 100], 2000),
    ([16385, 65536], 30000),               # 64 tokens a lane
    ([65537, 140000, 5], 50001),           # in segments
])
def test_choose_long(lens, keep):
    """On both sides of each size of workgroup, and past the longest one's."""
    w = World(keep, 2, 16, 64, lens, [0] * len(lens), holes=0.02)
    m = np.exp(2 * w.rng.normal(size=(w.ref.pages, 2, 64))).astype(np.float32)
    m[w.rng.random(m.shape) < 0.3] = 0.0
    m[w.rng.random(m.shape) < 0.2] = np.float32(0.75)
    want = plain.choose(w.ref, m, keep, 5, 700)
    for bound in (max(lens), 0, 10):
        w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=bound)
        say(f"choose lens={lens} keep={keep} max_len={bound}")
        for a, b in zip(kv8_scores.kv8_choose(w.cache, w.batch, dev(m), keep, first=5, recent=700), want):
            assert np.array_equal(host(a), b)


def test_choose_of_many_sequences():
    w = World(77, 8, 16, 64, list(range(8300, 8300 + 40 * 40, 40)), [0] * 40)
    m = w.rng.exponential(size=(w.ref.pages, 8, 64)).astype(np.float32)
    want = plain.choose(w.ref, m, 1500, 4, 64)
    for a, b in zip(kv8_scores.kv8_choose(w.cache, w.batch, dev(m), 1500, first=4, recent=64), want):
        assert np.array_equal(host(a), b)
