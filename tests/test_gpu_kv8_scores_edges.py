"""Scores, weights and eviction over the int8 K/V cache where kernels and
binding meet their edges, against the plain 64-bit forms; tolerances as derived
in test_gpu_kv8_scores, whose checks are used."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import kv8, kv8_scores
from ternary_weight_integer_amd.i2s import I2SError

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import kv8_plain as plain  # noqa: E402
from test_gpu_kv8 import BF16, DEV, F16, F32, U, World, bits, dev, host, say  # noqa: E402
from test_gpu_kv8_scores import check_move, check_scored, check_weigh, masses, movable, noise, shape_of  # noqa: E402


@pytest.mark.parametrize("seqs", [63, 64, 65, 300])
def test_many_sequences(seqs):
    """On both sides of the one-load search, with sequences that bring no rows."""
    rng = np.random.default_rng(seqs)
    news = rng.integers(0, 4, size=seqs) * (rng.random(seqs) < 0.7)
    news[:2] = news[-3:] = 0
    news[7] = 40
    lens = news + rng.integers(0, 60, size=seqs)
    prefix = rng.integers(-5, 60, size=seqs)
    for dtype in (F32, BF16):
        check_scored(World(seqs, 1, 32, 16, lens, news, lead=2), 3, dtype, cap=4.0, slopes=True, prefix=prefix, tag=f"{seqs} sequences")
        check_weigh(World(seqs, 1, 32, 16, lens, news, lead=2), 3, dtype, cap=4.0, slopes=True, prefix=prefix, tag=f"{seqs} sequences")


def test_batches_without_starts():
    for n in (1, 5, 33):
        w = World(n, 2, 64, 16, [40, 33, 90, 64], [n] * 4, starts=False)
        check_scored(w, 3, F32, rows=w.rows, slopes=True, prefix=[10, 0, 90, 3], tag="no starts")
        w = World(n, 2, 64, 16, [40, 33, 90, 64], [n] * 4, starts=False)
        check_weigh(w, 3, F32, rows=w.rows, slopes=True, prefix=[10, 0, 90, 3], tag="no starts")


def test_a_very_wide_group():
    check_scored(World(64, 1, 64, 64, [400, 30], [2, 1]), 1000, F32, cap=9.0, slopes=True, tag="1000 heads over one")
    check_weigh(World(64, 1, 64, 64, [400, 30], [2, 1]), 1000, F32, cap=9.0, slopes=True, tag="1000 heads over one")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,group,seqs,rows", [(8, 64, 4, 60, 70), (8, 128, 4, 60, 70), (8, 112, 7, 40, 66)])
def test_scored_many_rows(heads, D, group, seqs, rows, dtype):
    """Waves of two row tiles."""
    rng = np.random.default_rng(seqs + D)
    news = rng.integers(rows - 40, rows + 20, size=seqs)
    news[3] = 0
    lens = news + rng.integers(0, 50, size=seqs) * (rng.random(seqs) < 0.5)
    check_scored(World(D, heads, D, 32, lens, news, lead=1), group, dtype, cap=6.0, slopes=True, prefix=rng.integers(0, 90, size=seqs))
    check_weigh(World(D, heads, D, 32, lens, news, lead=1), group, dtype, window=40)


@pytest.mark.parametrize("news", [[3, 1], [1900, 30]])
def test_a_bound_of_the_lengths_only_steers(news):
    """Lengths past max_len, tables far longer than any length, and no bound at all: the same masses."""
    for bound in (1, 300, 0, 4000):
        w = World(61, 2, 128, 64, [2600, 40], news, blocks=700)
        w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=bound)
        check_weigh(w, 3, F32, tag=f"max_len={bound}")
        check_scored(w, 3, F32, cap=20.0, tag=f"max_len={bound}")


def test_weigh_without_a_bound_and_many_sequences():
    """Fewer workgroups than token blocks, each with several."""
    w = World(5, 8, 32, 64, list(range(300, 300 + 64 * 20, 20)), [2] * 64, blocks=3000)
    w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=0)
    check_weigh(w, 2, BF16, tag="no bound")


def test_weigh_a_page_twice_in_a_sequence():
    w = World(24, 2, 64, 16, [100], [1])
    w.ref.table[0, 1] = w.ref.table[0, 3]
    w.batch.table.copy_(dev(w.ref.table))
    check_weigh(w, 4, F32, rows=w.rows)


def test_weigh_is_the_same_every_time():
    for news in ([1, 1], [2000, 90]):
        w = World(16, 2, 128, 64, [3000, 100], news)
        rows = sum(news)
        q = dev(w.values(rows, F32, heads=12))
        _, lse = kv8.kv8_attention(w.cache, w.batch, q, lse=True)
        first = None
        for _ in range(5):
            mass = kv8_scores.new_mass(w.cache)
            kv8_scores.kv8_weigh(w.cache, w.batch, q, lse, mass)
            first = mass if first is None else first
            assert torch.equal(mass, first)


def test_weigh_large_bf16_queries():
    """Products with the codes past F32's range, exponents inside it."""
    w = World(25, 1, 128, 64, [200], [3])
    q = w.values(3, BF16, heads=2, spread=0.0)
    for size, scale in ((2.0 ** 120, 2.0 ** -123), (2.0 ** -80, 2.0 ** 77)):
        check_weigh(w, 2, BF16, q=(q * size).astype(np.float32), scale=scale, rows=3, tag=f"size={size}")


def test_a_wide_channel_takes_nothing_from_the_others():
    """F32 queries with one component 1000 times the rest, and the key channel to it zero."""
    w = World(26, 2, 128, 64, [300], [70])
    w.ref.k[:, :, :, 5] = 0
    w.cache.k.copy_(dev(w.ref.k))
    q = w.values(w.rows, F32, heads=4, spread=0.0)
    q[:, :, 5] = 1000.0
    theirs, ours = shape_of(w, 2, cap=30.0)
    scale = float(np.float32(128 ** -0.5))
    lse = plain.attention(w.ref, q, scale, cap=30.0)["lse"].astype(np.float32)
    got = kv8_scores.new_mass(w.cache)
    kv8_scores.kv8_weigh(w.cache, w.batch, dev(q), dev(lse), got, scale=scale, cap=30.0)
    small = q.copy()
    small[:, :, 5] = 0
    want, off = plain.weigh(w.ref, small, lse, np.zeros(got.shape, np.float32), scale, cap=30.0,
                            noise=lambda parts, spread, s: noise(128, F32)(parts, spread) + 8 * U * parts + 4 * U * np.abs(s) + 8 * U)
    assert (np.abs(host(got) - want) <= 2 * off + 1e-37).all()


def test_strided_queries():
    """Queries as a view of a fused projection's rows, outputs into one."""
    w = World(9, 2, 64, 16, [100, 90, 100], [3, 2, 3])
    line = w.rng.normal(0, 1, size=(w.rows, 1000)).astype(np.float32)
    q, t = line[:, 40:552].reshape(w.rows, 8, 64), dev(line)
    view = t[:, 40:552].view(w.rows, 8, 64)
    _, ours = shape_of(w, 4, cap=5.0, slopes=True)
    out = torch.full((w.rows, 600), 3.0, device=DEV)
    _, lse = kv8_scores.kv8_attention_scored(w.cache, w.batch, view, out=out[:, 4:516].view(w.rows, 8, 64), lse=True, **ours)
    dense, same = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q), lse=True, **ours)
    o = host(out)
    assert np.array_equal(o[:, 4:516].reshape(w.rows, 8, 64), host(dense)) and torch.equal(lse, same)
    assert (o[:, :4] == 3).all() and (o[:, 516:] == 3).all()
    a, b = kv8_scores.new_mass(w.cache), kv8_scores.new_mass(w.cache)
    kv8_scores.kv8_weigh(w.cache, w.batch, view, lse, a, **ours)
    kv8_scores.kv8_weigh(w.cache, w.batch, dev(q), lse, b, **ours)
    assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 bytes: chosen tokens out of its last pages into others of its last."""
    heads, D, P, pages = 8, 256, 64, 17000
    small, index, kept, to = movable(3, heads, D, P, [130], 70)
    used = np.concatenate([small.ref.table[0, :3], to[0, :2]])
    far = np.array([pages - 1, 3, pages - 2, pages - 4, pages - 3], np.int32)
    k = torch.zeros((pages, heads, P, D), dtype=torch.int8, device=DEV)
    v = torch.zeros((pages, heads, D, P), dtype=torch.int8, device=DEV)
    ks, vs = torch.zeros((pages, heads), device=DEV), torch.zeros((pages, heads), device=DEV)
    for a, b in zip(used, far):
        k[b], v[b], ks[b], vs[b] = (x[a] for x in (small.cache.k, small.cache.v, small.cache.k_scale, small.cache.v_scale))
    cache = kv8.KV8Cache(k, v, ks, vs)
    batch = kv8.KV8Batch(dev(far[None, :3]), dev(np.array([130], np.int32)), dev(np.array([0, 66], np.int32)))
    small.ref.starts[:] = [0, 66]
    q = small.values(66, F32, heads=16, spread=0.2)
    got, lse = kv8_scores.kv8_attention_scored(cache, batch, dev(q), cap=10.0, lse=True)
    ref = plain.attention(small.ref, q, 1 / 16, cap=10.0)
    assert np.allclose(host(got), ref["out"], rtol=1e-4, atol=1e-4 * np.abs(ref["out"]).max())
    mass = kv8_scores.new_mass(cache)
    kv8_scores.kv8_weigh(cache, batch, dev(q), lse, mass, cap=10.0)
    want, _ = plain.weigh(small.ref, q, host(lse), np.zeros((small.ref.pages, heads, P)), 1 / 16, cap=10.0)
    for a, b in zip(used[:3], far[:3]):
        assert np.allclose(host(mass[int(b)]), want[a], rtol=1e-4, atol=1e-7)
    plain.move(small.ref, index, kept, to)
    there = np.full_like(to, -1)
    there[0, :2] = far[3:]
    kv8_scores.kv8_move(cache, batch, dev(index), dev(kept), dev(there), mass=mass)
    for a, b in zip(to[0, :2], far[3:]):
        assert np.array_equal(host(k[int(b)]), small.ref.k[a]) and np.array_equal(host(v[int(b)]), small.ref.v[a])
        assert np.array_equal(bits(host(ks[int(b)])), bits(small.ref.ks[a])) and np.array_equal(bits(host(vs[int(b)])), bits(small.ref.vs[a]))


def test_move_near_ties_and_extremes():
    """Scales a rounding apart, so that quotients lie around the middle of two integers; tiny, zero and huge scales."""
    for seed, scales in enumerate(([0.01, 0.02, 0.005], [1.0, np.nextafter(np.float32(1), np.float32(2)), 0.5], [1e-40, 1e-9, 0.0],
                                   [1e36, 1e30, 2.0 ** 100], [3.0, 1.5, 127 / 254.0])):
        w, index, kept, to = movable(90 + seed, 2, 128, 16, [200, 60], 100)
        w.ref.ks[:] = w.rng.choice(np.float32(scales), size=w.ref.ks.shape)
        w.ref.vs[:] = w.rng.choice(np.float32(scales), size=w.ref.vs.shape)
        w.cache.k_scale.copy_(dev(w.ref.ks))
        w.cache.v_scale.copy_(dev(w.ref.vs))
        say(f"move scales={scales}")
        check_move(w, index, kept, to)


@pytest.mark.parametrize("D,P", [(16, 16), (256, 16), (80, 16), (48, 32), (112, 64), (256, 64), (16, 128), (256, 128), (16, 256), (64, 256)])
def test_move_every_layout(D, P):
    """Items of one, two and four waves, staged and not, held in registers and gathered twice; few and many pages to a page."""
    for lens, keep in (([900, 333], 300), ([5000], 70), ([40, 3], 40)):
        check_move(*movable(D + P, 2, D, P, lens, keep))


# ---------------------------------------------------------------------------
# Streams and graphs

def one_step(w, q, lse_in, mass, keep, ours, to, **kw):
    out, lse = kv8_scores.kv8_attention_scored(w.cache, w.batch, q, lse=True, **ours, **kw)
    kv8_scores.kv8_weigh(w.cache, w.batch, q, lse_in, mass, **ours, **kw)
    index, kept = kv8_scores.kv8_choose(w.cache, w.batch, mass, keep, first=2, recent=16, **kw)
    kv8_scores.kv8_move(w.cache, w.batch, index, kept, to, mass=mass, **kw)
    return out, lse, index, kept


def test_calls_on_another_stream():
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side.cuda_stream):
        w, _, _, to = movable(70, 2, 128, 64, [3000, 900], 200)
        w.ref.starts[:] = [0, 40, 41]
        w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, dev(w.ref.starts), max_len=3000)
        _, ours = shape_of(w, 6, cap=8.0, slopes=True)
        q, mass = dev(w.values(41, F32, heads=12)), kv8_scores.new_mass(w.cache)
        lse = dev(w.rng.normal(3, 0.1, size=(41, 12)).astype(np.float32))
        torch.cuda.synchronize()
        r = one_step(w, q, lse, mass, 200, ours, dev(to), stream=stream)
        torch.cuda.synchronize()
        got.append([host(x) for x in (*r, mass, w.cache.k, w.cache.v, w.cache.k_scale)])
    for other in got[1:]:
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got[0], other))


def test_captured_steps_follow_the_device():
    """Two steps captured, each with a workspace of its own, replayed with new queries, masses and lengths; eager work between the
    replays, and every replay against the eager result."""
    worlds, graphs = [], []
    for seed in (71, 72):
        w, _, _, to = movable(seed, 2, 64, 16, [900, 400], 120, holes=0.0)
        w.ref.starts[:] = [0, 30, 33]
        w.batch = kv8.KV8Batch(w.batch.table, dev(w.ref.lens), dev(w.ref.starts), max_len=1000)
        _, ours = shape_of(w, 4, cap=8.0, prefix=[100, 5])
        worlds.append((w, ours, dev(w.values(33, BF16, heads=8), BF16), dev(np.full((33, 8), 4.0, np.float32)),
                       kv8_scores.new_mass(w.cache), dev(to)))
    side = torch.cuda.Stream()
    for w, ours, q, lse, mass, to in worlds:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            one_step(w, q, lse, mass, 120, ours, to)  # libraries and kernels loaded
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = one_step(w, q, lse, mass, 120, ours, to)
        graphs.append((g, held))
    rng = np.random.default_rng(5)
    for replay in range(4):
        for (w, ours, q, lse, mass, to), (g, held) in zip(worlds, graphs):
            q.copy_(dev(rng.normal(0, 1, size=q.shape).astype(np.float32), BF16))
            mass.copy_(dev(rng.exponential(size=mass.shape).astype(np.float32)))
            w.batch.lens.copy_(dev(np.array([900 - 100 * replay, 400 - 3 * replay], np.int32)))
        torch.cuda.synchronize()
        before = [[t.clone() for t in (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale, mass)] for w, _, _, _, mass, _ in worlds]
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (w, ours, q, lse, mass, to), (_, held), start in zip(worlds, graphs, before):
            got = [host(x) for x in (*held, mass, w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)]
            for t, s in zip((w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale, mass), start):
                t.copy_(s)
            eager = one_step(w, q, lse, mass, 120, ours, to)
            want = [host(x) for x in (*eager, mass, w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)]
            assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# Refusals of the binding

def test_refusals():
    w, index, kept, to = movable(80, 2, 64, 16, [100, 40], 30)
    q, mass = dev(w.values(2, F32, heads=8)), kv8_scores.new_mass(w.cache)
    lse = torch.zeros((2, 8), device=DEV)
    index, kept, to = dev(index), dev(kept), dev(to)
    batch = kv8.KV8Batch(w.batch.table, w.batch.lens)
    weigh = lambda **kw: kv8_scores.kv8_weigh(**{**dict(cache=w.cache, batch=batch, q=q, lse=lse, mass=mass), **kw})  # noqa: E731
    scored = lambda **kw: kv8_scores.kv8_attention_scored(w.cache, batch, q, **kw)  # noqa: E731
    for call in (weigh, scored):
        for kw in (dict(slopes=torch.ones(7, device=DEV)), dict(slopes=torch.ones(8)), dict(slopes=torch.ones(8, dtype=F16, device=DEV)),
                   dict(prefix=torch.ones(2, device=DEV)), dict(prefix=torch.ones(3, dtype=torch.int32, device=DEV)),
                   dict(workspace=torch.zeros(64, device=DEV))):
            with pytest.raises(ValueError):
                call(**kw)
        for kw in (dict(cap=-1.0), dict(cap=float("nan")), dict(window=-1), dict(scale=float("inf"))):
            with pytest.raises(I2SError):
                call(**kw)
    for kw in (dict(lse=lse[:1]), dict(lse=lse.double()), dict(lse=lse.t().contiguous().t()), dict(mass=mass[:-1]), dict(mass=mass.cpu()),
               dict(mass=mass.transpose(0, 1))):
        with pytest.raises(ValueError):
            weigh(**kw)
    with pytest.raises(TypeError):
        weigh(q=q.double())
    for kw in (dict(keep=-1), dict(keep=10, first=6, recent=5), dict(keep=10, first=-1)):
        with pytest.raises(I2SError):
            kv8_scores.kv8_choose(w.cache, batch, mass, **kw)
    for kw in (dict(index=index[:, :, :5]), dict(kept=kept[:1]), dict(mass=mass[1:])):
        with pytest.raises(ValueError):
            kv8_scores.kv8_choose(w.cache, batch, **{**dict(mass=mass, keep=30, index=index, kept=kept), **kw})
    for bad in (to[:1], to.t().contiguous().t(), to[:, :1].expand(2, 3)):
        with pytest.raises(ValueError):
            kv8_scores.kv8_move(w.cache, batch, index, kept, bad)
    for bad in ((index[:1], kept, to), (index[:, :1], kept, to), (index, kept[:1], to), (index.long(), kept, to)):
        with pytest.raises((ValueError, TypeError)):
            kv8_scores.kv8_move(w.cache, batch, *bad)
    w.same_cache()


def test_nothing_kept_and_nothing_there():
    w, index, kept, to = movable(81, 2, 64, 16, [100, 0], 30)
    mass = kv8_scores.new_mass(w.cache)
    none, count = kv8_scores.kv8_choose(w.cache, w.batch, mass, 0)
    assert none.shape == (2, 2, 0) and host(count).tolist() == [0, 0]
    kv8_scores.kv8_move(w.cache, w.batch, none, count, dev(to))
    kv8_scores.kv8_move(w.cache, w.batch, dev(index), torch.zeros(2, dtype=torch.int32, device=DEV), dev(to), mass=mass)
    kv8_scores.kv8_weigh(w.cache, w.batch, torch.zeros((0, 4, 64), device=DEV), torch.zeros((0, 4), device=DEV), mass)
    w.same_cache()
    assert not host(mass).any()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_weigh_few_rows_on_average(D, dtype):
    """A decode step's kernel where one sequence has several stages of rows, with windows that leave blocks behind, a prefix that
    reaches past them, and holes."""
    lens, news = [1300] + list(range(250, 700, 45)) * 2, [90] + [1] * 20
    for kw in ({}, dict(window=100), dict(window=300, prefix=[1290] + [240] * 20, cap=5.0), dict(causal=False, slopes=True, holes=0.2)):
        w = World(D, 2, D, 32, lens, news, holes=kw.pop("holes", 0.0))
        assert w.rows * 3 <= 16 * len(lens)
        check_weigh(w, 3, dtype, **kw)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_weigh_many_rows_among_many_sequences(dtype):
    """So many sequences that a workgroup takes all the blocks of one, more than it holds the sums of, and one with several stages."""
    lens, news = [9 + i % 20 for i in range(1023)] + [2700], [1] * 1023 + [50]
    w = World(28, 4, 64, 16, lens, news)
    assert w.rows * 3 <= 16 * len(lens) and len(lens) * 4 >= 16 * 256
    check_weigh(w, 3, dtype, window=2300, cap=5.0, tag="among")


def test_weigh_one_row_far_behind_its_window():
    for bound in (20000, 0):
        w = World(27, 1, 64, 64, [20000, 90], [1, 2])
        w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=bound)
        check_weigh(w, 4, F32, window=700, tag="far")
