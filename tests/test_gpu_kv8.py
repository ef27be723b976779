"""GPU parity of attention over the int8 K/V cache against the CPU oracle: the
quantizing append and the read-back bit for bit (whole pools are compared, so
a byte written out of place fails), rotation and attention against 64 bits
with tolerances that the arithmetic gives.

u = 2^-24 below: half a step of F32, relative.  Attention in F32 rows:
  - a query is held as a fixed-point number of 23 bits of its row's largest
    magnitude: |dq| <= 1.5 steps of max|q| / (127 * 65536) = 3 u max|q|, so an
    exponent e is off by at most 3 u spread, spread = |scale| k_scale
    sum|code| max|q| (the oracle gives its maximum over the row);
  - four roundings of partial sums (each at most u spread), and roundings of
    e in base 2 with the value scale's logarithm added (|log2| <= 25 here) and
    the maximum taken off: 8 u (2 max|e| + 25) covers them;
    so a weight's relative error is at most
    w = 7 u spread + 8 u (2 top + 25) + 4 u (the exponential itself);
  - sums over n tokens in any order: n u of the sum of magnitudes, for the
    numerator (mag = sum p |v| / sum p) and for the denominator;
  - weights are held as two F16 numbers, 2^-22 relative and 2^-40 of the
    largest weight absolutely: n 2^-40 * 127 max(v_scale).
16-bit rows: the fixed-point query has 15 bits (1.1 * 2^-15 max|q|), the
weight one F16 number (2^-11), and the result is rounded by half a step."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from ternary_weight_integer_amd import i2s, kv8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

DEV = torch.device("cuda:0")
U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def say(msg):
    print(msg, flush=True)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype in (F16, BF16) else t.cpu().numpy()


def bits(a):
    return np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)


def rounded(a, dtype):
    """F32 values that `dtype` holds."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype).float().numpy()


class World:
    """A cache with random contents and a batch over it, on the host (oracle)
    and on the device.  holes: share of table entries that are -1."""

    def __init__(self, seed, heads, D, P, lens, news, *, spare=3, holes=0.0, starts=True, lead=0, blocks=None):
        rng = self.rng = np.random.default_rng(seed)
        lens, news = np.asarray(lens, np.int32), np.asarray(news, np.int32)
        need = [-(-max(int(n), 0) // P) for n in lens]
        pages = sum(need) + spare
        blocks = max(need) + 2 if blocks is None else blocks
        order = rng.permutation(pages).astype(np.int32)
        table = rng.choice(np.array([-1, 2 ** 31 - 1, pages, -2 ** 31], np.int32), size=(len(lens), blocks))  # never to be used
        at = 0
        for b, n in enumerate(need):
            n = min(n, blocks)
            table[b, :n] = order[at:at + n]
            at += n
            drop = rng.random(n) < holes
            table[b, :n][drop] = rng.choice([-1, pages + 5], size=int(drop.sum()))
        st = np.concatenate([[lead], lead + np.cumsum(news)]).astype(np.int32)
        k = rng.integers(-127, 128, size=(pages, heads, P, D), dtype=np.int8)
        v = rng.integers(-127, 128, size=(pages, heads, D, P), dtype=np.int8)
        ks = rng.uniform(0.005, 0.03, size=(pages, heads)).astype(np.float32)
        vs = (2.0 ** rng.uniform(-8, -3, size=(pages, heads))).astype(np.float32)
        idle = np.setdiff1d(np.arange(pages), table[(table >= 0) & (table < pages)])
        ks[idle], vs[idle] = np.nan, np.nan  # scales of pages that nothing names
        self.ref = oracle.KV8(k, v, ks, vs, table, lens, st)
        self.rows = int(st[-1])
        self.cache = kv8.KV8Cache(dev(k), dev(v), dev(ks), dev(vs))
        self.batch = kv8.KV8Batch(dev(table), dev(lens), dev(st) if starts else None, max_len=int(max(0, lens.max())))

    def set_lens(self, lens):
        self.ref.lens[:] = lens
        self.batch.lens.copy_(dev(np.asarray(lens, np.int32)))

    def values(self, rows, dtype, heads=None, spread=1.0):
        x = self.rng.normal(0, 1, size=(rows, self.ref.heads if heads is None else heads, self.ref.D))
        x *= np.exp(spread * self.rng.normal(0, 1, size=x.shape[:2]))[:, :, None]
        return rounded(x, dtype)

    def same_cache(self):
        same = [np.array_equal(host(self.cache.k), self.ref.k), np.array_equal(host(self.cache.v), self.ref.v),
                np.array_equal(bits(host(self.cache.k_scale)), bits(self.ref.ks)),
                np.array_equal(bits(host(self.cache.v_scale)), bits(self.ref.vs))]
        assert same == [True] * 4, "k, v, k_scale, v_scale"


# (heads, D, P, lens, news)
BATCHES = [
    (1, 16, 16, [1], [1]),
    (2, 128, 64, [777], [1]),
    (2, 128, 64, [64, 65, 1, 128, 127], [1, 1, 1, 1, 1]),
    (3, 80, 32, [100, 31, 33, 0, 64], [100, 5, 33, 0, 32]),
    (2, 128, 64, [300, 64, 129], [300, 64, 64]),
    (1, 256, 16, [50, 17], [33, 17]),
    (2, 48, 256, [600, 256, 3], [400, 1, 3]),
    (1, 256, 256, [300, 511], [300, 200]),
    (4, 64, 128, [129, 500], [129, 77]),
    (1, 128, 64, [5, 0, 70], [9, 4, 3]),           # more rows than tokens
    (2, 96, 32, [40, 0, -7, 33], [8, 0, 0, 32]),   # empty and negative lengths
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,P,lens,news", BATCHES)
def test_append_and_read(heads, D, P, lens, news, dtype):
    say(f"kv8 append/read heads={heads} D={D} P={P} lens={lens} news={news} {dtype}")
    for holes, lead in ((0.0, 0), (0.3, 5)):
        w = World(1 + D + P, heads, D, P, lens, news, holes=holes, lead=lead)
        rows = w.rows + 3  # rows behind the last sequence: not to be read or written
        k, v = w.values(rows, dtype), w.values(rows, dtype)
        k[w.rows:], v[w.rows:] = np.nan, np.nan
        k[:lead] = np.nan
        w.ref.append(k, v)
        kv8.kv8_append(w.cache, w.batch, dev(k, dtype), dev(v, dtype))
        w.same_cache()
        got_k, got_v = (torch.full((rows, heads, D), 9.0, dtype=dtype, device=DEV) for _ in range(2))
        kv8.kv8_read(w.cache, w.batch, rows, k=got_k, v=got_v)
        for got, ref in zip((got_k, got_v), w.ref.read(rows)):
            want = np.where(np.isnan(ref), np.float32(9.0), rounded(ref, dtype))
            assert np.array_equal(bits(host(got)), bits(want))
        w.same_cache()


def test_append_uniform_batches_without_starts():
    for n in (1, 2, 16, 33):
        say(f"kv8 append without starts, {n} rows each")
        w = World(n, 2, 64, 16, [40, 33, 90, 64], [n] * 4, starts=False)
        k, v = w.values(4 * n, F32), w.values(4 * n, F32)
        w.ref.append(k, v)
        kv8.kv8_append(w.cache, w.batch, dev(k), dev(v))
        w.same_cache()
        got = kv8.kv8_read(w.cache, w.batch, 4 * n)
        for g, r in zip(got, w.ref.read(4 * n)):
            assert np.array_equal(bits(host(g)), bits(r))


def test_token_by_token_with_growing_scales():
    """Decode steps into the same pages: scales that grow, stay and are begun
    anew at a page's first token, codes that are rescaled again and again."""
    w = World(4, 2, 128, 16, [1, 14], [1, 1], spare=9, blocks=4)
    for b in range(2):
        w.ref.table[b] = np.arange(4) + 4 * b
    w.batch.table.copy_(dev(w.ref.table))
    for step in range(40):
        w.set_lens([1 + step, 14 + step])
        k, v = w.values(2, BF16, spread=1.5), w.values(2, BF16, spread=1.5)
        w.ref.append(k, v)
        kv8.kv8_append(w.cache, w.batch, dev(k, BF16), dev(v, BF16))
    w.same_cache()


def test_append_near_ties_and_extremes():
    """Quotients around half-integers, the floor, huge and tiny magnitudes."""
    w = World(8, 1, 64, 16, [16, 3], [16, 3])
    k, v = np.zeros((19, 1, 64), np.float32), np.zeros((19, 1, 64), np.float32)
    s = np.float32(np.float32(3.3) / np.float32(127))
    halves = (np.arange(64) - 32 + 0.5).astype(np.float32) * s
    for r in range(16):
        k[r, 0] = halves
        for _ in range(r):
            k[r, 0] = np.nextafter(k[r, 0], np.float32(np.inf if r % 2 else -np.inf))
    k[0, 0, 0] = 3.3
    k[0, 0, 1:] = np.clip(k[0, 0, 1:], -3.2, 3.2)
    v[:8], v[8:16] = 1e-30, 1e-7
    k[16:], v[16:] = 3e37, -1e-38
    w.ref.append(k, v)
    kv8.kv8_append(w.cache, w.batch, dev(k), dev(v))
    w.same_cache()


def test_strided_rows():
    """Keys and values as views of a fused projection's rows."""
    for dtype in (F32, BF16):
        w = World(6, 2, 64, 32, [50, 40], [50, 7])
        line = rounded(w.rng.normal(0, 1, size=(57, 12 * 64)), dtype)
        k, v = line[:, 512:640].reshape(57, 2, 64), line[:, 640:768].reshape(57, 2, 64)
        w.ref.append(k, v)
        t = dev(line, dtype)
        kv8.kv8_append(w.cache, w.batch, t[:, 512:640].view(57, 2, 64), t[:, 640:768].view(57, 2, 64))
        w.same_cache()
        out = torch.full((57, 300), 7.0, dtype=F32, device=DEV)
        kv8.kv8_read(w.cache, w.batch, 57, k=out[:, 8:136].view(57, 2, 64), v=out[:, 140:268].view(57, 2, 64))
        o, (rk, rv) = host(out), w.ref.read(57)
        assert np.array_equal(o[:, 8:136], rk.reshape(57, 128)) and np.array_equal(o[:, 140:268], rv.reshape(57, 128))
        assert (o[:, :8] == 7).all() and (o[:, 136:140] == 7).all() and (o[:, 268:] == 7).all()


# ---------------------------------------------------------------------------
# Attention

def attention_bound(ref, world, dtype, n):
    """(of out, of lse): see the module's head."""
    eps = {F32: 0.0, F16: 2.0 ** -11, BF16: 2.0 ** -8}[dtype]
    fixed, weight = (3 * U, 2.0 ** -22) if dtype == F32 else (1.1 * 2.0 ** -15, 2.0 ** -11)
    w = (fixed + 4 * U) * ref["spread"] + 8 * U * (2 * ref["top"] + 25) + 4 * U
    vs = world.ref.vs[np.isfinite(world.ref.vs)].max()
    out = ref["mag"] * (2 * w + 2 * n * U + weight)[..., None] + 127 * vs * n * 2.0 ** -40
    out = out + eps * np.abs(ref["out"]) + (2.0 ** -25 if dtype == F16 else 0.0)
    return out, w + 2 * n * U + 4 * U * np.abs(ref["lse"])


def check_attention(w, group, dtype, *, causal=True, window=0, scale=None, tag="", rows=None, kw=None, q=None):
    heads = w.ref.heads * group
    rows = w.rows + 2 if rows is None else rows
    q = w.values(rows, dtype, heads=heads, spread=0.4) if q is None else q
    q[w.rows:] = np.nan
    scale = float(np.float32(w.ref.D ** -0.5)) if scale is None else scale
    say(f"kv8 attention {tag} heads={heads}/{w.ref.heads} D={w.ref.D} P={w.ref.P} lens={list(w.ref.lens)[:8]} "
        f"starts={list(w.ref.starts)[:8]} {dtype} causal={causal} window={window}")
    ref = w.ref.attention(q, scale, causal, window)
    out = torch.full((rows, heads, w.ref.D), 5.0, dtype=dtype, device=DEV)
    lse = torch.full((rows, heads), 5.0, dtype=F32, device=DEV)
    kv8.kv8_attention(w.cache, w.batch, dev(q, dtype), scale=scale, causal=causal, window=window, out=out, lse=lse, **(kw or {}))
    o, s = host(out), host(lse)
    idle = np.isnan(ref["lse"])
    assert (o[idle] == 5.0).all() and (s[idle] == 5.0).all()
    none = np.isneginf(ref["lse"])
    assert not o[none].any() and np.isneginf(s[none]).all()
    live = ~idle & ~none
    tol, tol_lse = attention_bound(ref, w, dtype, max(1, int(w.ref.lens.max())))
    err, err_lse = np.abs(o[live] - ref["out"][live]), np.abs(s[live] - ref["lse"][live])
    assert (err <= tol[live]).all(), f"out: worst {np.max(err / tol[live]):.3g} of the bound"
    assert (err_lse <= tol_lse[live]).all(), f"lse: worst {np.max(err_lse / tol_lse[live]):.3g} of the bound"
    return out


# (heads, D, P, group, lens, news)
ATTEND = [
    (1, 16, 16, 1, [1], [1]),
    (2, 128, 64, 6, [777], [1]),
    (2, 128, 64, 6, [64, 65, 1, 0, 63, 200], [1, 1, 1, 1, 1, 1]),
    (1, 64, 16, 1, [15, 16, 17, 100], [1, 1, 1, 1]),
    (2, 80, 32, 3, [70, 33, 5], [4, 2, 5]),
    (2, 256, 64, 2, [300, 20], [3, 20]),
    (1, 112, 128, 16, [260, 128], [2, 1]),
    (1, 128, 16, 33, [90, 40], [1, 2]),            # a group wider than a tile
    (2, 128, 64, 6, [130, 64, 200], [130, 64, 70]),
    (3, 48, 16, 7, [100, 37], [100, 37]),
    (2, 96, 256, 4, [300, 257], [290, 30]),
    (2, 64, 32, 8, [150, 0, 40], [150, 0, 3]),
    (1, 128, 64, 4, [3, 0, 70], [9, 4, 3]),        # rows in front of position 0
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,P,group,lens,news", ATTEND)
def test_attention(heads, D, P, group, lens, news, dtype):
    for causal, window, holes in ((True, 0, 0.0), (True, 20, 0.0), (False, 0, 0.2), (False, 33, 0.0)):
        w = World(D + P + group, heads, D, P, lens, news, holes=holes, lead=0 if causal else 3)
        check_attention(w, group, dtype, causal=causal, window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_long_and_split(dtype):
    """Long sequences next to short ones, so that work is split over the axis
    and joined, with and without a window."""
    for lens, news, window in (([5000], [1], 0), ([3, 4100, 0, 1200], [1, 1, 1, 1], 0), ([2500, 700], [40, 3], 600),
                               ([1500], [1500], 0), ([2100, 30], [2, 2], 64)):
        w = World(7, 2, 128, 64, lens, news)
        check_attention(w, 6, dtype, window=window, tag="long")


def test_attention_every_page_size_at_each_offset():
    for P in (16, 32, 64, 128, 256):
        w = World(P, 1, 64, P, [P - 1, P, P + 1, 2 * P - 1, 2 * P, 3 * P + 7], [1] * 6, starts=False)
        check_attention(w, 4, F32, rows=w.rows, tag="no starts")


def test_attention_peaked_and_flat():
    """One token that takes nearly all the weight, with a tiny value scale, and
    equal weights; large scales of e."""
    for scale in (1e-6, 0.0, 3.0, -0.5):
        w = World(12, 2, 128, 32, [513, 100], [2, 1])
        w.ref.vs[w.ref.table[0, 3]] = np.float32(1e-5 / 127)
        w.cache.v_scale.copy_(dev(w.ref.vs))
        check_attention(w, 4, F32, scale=scale, tag=f"scale={scale}")
        check_attention(w, 4, BF16, scale=scale, tag=f"scale={scale}")


def test_attention_strides_and_shared_pages():
    """Queries as a view of a fused row, outputs into one, two sequences whose
    first pages are the same, and the same table row twice."""
    w = World(9, 2, 64, 16, [100, 90, 100], [3, 2, 3])
    w.ref.table[1, :4] = w.ref.table[0, :4]
    w.ref.table[2] = w.ref.table[0]
    w.batch.table.copy_(dev(w.ref.table))
    rows, heads = w.rows, 8
    line = w.rng.normal(0, 1, size=(rows, 1000)).astype(np.float32)
    q = line[:, 40:40 + 512].reshape(rows, 8, 64)
    out = torch.full((rows, 600), 3.0, dtype=F32, device=DEV)
    kv8.kv8_attention(w.cache, w.batch, dev(line)[:, 40:552].view(rows, 8, 64), out=out[:, 4:516].view(rows, 8, 64))
    ref = w.ref.attention(q, 0.125)
    o = host(out)
    tol, _ = attention_bound(ref, w, F32, 100)
    assert (np.abs(o[:, 4:516].reshape(rows, 8, 64) - ref["out"]) <= tol).all()
    assert (o[:, :4] == 3).all() and (o[:, 516:] == 3).all()


@pytest.mark.parametrize("seqs", [63, 64, 65, 700])
def test_many_sequences(seqs):
    """Batches on both sides of the one-load search, with sequences that bring
    no rows, at the front, between and at the end."""
    rng = np.random.default_rng(seqs)
    news = rng.integers(0, 4, size=seqs) * (rng.random(seqs) < 0.7)
    news[:2] = news[-3:] = 0
    news[7] = 40
    lens = news + rng.integers(0, 60, size=seqs)
    w = World(seqs, 1, 32, 16, lens, news, lead=2)
    rows = w.rows + 5
    k, v = w.values(rows, F32), w.values(rows, F32)
    w.ref.append(k, v)
    kv8.kv8_append(w.cache, w.batch, dev(k), dev(v))
    w.same_cache()
    got = [torch.full((rows, 1, 32), 9.0, device=DEV) for _ in range(2)]
    kv8.kv8_read(w.cache, w.batch, rows, k=got[0], v=got[1])
    for g, ref in zip(got, w.ref.read(rows)):
        assert np.array_equal(bits(host(g)), bits(np.where(np.isnan(ref), np.float32(9.0), ref)))
    check_attention(w, 3, F32, tag=f"{seqs} sequences")
    check_attention(w, 40, BF16, tag=f"{seqs} sequences, wide group")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("heads,D,group,seqs,rows", [(8, 64, 4, 60, 70), (8, 128, 4, 60, 70), (16, 48, 2, 40, 67), (8, 112, 7, 40, 66)])
def test_attention_of_many_rows(heads, D, group, seqs, rows, dtype):
    """More workgroups of 128 rows (rows / 128 + 1 of each sequence and head)
    than four times the compute units: waves of two row tiles, some of which
    end inside the second, or before it."""
    rng = np.random.default_rng(seqs + D)
    news = rng.integers(rows - 40, rows + 20, size=seqs)
    news[3] = 0
    assert heads * (int(news.sum()) * group // 128 + seqs) >= 1024
    w = World(D, heads, D, 32, news + rng.integers(0, 50, size=seqs) * (rng.random(seqs) < 0.5), news, lead=1)
    check_attention(w, group, dtype, tag="many rows")
    check_attention(w, group, dtype, window=40, tag="many rows")


def test_attention_of_a_very_wide_group():
    w = World(64, 1, 64, 64, [400, 30], [2, 1])
    check_attention(w, 1000, F32, tag="1000 heads over one")


def test_attention_with_a_wrong_bound_of_the_lengths():
    """max_len only steers the split: lengths past it, and tables far longer
    than any length, give the same values."""
    w = World(61, 2, 128, 64, [2600, 40], [1, 1], blocks=70)
    for bound in (1, 100, 0, 4000):
        w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=bound)
        check_attention(w, 6, F32, tag=f"max_len={bound}")


def test_attention_rows_before_holes_only():
    """Rows that see nothing but holes give zeros, whatever their queries."""
    w = World(62, 2, 64, 16, [40, 33], [3, 2])
    w.ref.table[0] = -1
    w.batch.table.copy_(dev(w.ref.table))
    q = w.values(w.rows, F32, heads=8)
    q[1, 2, 3], q[4, 1, 0] = np.nan, np.inf
    out, lse = kv8.kv8_attention(w.cache, w.batch, dev(q), lse=True)
    o, s = host(out), host(lse)
    assert not o[:3].any() and np.isneginf(s[:3]).all()
    bad = np.zeros((5, 8), bool)
    bad[4, 1] = True
    assert np.isnan(o[bad]).all() and np.isnan(s[bad]).all() and np.isfinite(o[3:][~bad[3:]]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_bad_queries_stay_in_their_rows(dtype):
    w = World(15, 2, 128, 64, [200, 90], [2, 20])
    heads = 12
    q = w.values(w.rows, dtype, heads=heads, spread=0.0)
    clean = kv8.kv8_attention(w.cache, w.batch, dev(q, dtype))
    bad = q.copy()
    bad[1, 3, 5], bad[4, 0, 127], bad[20, 11, 0] = np.nan, np.inf, -np.inf
    got = kv8.kv8_attention(w.cache, w.batch, dev(bad, dtype))
    a, b = host(clean), host(got)
    hit = np.zeros(a.shape[:2], bool)
    hit[1, 3] = hit[4, 0] = hit[20, 11] = True
    assert np.isnan(b[hit]).all() and np.array_equal(a[~hit], b[~hit])


def test_attention_is_the_same_every_time():
    w = World(16, 2, 128, 64, [3000, 100, 900], [1, 1, 1])
    q = dev(w.values(3, F32, heads=12))
    first = kv8.kv8_attention(w.cache, w.batch, q)
    for _ in range(5):
        assert torch.equal(kv8.kv8_attention(w.cache, w.batch, q), first)
    # A longer bound of the lengths splits the work differently: equal within the sums' rounding.
    wide = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=0)
    torch.testing.assert_close(kv8.kv8_attention(w.cache, wide, q), first, rtol=0, atol=3000 * 2 * U * 127 * 0.125)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 bytes, the sequence in its last pages."""
    heads, D, P, pages = 8, 256, 64, 17000  # 2.2e9 bytes each of K and V
    small = World(3, heads, D, P, [130], [66], spare=0)
    need = small.ref.table[0, :3].copy()
    k = torch.zeros((pages, heads, P, D), dtype=torch.int8, device=DEV)
    v = torch.zeros((pages, heads, D, P), dtype=torch.int8, device=DEV)
    ks, vs = torch.zeros((pages, heads), device=DEV), torch.zeros((pages, heads), device=DEV)
    far = np.array([pages - 1, 3, pages - 2], np.int32)
    for a, b in zip(need, far):
        k[b], v[b], ks[b], vs[b] = (x[a] for x in (small.cache.k, small.cache.v, small.cache.k_scale, small.cache.v_scale))
    cache = kv8.KV8Cache(k, v, ks, vs)
    batch = kv8.KV8Batch(dev(far[None, :]), small.batch.lens, small.batch.starts)
    x, y = small.values(66, F32), small.values(66, F32)
    small.ref.append(x, y)
    kv8.kv8_append(cache, batch, dev(x), dev(y))
    for a, b in zip(need, far):
        assert np.array_equal(host(k[b]), small.ref.k[a]) and np.array_equal(host(v[b]), small.ref.v[a])
    got = kv8.kv8_read(cache, batch, 66)
    for g, r in zip(got, small.ref.read(66)):
        assert np.array_equal(bits(host(g)), bits(r))
    q = small.values(66, F32, heads=16, spread=0.2)
    out = kv8.kv8_attention(cache, batch, dev(q))
    ref = small.ref.attention(q, 1 / 16)
    tol, _ = attention_bound(ref, small, F32, 130)
    assert (np.abs(host(out) - ref["out"]) <= tol).all()


# ---------------------------------------------------------------------------
# Norm and rotation

def rope_bound(x, ref, pairs, neighbours, weight, dtype):
    """A rotated component comes from two: the norm's factor has at most 16 u
    (a sum of at most 16 terms in a lane and 5 steps across, halved by the
    root, then root, quotient and two products), cosine and sine 4 u of
    themselves and 3.2 u of the angle (2^-25 of a turn's fraction), product and
    sum 3 u: 32 u (|a| + |b|) covers them; then half a step of the type."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(np.square(y), -1, keepdims=True) + 1e-6) * weight
    mag = np.abs(y)
    iu, iv = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if neighbours else (slice(0, pairs), slice(pairs, 2 * pairs))
    both = mag[..., iu] + mag[..., iv]
    mag[..., iu], mag[..., iv] = both, both
    return 32 * U * mag + torch.finfo(dtype).eps / 2 * np.abs(ref) + (2.0 ** -25 if dtype == F16 else 0.0)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,hq,hk,D,pairs", [(1, 12, 2, 128, 64), (1, 1, 1, 16, 8), (5, 3, 1, 64, 32), (33, 28, 4, 128, 32),
                                               (7, 5, 5, 96, 48), (3, 2, 1, 256, 128), (2500, 2, 1, 48, 16), (9, 16, 0, 80, 0),
                                               (4, 0, 3, 112, 56), (70, 9, 3, 160, 64), (9001, 2, 1, 16, 8), (4100, 3, 2, 64, 32)])
def test_norm_and_rotation(rows, hq, hk, D, pairs, dtype):
    rng = np.random.default_rng(rows + D)
    q, k = (rounded(rng.normal(0, 1, size=(rows, h, D)), dtype) for h in (hq, hk))
    pos = rng.integers(0, 131072, size=rows).astype(np.int32)
    pos[0], pos[-1] = 0 if rows > 1 else 7, 2 ** 20
    freq = (1e6 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    qw, kw = (1 + 0.3 * rng.normal(0, 1, size=D)).astype(np.float32), rng.uniform(-2, 2, size=D).astype(np.float32)
    for neighbours in (False, True):
        for weights in ((None, None), (qw, kw), (qw, None)):
            say(f"kv8 rope rows={rows} heads={hq}/{hk} D={D} pairs={pairs} {dtype} neighbours={neighbours} "
                f"norm={[x is not None for x in weights]}")
            got = kv8.kv8_qk_norm_rope(dev(q, dtype), dev(k, dtype), dev(pos), dev(freq), eps=1e-6, neighbours=neighbours,
                                       q_weight=None if weights[0] is None else dev(weights[0]),
                                       k_weight=None if weights[1] is None else dev(weights[1]))
            for x, g, wt in zip((q, k), got, weights):
                if not x.size:
                    continue
                ref = oracle.kv8_norm_rope(x, pos, freq, neighbours, wt, 1e-6)
                assert (np.abs(host(g) - ref) <= rope_bound(x, ref, pairs, neighbours, wt, dtype)).all()


def test_rotation_in_place_and_strided():
    rng = np.random.default_rng(2)
    rows = 37
    line = rng.normal(0, 1, size=(rows, 10 * 64)).astype(np.float32)
    pos, freq = np.arange(rows, dtype=np.int32), (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    q, k = line[:, :384].reshape(rows, 6, 64), line[:, 384:512].reshape(rows, 2, 64)
    refs = [oracle.kv8_norm_rope(x, pos, freq) for x in (q, k)]
    t = dev(line)
    qv, kv = t[:, :384].view(rows, 6, 64), t[:, 384:512].view(rows, 2, 64)
    apart = kv8.kv8_qk_norm_rope(qv, kv, dev(pos), dev(freq))
    kv8.kv8_qk_norm_rope(qv, kv, dev(pos), dev(freq), q_out=qv, k_out=kv)
    o = host(t)
    assert np.array_equal(o[:, :384].reshape(rows, 6, 64), host(apart[0])) and np.array_equal(o[:, 384:512].reshape(rows, 2, 64), host(apart[1]))
    assert np.array_equal(o[:, 512:], line[:, 512:])
    for x, g, ref in zip((q, k), apart, refs):
        assert (np.abs(host(g) - ref) <= rope_bound(x, ref, 32, False, None, F32)).all()


# ---------------------------------------------------------------------------
# Together, streams and graphs

def test_decoder_layer_attention_step_by_step():
    """What a decoder layer runs between its norms, with the I2_S projections
    around it: q/k/v (one group call, biased) -> rotation -> append ->
    attention -> o, for a prompt and then single tokens; each operator is
    checked on the inputs the device gave it."""
    rng = np.random.default_rng(20)
    H, heads, kv_heads, D, P = 512, 8, 2, 64, 16
    ternary = lambda o: rng.choice(np.array([-1, 0, 1], np.int8), size=(o, H))  # noqa: E731
    packed = [i2s.i2s_pack(dev(ternary(o)), 0.05) for o in (heads * D, kv_heads * D, kv_heads * D, H)]
    biases = [dev(rng.normal(0, 0.5, size=o).astype(np.float32)) for o in (heads * D, kv_heads * D, kv_heads * D)]
    freq = (1e6 ** (-np.arange(32) / 32)).astype(np.float32)
    w = World(21, kv_heads, D, P, [50, 23], [50, 23])
    w.ref.table = np.arange(10, dtype=np.int32).reshape(2, 5)
    pages = 12
    w.ref = oracle.KV8(np.zeros((pages, kv_heads, P, D)), np.zeros((pages, kv_heads, D, P)), np.zeros((pages, kv_heads)),
                       np.zeros((pages, kv_heads)), w.ref.table, w.ref.lens, w.ref.starts)
    cache = w.cache = kv8.new_cache(pages, kv_heads, D, P, device=DEV)
    table = dev(w.ref.table)
    lens = np.array([50, 23], np.int32)
    for step in range(4):
        news = lens.copy() if step == 0 else np.array([1, 1], np.int32)
        if step:
            lens = lens + 1
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        pos = np.concatenate([np.arange(a - n, a) for a, n in zip(lens, news)]).astype(np.int32)
        rows = int(starts[-1])
        say(f"kv8 layer step {step}: rows={rows} lens={list(lens)}")
        x = dev(rng.normal(0, 1, size=(rows, H)).astype(np.float32))
        q, k, v = i2s.i2s_mul_mat_group([(p, b.numel()) for p, b in zip(packed[:3], biases)], H, x, biases=biases)
        q, k, v = q.view(rows, heads, D), k.view(rows, kv_heads, D), v.view(rows, kv_heads, D)
        batch = kv8.KV8Batch(table, dev(lens), dev(starts) if step == 0 else None)
        qr, kr = kv8.kv8_qk_norm_rope(q, k, dev(pos), dev(freq))
        kv8.kv8_append(cache, batch, kr, v)
        o = kv8.kv8_attention(cache, batch, qr)
        y = i2s.i2s_mul_mat(packed[3], H, H, o.view(rows, H))
        for a, g in ((q, qr), (k, kr)):
            ref = oracle.kv8_norm_rope(host(a), pos, freq)
            assert (np.abs(host(g) - ref) <= rope_bound(host(a), ref, 32, False, None, F32)).all()
        w.ref.lens, w.ref.starts = lens, starts
        w.ref.append(host(kr), host(v))
        w.same_cache()
        ref = w.ref.attention(host(qr), 0.125)
        tol, _ = attention_bound(ref, w, F32, int(lens.max()))
        assert (np.abs(host(o) - ref["out"]) <= tol).all()
        assert np.array_equal(bits(host(y)), bits(oracle.mul_mat(host(packed[3]), H, H, host(o.view(rows, H)))))


@pytest.mark.parametrize("poisoned", [True, False])
def test_captured_steps_follow_lengths_on_the_device(poisoned):
    """Rotation, append and attention captured once, replayed with new tokens,
    positions and lengths; eager work and a second graph with a workspace of
    its own in between.  Every replay equals the eager calls bit for bit, also
    where scales that are NaN (poisoned) make outputs NaN."""
    w = World(30, 2, 128, 64, [900, 70], [1, 1], starts=False)
    if not poisoned:
        w.cache.k_scale.nan_to_num_(0.01), w.cache.v_scale.nan_to_num_(0.01)
    heads = 12
    twin = kv8.KV8Cache(*(t.clone() for t in (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)))
    table = w.batch.table.clone()
    table[:, :] = torch.arange(2 * table.shape[1], dtype=torch.int32, device=DEV).view(2, -1) % w.cache.pages
    lens = torch.tensor([800, 40], dtype=torch.int32, device=DEV)
    pos, freq = lens - 1, dev((1e6 ** (-np.arange(64) / 64)).astype(np.float32))
    q, k, v = (torch.zeros((2, h, 128), device=DEV) for h in (heads, 2, 2))
    batch = kv8.KV8Batch(table, lens, max_len=1000)

    def step(cache, ws):
        qr, kr = kv8.kv8_qk_norm_rope(q, k, pos, freq)
        kv8.kv8_append(cache, batch, kr, v)
        return kv8.kv8_attention(cache, batch, qr, workspace=ws)

    n = max(1, kv8.kv8_attention_workspace_bytes(w.cache, batch, heads, 2))
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(3)]
    step(w.cache, ws[0])
    torch.cuda.synchronize()
    twin.k.copy_(w.cache.k), twin.v.copy_(w.cache.v), twin.k_scale.copy_(w.cache.k_scale), twin.v_scale.copy_(w.cache.v_scale)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(w.cache, ws[0])
    with torch.cuda.graph(other):
        kv8.kv8_attention(twin, batch, q, workspace=ws[1])
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    for i in range(4):
        lens.add_(1 if i != 2 else 30)
        pos.copy_(lens - 1)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV) * (1 + i))
        graph.replay()
        other.replay()
        eager = step(twin, ws[2])
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int32), eager.view(torch.int32)) and (poisoned or not got.isnan().any())
        for a, b in ((w.cache.k, twin.k), (w.cache.v, twin.v)):
            assert torch.equal(a, b)


def test_side_stream_and_raw_handle():
    w = World(40, 2, 128, 64, [1500, 300], [1, 1])
    q = dev(w.values(2, F32, heads=12))
    want = kv8.kv8_attention(w.cache, w.batch, q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        out = kv8.kv8_attention(w.cache, w.batch, q, stream=stream)
        side.synchronize()
        assert torch.equal(out, want)
    with torch.cuda.stream(side):
        out = kv8.kv8_attention(w.cache, w.batch, q)
    side.synchronize()
    assert torch.equal(out, want)


def test_two_calls_at_once():
    """Attention of two batches over one cache, and an append to another, on
    three streams together: each as when it runs alone."""
    w, x = World(41, 2, 128, 64, [2500, 300, 900], [1, 1, 1]), World(42, 2, 128, 64, [200, 90], [100, 90])
    one = kv8.KV8Batch(w.batch.table[:1], w.batch.lens[:1].clone(), max_len=2500)
    q = [dev(w.values(n, F32, heads=12)) for n in (3, 1)]
    want = [kv8.kv8_attention(w.cache, w.batch, q[0]), kv8.kv8_attention(w.cache, one, q[1])]
    k, v = x.values(190, F32), x.values(190, F32)
    x.ref.append(k, v)
    kd, vd = dev(k), dev(v)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for turn in range(8):
        with torch.cuda.stream(streams[0]):
            a = kv8.kv8_attention(w.cache, w.batch, q[0])
        with torch.cuda.stream(streams[1]):
            b = kv8.kv8_attention(w.cache, one, q[1])
        if turn == 0:
            kv8.kv8_append(x.cache, x.batch, kd, vd, stream=streams[2])
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    x.same_cache()


def test_binding_refusals():
    w = World(50, 2, 64, 16, [20, 20], [1, 1])
    q = torch.zeros((2, 4, 64), device=DEV)
    with pytest.raises(TypeError):
        kv8.kv8_attention(w.cache, w.batch, q.double())
    with pytest.raises(ValueError):
        kv8.kv8_attention(w.cache, w.batch, torch.zeros((2, 4, 32), device=DEV))
    with pytest.raises(ValueError):
        kv8.kv8_attention(w.cache, w.batch, q.transpose(0, 1).contiguous().transpose(0, 1))  # heads not dense
    with pytest.raises(ValueError):
        kv8.kv8_attention(w.cache, w.batch, q, out=torch.zeros((3, 4, 64), device=DEV))
    with pytest.raises(i2s.I2SError) as e:
        kv8.kv8_attention(w.cache, w.batch, torch.zeros((2, 3, 64), device=DEV))  # 3 query heads over 2
    assert e.value.status == i2s.I2S_EINVAL
    with pytest.raises(ValueError):
        kv8.kv8_append(w.cache, w.batch, q[:, :2], q[:, :2].cpu())
    with pytest.raises(ValueError):
        kv8.kv8_append(w.cache, w.batch, q[:1, :2], q[:, :2])
    with pytest.raises(ValueError):
        kv8.KV8Batch(w.batch.table, w.batch.lens[:1])
    with pytest.raises(ValueError):
        kv8.KV8Cache(w.cache.k, w.cache.k, w.cache.k_scale, w.cache.v_scale)
    with pytest.raises(ValueError):
        kv8.kv8_qk_norm_rope(q, q, torch.zeros(3, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV))
