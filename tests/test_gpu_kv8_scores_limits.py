"""Scores, weights and eviction over the int8 K/V cache at the limits of what
include/kv8_scores.h promises: roundings, numbers at the ends of their range,
masses of pages taken anew, workspaces of the size asked for.  Tolerances as
derived in test_gpu_kv8_scores."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ternary_weight_integer_amd import i2s, kv8, kv8_scores
from ternary_weight_integer_amd.i2s import I2SError

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import kv8_plain as plain  # noqa: E402
from test_gpu_kv8 import BF16, DEV, F16, F32, U, World, dev, host, rounded, say  # noqa: E402
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


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("lens,news", [([70, 33], [1, 1]), ([200, 150], [200, 90])])
def test_slopes_up_to_the_largest_number(lens, news, dtype):
    """A row sees its own token, at distance 0, and the one before, whose exponent is as good as none.  Exponents are off by at most
    (3 + 64 / 16 + 8) u spread, spread < 0.125 * 0.03 * 127 * 64 * 4 = 122: 1.1e-4, and as much of a weight."""
    for steep in (2.5e38, np.finfo(np.float32).max):
        for cap in (0.0, 5.0):
            w = World(3, 2, 64, 16, lens, news)
            q = w.values(w.rows, dtype, heads=4)
            slopes = np.array([steep, 0.5, 0.0, steep], np.float32)
            say(f"slopes {steep} cap={cap} lens={lens} {dtype}")
            kw = dict(window=2, cap=cap)
            ref = plain.attention(w.ref, q, 0.125, slopes=slopes, **kw)
            out, lse = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q, dtype), slopes=dev(slopes), lse=True, **kw)
            assert np.allclose(host(lse), ref["lse"], rtol=1e-5, atol=1.2e-4)
            assert np.allclose(host(out), ref["out"], rtol=2.0 ** -8, atol=3e-4 * np.abs(ref["mag"]).max())
            mass = kv8_scores.new_mass(w.cache)
            kv8_scores.kv8_weigh(w.cache, w.batch, dev(q, dtype), lse, mass, slopes=dev(slopes), **kw)
            want, _ = plain.weigh(w.ref, q, host(lse), np.zeros(mass.shape, np.float32), 0.125, slopes=slopes, **kw)
            assert np.allclose(host(mass), want, rtol=1.5e-4, atol=1e-6)


def test_rows_that_add_nothing_whatever_their_slope():
    w = World(5, 2, 64, 16, [200], [3])
    q, lse = w.values(3, F32, heads=4), np.full((3, 4), 3.0, np.float32)
    lse[:, 1] = [np.nan, -np.inf, np.inf]
    for steep in (3e38, -3e38):
        slopes, mass = np.array([0.5, steep, 0.25, 0.125], np.float32), kv8_scores.new_mass(w.cache)
        kv8_scores.kv8_weigh(w.cache, w.batch, dev(q), dev(lse), mass, slopes=dev(slopes))
        with np.errstate(invalid="ignore"):
            want, _ = plain.weigh(w.ref, q, lse, np.zeros(mass.shape, np.float32), 0.125, slopes=slopes)
        assert np.allclose(host(mass), want, rtol=1.5e-4, atol=1e-6)


@pytest.mark.parametrize("dtype,size,scale,ks", [
    (F32, 1e20, 1e36, 0.02),      # the row's factor past F32's range
    (F32, 1.0, 1e36, 1e5),        # its product with a key's scale
    (F32, 1e38, 2.0 ** 126, 1e35),
    (F16, 6e4, 1e36, 1e5),
    (BF16, 1e30, -1e36, 0.02),
    (BF16, 1.0, 1e36, 1e5),
])
@pytest.mark.parametrize("lens,news", [([70, 33], [1, 1]), ([200, 150], [200, 90])])
def test_a_key_of_zeros_under_scores_past_the_range(lens, news, dtype, size, scale, ks):
    """Scores of any size are capped, one of 0 stays 0: every third key is zeros, and one page has the scale 0.  Scores
    are 0 or the cap, so exponents are off by 10 u of it and by 8 u (2 * 5 + 25), 2e-5, and a sum of 200 adds 1.2e-5."""
    D, cap = 64, 5.0
    w = World(4, 2, D, 16, lens, news)
    w.ref.k[:, :, ::3] = 0
    w.ref.ks[:] = np.float32(ks)
    w.ref.ks[w.ref.table[0, 1]] = 0.0
    w.cache.k.copy_(dev(w.ref.k))
    w.cache.k_scale.copy_(dev(w.ref.ks))
    # One component a query, so that a dot is no difference of large terms.
    q = np.zeros((w.rows, 4, D), np.float32)
    q[:, :, 7] = np.where(w.rng.random((w.rows, 4)) < 0.5, -1, 1) * size
    q = rounded(q, dtype)
    say(f"past the range: size={size} scale={scale} ks={ks} lens={lens} {dtype}")
    ref = plain.attention(w.ref, q, scale, cap=cap)
    out, lse = kv8_scores.kv8_attention_scored(w.cache, w.batch, dev(q, dtype), scale=scale, cap=cap, lse=True)
    assert np.allclose(host(lse), ref["lse"], rtol=1e-5, atol=3.2e-5)
    assert np.allclose(host(out), ref["out"], rtol=2.0 ** -8, atol=1e-4 * np.abs(ref["mag"]).max())
    mass = kv8_scores.new_mass(w.cache)
    kv8_scores.kv8_weigh(w.cache, w.batch, dev(q, dtype), lse, mass, scale=scale, cap=cap)
    want, _ = plain.weigh(w.ref, q, host(lse), np.zeros(mass.shape, np.float32), scale, cap=cap)
    assert np.allclose(host(mass), want, rtol=5e-5, atol=1e-7)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_prompt_of_which_only_the_last_rows_are_weighed(dtype):
    """Its pages are taken anew and hold another sequence's masses: they are added to where they are left, and count for nothing where
    they are zeroed as the header asks, up to the choice."""
    w = World(6, 2, 64, 16, [250, 37], [32, 32])
    q = w.values(w.rows, dtype, heads=8)
    _, lse = kv8.kv8_attention(w.cache, w.batch, dev(q, dtype), lse=True)
    old = (1000 * w.rng.exponential(size=(w.ref.pages, 2, 16))).astype(np.float32)
    begun = [int(p) for b, n in enumerate(w.ref.lens) for p in w.ref.table[b, :-(-int(n) // 16)]]
    for zeroed in (False, True):
        if zeroed:
            old[begun] = 0.0
        mass = dev(old)
        kv8_scores.kv8_weigh(w.cache, w.batch, dev(q, dtype), lse, mass)
        bound = noise(64, dtype)
        want, off = plain.weigh(w.ref, q, host(lse), old, 0.125, noise=lambda parts, spread, s: bound(parts, spread) + 8 * U * parts
                                + 4 * U * np.abs(s) + 8 * U)
        assert (np.abs(host(mass) - want) <= off + 1e-37).all()
        got = kv8_scores.kv8_choose(w.cache, w.batch, mass, 60, first=2, recent=8)
        assert all(np.array_equal(host(a), b) for a, b in zip(got, plain.choose(w.ref, host(mass), 60, 2, 8)))


def guarded(size):
    """(workspace of `size` bytes that are NaN, all of what it lies in)."""
    whole = torch.full((256 + size + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    assert whole.data_ptr() % 256 == 0
    return whole[256:256 + size], whole


@pytest.mark.parametrize("lens,news,bound", [([4096], [4096], 4096), ([900, 1300, 64, 0], [300, 250, 64, 0], 1300), ([3000], [700], 500)])
def test_workspaces_of_the_size_asked_for(lens, news, bound):
    """Nothing is written beside them, nothing is read of them that the call has not written, and one byte less is refused."""
    w = World(8, 2, 128, 64, lens, news)
    w.batch = kv8.KV8Batch(w.batch.table, w.batch.lens, w.batch.starts, max_len=bound)
    q = dev(w.values(w.rows, F32, heads=12))
    _, lse = kv8.kv8_attention(w.cache, w.batch, q, lse=True)
    size = kv8_scores.kv8_weigh_workspace_bytes(w.cache, w.batch, 12, w.rows)
    say(f"workspace lens={lens} bytes={size}")
    assert size > 0
    workspace, whole = guarded(size)
    masses = [kv8_scores.new_mass(w.cache) for _ in range(3)]
    kv8_scores.kv8_weigh(w.cache, w.batch, q, lse, masses[0], workspace=workspace)
    kv8_scores.kv8_weigh(w.cache, w.batch, q, lse, masses[1])
    assert torch.equal(masses[0], masses[1]) and host(masses[0]).sum() > 0
    edge = host(whole)
    assert (edge[:256] == 0xFF).all() and (edge[-256:] == 0xFF).all()
    with pytest.raises(I2SError) as refused:
        kv8_scores.kv8_weigh(w.cache, w.batch, q, lse, masses[2], workspace=workspace[:-1])
    assert refused.value.status == i2s.I2S_EWORKSPACE and not host(masses[2]).any()


@pytest.mark.parametrize("lens,news", [([5000], [1]), ([3000, 20], [40, 2])])
def test_scored_attention_in_a_workspace_of_the_size_asked_for(lens, news):
    w = World(9, 2, 128, 64, lens, news)
    q = dev(w.values(w.rows, F32, heads=12))
    size = kv8.kv8_attention_workspace_bytes(w.cache, w.batch, 12, w.rows)
    assert size > 0
    workspace, whole = guarded(size)
    want = kv8_scores.kv8_attention_scored(w.cache, w.batch, q, cap=9.0, lse=True)
    got = kv8_scores.kv8_attention_scored(w.cache, w.batch, q, cap=9.0, lse=True, workspace=workspace)
    edge = host(whole)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (edge[:256] == 0xFF).all() and (edge[-256:] == 0xFF).all()


def test_a_cap_that_rounds_to_none_is_refused():
    w = World(10, 1, 64, 16, [20], [1])
    q, lse, mass = dev(w.values(1, F32, heads=2)), torch.zeros((1, 2), device=DEV), kv8_scores.new_mass(w.cache)
    with pytest.raises(I2SError):
        kv8_scores.kv8_attention_scored(w.cache, w.batch, q, cap=1e-50)
    with pytest.raises(I2SError):
        kv8_scores.kv8_weigh(w.cache, w.batch, q, lse, mass, cap=1e-50)
    assert not host(mass).any()
