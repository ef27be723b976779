"""Scores, weights, choices and moves over an int8 K/V cache in plain numpy,
64 bits, written from the formulas: what the kv8_scores tests compare with.
`ref` is an oracle.KV8 (a cache and a batch on the host)."""

from __future__ import annotations

import numpy as np


def pages_of(ref, b, n):
    """(page, slot, in no hole) of tokens 0 .. n - 1 of sequence b; page 0 stands in for a hole's."""
    t = np.arange(n)
    j = t // ref.P
    page = np.where(j < ref.table.shape[1], ref.table[b, np.minimum(j, max(0, ref.table.shape[1] - 1))] if ref.table.shape[1] else -1, -1)
    there = (page >= 0) & (page < ref.pages)
    return np.where(there, page, 0), t % ref.P, there


def length(ref, b):
    return max(0, int(ref.lens[b]))


def walk(ref, q, scale, causal, window, cap, slopes, prefix):
    """For each sequence with rows and each K/V head: (b, h, rows' slice, heads' slice, e [rows][group][L] before -inf is put
    anywhere, seen [rows][L], |bias| and |score before the bias|, spread) in 64 bits."""
    heads = q.shape[1]
    group = heads // ref.heads
    q = np.asarray(q, np.float64)
    for b in range(len(ref.lens)):
        lo, hi = int(ref.starts[b]), int(ref.starts[b + 1])
        L = length(ref, b)
        if hi == lo:
            continue
        page, slot, there = pages_of(ref, b, L)
        t = np.arange(L)[None, :]
        pos = (L - (hi - lo) + np.arange(hi - lo))[:, None]
        seen = np.broadcast_to(there, (hi - lo, L)).copy()
        if causal:
            seen &= (t <= pos) | (t < (0 if prefix is None else int(prefix[b])))
        if window:
            seen &= t > pos - window
        for h in range(ref.heads):
            of = slice(h * group, (h + 1) * group)
            code = ref.k[page, h, slot].astype(np.float64)
            ks = np.where(there, ref.ks[page, h], 0).astype(np.float64)
            x = q[lo:hi, of]
            with np.errstate(invalid="ignore", over="ignore"):
                e = scale * (np.matmul(x, code.T) * ks)
                most = np.abs(x).max(-1, initial=0.0)
                spread = abs(scale) * most[..., None] * (np.abs(code).sum(-1) * ks)
                if cap:
                    e = cap * np.tanh(e / cap)
            first = np.abs(e)
            bias = np.zeros_like(e)
            if slopes is not None:
                bias = np.asarray(slopes, np.float64)[of][None, :, None] * np.abs(pos - t)[:, None, :]
                e = e - bias
            yield b, h, slice(lo, hi), of, e, seen, np.abs(bias) + first, spread


def attention(ref, q, scale, causal=True, window=0, cap=0.0, slopes=None, prefix=None):
    """dict of float64 arrays: out, mag [rows][q_heads][D], lse, top (max |e|), parts (max |bias| + |score|), spread [rows][q_heads];
    rows outside the batch's are NaN."""
    rows, heads, D = q.shape
    r = {n: np.full((rows, heads, D) if n in ("out", "mag") else (rows, heads), np.nan)
         for n in ("out", "mag", "lse", "top", "parts", "spread")}
    for b, h, at, of, e, seen, parts, spread in walk(ref, q, scale, causal, window, cap, slopes, prefix):
        page, slot, there = pages_of(ref, b, e.shape[-1])
        v = ref.v[page, h, :, slot].astype(np.float64) * np.where(there, ref.vs[page, h], 0).astype(np.float64)[:, None]
        mask = seen[:, None, :]
        e = np.where(mask, e, -np.inf)
        with np.errstate(invalid="ignore", divide="ignore"):
            top = e.max(-1, initial=-np.inf)
            p = np.where(mask, np.exp(e - np.where(np.isneginf(top), 0, top)[..., None]), 0.0)
            total = p.sum(-1)
            p = p / np.where(total == 0, 1, total)[..., None]
            r["lse"][at, of] = np.where(total == 0, -np.inf, np.where(np.isneginf(top), 0, top) + np.log(total))
            r["out"][at, of], r["mag"][at, of] = np.matmul(p, v), np.matmul(p, np.abs(v))
            r["top"][at, of] = np.where(mask, np.abs(e), 0).max(-1, initial=0)
            r["parts"][at, of] = np.where(mask, parts, 0).max(-1, initial=0)
            r["spread"][at, of] = np.where(mask, spread, 0).max(-1, initial=0)
    return r


def weigh(ref, q, lse, mass, scale, causal=True, window=0, cap=0.0, slopes=None, prefix=None, noise=None):
    """The masses afterwards, and a bound of what F32 kernels may add: noise(parts, spread, lse) is a weight's relative error."""
    out = np.asarray(mass, np.float64).copy()
    off = np.zeros_like(out)
    lse = np.asarray(lse, np.float64)
    for b, h, at, of, e, seen, parts, spread in walk(ref, q, scale, causal, window, cap, slopes, prefix):
        L = e.shape[-1]
        page, slot, there = pages_of(ref, b, L)
        s = lse[at, of][..., None]
        adds = seen[:, None, :] & np.isfinite(s)
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(adds, np.exp(e - s), 0.0)
            err = np.where(adds, p * noise(parts, spread, np.where(np.isfinite(s), s, 0)), 0.0) if noise else 0 * p
        w, err = p.sum((0, 1)), err.sum((0, 1))
        own = np.arange(L) >= L - (at.stop - at.start)
        err = err + p.shape[0] * p.shape[1] * 2.0 ** -24 * w
        for t in np.nonzero(there)[0]:
            i = page[t], h, slot[t]
            out[i] = w[t] if own[t] else out[i] + w[t]
            off[i] = err[t] + 2.0 ** -23 * abs(out[i]) + (off[i] if not own[t] else 0)
    return out, off


def choose(ref, mass, keep, first, recent):
    """(index int32 [seqs][heads][keep], kept int32 [seqs])."""
    seqs = len(ref.lens)
    index, kept = np.full((seqs, ref.heads, keep), -1, np.int32), np.zeros(seqs, np.int32)
    for b in range(seqs):
        L = length(ref, b)
        page, slot, there = pages_of(ref, b, L)
        t = np.nonzero(there)[0]
        kept[b] = min(keep, len(t))
        for h in range(ref.heads):
            m = np.asarray(mass, np.float64)[page[t], h, slot[t]]
            rank = np.where(np.isnan(m), -np.inf, np.maximum(m, -1e300))  # a NaN under every number, -inf among them
            always = (t < first) | (t >= L - recent)
            order = np.lexsort((t, -rank, ~always))
            index[b, h, :kept[b]] = np.sort(t[order[:kept[b]]])
    return index, kept


def half_away(x):
    return np.copysign(np.floor(np.abs(x) + 0.5), x)


def move(ref, index, kept, to, mass=None):
    """Moves in place in ref's arrays (and mass): each F32 step computed in 64 bits and rounded."""
    keep = index.shape[2]
    f32 = lambda x: np.asarray(x, np.float64).astype(np.float32).astype(np.float64)  # noqa: E731
    k0, v0, ks0, vs0 = ref.k.copy(), ref.v.copy(), ref.ks.copy(), ref.vs.copy()
    m0 = None if mass is None else mass.copy()
    for b in range(len(ref.lens)):
        n, L = min(max(0, int(kept[b])), keep), length(ref, b)
        page, slot, there = pages_of(ref, b, L)
        for j in range(min(to.shape[1], -(-n // ref.P))):
            dest = int(to[b, j])
            if not 0 <= dest < ref.pages:
                continue
            t0, t1 = j * ref.P, min(n, (j + 1) * ref.P)
            for h in range(ref.heads):
                t = index[b, h, t0:t1]
                ok = (t >= 0) & (t < L)
                ok &= there[np.where(ok, t, 0)] if L else False
                p, s = (page[np.where(ok, t, 0)], slot[np.where(ok, t, 0)]) if L else (0 * t, 0 * t)
                for x, scale, codes, out in ((k0[p, h, s], ks0, ref.k, ref.ks), (v0[p, h, :, s], vs0, ref.v, ref.vs)):
                    value = np.where(ok[:, None], f32(x.astype(np.float64) * scale[p, h].astype(np.float64)[:, None]), 0.0)
                    now = f32(max(np.abs(value).max(initial=0), np.float64(np.float32(1e-5))) / 127.0)
                    q = np.clip(half_away(f32(value / now)), -127, 127).astype(np.int8)
                    if codes is ref.k:
                        codes[dest, h, :t1 - t0] = q
                    else:
                        codes[dest, h, :, :t1 - t0] = q.T
                    out[dest, h] = now
                if mass is not None:
                    mass[dest, h, :t1 - t0] = np.where(ok, m0[p, h, s], 0)
