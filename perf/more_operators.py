"""What is measured of the operators that score, weigh and thin out the int8 K/V cache (the kv8_scores family):

  attend   kv8_attention_scored: attention with capped scores, a bias by distance, a prefix that all rows see
  weigh    kv8_weigh: the attention weight that each cached token gets, added to its mass
  choose   kv8_choose: the tokens of each sequence and head that stay, by mass
  move     kv8_move, then kv8_read: the chosen tokens in fresh pages

Each case is a dict of plain values.  With ``own`` false ``run`` computes the operator in elementary
torch operations; with ``own`` true it makes the framework's calls.  The cache is paged: pages of
``page`` tokens, K codes [pages][Hk][page][D], V codes [pages][Hk][D][page], one F32 scale per page and
head for each, and F32 masses [pages][Hk][page]; ``table`` holds each sequence's pages in order.
"""

from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
FLOOR = 1e-5  # of a block's largest magnitude, before it is divided by 127


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # One sequence, one token, capped scores, decoder geometry: latency.
        scored("attend", "attend one, capped", "f32", 12, 2, 128, 64, 1, lo=1500, hi=1500, new=1, cap=30.0),
        # A serving batch at one token each whose scores fall with the distance.
        scored("attend", "attend 48 by distance", "bf16", 32, 8, 128, 64, 48, lo=400, hi=6000, new=1, slopes=True),
        # Prompts that begin with frames which all rows see (audio, a document), in the framework's activation type.
        scored("attend", "attend behind a prefix", "f32", 12, 2, 128, 64, 5, lo=200, hi=2600, prefix=0.4),
        # Prompts with capped scores and a sliding window.
        scored("attend", "attend capped prompts", "bf16", 16, 8, 128, 32, 4, lo=500, hi=4000, cap=50.0, window=1024),
        # One sequence, one token: what a decode step adds to the masses.
        scored("weigh", "weigh one", "f32", 12, 2, 128, 64, 1, lo=3000, hi=3000, new=1),
        # A serving batch at one token each, lengths ragged.
        scored("weigh", "weigh a batch of 64", "bf16", 32, 8, 128, 64, 64, lo=500, hi=8000, new=1),
        # A whole prompt's weights, in the framework's activation type.
        scored("weigh", "weigh a prompt of 4096", "f32", 12, 2, 128, 64, 1, lo=4096, hi=4096),
        # The last 32 rows of prompts decide what stays; an odd group, small pages, capped scores.
        scored("weigh", "weigh the last 32 rows", "f16", 28, 4, 128, 16, 10, lo=900, hi=5000, new=32, cap=50.0),
        # The decoder's full context, one sequence: a long axis and few rows of it.
        choice("choose of one", 2, 64, 1, lo=65536, hi=65536, keep=8192, first=4, recent=512),
        # A batch of sequences that have outgrown their budget, two lengths of it apart.
        choice("choose of 48", 8, 64, 48, lo=1000, hi=9000, keep=2048, first=4, recent=256),
        # One sequence's chosen tokens in the decoder's geometry, handed back in F32.
        moved("move one", "f32", 2, 128, 64, 1, lo=6000, hi=6000, keep=1024),
        # A batch's chosen tokens.
        moved("move 40", "bf16", 8, 128, 64, 40, lo=1500, hi=8000, keep=2048),
    ]


def named(name, case):
    return case if name is None else {"name": name, **case}


def scored(op, name, kind, hq, hk, d, page, seqs, *, lo, hi, new=0, cap=0.0, slopes=False, prefix=0.0, window=0, causal=True, gap=0):
    """Sequences of lo..hi cached tokens; the newest `new` of each (all, if 0) are the call's rows.  prefix: share of a sequence
    that all of its rows see; gap: blocks behind the first whose pages were handed on."""
    return named(name, {"op": op, "type": kind, "hq": hq, "hk": hk, "d": d, "page": page, "seqs": seqs, "lo": lo, "hi": hi, "new": new,
                        "cap": cap, "slopes": slopes, "prefix": prefix, "window": window, "causal": causal, "gap": gap})


def choice(name, hk, page, seqs, *, lo, hi, keep, first, recent, gap=0):
    return named(name, {"op": "choose", "hk": hk, "page": page, "seqs": seqs, "lo": lo, "hi": hi, "keep": keep, "first": first,
                        "recent": recent, "gap": gap})


def moved(name, kind, hk, d, page, seqs, *, lo, hi, keep):
    return named(name, {"op": "move", "type": kind, "hk": hk, "d": d, "page": page, "seqs": seqs, "lo": lo, "hi": hi, "keep": keep})


def log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weigh", "weigh", "choose", "move"])
    kind = rng.choice(["f32", "bf16", "f16"])
    d = rng.choice([64, 96, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "choose":
        seqs = log_between(rng, 1, 48)
        hi = log_between(rng, 20, min(65536, max(21, 48 * 5000 * 8 // (seqs * hk))))
        keep = log_between(rng, 4, hi + 10)
        first = rng.randint(0, keep // 2)
        return choice(None, hk, page, seqs, lo=rng.randint(1, hi), hi=hi, keep=keep, first=first, recent=rng.randint(0, keep - first),
                      gap=rng.choice([0, 0, 3]))
    if op == "move":
        seqs = log_between(rng, 1, 40)
        hi = log_between(rng, 20, min(16000, max(21, 40 * 4750 * 8 * 128 // (seqs * hk * d))))
        keep = log_between(rng, 4, min(hi, max(5, 40 * 2048 * 8 * 128 // (seqs * hk * d))))
        return moved(None, kind, hk, d, page, seqs, lo=rng.randint(1, hi), hi=hi, keep=keep)
    hq = hk * rng.choice([1, 2, 4, 6, 7, 8, 16])
    shape = {"cap": rng.choice([0.0, 20.0, 50.0]), "slopes": rng.random() < 0.4, "prefix": rng.choice([0.0, 0.0, 0.3, 0.8]),
             "causal": rng.random() < 0.85}
    if op == "attend" and not shape["cap"] and not shape["slopes"] and not shape["prefix"]:
        shape["cap"] = 30.0
    way = rng.choice(["one", "few", "prompt", "chunk"])
    most_read = 48 * 3200 * 8 * 128  # token places a call streams: the listed batches at one token
    most_work = 12 * 128 * 4096 * 4096 // 2  # pairs times width of the listed prompt of 4096
    if way in ("one", "few"):
        seqs = log_between(rng, 1, 64)
        hi = log_between(rng, 1, max(2, min(65536, most_read // (seqs * hk * d))))
        new = 1 if way == "one" else rng.randint(2, 12)
        return scored(op, None, kind, hq, hk, d, page, seqs, lo=rng.randint(max(1, hi // 8), hi), hi=hi, new=new,
                      window=rng.choice([0, 0, 0, 500, 4096]), gap=rng.choice([0, 0, 0, 2]), **shape)
    seqs = rng.randint(1, 6)
    shared = 2 if shape["prefix"] < 0.5 and shape["causal"] else 1  # about half of the pairs are seen then
    hi = log_between(rng, 16, max(17, min(4096, int(math.sqrt(shared * most_work / (seqs * hq * d))))))
    new = 0 if way == "prompt" else rng.randint(1, max(1, hi // 2))
    return scored(op, None, kind, hq, hk, d, page, seqs, lo=rng.randint(max(1, hi // 10), hi), hi=hi, new=new,
                  window=rng.choice([0, 0, 100, 1000]), gap=0, **shape)


def lengths(case):
    """Tokens in the cache of each sequence, scattered evenly over lo..hi, the first hi: of the case, not of the seed."""
    return [case["hi"] - int((case["hi"] - case["lo"]) * (i * 0.6180339887 % 1.0) + 0.5) for i in range(case["seqs"])]


def rows_of(case, lens):
    return [min(case["new"], n) if case["new"] else n for n in lens]


def prefixes(case, lens):
    return [int(case["prefix"] * n) for n in lens]


def absent(case, have):
    """Tokens [first, last) of a sequence whose pages were handed on: whole blocks, never the newest one."""
    first = case["page"]
    last = min(first + case.get("gap", 0) * case["page"], (have - 1) // case["page"] * case["page"])
    return first, max(first, last)


def reach(case, have, rows, prefix):
    """(query, token) pairs of one head, and the tokens that any of the rows reads."""
    pairs, lowest, highest = 0, have, 0
    for p in range(have - rows, have):
        end = max(p + 1, prefix) if case["causal"] else have
        begin = max(0, p - case["window"] + 1) if case["window"] else 0
        pairs += max(0, end - begin)
        if end > begin:
            lowest, highest = min(lowest, begin), max(highest, end)
    return pairs, max(0, highest - lowest)


def work(case):
    lens, hk = lengths(case), case["hk"]
    if case["op"] == "choose":
        n = sum(lens) * hk
        kept = sum(min(case["keep"], a) for a in lens) * hk
        return {"bytes": 4 * n + 4 * kept, "flops": n}
    d, size = case["d"], SIZE[case["type"]]
    if case["op"] == "move":
        kept = sum(min(case["keep"], a) for a in lens) * hk
        n = 2 * kept * d
        return {"bytes": 2 * n + 12 * kept + n * (1 + size), "flops": 4 * n}
    hq, news = case["hq"], rows_of(case, lens)
    pairs, tokens = (sum(x) for x in zip(*(reach(case, a, b, c) for a, b, c in zip(lens, news, prefixes(case, lens)))))
    queries = sum(news) * hq
    if case["op"] == "weigh":
        return {"bytes": tokens * hk * (d + 8) + queries * (d * size + 4), "flops": 2 * pairs * hq * d}
    return {"bytes": 2 * tokens * hk * d + 8 * hk * tokens // case["page"] + 2 * queries * d * size, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------
# What a program has in hand

def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def prepare(case, seed):
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 6011 + 29)
    hk, page, seqs, lens = case["hk"], case["page"], case["seqs"], lengths(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def pages_for(counts, order, at, gaps):
        table = torch.full((seqs, max(1, max(-(-n // page) for n in counts))), -1, dtype=torch.int32)
        for b, n in enumerate(counts):
            blocks = -(-n // page)
            table[b, :blocks] = order[at:at + blocks]
            at += blocks
            if gaps:
                lo, hi = absent(case, n)
                table[b, lo // page:hi // page] = -1
        return table.to(dev), at

    stay = [min(case["keep"], n) for n in lens] if case["op"] == "move" else [0] * seqs
    pages = sum(-(-n // page) for n in lens) + sum(-(-n // page) for n in stay) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table, at = pages_for(lens, order, 0, True)
    s = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "longest": max(lens), "pages": pages}
    # Masses as sums of softmax weights leave them: some tokens have most, many next to nothing, some nothing at all.
    mass = torch.exp(2.0 * normal(pages, hk, page) - 4.0)
    s["mass"] = torch.where(torch.rand(pages, hk, page, generator=g, device=dev) < 0.15, 0.0, mass)
    if case["op"] == "choose":
        # Codes are not looked at: the cache's tensors are there, as in a program, and small.
        s["k"] = torch.zeros(pages, hk, page, 16, dtype=torch.int8, device=dev)
        s["v"] = torch.zeros(pages, hk, 16, page, dtype=torch.int8, device=dev)
        s["ks"] = s["vs"] = torch.ones(pages, hk, device=dev)
        return s
    d, kind = case["d"], TYPES[case["type"]]
    # Keys carry a few wide channels, as the biases of key projections leave them; values are plain.
    wide = torch.ones(hk, 1, d, device=dev)
    wide[:, :, torch.randperm(d, generator=g, device=dev)[:max(1, d // 32)]] = 5.0
    s["k"] = (normal(pages, hk, page, d) * (18.0 * wide)).round_().clamp_(-127, 127).to(torch.int8)
    s["v"] = (normal(pages, hk, d, page) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
    s["ks"] = torch.exp(0.15 * normal(pages, hk)) / 22.0
    s["vs"] = torch.exp(0.25 * normal(pages, hk)) / 32.0
    if case["op"] == "move":
        s["to"], _ = pages_for(stay, order, at, False)
        # A choice for each sequence and head: the first 4 tokens, then any, ascending.
        worth = torch.rand(seqs, hk, max(lens), generator=g, device=dev)
        worth[:, :, :4] = 2.0
        worth.masked_fill_(torch.arange(max(lens), device=dev) >= s["lens"][:, None, None], -1.0)
        s["kept"] = torch.tensor(stay, dtype=torch.int32, device=dev)
        best = worth.topk(min(case["keep"], max(lens)), dim=-1).indices
        live = torch.arange(best.shape[-1], device=dev) < s["kept"][:, None, None]
        best = torch.where(live, best, max(lens)).sort(dim=-1).values
        index = torch.full((seqs, hk, case["keep"]), -1, dtype=torch.int32, device=dev)
        index[:, :, :best.shape[-1]] = torch.where(live, best, -1).to(torch.int32)
        s["index"] = index
        s["rows"] = sum(stay)
        starts = [0]
        for n in stay:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        s["row_seq"] = torch.cat([torch.full((n,), b) for b, n in enumerate(stay)]).to(dev)
        s["row_tok"] = torch.cat([torch.arange(n) for n in stay]).to(dev)
        return s
    hq, news = case["hq"], rows_of(case, lens)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s["rows"], s["most"] = starts[-1], max(news)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["q"] = normal(starts[-1], hq, d).to(kind)
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=dev) / hq) if case["slopes"] else None
    s["prefix"] = torch.tensor(prefixes(case, lens), dtype=torch.int32, device=dev) if case["prefix"] else None
    if case["op"] == "weigh":  # the attention has left its log-sums, and the masses of the call's own tokens are anything
        s["tok_seq"] = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(dev)
        s["tok"] = torch.cat([torch.arange(n) for n in lens]).to(dev)
        e, src, live = scores(s)
        lse = torch.logsumexp(e, -1).permute(0, 3, 1, 2).reshape(seqs, s["most"], hq)
        s["lse"] = torch.zeros(s["rows"], hq, device=dev)
        s["lse"][src[live]] = lse[live]
    return s


# ---------------------------------------------------------------------------
# One pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attend": own_attend, "weigh": own_weigh, "choose": own_choose, "move": own_move}[op](s)
    return {"attend": plain_attend, "weigh": plain_weigh, "choose": plain_choose, "move": plain_move}[op](s)


def handles(s):
    """The cache's and the batch's handles: a program makes them where it makes the tensors that they name."""
    if "handles" not in s:
        from ternary_weight_integer_amd import kv8, kv8_scores
        cache = kv8.KV8Cache(s["k"], s["v"], s["ks"], s["vs"])
        batch = kv8.KV8Batch(s["table"], s["lens"], s.get("starts") if s["case"]["op"] != "move" else None, max_len=s["longest"])
        back = kv8.KV8Batch(s["to"], s["kept"], s["starts"], max_len=s["case"]["keep"]) if "to" in s else None
        s["handles"] = kv8, kv8_scores, cache, batch, back
    return s["handles"]


def own_attend(s):
    _, kv8_scores, cache, batch, _ = handles(s)
    c = s["case"]
    return kv8_scores.kv8_attention_scored(cache, batch, s["q"], causal=c["causal"], window=c["window"], cap=c["cap"],
                                           slopes=s["slopes"], prefix=s["prefix"])


def own_weigh(s):
    _, kv8_scores, cache, batch, _ = handles(s)
    c = s["case"]
    kv8_scores.kv8_weigh(cache, batch, s["q"], s["lse"], s["mass"], causal=c["causal"], window=c["window"], cap=c["cap"],
                         slopes=s["slopes"], prefix=s["prefix"])
    return s["mass"]


def own_choose(s):
    _, kv8_scores, cache, batch, _ = handles(s)
    c = s["case"]
    return kv8_scores.kv8_choose(cache, batch, s["mass"], c["keep"], first=c["first"], recent=c["recent"])


def own_move(s):
    kv8, kv8_scores, cache, batch, back = handles(s)
    kv8_scores.kv8_move(cache, batch, s["index"], s["kept"], s["to"], mass=s["mass"])
    k, v = kv8.kv8_read(cache, back, s["rows"], dtype=TYPES[s["case"]["type"]])
    return k, v, s["mass"]


def scores(s):
    """The scores e [seqs][Hk][group][rows][tokens] in F32, -inf where a row does not see a token; each place's row of the call,
    and which places there are."""
    c = s["case"]
    hq, hk, d, page, q = c["hq"], c["hk"], c["d"], c["page"], s["q"]
    group, dev, rows = hq // hk, q.device, s["most"]
    starts, lens, table = s["starts"].long(), s["lens"].long(), s["table"].long()
    seqs, blocks = table.shape
    at = table.clamp(min=0)
    row = torch.arange(rows, device=dev)
    new = starts[1:] - starts[:-1]
    live = row[None, :] < new[:, None]  # [B][rows]
    src = (starts[:-1, None] + row[None, :]).clamp(max=max(0, q.shape[0] - 1))
    x = q.float()[src].view(seqs, rows, hk, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, hk, group * rows, d)
    k = (s["k"][at].float() * s["ks"][at][..., None, None]).permute(0, 2, 1, 3, 4).reshape(seqs, hk, blocks * page, d)
    e = torch.matmul(x, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(seqs, hk, group, rows, blocks * page)
    if c["cap"]:
        e = e.div_(c["cap"]).tanh_().mul_(c["cap"])
    tok = torch.arange(blocks * page, device=dev)
    place = lens[:, None] - new[:, None] + row[None, :]  # [B][rows]
    if s["slopes"] is not None:
        away = (place[:, :, None] - tok[None, None, :]).abs().float()
        e = e.sub_(s["slopes"].view(1, hk, group, 1, 1) * away[:, None, None])
    seen = (tok[None, None, :] < lens[:, None, None]) & live[:, :, None]
    seen &= (table >= 0).repeat_interleave(page, 1)[:, None, :]
    if c["causal"]:
        early = tok[None, None, :] <= place[:, :, None]
        if s["prefix"] is not None:
            early |= tok[None, None, :] < s["prefix"].long()[:, None, None]
        seen &= early
    if c["window"]:
        seen &= tok[None, None, :] > place[:, :, None] - c["window"]
    return e.masked_fill_(~seen[:, None, None], -math.inf), src, live


def plain_attend(s):
    c, q = s["case"], s["q"]
    e, src, live = scores(s)
    at = s["table"].long().clamp(min=0)
    seqs, hk, group, rows, tokens = e.shape
    v = (s["v"][at].float() * s["vs"][at][..., None, None]).permute(0, 2, 1, 4, 3).reshape(seqs, hk, tokens, c["d"])
    top = e.amax(-1, keepdim=True)
    p = torch.exp(e.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hk, group * rows, tokens), v).view(seqs, hk, group, rows, c["d"])
    o = o / torch.where(total == 0, 1.0, total)
    out = torch.zeros(q.shape, dtype=torch.float32, device=q.device)
    out[src[live]] = o.permute(0, 3, 1, 2, 4).reshape(seqs, rows, c["hq"], c["d"])[live]
    return out.to(q.dtype)


def plain_weigh(s):
    c = s["case"]
    e, src, live = scores(s)
    seqs, hk, group, rows, tokens = e.shape
    lse = s["lse"][src].view(seqs, rows, hk, group).permute(0, 2, 3, 1)[..., None]
    some = torch.isfinite(lse) & live[:, None, None, :, None]
    w = torch.exp(e.sub_(torch.where(some, lse, math.inf))).view(seqs, hk, group * rows, tokens).sum(2)  # [B][Hk][tokens]
    b, t = s["tok_seq"], s["tok"]
    page = s["table"].long()[b, t // c["page"]]
    b, t, page = b[page >= 0], t[page >= 0], page[page >= 0]
    fresh = t >= (s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long())[b]
    before = torch.where(fresh[:, None], 0.0, s["mass"][page, :, t % c["page"]])
    s["mass"][page, :, t % c["page"]] = before + w[b, :, t]
    return s["mass"]


def plain_choose(s):
    c = s["case"]
    page, keep, lens, table = c["page"], c["keep"], s["lens"].long(), s["table"].long()
    seqs, blocks = table.shape
    m = s["mass"][table.clamp(min=0)].permute(0, 2, 1, 3).reshape(seqs, c["hk"], blocks * page)
    t = torch.arange(blocks * page, device=m.device)
    there = (t < lens[:, None]) & (table >= 0).repeat_interleave(page, 1)  # [B][tokens]
    forced = (t < c["first"]) | (t >= lens[:, None] - c["recent"])
    m = torch.where(forced[:, None], math.inf, m)
    m = torch.where(there[:, None], m, -math.inf)
    kept = there.sum(-1).clamp(max=keep)
    best = m.sort(dim=-1, descending=True, stable=True).indices[:, :, :keep]  # stable: ties go to the lowest index
    live = torch.arange(best.shape[-1], device=m.device) < kept[:, None, None]
    best = torch.where(live, best, blocks * page).sort(dim=-1).values
    index = torch.full((seqs, c["hk"], keep), -1, dtype=torch.int32, device=m.device)
    index[:, :, :best.shape[-1]] = torch.where(live, best, -1).to(torch.int32)
    return index, kept.to(torch.int32)


def half_away(x):
    """Rounded half away from zero, in 64 bits (where adding a half is exact)."""
    x = x.double()
    return torch.sign(x) * torch.floor(x.abs() + 0.5)


def plain_move(s):
    c = s["case"]
    page, keep, hk, d = c["page"], c["keep"], c["hk"], c["d"]
    to, table, kept = s["to"].long(), s["table"].long(), s["kept"].long()
    seqs, blocks = to.shape
    dev = to.device
    index = torch.full((seqs, hk, blocks * page), -1, dtype=torch.int64, device=dev)
    n = min(keep, blocks * page)
    index[:, :, :n] = s["index"][:, :, :n]
    live = torch.arange(blocks * page, device=dev) < kept[:, None, None]
    index = torch.where(live, index, 0)
    b = torch.arange(seqs, device=dev)[:, None, None]
    h = torch.arange(hk, device=dev)[None, :, None]
    at, slot = table[b, index // page], index % page  # [B][Hk][places]
    used = (torch.arange(blocks, device=dev)[None, :] * page < kept[:, None]).nonzero()
    ub, uj = used[:, 0], used[:, 1]
    dest = to[ub, uj]
    there = live.expand(seqs, hk, -1).reshape(seqs, hk, blocks, page)[ub, :, uj]  # [used][Hk][page]
    for codes, scale, turn in ((s["k"], s["ks"], False), (s["v"], s["vs"], True)):
        x = (codes[at, h, :, slot] if turn else codes[at, h, slot]).float() * scale[at, h][..., None]  # [B][Hk][places][D]
        x = x.view(seqs, hk, blocks, page, d)[ub, :, uj]
        x = torch.where(there[..., None], x, 0.0)
        top = x.abs().amax((-1, -2)).clamp(min=FLOOR)
        now = (top.double() / 127.0).float()  # two F32 values divided in 64 bits round as in 32
        q = half_away((x.double() / now.double()[:, :, None, None]).float()).clamp(-127, 127).to(torch.int8)
        old = codes[dest].transpose(-1, -2) if turn else codes[dest]
        q = torch.where(there[..., None], q, old)
        codes[dest] = q.transpose(-1, -2) if turn else q
        scale[dest] = now
    m = s["mass"][at, h, slot].view(seqs, hk, blocks, page)[ub, :, uj]
    s["mass"][dest] = torch.where(there, m, s["mass"][dest])
    rb, rt = s["row_seq"], s["row_tok"]
    at, slot = to[rb, rt // page], rt % page
    k = s["k"][at, :, slot, :].float() * s["ks"][at][:, :, None]
    v = s["v"][at, :, :, slot].float() * s["vs"][at][:, :, None]
    return k.to(TYPES[c["type"]]), v.to(TYPES[c["type"]]), s["mass"]


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": exact_attend, "weigh": exact_weigh, "choose": exact_choose, "move": exact_move}[case["op"]](case, s)


def walk(c, s):
    """Sequence by sequence and head by head, with torch in 64 bits on the device that holds the inputs: (rows' places, head, tokens,
    scores [rows][group][tokens], mask of what a row does not see)."""
    group, dev = c["hq"] // c["hk"], s["q"].device
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    prefix = s["prefix"].tolist() if s["prefix"] is not None else [0] * len(lens)
    for b, have in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        at = s["table"][b, :-(-have // c["page"])].long()
        gone = (at < 0).repeat_interleave(c["page"])[:have]
        at = torch.where(at < 0, 0, at)
        t = torch.arange(have, device=dev, dtype=torch.float64)
        for h in range(c["hk"]):
            k = (s["k"][at, h].double() * s["ks"][at, h].double()[:, None, None]).reshape(-1, c["d"])[:have]
            for r0 in range(lo, hi, 1024):
                r1 = min(hi, r0 + 1024)
                x = s["q"][r0:r1, h * group:(h + 1) * group].double()
                e = (x.reshape(-1, c["d"]) @ k.t()).view(r1 - r0, group, have) / math.sqrt(c["d"])
                p = have - (hi - lo) + torch.arange(r0 - lo, r1 - lo, device=dev, dtype=torch.float64)[:, None]
                if c["cap"]:
                    e = c["cap"] * (1.0 - 2.0 / (torch.exp(2.0 * e / c["cap"]) + 1.0))
                if s["slopes"] is not None:
                    e = e - s["slopes"][h * group:(h + 1) * group].double()[None, :, None] * (p - t)[:, None, :].abs()
                hidden = gone[None, :].expand(r1 - r0, -1).clone()
                if c["causal"]:
                    hidden |= (t > p) & (t >= prefix[b])
                if c["window"]:
                    hidden |= t <= p - c["window"]
                yield b, h, at, r0, r1, e, hidden


def exact_attend(c, s):
    group, d = c["hq"] // c["hk"], c["d"]
    out = torch.zeros(s["rows"], c["hq"], d, dtype=torch.float64, device=s["q"].device)
    for b, h, at, r0, r1, e, hidden in walk(c, s):
        have = e.shape[-1]
        v = (s["v"][at, h].double() * s["vs"][at, h].double()[:, None, None]).transpose(-1, -2).reshape(-1, d)[:have]
        e = e.masked_fill(hidden[:, None, :], -math.inf)
        top = e.amax(-1, keepdim=True)
        p = torch.where(torch.isneginf(top), 0.0, torch.exp(e - top))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total == 0, torch.ones_like(total), total)
        out[r0:r1, h * group:(h + 1) * group] = (p.reshape(-1, have) @ v).view(r1 - r0, group, d)
    return out


def exact_weigh(c, s):
    group, page = c["hq"] // c["hk"], c["page"]
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = s["mass"].double()
    sums = [torch.zeros(c["hk"], n, dtype=torch.float64, device=out.device) for n in lens]
    for b, h, at, r0, r1, e, hidden in walk(c, s):
        lse = s["lse"][r0:r1, h * group:(h + 1) * group].double()[:, :, None]
        w = torch.exp(e - lse)
        w = torch.where(hidden[:, None, :] | torch.isinf(lse), 0.0, w)
        sums[b][h] += w.sum((0, 1))
    for b, have in enumerate(lens):
        own_from = have - (starts[b + 1] - starts[b])
        for j in range(-(-have // page)):
            p, t0, t1 = int(s["table"][b, j]), j * page, min(have, (j + 1) * page)
            if p < 0:
                continue
            part = sums[b][:, t0:t1]
            cut = min(max(own_from - t0, 0), t1 - t0)  # earlier tokens of the block
            out[p, :, :cut] += part[:, :cut]
            out[p, :, cut:t1 - t0] = part[:, cut:]
    return out


def exact_choose(c, s):
    import numpy as np
    mass, table, page = s["mass"].cpu().numpy(), s["table"].cpu().numpy(), c["page"]
    lens = s["lens"].tolist()
    index = np.full((c["seqs"], c["hk"], c["keep"]), -1, np.int32)
    kept = np.zeros(c["seqs"], np.int32)
    for b, have in enumerate(lens):
        t = np.arange(have)
        t = t[table[b, t // page] >= 0]
        kept[b] = min(c["keep"], len(t))
        always = (t < c["first"]) | (t >= have - c["recent"])
        for h in range(c["hk"]):
            order = np.lexsort((t, -mass[table[b, t // page], h, t % page], ~always))
            index[b, h, :kept[b]] = np.sort(t[order[:kept[b]]])
    return index, kept


def exact_move(c, s):
    """The operator's own F32 steps (value, scale, quotient) are part of its definition: each is computed in 64 bits and rounded to 32."""
    import numpy as np
    page, table, to = c["page"], s["table"].cpu().numpy(), s["to"].cpu().numpy()
    index, kept = s["index"].cpu().numpy(), s["kept"].tolist()
    codes = [s["k"].cpu().numpy(), s["v"].cpu().numpy().swapaxes(-1, -2)]
    scale = [s["ks"].cpu().numpy(), s["vs"].cpu().numpy()]
    mass = s["mass"].cpu().numpy()
    out = [np.zeros((s["rows"], c["hk"], c["d"])) for _ in range(2)]
    new_mass = mass.astype(np.float64)
    row = 0
    for b, n in enumerate(kept):
        for j in range(-(-n // page)):
            t0, t1 = j * page, min(n, (j + 1) * page)
            for h in range(c["hk"]):
                src = index[b, h, t0:t1]
                p, slot = table[b, src // page], src % page
                for x, f, o in zip(codes, scale, out):
                    v = (x[p, h, slot].astype(np.float64) * f[p, h].astype(np.float64)[:, None]).astype(np.float32).astype(np.float64)
                    now = np.float64(np.float32(max(np.abs(v).max(), np.float64(np.float32(FLOOR))) / 127.0))
                    q = (v / now).astype(np.float32).astype(np.float64)
                    q = np.clip(np.copysign(np.floor(np.abs(q) + 0.5), q), -127, 127)
                    o[row + t0:row + t1, h] = q * now
                new_mass[to[b, j], h, :t1 - t0] = mass[p, h, slot]
        row += n
    return out[0], out[1], new_mass
