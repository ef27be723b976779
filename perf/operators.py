"""What is measured of the decoder's attention operators (the kv8 family):

  rotate   kv8_qk_norm_rope: RMS norms of queries and keys per head, with the position rotation
  write    kv8_append, then kv8_read of the pages written: new K/V rows into the int8 cache
  read     kv8_read: cached tokens back as values
  attend   kv8_attention: queries over the int8 cache, one token or many, causal, windowed

Each case is a dict of plain values.  With ``own`` false ``run`` computes the operator in elementary
torch operations; with ``own`` true it makes the framework's calls.  The cache is paged: pages of
``page`` tokens, K codes [pages][Hk][page][D], V codes [pages][Hk][D][page], one F32 scale per page and
head for each; ``table`` holds each sequence's pages in order.
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
        # One token's queries and keys in the decoder's own geometry: the call's latency.
        rotate("rotate one token", 1, 12, 2, 128, "f32", norm=False),
        # A long prompt, normed, read out of the rows of a fused projection.
        rotate("rotate a long prompt", 8192, 32, 8, 128, "bf16", norm=True, fused=True),
        # A decode step of a batch: one token per sequence into pages partly filled.
        paged("write", "write one token of 48", "bf16", 8, 8, 128, 64, 48, lo=90, hi=2300, new_lo=1, new_hi=1),
        # Prompts of several lengths, some behind a cached prefix, in the decoder's geometry.
        paged("write", "write ragged prompts", "f32", 2, 2, 128, 64, 7, lo=700, hi=3900, new_lo=150, new_hi=3400),
        # A few short sequences handed back in F32.
        paged("read", "read a few back", "f32", 2, 2, 128, 64, 3, lo=60, hi=700, whole=True),
        # A whole batch's cache handed back (a move to another engine, a check).
        paged("read", "read a batch back", "bf16", 8, 8, 128, 32, 16, lo=1800, hi=6000, whole=True),
        # One sequence, one token, decoder geometry: latency.
        paged("attend", "attend one short", "f32", 12, 2, 128, 64, 1, lo=777, hi=777, new_lo=1, new_hi=1),
        # The decoder's full context, one sequence: a long axis and few rows.
        paged("attend", "attend one at 65536", "f32", 12, 2, 128, 64, 1, lo=65536, hi=65536, new_lo=1, new_hi=1),
        # A serving batch at one token each, lengths ragged.
        paged("attend", "attend a batch of 64", "bf16", 32, 8, 128, 64, 64, lo=500, hi=8000, new_lo=1, new_hi=1),
        # Drafted tokens verified: a few rows per sequence, an odd group, small pages.
        paged("attend", "attend 5 drafted of 24", "f16", 28, 4, 128, 16, 24, lo=300, hi=4000, new_lo=5, new_hi=5),
        # A prompt in one go, in the framework's own activation type.
        paged("attend", "attend a prompt of 4096", "f32", 12, 2, 128, 64, 1, lo=4096, hi=4096, whole=True),
        # Ragged prompts with a sliding window, narrow heads.
        paged("attend", "attend windowed prompts", "bf16", 16, 4, 64, 32, 6, lo=150, hi=5000, whole=True, window=1024),
    ]


def rotate(name, rows, hq, hk, d, kind, *, norm, fused=False, part=False, neighbours=False, top=60000):
    """top: the largest position; part: the rotation covers the first half of a head only."""
    c = {"op": "rotate", "rows": rows, "hq": hq, "hk": hk, "d": d, "type": kind, "norm": norm, "fused": fused, "part": part,
         "neighbours": neighbours, "top": top}
    return c if name is None else {"name": name, **c}


def paged(op, name, kind, hq, hk, d, page, seqs, *, lo, hi, new_lo=0, new_hi=0, whole=False, window=0, causal=True):
    """Sequences of lo..hi tokens in the cache; the newest new_lo..new_hi of them (all, if whole) are the call's rows."""
    c = {"op": op, "type": kind, "hq": hq, "hk": hk, "d": d, "page": page, "seqs": seqs, "lo": lo, "hi": hi, "new_lo": new_lo,
         "new_hi": new_hi, "whole": whole, "window": window, "causal": causal}
    return c if name is None else {"name": name, **c}


def log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "write", "read", "attend", "attend", "attend"])
    kind = rng.choice(["f32", "bf16", "f16"])
    d = rng.choice([64, 96, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotate":
        group = rng.choice([1, 2, 4, 5, 7])
        rows = log_between(rng, 1, max(1, 8192 * 40 * 128 // (hk * (group + 1) * d * 2)))
        return rotate(None, rows, hk * group, hk, d, kind, norm=rng.random() < 0.6, fused=rng.random() < 0.5,
                      part=d == 128 and rng.random() < 0.3, neighbours=rng.random() < 0.3, top=log_between(rng, 100, 120000))
    if op in ("write", "read"):
        seqs = log_between(rng, 1, 48)
        tokens = 65536 * 8 * 128 // (hk * d) // (4 if op == "write" else 1)
        hi = log_between(rng, 20, max(21, min(8000, tokens // seqs)))
        lo = rng.randint(1, hi)
        if op == "read":
            return paged("read", None, kind, hk, hk, d, page, seqs, lo=lo, hi=hi, whole=True)
        new_hi = 1 if rng.random() < 0.4 else log_between(rng, 1, hi)
        return paged("write", None, kind, hk, hk, d, page, seqs, lo=lo, hi=hi, new_lo=rng.randint(1, new_hi), new_hi=new_hi)
    group = rng.choice([1, 2, 4, 6, 7, 8, 16])
    way = rng.choice(["one", "one", "few", "prompt", "chunk"])
    hq = hk * group
    most_read = 64 * 4250 * 8 * 128  # token places a call streams: the largest listed decode case
    most_work = 12 * 128 * 4096 * 4096 // 2  # pairs times width of the listed prompt of 4096
    if way in ("one", "few"):
        seqs = log_between(rng, 1, 64)
        hi = log_between(rng, 1, max(2, min(65536, most_read // (seqs * hk * d))))
        new = 1 if way == "one" else rng.randint(2, 12)
        lo = rng.randint(max(1, hi // 8), hi)
        return paged("attend", None, kind, hq, hk, d, page, seqs, lo=lo, hi=hi, new_lo=1 if way == "one" else rng.randint(1, new),
                     new_hi=new, window=rng.choice([0, 0, 0, 500, 4096]), causal=way == "one" or rng.random() < 0.8)
    seqs = rng.randint(1, 6)
    hi = log_between(rng, 16, max(17, min(4096, int(math.sqrt(2 * most_work / (seqs * hq * d))))))
    lo = rng.randint(max(1, hi // 10), hi)
    window = rng.choice([0, 0, 100, 1000])
    if way == "prompt":
        return paged("attend", None, kind, hq, hk, d, page, seqs, lo=lo, hi=hi, whole=True, window=window)
    new_hi = rng.randint(1, max(1, hi // 2))
    return paged("attend", None, kind, hq, hk, d, page, seqs, lo=lo, hi=hi, new_lo=rng.randint(1, new_hi), new_hi=new_hi, window=window,
                 causal=rng.random() < 0.9)


def spread(count, lo, hi, step):
    """count whole numbers over lo..hi, scattered evenly; the first is hi."""
    return [hi - int((hi - lo) * (i * step % 1.0) + 0.5) for i in range(count)]


def lengths(case):
    """(tokens in the cache, rows of the call) of each sequence: of the case, not of the seed."""
    lens = spread(case["seqs"], case["lo"], case["hi"], 0.6180339887)
    if case["whole"]:
        return lens, list(lens)
    news = spread(case["seqs"], case["new_lo"], case["new_hi"], 0.7548776662)
    return lens, [min(n, have) for n, have in zip(news, lens)]


def reach(case, have, rows):
    """(query, token) pairs of one head, and the tokens that any of the rows reads."""
    if not case["causal"]:
        w = case["window"]
        spans = [(max(0, have - rows + i - w + 1) if w else 0, have) for i in range(rows)]
    else:
        w = case["window"]
        spans = [(max(0, have - rows + i + 1 - w) if w else 0, have - rows + i + 1) for i in range(rows)]
    pairs = sum(max(0, hi - lo) for lo, hi in spans)
    return pairs, (max(hi for _, hi in spans) - min(lo for lo, _ in spans)) if spans else 0


def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "rotate":
        n = case["rows"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * n * size, "flops": 6 * n}
    lens, news = lengths(case)
    hk, hq, d, page = case["hk"], case["hq"], case["d"], case["page"]
    if case["op"] == "attend":
        pairs, tokens = (sum(x) for x in zip(*(reach(case, a, b) for a, b in zip(lens, news))))
        return {"bytes": 2 * tokens * hk * d + 8 * hk * tokens // page + 2 * sum(news) * hq * d * size, "flops": 4 * pairs * hq * d}
    rows = sum(news) if case["op"] == "read" else sum(a - (a - b) // page * page for a, b in zip(lens, news))
    n = 2 * rows * hk * d
    m = 2 * sum(news) * hk * d if case["op"] == "write" else 0
    return {"bytes": n * (1 + size) + m * (1 + size), "flops": n + 4 * m}


# ---------------------------------------------------------------------------
# What a program has in hand

def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def prepare(case, seed):
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 17)
    kind = TYPES[case["type"]]
    hq, hk, d = case["hq"], case["hk"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "rotate":
        rows, turned = case["rows"], d // 2 if case["part"] else d
        if case["fused"]:  # the rows of one projection for queries, keys and values
            line = normal(rows, (hq + 2 * hk) * d).to(kind)
            q, k = line[:, :hq * d].view(rows, hq, d), line[:, hq * d:(hq + hk) * d].view(rows, hk, d)
        else:
            q, k = normal(rows, hq, d).to(kind), normal(rows, hk, d).to(kind)
        # Runs of positions of sequences that lie one behind another.
        begin = torch.randint(0, max(1, case["top"] - rows), (1,), generator=g, device=dev)
        pos = (begin + torch.arange(rows, device=dev)).to(torch.int32)
        freq = 1e6 ** (-torch.arange(0, turned, 2, dtype=torch.float64, device=dev) / turned)
        weights = [1 + 0.2 * normal(d) if case["norm"] else None for _ in range(2)]
        return {"case": case, "q": q, "k": k, "pos": pos, "freq": freq.float(), "qw": weights[0], "kw": weights[1]}

    lens, news = lengths(case)
    page, seqs = case["page"], case["seqs"]
    blocks = [-(-n // page) for n in lens]
    total = sum(blocks)
    order = torch.randperm(total + 3, generator=g, device=dev).to(torch.int32)
    table = torch.full((seqs, max(1, max(blocks))), -1, dtype=torch.int32)
    order_h, at = order.cpu(), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order_h[at:at + n]
        at += n
    pages = total + 3
    # Keys carry a few wide channels, as the biases of key projections leave them; values are plain.
    wide = torch.ones(hk, 1, d, device=dev)
    wide[:, :, torch.randperm(d, generator=g, device=dev)[:max(1, d // 32)]] = 5.0
    kcodes = (normal(pages, hk, page, d) * (18.0 * wide)).round_().clamp_(-127, 127).to(torch.int8)
    vcodes = (normal(pages, hk, d, page) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
    kscale = torch.exp(0.15 * normal(pages, hk)) / 22.0
    vscale = torch.exp(0.25 * normal(pages, hk)) / 32.0
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s = {"case": case, "k": kcodes, "v": vcodes, "ks": kscale, "vs": vscale, "table": table.to(dev),
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "starts": torch.tensor(starts, dtype=torch.int32, device=dev),
         "rows": starts[-1], "longest": max(lens)}
    if case["op"] == "attend":
        s["q"] = normal(starts[-1], hq, d).to(kind)
        return s
    back = news if case["op"] == "read" else [a - (a - b) // page * page for a, b in zip(lens, news)]
    s["row_seq"] = torch.cat([torch.full((n,), b) for b, n in enumerate(back)]).to(dev)
    s["row_tok"] = torch.cat([torch.arange(a - n, a) for a, n in zip(lens, back)]).to(dev)
    if case["op"] == "write":
        s["new_k"] = (normal(starts[-1], hk, d) * wide.view(1, hk, d)).to(kind)
        s["new_v"] = normal(starts[-1], hk, d).to(kind)
        ends = [0]
        for n in back:
            ends.append(ends[-1] + n)
        s["back"], s["back_rows"] = torch.tensor(ends, dtype=torch.int32, device=dev), ends[-1]
        touched = [(b, j) for b, (a, n) in enumerate(zip(lens, news)) if n for j in range((a - n) // page, (a - 1) // page + 1)]
        s["touched_seq"] = torch.tensor([b for b, _ in touched], device=dev)
        s["touched_block"] = torch.tensor([j for _, j in touched], device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rotate": own_rotate, "write": own_write, "read": own_read, "attend": own_attend}[op](s)
    return {"rotate": plain_rotate, "write": plain_write, "read": plain_read, "attend": plain_attend}[op](s)


def handles(s):
    """The cache's and the batch's handles: a program makes them where it makes the tensors that they name."""
    if "handles" not in s:
        from ternary_weight_integer_amd import kv8
        cache = kv8.KV8Cache(s["k"], s["v"], s["ks"], s["vs"])
        batch = kv8.KV8Batch(s["table"], s["lens"], s["starts"], max_len=s["longest"])
        back = kv8.KV8Batch(s["table"], s["lens"], s["back"], max_len=s["longest"]) if "back" in s else batch
        s["handles"] = kv8, cache, batch, back
    return s["handles"]


def own_rotate(s):
    from ternary_weight_integer_amd import kv8
    return kv8.kv8_qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                neighbours=s["case"]["neighbours"])


def own_write(s):
    kv8, cache, batch, back = handles(s)
    kv8.kv8_append(cache, batch, s["new_k"], s["new_v"])
    return kv8.kv8_read(cache, back, s["back_rows"], dtype=TYPES[s["case"]["type"]])


def own_read(s):
    kv8, cache, batch, _ = handles(s)
    return kv8.kv8_read(cache, batch, s["rows"], dtype=TYPES[s["case"]["type"]])


def own_attend(s):
    kv8, cache, batch, _ = handles(s)
    return kv8.kv8_attention(cache, batch, s["q"], causal=s["case"]["causal"], window=s["case"]["window"])


def plain_rotate(s):
    c, out = s["case"], []
    angle = s["pos"].double()[:, None] * s["freq"].double()[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    turned = 2 * s["freq"].numel()
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        a, rest = y[..., :turned], y[..., turned:]
        if c["neighbours"]:
            u, v = a[..., 0::2], a[..., 1::2]
            a = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
        else:
            u, v = a[..., :turned // 2], a[..., turned // 2:]
            a = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
        out.append(torch.cat((a, rest), -1).to(x.dtype))
    return tuple(out)


def half_away(x):
    """Rounded half away from zero, in 64 bits (where adding a half is exact)."""
    x = x.double()
    return torch.sign(x) * torch.floor(x.abs() + 0.5)


def plain_write(s):
    c = s["case"]
    page = c["page"]
    b, j = s["touched_seq"], s["touched_block"]
    have, first = s["lens"].long()[b], s["starts"].long()[b]
    rows = s["starts"].long()[b + 1] - first
    tok = j[:, None] * page + torch.arange(page, device=b.device)[None, :]
    old = tok < (have - rows)[:, None]
    new = ~old & (tok < have[:, None])
    src = (first[:, None] + tok - (have - rows)[:, None]).clamp(0, s["rows"] - 1)
    at = s["table"].long()[b, j]
    fresh = (j * page >= have - rows)[:, None]
    for x, codes, scale, turn in ((s["new_k"], s["k"], s["ks"], False), (s["new_v"], s["v"], s["vs"], True)):
        x = x.float()[src]  # [touched][page][Hk][D]
        x = torch.where(new[:, :, None, None], x, 0.0).permute(0, 2, 1, 3)
        q = codes[at].transpose(-1, -2) if turn else codes[at]
        top = x.abs().amax((-1, -2))
        need = (torch.clamp(top, min=FLOOR).double() / 127.0).float()  # two F32 values divided in 64 bits round as in 32
        before = scale[at]
        now = torch.where(fresh, need, torch.maximum(before, need))
        shrink = (before.double() / now.double()).float()
        moved = half_away(q.float() * shrink[:, :, None, None])
        moved = torch.where((now > before)[:, :, None, None], moved, q.double())
        fit = half_away((x.double() / now.double()[:, :, None, None]).float()).clamp(-127, 127)
        q = torch.where(new[:, None, :, None], fit, torch.where(old[:, None, :, None], moved, q.double())).to(torch.int8)
        codes[at] = q.transpose(-1, -2) if turn else q
        scale[at] = now
    return plain_read(s)


def plain_read(s):
    c = s["case"]
    at = s["table"].long()[s["row_seq"], s["row_tok"] // c["page"]]
    slot = s["row_tok"] % c["page"]
    k = s["k"][at, :, slot, :].float() * s["ks"][at][:, :, None]
    v = s["v"][at, :, :, slot].float() * s["vs"][at][:, :, None]
    return k.to(TYPES[c["type"]]), v.to(TYPES[c["type"]])


def plain_attend(s):
    c = s["case"]
    hq, hk, d, page, q = c["hq"], c["hk"], c["d"], c["page"], s["q"]
    group, dev = hq // hk, q.device
    starts, lens, at = s["starts"].long(), s["lens"].long(), s["table"].long().clamp(min=0)
    seqs, blocks = at.shape
    rows = int(max(lengths(c)[1]))
    row = torch.arange(rows, device=dev)
    new = starts[1:] - starts[:-1]
    live = row[None, :] < new[:, None]  # [B][rows]
    src = (starts[:-1, None] + row[None, :]).clamp(max=max(0, q.shape[0] - 1))
    x = q.float()[src].view(seqs, rows, hk, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, hk, group * rows, d)
    k = (s["k"][at].float() * s["ks"][at][..., None, None]).permute(0, 2, 1, 3, 4).reshape(seqs, hk, blocks * page, d)
    v = (s["v"][at].float() * s["vs"][at][..., None, None]).permute(0, 2, 1, 4, 3).reshape(seqs, hk, blocks * page, d)
    logits = torch.matmul(x, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(seqs, hk, group, rows, blocks * page)
    tok = torch.arange(blocks * page, device=dev)
    place = lens[:, None] - new[:, None] + row[None, :]  # [B][rows]
    seen = (tok[None, None, :] < lens[:, None, None]) & live[:, :, None]
    if c["causal"]:
        seen &= tok[None, None, :] <= place[:, :, None]
    if c["window"]:
        seen &= tok[None, None, :] > place[:, :, None] - c["window"]
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hk, group * rows, blocks * page), v).view(seqs, hk, group, rows, d)
    o = o / torch.where(total == 0, 1.0, total)
    out = torch.zeros(q.shape, dtype=torch.float32, device=dev)
    out[src[live]] = o.permute(0, 3, 1, 2, 4).reshape(seqs, rows, hq, d)[live]
    return out.to(q.dtype)


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": exact_rotate, "write": exact_write, "read": exact_read, "attend": exact_attend}[case["op"]](case, s)


def exact_rotate(c, s):
    import numpy as np
    pos, f = s["pos"].cpu().numpy().astype(np.float64), s["freq"].cpu().numpy().astype(np.float64)
    turn = np.exp(1j * pos[:, None] * f[None, :])[:, None, :]
    n, out = len(f), []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.float().cpu().numpy().astype(np.float64)
        if w is not None:
            y = y / np.sqrt(np.mean(np.square(y), -1, keepdims=True) + 1e-6) * w.cpu().numpy().astype(np.float64)
        first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if c["neighbours"] else (slice(0, n), slice(n, 2 * n))
        z = (y[..., first] + 1j * y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def exact_write(c, s):
    """The operator's own F32 steps (scale, quotient, product) are part of its definition: each is computed in 64 bits and rounded to 32."""
    import numpy as np
    page, lens, starts = c["page"], s["lens"].tolist(), s["starts"].tolist()
    table = s["table"].cpu().numpy()
    for x, codes, scale, turn in ((s["new_k"], s["k"], s["ks"], False), (s["new_v"], s["v"], s["vs"], True)):
        x, q, sc = x.float().cpu().numpy(), codes.cpu().numpy(), scale.cpu().numpy()
        for b, have in enumerate(lens):
            done = have - (starts[b + 1] - starts[b])
            for j in range(done // page, -(-have // page) if have > done else 0):
                t0, t1 = max(done, j * page), min(have, (j + 1) * page)
                part = x[starts[b] + t0 - done:starts[b] + t1 - done].astype(np.float64)  # [n][Hk][D]
                p = table[b, j]
                block = q[p].swapaxes(-1, -2) if turn else q[p]
                need = (np.maximum(np.abs(part).max((0, 2)), np.float64(np.float32(FLOOR))) / 127.0).astype(np.float32)
                if t0 > j * page:
                    grown = np.maximum(need, sc[p])
                    ratio = (sc[p].astype(np.float64) / grown.astype(np.float64)).astype(np.float32)
                    kept = block[:, :t0 - j * page].astype(np.float64)
                    again = (kept * ratio[:, None, None].astype(np.float64)).astype(np.float32).astype(np.float64)
                    again = np.copysign(np.floor(np.abs(again) + 0.5), again)
                    block[:, :t0 - j * page] = np.where((grown > sc[p])[:, None, None], again, kept).astype(np.int8)
                    need = grown
                sc[p] = need
                v = (part / need[None, :, None].astype(np.float64)).astype(np.float32).astype(np.float64)
                v = np.clip(np.copysign(np.floor(np.abs(v) + 0.5), v), -127, 127)
                block[:, t0 - j * page:t1 - j * page] = v.astype(np.int8).swapaxes(0, 1)
        codes.copy_(torch.from_numpy(q))
        scale.copy_(torch.from_numpy(sc))
    return exact_read(c, s)


def exact_read(c, s):
    import numpy as np
    page, table = c["page"], s["table"].cpu().numpy()
    seq, tok = s["row_seq"].cpu().numpy(), s["row_tok"].cpu().numpy()
    p, slot = table[seq, tok // page], tok % page
    k, v = s["k"].cpu().numpy(), s["v"].cpu().numpy().swapaxes(-1, -2)
    ks, vs = s["ks"].cpu().numpy(), s["vs"].cpu().numpy()
    out = []
    for codes, scale in ((k, ks), (v, vs)):
        out.append(codes[p, :, slot, :].astype(np.float64) * scale[p][:, :, None].astype(np.float64))
    return tuple(out)


def exact_attend(c, s):
    """Sequence by sequence and head by head, with torch in 64 bits on the device that holds the inputs."""
    hq, hk, d, page = c["hq"], c["hk"], c["d"], c["page"]
    group = hq // hk
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device=s["q"].device)
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    for b, have in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi or have == 0:
            continue
        at = s["table"][b, :-(-have // page)].long()
        t = torch.arange(have, device=out.device)
        for h in range(hk):
            k = (s["k"][at, h].double() * s["ks"][at, h].double()[:, None, None]).reshape(-1, d)[:have]
            v = (s["v"][at, h].double() * s["vs"][at, h].double()[:, None, None]).transpose(-1, -2).reshape(-1, d)[:have]
            for r0 in range(lo, hi, 1024):
                r1 = min(hi, r0 + 1024)
                x = s["q"][r0:r1, h * group:(h + 1) * group].double()  # [rows][group][D]
                e = (x.reshape(-1, d) @ k.t()).view(r1 - r0, group, have) / math.sqrt(d)
                place = have - (hi - lo) + torch.arange(r0 - lo, r1 - lo, device=out.device)
                hidden = torch.zeros(r1 - r0, have, dtype=torch.bool, device=out.device)
                if c["causal"]:
                    hidden |= t[None, :] > place[:, None]
                if c["window"]:
                    hidden |= t[None, :] <= place[:, None] - c["window"]
                e = e.masked_fill(hidden[:, None, :], -math.inf)
                top = e.amax(-1, keepdim=True)
                p = torch.where(torch.isneginf(top), 0.0, torch.exp(e - top))
                total = p.sum(-1, keepdim=True)
                p = p / torch.where(total == 0, torch.ones_like(total), total)
                out[r0:r1, h * group:(h + 1) * group] = (p.reshape(-1, have) @ v).view(r1 - r0, group, d)
    return out
