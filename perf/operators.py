"""Measured cases of the paged-cache operators: kvsel_paged_append, kvsel_paged_attention,
kvsel_paged_compact and kvsel_pages_update.

A cache lies in pages: K and V [layers, pages, page_size, kv_heads, dim], a table of page
numbers per sequence and its length in rows. Each case below is one call of one operator, in
plain torch operations (own = False) or through the library (own = True).
"""

import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of one short conversation: the call's latency
        dict(name="attention, one short cache", op="attention", dtype="bf16", layers=1, seqs=1,
             heads=32, kv_heads=8, dim=128, page=16, lo=293, hi=293, lens_seed=1),
        # a serving batch of mixed lengths, some slots of the batch empty
        dict(name="attention, ragged batch", op="attention", dtype="bf16", layers=1, seqs=48,
             heads=32, kv_heads=8, dim=128, page=16, lo=0, hi=8192, lens_seed=2),
        # the full caches of long prompts, before any eviction; eight queries share a head
        dict(name="attention, long caches", op="attention", dtype="bf16", layers=1, seqs=8,
             heads=64, kv_heads=8, dim=128, page=64, lo=120000, hi=131072, lens_seed=3),
        # every layer's compacted fp32 cache at once (retained-mass studies), no shared heads
        dict(name="attention, fp32 own heads", op="attention", dtype="f32", layers=4, seqs=5,
             heads=16, kv_heads=16, dim=64, page=8, lo=200, hi=3001, lens_seed=4),
        # one decode step of a batch: norms, rotation and the rows' places in one call
        dict(name="append, decode step", op="append", dtype="bf16", layers=1, tokens=16, heads=32,
             kv_heads=8, dim=128, page=16, rot=128, interleaved=False, norm=True, far=40000),
        # a prompt's queries and keys, written into pages as the projection left them
        dict(name="append, long prompt", op="append", dtype="bf16", layers=1, tokens=16384, heads=32,
             kv_heads=8, dim=128, page=64, rot=128, interleaved=False, norm=True, far=16384),
        # interleaved pairs on half of each head, far positions, 32-bit rows, no norm
        dict(name="append, fp32 interleaved", op="append", dtype="f32", layers=2, tokens=777, heads=12,
             kv_heads=4, dim=64, page=8, rot=32, interleaved=True, norm=False, far=1000000),
        # a long prompt's cache cut to its budget, every layer, right after the selection
        dict(name="compact, whole prompt", op="compact", dtype="bf16", layers=32, seqs=1, kv_heads=8,
             dim=128, page=16, lo=16384, hi=16384, keep=2048, lens_seed=5),
        # a batch of sequences cut during decoding, odd lengths, some already within the budget
        dict(name="compact, ragged batch", op="compact", dtype="f32", layers=3, seqs=7, kv_heads=6,
             dim=64, page=32, lo=90, hi=3501, keep=517, lens_seed=6),
        # four beams exchange their parents before the next token
        dict(name="update, four beams", op="update", dtype="bf16", layers=32, seqs=4, kv_heads=8,
             dim=128, page=16, pages=1200, lo=2001, hi=2001, forks=4, drop=0, lens_seed=7),
        # every prompt forked into eight samples
        dict(name="update, eight samples", op="update", dtype="bf16", layers=4, seqs=32, kv_heads=8,
             dim=128, page=64, pages=2400, lo=500, hi=4100, forks=8, drop=0, lens_seed=8),
        # a step of a large server: every sequence grows by a row, some end and free their pages
        dict(name="update, one step of many", op="update", dtype="bf16", layers=1, seqs=700,
             kv_heads=1, dim=64, page=16, pages=150000, lo=1, hi=3000, forks=0, drop=9, lens_seed=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "compact", "update"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype, dim=rng.choice([64, 128]), page=rng.choice([1, 2, 8, 16, 32, 64, 128]),
             lens_seed=rng.randrange(1 << 30))
    if op == "attention":
        kv = rng.choice([1, 2, 3, 4, 8, 8])
        rows = _log(rng, 1, 100000 if dtype == "bf16" else 40000)
        c.update(layers=rng.choice([1, 1, 2, 5]), seqs=max(1, min(_log(rng, 1, 128), 300000 // rows)),
                 kv_heads=kv, heads=kv * rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 24]),
                 lo=rng.choice([0, 1, rows]), hi=rows)
        while c["layers"] * c["seqs"] * rows * c["heads"] > 40000000:
            c["seqs"] = max(1, c["seqs"] // 2)
            c["layers"] = 1
            if c["seqs"] == 1:
                rows //= 2
                c.update(lo=rows, hi=rows)
    elif op == "append":
        kv = rng.choice([1, 2, 3, 4, 8, 16])
        c.update(layers=rng.choice([1, 1, 3]), kv_heads=kv, heads=kv * rng.choice([1, 2, 4, 5, 8]),
                 tokens=_log(rng, 1, 4000), rot=rng.choice([0, 16, 32, 48, 64]),
                 interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, far=_log(rng, 10, 3000000))
    elif op == "compact":
        c.update(layers=rng.choice([1, 2, 5]), seqs=_log(rng, 1, 12), kv_heads=rng.choice([1, 2, 3, 8]),
                 lo=_log(rng, 1, 3000), keep=_log(rng, 1, 3000))
        c["hi"] = c["lo"] + _log(rng, 1, 6000)
    else:
        c.update(layers=rng.choice([1, 2, 7]), seqs=_log(rng, 1, 100), kv_heads=rng.choice([1, 2, 8]),
                 lo=0, hi=_log(rng, 1, 1500), forks=rng.choice([0, 0, 1, 3]), drop=rng.choice([0, 2, 5]))
        c["pages"] = c["seqs"] * (2 + c["hi"] // c["page"]) * (1 + c["forks"]) + rng.randrange(50)
        while c["pages"] * c["page"] * c["kv_heads"] * c["dim"] * c["layers"] > 400000000:
            c["layers"], c["kv_heads"], c["dim"] = 1, 1, 64
            c["page"] = max(1, c["page"] // 2)
            c["seqs"] = max(1, c["seqs"] * 3 // 4)
            c["pages"] = c["seqs"] * (2 + c["hi"] // c["page"]) * (1 + c["forks"])
    return c


def _lens(c):
    """The sequences' lengths: lo .. hi by the case's own seed, the first at hi; where lo is 0, about
    one in six empty."""
    r = random.Random(c["lens_seed"])
    n = []
    for i in range(c["seqs"]):
        x = c["hi"] if i == 0 else int(round(math.exp(r.uniform(math.log(max(1, c["lo"])),
                                                                 math.log(max(1, c["hi"]))))))
        n.append(0 if c["lo"] == 0 and i and r.random() < 1 / 6 else x)
    return n


def _kept(c):
    return [min(n, c["keep"]) for n in _lens(c)]


def _new(c):
    """(parents, new lengths) of an update case."""
    r = random.Random(c["lens_seed"] + 1)
    lens = _lens(c)
    if c["forks"]:
        parents = [b for b in range(c["seqs"]) for _ in range(c["forks"])]
        if c["forks"] == c["seqs"]:                     # beams: every slot takes some beam's place
            parents = [r.randrange(c["seqs"]) for _ in range(c["seqs"])]
    else:
        parents = list(range(c["seqs"]))
    if c["drop"]:
        parents = [-1 if i % c["drop"] == c["drop"] - 1 else p for i, p in enumerate(parents)]
    return parents, [0 if p < 0 else lens[p] + 1 for p in parents]


def work(c):
    e, op = BYTES[c["dtype"]], c["op"]
    row = c["dim"] * e
    if op == "attention":
        rows = sum(_lens(c)) * c["layers"]
        inst = c["layers"] * c["seqs"] * c["heads"]
        return dict(bytes=rows * c["kv_heads"] * 2 * row + inst * (row + 4 * c["dim"] + 4)
                    + 4 * sum(-(-n // c["page"]) for n in _lens(c)),
                    flops=4 * rows * c["heads"] * c["dim"])
    if op == "append":
        rows = c["layers"] * c["tokens"] * (c["heads"] + 2 * c["kv_heads"])
        return dict(bytes=2 * rows * row + 12 * c["tokens"], flops=10 * rows * c["dim"])
    if op == "compact":
        moved = sum(n * (1 - n / l) for n, l in zip(_kept(c), _lens(c)))
        inst = c["layers"] * c["kv_heads"]
        return dict(bytes=inst * (4 * row * moved + 8 * sum(_kept(c))), flops=inst * sum(_kept(c)))
    parents, new = _new(c)
    lens, page = _lens(c), c["page"]
    cols = sum(-(-n // page) for n in new)
    old = sum(-(-n // page) for n in lens)
    copied, seen = 0, set()
    for p in parents:
        if p >= 0 and p in seen:
            copied += lens[p] % page
        seen.add(p)
    return dict(bytes=4 * (old + cols + c["pages"]) + 4 * copied * c["layers"] * c["kv_heads"] * row,
                flops=cols + c["pages"])


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _tables(lens, page, pages, gen, extra=0):
    """A table of distinct page numbers in random order: [seqs, width] int32, -1 past the end."""
    need = [-(-n // page) for n in lens]
    width = max(max(need) + extra, 1)
    order = torch.randperm(pages, generator=gen)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return table.to(DEV)


def prepare(c, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, op = DTYPES[c["dtype"]], c["op"]

    def normal(*shape, scale=1.0):
        out = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)
        return out * scale if scale != 1.0 else out

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    s = dict(c)
    D, kv, page, layers = c["dim"], c["kv_heads"], c["page"], c["layers"]
    if op == "append":
        n = c["tokens"]
        # as many sequences as fit a page-count of about n / 4 tokens each, or one token a sequence
        per = 1 if n <= 64 else -(-n // 4)
        seqs = -(-n // per)
        start = [random.Random(c["tokens"] + b).randrange(0, 50) for b in range(seqs)]
        lens = [start[b] + per for b in range(seqs)]
        pages = sum(-(-x // page) for x in lens) + 3
        s["table"] = _tables(lens, page, pages, gen)
        tok = torch.arange(n)
        s["seqs"] = (tok // per).to(torch.int32).to(DEV)
        s["cache_pos"] = (torch.tensor(start)[tok // per] + tok % per).to(torch.int32).to(DEV)
        s["positions"] = torch.randint(0, c["far"], (n,), generator=gen).to(torch.int32).to(DEV)
        # the fused projection's rows: queries, keys and values side by side
        s["qkv"] = normal(layers, n, (c["heads"] + 2 * kv) * D)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64)
                                     / max(1, c["rot"]))).to(torch.float32).to(DEV)
        for w in ("q_weight", "k_weight"):
            s[w] = (1 + 0.2 * torch.randn((layers, D), generator=gen)).to(dt).to(DEV) if c["norm"] else None
    else:
        lens = _lens(c)
        if op == "update":
            parents, new = _new(c)
            pages, extra = c["pages"], 2
            s["parents"], s["new_lens"] = ints(parents), ints(new)
        else:
            pages, extra = sum(-(-n // page) for n in lens) + 5, 0
        s["table"] = _tables(lens, page, pages, gen, extra)
        s["lens"] = ints(lens)
        s["max_len"] = max(lens)
    s["K"], s["V"] = normal(layers, pages, page, kv, D), normal(layers, pages, page, kv, D)
    if op == "attention":
        s["q"] = normal(layers, c["seqs"], c["heads"], D, scale=2.0)
    if op == "compact":
        kept = _kept(c)
        window = 32
        parts = []
        for n, l in zip(kept, lens):
            w = min(window, n)
            score = torch.rand((layers, kv, l - w), device=DEV, generator=g)
            top = score.topk(n - w, dim=2).indices
            tail = torch.arange(l - w, l, device=DEV).expand(layers, kv, w)
            parts.append(torch.cat([top, tail], dim=2).transpose(1, 2))
        s["keep_idx"] = torch.cat(parts, dim=1).to(torch.int32).contiguous()
        offs = [0]
        for n in kept:
            offs.append(offs[-1] + n)
        s["keep_offsets"] = ints(offs)
        s["max_keep"] = max(kept)
        s["ref"] = torch.ones(pages, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"attention": _attention, "append": _append, "compact": _compact, "update": _update}[s["op"]](s)


def _split(s):
    """The fused projection's queries, keys and values: [layers, tokens, heads, dim] views."""
    H, kv, D = s["heads"], s["kv_heads"], s["dim"]
    t = s["qkv"].unflatten(2, (H + 2 * kv, D))
    return t[:, :, :H], t[:, :, H:H + kv], t[:, :, H + kv:]


def _own(s):
    from kv_cache_eviction_snapkv_gb300 import api
    op = s["op"]
    if op == "attention":
        out, lse = api.kvsel_paged_attention(s["q"], s["K"], s["V"], s["table"], s["lens"])
        return {"out": out, "lse": lse}
    if op == "append":
        q, k, v = _split(s)
        q = api.kvsel_paged_append(q, k, v, s["K"], s["V"], s["cache_pos"], positions=s["positions"],
                                   table=s["table"], seqs=s["seqs"], q_weight=s["q_weight"],
                                   k_weight=s["k_weight"], eps=1e-6, inv_freq=s["inv_freq"],
                                   interleaved=s["interleaved"])
        return {"q": q, "K": s["K"], "V": s["V"]}
    if op == "compact":
        pos = api.kvsel_paged_compact(s["K"], s["V"], s["table"], s["lens"], s["keep_idx"],
                                      s["keep_offsets"], s["max_keep"], ref=s["ref"])
        return {"pos": pos, "K": s["K"], "V": s["V"]}
    table, ref, free = api.kvsel_pages_update(s["K"], s["V"], s["table"], s["lens"], s["new_lens"],
                                              parents=s["parents"])
    return {"table": table, "ref": ref, "free": free, "K": s["K"], "V": s["V"]}


def _rows(t, table, at, page):
    """Row numbers in the pool of rows `at` of each sequence: table [seqs, width], at [seqs, n]."""
    return table.long().clamp(min=0).gather(1, at // page) * page + at % page


def _attention(s):
    q, K, V, page = s["q"], s["K"], s["V"], s["page"]
    layers, S, H, D = q.shape
    kv = K.shape[3]
    n = max(1, s["max_len"])
    at = torch.arange(n, device=q.device).expand(S, n)
    rows = _rows(K, s["table"], at, page)
    k = K.flatten(1, 2)[:, rows].float().permute(0, 1, 3, 4, 2)             # [layers, S, kv, D, n]
    z = (q.float().view(layers, S, kv, H // kv, D) @ k) * (1.0 / math.sqrt(D))
    del k
    z = z.masked_fill((at >= s["lens"][:, None])[None, :, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (z - m).exp()
    total = p.sum(-1, keepdim=True)
    v = V.flatten(1, 2)[:, rows].float().permute(0, 1, 3, 2, 4)             # [layers, S, kv, n, D]
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return {"out": out.reshape(layers, S, H, D), "lse": (m + total.log()).reshape(layers, S, H)}


def _rotate(x, cos, sin, rot, interleaved):
    """x [layers, tokens, heads, dim] fp32; cos, sin [tokens, 1, rot / 2]."""
    if not rot:
        return x
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _append(s):
    q, k, v = _split(s)
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()[:, None, None]
        return _rotate(y, cos, sin, s["rot"], s["interleaved"]).to(x.dtype)

    at, seq = s["cache_pos"].long(), s["seqs"].long()
    row = s["table"].long()[seq, at // s["page"]] * s["page"] + at % s["page"]
    s["K"].flatten(1, 2)[:, row] = one(k, s["k_weight"])
    s["V"].flatten(1, 2)[:, row] = v
    return {"q": one(q, s["q_weight"]), "K": s["K"], "V": s["V"]}


def _compact(s):
    K, V, page, width = s["K"], s["V"], s["page"], s["max_keep"]
    layers, kv = K.shape[0], K.shape[3]
    offs = s["keep_offsets"].long()
    S, dev = offs.numel() - 1, K.device
    n = (offs[1:] - offs[:-1])[None, :, None, None]                          # rows kept: [1, S, 1, 1]
    slot = torch.arange(width, device=dev)
    valid = slot < n                                                         # [1, S, 1, width]
    entry = (offs[:-1, None] + slot).clamp(max=s["keep_idx"].shape[1] - 1)   # [S, width]
    idx = s["keep_idx"].long()[:, entry].permute(0, 1, 3, 2)                 # [layers, S, kv, width]
    stays = valid & (idx < n)
    kept = torch.zeros((layers, S, kv, width + 1), dtype=torch.bool, device=dev)
    kept.scatter_(3, torch.where(stays, idx, width), True)
    kept = kept[..., :width]
    hole, moves = valid & ~kept, valid & (idx >= n)
    rank = lambda m: m.long().cumsum(3) - 1  # noqa: E731
    movers = torch.zeros((layers, S, kv, width + 1), dtype=torch.long, device=dev)
    movers.scatter_(3, torch.where(moves, rank(moves), width), idx)
    src = torch.where(hole, movers.gather(3, rank(hole).clamp(min=0)), slot)  # the row that each slot takes
    pos = torch.zeros_like(s["keep_idx"])
    out = torch.where(valid.expand_as(src), src, -1).permute(0, 1, 3, 2)      # [layers, S, width, kv]
    flat = valid[0, :, 0].nonzero()
    pos[:, entry[flat[:, 0], flat[:, 1]]] = out[:, flat[:, 0], flat[:, 1]].int()
    # a slot past the end writes slot 0's row once more
    first = src[..., :1]
    src = torch.where(valid, src, first)
    dst = torch.where(valid, slot, 0).expand_as(src)
    table = s["table"].long().clamp(min=0)[None, :, None].expand(layers, S, kv, -1)
    src = table.gather(3, src // page) * page + src % page
    dst = table.gather(3, dst // page) * page + dst % page
    layer = torch.arange(layers, device=dev)[:, None, None, None]
    head = torch.arange(kv, device=dev)[None, None, :, None]
    for pool in (K.flatten(1, 2), V.flatten(1, 2)):
        pool[layer, dst, head] = pool[layer, src, head]
    return {"pos": pos, "K": K, "V": V}


def _update(s):
    K, V, page = s["K"], s["V"], s["page"]
    pages, table, parents, new = K.shape[1], s["table"].long(), s["parents"].long(), s["new_lens"].long()
    S, width, dev = parents.numel(), table.shape[1], K.device
    old = torch.where(parents < 0, 0, s["lens"].long()[parents.clamp(min=0)])
    old_table = table[parents.clamp(min=0)]
    rows = torch.minimum(old, new)                                # rows taken over
    whole, rest, need = rows // page, rows % page, -(-new // page)
    col = torch.arange(width, device=dev)[None]
    full = col < whole[:, None]
    part = (col == whole[:, None]) & (rest > 0)[:, None]
    spare = lambda m: torch.where(m, old_table, pages)  # noqa: E731
    fulls = torch.zeros(pages + 1, dtype=torch.long, device=dev).index_add_(
        0, spare(full).flatten(), torch.ones(S * width, dtype=torch.long, device=dev))
    seq = torch.arange(S, device=dev)[:, None].expand(S, width)
    owner = torch.full((pages + 1,), S, dtype=torch.long, device=dev).scatter_reduce_(
        0, spare(part).flatten(), seq.flatten(), "amin")
    at = old_table.clamp(min=0)
    keeps = part & (fulls[at] == 0) & (owner[at] == seq)
    held = full | keeps
    ref = torch.zeros(pages + 1, dtype=torch.long, device=dev).index_add_(
        0, spare(held).flatten(), torch.ones(S * width, dtype=torch.long, device=dev))
    free = ref[:pages] == 0
    rank = free.long().cumsum(0) - 1
    number = torch.full((pages + 1,), -1, dtype=torch.long, device=dev)
    number.scatter_(0, torch.where(free, rank, pages), torch.arange(pages, device=dev))
    number[pages] = -1
    fresh = (col < need[:, None]) & ~held
    order = (fresh.flatten().long().cumsum(0) - 1).view(S, width)
    got = torch.where(fresh, number[order.clamp(min=0, max=pages)], -1)
    out = torch.where(held, old_table, got)
    ref.index_add_(0, torch.where(got >= 0, got, pages).flatten(), torch.ones(S * width, dtype=torch.long,
                                                                              device=dev))
    b = (part & ~keeps & (got >= 0)).any(1).nonzero()[:, 0]       # sequences that get a copy
    src, dst = old_table[b, whole[b]], got[b, whole[b]]
    r = torch.arange(page, device=dev)
    take = (r < rest[b][:, None])[None, :, :, None, None]
    for pool in (K, V):
        pool[:, dst] = torch.where(take, pool[:, src], pool[:, dst])
    return {"table": out.int(), "ref": ref[:pages].int(), "free": (free.sum() - fresh.sum()).int().view(1),
            "K": K, "V": V}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return {"attention": _exact_attention, "append": _exact_append, "compact": _exact_compact,
            "update": _exact_update}[c["op"]](s)


def _exact_attention(s):
    q = s["q"].double()
    layers, S, H, D = q.shape
    G = H // s["kv_heads"]
    out = torch.zeros((layers, S, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((layers, S, H), -math.inf, dtype=torch.float64, device=q.device)
    lens = s["lens"].tolist()
    for l in range(layers):
        for b in range(S):
            if lens[b] == 0:
                continue
            j = torch.arange(lens[b], device=q.device)
            pages = s["table"][b].long()[torch.div(j, s["page"], rounding_mode="floor")]
            for h in range(s["kv_heads"]):
                k = s["K"][l, pages, j % s["page"], h].double()
                v = s["V"][l, pages, j % s["page"], h].double()
                z = q[l, b, h * G:(h + 1) * G] @ k.T / math.sqrt(D)
                lse[l, b, h * G:(h + 1) * G] = z.logsumexp(1)
                out[l, b, h * G:(h + 1) * G] = z.softmax(1) @ v
    return {"out": out, "lse": lse}


def _exact_append(s):
    H, kv, D, half = s["heads"], s["kv_heads"], s["dim"], s["rot"] // 2
    x = s["qkv"].double().unflatten(2, (H + 2 * kv, D))
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[None, :, None]          # e^(i angle)

    def one(y, w):
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()[:, None, None]
        y = y.clone()
        if half:
            first = slice(0, 2 * half, 2) if s["interleaved"] else slice(0, half)
            second = slice(1, 2 * half, 2) if s["interleaved"] else slice(half, 2 * half)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
        return y

    K, V = s["K"].double(), s["V"].double()
    at = s["cache_pos"].long()
    page = s["table"][s["seqs"].long(), at // s["page"]].long()
    K[:, page, at % s["page"]] = one(x[:, :, H:H + kv], s["k_weight"])
    V[:, page, at % s["page"]] = x[:, :, H + kv:]
    return {"q": one(x[:, :, :H], s["q_weight"]), "K": K, "V": V}


def _exact_compact(s):
    if s["K"].numel() > 650000000:
        return None
    K, V = s["K"].double(), s["V"].double()
    pos = torch.empty_like(s["keep_idx"])
    offs, page = s["keep_offsets"].tolist(), s["page"]
    lists = s["keep_idx"].cpu()
    for b in range(len(offs) - 1):
        n = offs[b + 1] - offs[b]
        pages = s["table"][b].cpu().long()
        for l in range(K.shape[0]):
            for h in range(K.shape[3]):
                want = lists[l, offs[b]:offs[b + 1], h].tolist()
                there = set(want)
                late = iter([j for j in want if j >= n])
                take = torch.tensor([j if j in there else next(late) for j in range(n)])
                slot = torch.arange(n)
                pos[l, offs[b]:offs[b + 1], h] = take.to(pos)
                for pool, old in ((K, s["K"]), (V, s["V"])):
                    pool[l, pages[slot // page], slot % page, h] = old[l, pages[take // page], take % page,
                                                                       h].double()
    return {"pos": pos, "K": K, "V": V}


def _exact_update(s):
    if s["K"].numel() > 650000000:
        return None
    page, pages, width = s["page"], s["K"].shape[1], s["table"].shape[1]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    parents, new = s["parents"].tolist(), s["new_lens"].tolist()
    rows = [0 if p < 0 else min(lens[p], n) for p, n in zip(parents, new)]
    out = [[-1] * width for _ in parents]
    ref, copies = [0] * pages, []
    for b, p in enumerate(parents):
        for i in range(rows[b] // page):
            out[b][i] = table[p][i]
            ref[table[p][i]] += 1
    for b, p in enumerate(parents):
        i = rows[b] // page
        if rows[b] % page and ref[table[p][i]] == 0:
            out[b][i] = table[p][i]
            ref[table[p][i]] = 1
    free = [x for x in range(pages) if ref[x] == 0]
    left = len(free)
    free = iter(free)
    for b, p in enumerate(parents):
        for i in range(-(-new[b] // page)):
            if out[b][i] >= 0:
                continue
            left -= 1
            out[b][i] = next(free, -1)
            if out[b][i] >= 0:
                ref[out[b][i]] = 1
                if i == rows[b] // page and rows[b] % page:
                    copies.append((table[p][i], out[b][i], rows[b] % page))
    K, V = s["K"].double(), s["V"].double()
    for src, dst, n in copies:
        K[:, dst, :n] = K[:, src, :n].clone()
        V[:, dst, :n] = V[:, src, :n].clone()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=s["K"].device)  # noqa: E731
    return {"table": ints(out), "ref": ints(ref), "free": ints([left]), "K": K, "V": V}
