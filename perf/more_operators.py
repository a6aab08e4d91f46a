"""Cases of the prompt and chunk attention and of the page operators: inputs, plain forms, 64-bit values.

What serving needs around a paged cache:
  prompt   causal attention of whole prompts packed one behind the other, grouped heads
  chunk    attention of chunks of new tokens over pages: a shared prefix, the sequence's cached tokens, the chunk itself
  fork     sequences that go on from another one: its full pages shared, its last one copied
  resize   sequences that grow (pages taken), shrink or end (pages given back), lengths given
  compact  the pages in use moved to the lowest places, the tables after them
"""
import math
import random

import torch

own = False  # False: the plain forms below; True: the framework's operators

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def _prompt(name, seqs, lo, hi, pad, Hq, Hkv, D, type_, window, lse, ragged):
    return dict(name=name, op="prompt", seqs=seqs, lo=lo, hi=hi, pad=pad, Hq=Hq, Hkv=Hkv, D=D, type=type_, window=window, lse=lse,
                ragged=ragged)


def _chunk(name, chunks, new_lo, new_hi, singles, old_hi, pad, prefix, Hq, Hkv, D, type_, page, layout, window, lse, ragged):
    return dict(name=name, op="chunk", chunks=chunks, new_lo=new_lo, new_hi=new_hi, singles=singles, old_hi=old_hi, pad=pad, prefix=prefix,
                Hq=Hq, Hkv=Hkv, D=D, type=type_, page=page, layout=layout, window=window, lse=lse, ragged=ragged)


def _pages(name, op, pages, seqs, n, len_hi, layers, Hkv, D, type_, page, layout, step, ragged):
    return dict(name=name, op=op, pages=pages, seqs=seqs, n=n, len_hi=len_hi, layers=layers, Hkv=Hkv, D=D, type=type_, page=page,
                layout=layout, step=step, ragged=ragged)


def listed():
    return [
        # four short questions without a context: latency
        _prompt("prompt_questions", 4, 20, 64, 0, 32, 8, 128, "bf16", 0, True, 1),
        # the ten chunks of a request computed each alone in a single call, as a chunk store takes them in
        _prompt("prompt_chunks", 10, 512, 512, 0, 32, 8, 128, "bf16", 0, False, 2),
        # the full prefill of a whole 35-chunk request of a 64-head layout
        _prompt("prompt_request", 1, 17984, 17984, 0, 64, 8, 128, "bf16", 0, False, 3),
        # one new question of 64 tokens over 5120 cached ones: latency
        _chunk("chunk_question", 1, 64, 64, 0, 5120, 0, 0, 32, 8, 128, "bf16", 16, "rows", 0, True, 4),
        # a serving step that mixes chunks of prompts with the single tokens of running answers, over a shared context,
        # rows padded behind the last one
        _chunk("chunk_mixed", 4, 300, 1024, 44, 1000, 19, 5120, 32, 8, 128, "f16", 32, "heads", 0, False, 5),
        # a chunk of 2048 tokens far inside a long prompt
        _chunk("chunk_long", 1, 2048, 2048, 0, 65536, 0, 0, 32, 8, 128, "bf16", 64, "rows", 0, False, 6),
        # fifteen more answers to one question over its whole context, 32 layers
        _pages("fork_answers", "fork", 480, 16, 15, 5191, 32, 8, 128, "bf16", 16, "rows", False, 8),
        # every one of 32 long sequences branches twice, pages kept head by head
        _pages("fork_branches", "fork", 4200, 96, 64, 8000, 2, 8, 128, "bf16", 64, "heads", False, 9),
        # a step of 64 running answers, one token more each: latency
        _pages("resize_step", "resize", 4096, 64, 64, 700, 4, 8, 128, "bf16", 16, "rows", True, 10),
        # the pages of a cache turned over: many sequences end, others are cut back, go on or grow by a chunk
        _pages("resize_turnover", "resize", 32768, 256, 200, 2000, 1, 4, 64, "f16", 16, "rows", False, 11),
        # a small cache made dense: latency
        _pages("compact_few", "compact", 600, 16, 0, 400, 8, 8, 128, "bf16", 16, "rows", False, 12),
        # a large one whose sequences left holes everywhere
        _pages("compact_cache", "compact", 12000, 96, 0, 1200, 4, 8, 128, "bf16", 16, "rows", False, 13),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "chunk", "chunk", "fork", "resize", "compact"])
    type_, ragged = rng.choice(["bf16", "f16"]), rng.randrange(1 << 20)
    if op in ("prompt", "chunk"):
        D = rng.choice([64, 80, 128, 128]) if op == "prompt" else rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 4, 8])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        pad = rng.choice([0, rng.randrange(1, 40)])
        if op == "prompt":
            seqs = _log(rng, 1, 64)
            hi = _log(rng, 1, max(2, 16384 // seqs))
            return _prompt(None, seqs, rng.choice([0, 1, (hi + 1) // 2]), hi, pad, Hq, Hkv, D, type_, window, pad == 0, ragged)
        chunks, singles = _log(rng, 1, 16), rng.choice([0, _log(rng, 1, 64)])
        return _chunk(None, chunks, 1, _log(rng, 1, max(2, 3000 // chunks)), singles, _log(rng, 1, max(2, 40000 // (chunks + singles))), pad,
                      rng.choice([0, 0, _log(rng, 1, 8192)]), Hq, Hkv, D, type_, rng.choice([8, 16, 32, 64, 128, 256]),
                      rng.choice(["rows", "heads"]), window, pad == 0, ragged)
    Hkv, D, page = rng.choice([1, 4, 8]), rng.choice([16, 64, 128]), rng.choice([8, 16, 32, 64])
    layers = _log(rng, 1, 32)
    pages = _log(rng, 64, min(40000, (3 << 29) // (layers * 4 * Hkv * D * page)))   # 1.6 GB at most
    seqs = _log(rng, 2, min(256, pages // 4))
    n = 0 if op == "compact" else rng.randint(1, max(1, seqs // 2 if op == "fork" else seqs))
    return _pages(None, op, pages, seqs, n, max(2, min(8000, pages * page // (3 * seqs))), layers, Hkv, D, type_, page,
                  rng.choice(["rows", "heads"]), op == "resize" and rng.random() < 0.3, ragged)


def _lengths(c):
    """New and own token counts of every sequence of an attention case."""
    r = random.Random(c["ragged"])
    if c["op"] == "prompt":
        new = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
        new[0] = max(new[0], 1)
        return new, list(new)
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["chunks"])] + [1] * c["singles"]
    r.shuffle(new)
    return new, [q + (c["old_hi"] if len(new) == 1 else r.randint(0, c["old_hi"])) for q in new]


def _held(c):
    """Of a page case: lengths of the sequences before the call; the pages that each holds, numbered 0, 1, .. (every second
    sequence has begun with the pages of the one before it); how many there are; the call's arguments: source and
    destination of fork, sequence and new length of resize."""
    r = random.Random(c["ragged"])
    S, hi, n, page = c["seqs"], c["len_hi"], c["n"], c["page"]
    lens = [r.randint((hi + 1) // 2, hi) for _ in range(S)]
    a = b = []
    if c["op"] == "fork":
        b = r.sample(range(S), n)
        for i in b:
            lens[i] = 0
        left = [i for i in range(S) if lens[i] > 0]
        a = [left[i % len(left)] for i in range(n)]
    elif c["op"] == "resize":
        a = r.sample(range(S), n)
        b = [lens[i] + 1 if c["step"] else r.choice([0, r.randint(0, lens[i]), lens[i] + 1, r.randint(lens[i], hi)]) for i in a]
    held, used = [], 0
    for i, m in enumerate(-(-x // page) for x in lens):
        same = held[-1][: min(len(held[-1]), m) // 2] if i % 2 and c["op"] != "fork" else []
        held.append(same + list(range(used, used + m - len(same))))
        used += m - len(same)
    return lens, held, used, a, b


def _places(c, used):
    """The pages of the cache that the numbers of _held stand for."""
    return random.Random(c["ragged"] + 1).sample(range(c["pages"]), used)


def _seen(q, n, prefix, window):
    """Keys that the rows of a sequence see, all together: q new of n own tokens."""
    first, last = prefix + n - q + 1, prefix + n
    if window == 0 or window >= last:
        return (first + last) * q // 2
    if window <= first:
        return window * q
    k = window - first
    return (first + window - 1) * k // 2 + window * (q - k)


def work(c):
    if c["op"] in ("prompt", "chunk"):
        new, lens = _lengths(c)
        prefix = c.get("prefix", 0)
        row = c["Hkv"] * c["D"] * 2
        seen = sum(_seen(q, n, prefix, c["window"]) for q, n in zip(new, lens))
        if c["window"]:
            reach = [min(prefix + n, q + c["window"] - 1) if q else 0 for q, n in zip(new, lens)]
            kv = min(prefix, max([x - n for x, n in zip(reach, lens)] + [0])) + sum(min(x, n) for x, n in zip(reach, lens))
        else:
            kv = prefix + sum(n for q, n in zip(new, lens) if q)
        return {"bytes": 2 * sum(new) * c["Hq"] * c["D"] * 2 + 2 * row * kv + (4 * sum(new) * c["Hq"] if c["lse"] else 0),
                "flops": 4 * c["Hq"] * c["D"] * seen}
    row = c["layers"] * 2 * c["Hkv"] * c["D"] * 2
    lens, held, used, a, b = _held(c)
    if c["op"] == "fork":
        return {"bytes": 2 * row * sum(lens[i] % c["page"] for i in a) + 4 * (4 * sum(len(held[i]) for i in a) + 5 * len(a)), "flops": 0}
    if c["op"] == "resize":
        return {"bytes": 4 * (3 * sum(abs(-(-t // c["page"]) - len(held[i])) for i, t in zip(a, b)) + 4 * len(a)), "flops": 0}
    moved = sum(p >= used for p in _places(c, used))
    return {"bytes": 2 * row * c["page"] * moved + 4 * (c["pages"] + 2 * sum(len(h) for h in held)), "flops": 0}


# ------------------------------------------------------------------ inputs

def _randn(shape, g, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _prepare_pages(c, g):
    s, T, page = {"case": c}, TYPES[c["type"]], c["page"]
    lens, held, used, a, b = _held(c)
    shape = (c["layers"], c["pages"], page, c["Hkv"], c["D"]) if c["layout"] == "rows" else (c["layers"], c["pages"], c["Hkv"], page, c["D"])
    s["k"], s["v"] = torch.empty(shape, dtype=T, device=DEV), torch.empty(shape, dtype=T, device=DEV)
    for t in (s["k"], s["v"]):
        for layer in t:
            layer.normal_(generator=g)
    wide = -(-c["len_hi"] // page) + 1
    place = torch.tensor(_places(c, used) + [0], dtype=torch.int32, device=DEV)
    place[:used] = place[:used][torch.randperm(used, generator=g, device=DEV)]
    table = place[torch.tensor([h + [used] * (wide - len(h)) for h in held], device=DEV)]
    table[torch.tensor([[i >= len(h) for i in range(wide)] for h in held], device=DEV)] = 0
    refs = torch.zeros(c["pages"] + 1, dtype=torch.int32, device=DEV)
    every = torch.tensor([i for h in held for i in h], device=DEV)
    refs.index_add_(0, place[every].long(), torch.ones(every.numel(), dtype=torch.int32, device=DEV))
    # counts, table and lengths side by side, so that one copy puts them back before a pass
    s["start"] = torch.cat([refs[:-1], table.flatten(), torch.tensor(lens, dtype=torch.int32, device=DEV)])
    s["now"] = s["start"].clone()
    n, m = c["pages"], c["seqs"] * wide
    s["refs"], s["table"], s["kv_len"] = s["now"][:n], s["now"][n: n + m].view(c["seqs"], wide), s["now"][n + m:]
    s["a"], s["b"] = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (a, b))
    if own:
        from rag_kv_cache_re_gb300 import qcf as Q
        caches = [Q.PagedKV(k, v, layout=c["layout"]) for k, v in zip(s["k"], s["v"])]
        s["pool"] = Q.PagePool(caches, s["refs"], s["table"], s["kv_len"])
    return s


def prepare(case, seed):
    c, g = dict(case), torch.Generator(device=DEV).manual_seed(seed)
    if c["op"] in ("fork", "resize", "compact"):
        return _prepare_pages(c, g)
    s, (new, lens) = {"case": c}, _lengths(c)
    T, Hq, Hkv, D = TYPES[c["type"]], c["Hq"], c["Hkv"], c["D"]
    n_rows = sum(new) + c["pad"]
    s["new"], s["lens"], s["rows"] = new, lens, sum(new)
    s["row_start"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["max_q"], s["max_len"] = max(new), max(lens)
    if c["op"] == "prompt":  # the packed q, k, v rows of the projection before
        rows = _randn((n_rows, Hq + 2 * Hkv, D), g, T, 1.2)
        s["q"], s["k"], s["v"] = rows.split([Hq, Hkv, Hkv], 1)
        s["out"] = torch.zeros((n_rows, Hq, D), dtype=T, device=DEV)
        return s
    page = c["page"]
    own_pages = [-(-n // page) for n in lens]
    n_prefix = -(-c["prefix"] // page)
    n_pages = n_prefix + sum(own_pages) + 3
    shape = (n_pages, page, Hkv, D) if c["layout"] == "rows" else (n_pages, Hkv, page, D)
    s["k_pages"], s["v_pages"] = _randn(shape, g, T), _randn(shape, g, T)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["prefix_pages"] = order[:n_prefix].contiguous()
    count = torch.tensor(own_pages, device=DEV)
    first = n_prefix + torch.cumsum(count, 0) - count
    col = torch.arange(max(own_pages), device=DEV)
    s["page_table"] = torch.where(col < count[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], 0).to(torch.int32)
    s["kv_len"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["q"] = _randn((n_rows, Hq, D), g, T, 1.5)
    s["out"] = torch.zeros_like(s["q"])
    if own:
        from rag_kv_cache_re_gb300 import qcf as Q
        s["cache"] = Q.PagedKV(s["k_pages"], s["v_pages"], layout=c["layout"])
        s["batch"] = Q.PagedBatch(s["row_start"], s["kv_len"], s["page_table"], n_rows=n_rows, max_q=s["max_q"], max_len=s["max_len"],
                                  prefix_pages=s["prefix_pages"], prefix_len=c["prefix"])
    return s


# ------------------------------------------------------------------ plain forms

def _rows(pages, layout):
    """The pages as [page][row][head][D]."""
    return pages if layout == "rows" else pages.transpose(-3, -2)


def _attend(q, K, V, first, window, scale, block=1 << 28):
    """q [n][Hq][D] at positions first, first + 1, ..; K, V [m][Hkv][D] at 0, 1, ..: output and log of the sum, 32 bits."""
    n, Hq, D = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    o, e = q.new_empty((n, Hkv, G, D)), q.new_empty((n, Hkv, G))
    K, V = K.transpose(0, 1), V.transpose(0, 1)
    step = max(1, block // (K.shape[1] * Hq))
    for i in range(0, n, step):
        m = min(n, i + step) - i
        p = (first + i + torch.arange(m, device=DEV))[:, None]
        a, b = max(0, first + i - window + 1) if window else 0, first + i + m   # the keys that any of them sees
        j = torch.arange(a, b, device=DEV)
        hidden = (j > p) | (j <= p - window) if window else j > p
        rows = q[i: i + m].view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D)
        x = (scale * rows @ K[:, a:b].transpose(1, 2)).view(Hkv, G, m, b - a).masked_fill_(hidden, -math.inf)
        top = x.amax(-1, keepdim=True)
        x = (x - top).exp_()
        total = x.sum(-1, keepdim=True)
        y = (x.view(Hkv, G * m, b - a) @ V[:, a:b]).view(Hkv, G, m, D) / total
        o[i: i + m] = y.permute(2, 0, 1, 3)
        e[i: i + m] = (top + total.log())[..., 0].permute(2, 0, 1)
    return o.view(n, Hq, D), e.view(n, Hq)


def _keys(s, b):
    """K and V of sequence b of a chunk case, the prefix before its own tokens, 32 bits."""
    c = s["case"]
    parts = []
    for pages in (s["k_pages"], s["v_pages"]):
        flat = _rows(pages, c["layout"])
        prefix = flat[s["prefix_pages"].long()].flatten(0, 1)[: c["prefix"]]
        mine = flat[s["page_table"][b, : -(-s["lens"][b] // c["page"])].long()].flatten(0, 1)[: s["lens"][b]]
        parts.append(torch.cat([prefix, mine]).float())
    return parts


def _plain_attn(s):
    c, r = s["case"], 0
    scale = 1.0 / math.sqrt(c["D"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV) if c["lse"] else None
    for b, n in enumerate(s["new"]):
        if n:
            at = slice(r, r + n)
            K, V = (s["k"][at].float(), s["v"][at].float()) if c["op"] == "prompt" else _keys(s, b)
            o, e = _attend(s["q"][at].float(), K, V, K.shape[0] - n, c["window"], scale)
            s["out"][at] = o.to(s["out"].dtype)
            if c["lse"]:
                lse[at] = e
        r += n
    return {"o": s["out"], "lse": lse} if c["lse"] else s["out"]


def _plain_fork(s):
    c, refs, table, kv_len, page = s["case"], s["refs"], s["table"], s["kv_len"], s["case"]["page"]
    src, dst = s["a"].long(), s["b"].long()
    free = torch.nonzero(refs == 0)[:, 0]
    col = torch.arange(table.shape[1], device=DEV)
    lens = kv_len[src].long()
    full, rest = (lens // page)[:, None], lens % page
    partly = rest > 0
    new = free[torch.where(partly, torch.cumsum(partly.int(), 0) - 1, 0)]
    old = table[src, (lens // page).clamp(max=table.shape[1] - 1)].long()
    held = col < ((kv_len[dst].long() + page - 1) // page)[:, None]
    refs.index_add_(0, table[dst].flatten().long(), -held.int().flatten())
    rows = torch.where(col < full, table[src], torch.where((col == full) & partly[:, None], new[:, None].int(), table[dst]))
    table[dst] = rows
    refs.index_add_(0, rows.flatten().long(), (col < full + partly[:, None]).int().flatten())
    kv_len[dst] = lens.int()
    pick = torch.nonzero(partly)[:, 0]
    new, old = new[pick], old[pick]
    copy = torch.arange(page, device=DEV) < rest[pick][:, None]
    for t in (s["k"], s["v"]):
        for layer in t:
            rows = _rows(layer, c["layout"])
            rows[new] = torch.where(copy[:, :, None, None], rows[old], rows[new])


def _plain_resize(s):
    c, refs, table, kv_len, page = s["case"], s["refs"], s["table"], s["kv_len"], s["case"]["page"]
    seq, to = s["a"].long(), s["b"].long()
    free = torch.nonzero(refs == 0)[:, 0]
    col = torch.arange(table.shape[1], device=DEV)
    now = kv_len[seq].long()
    kept = torch.minimum(now, to)
    have, need = (now + page - 1) // page, (to + page - 1) // page
    at = (kept // page).clamp(max=table.shape[1] - 1)
    old = table[seq, at].long()
    split = (kept % page > 0) & (now != to) & (refs[old] > 1)      # a page held in part by a sequence that changes is its own
    took = split.int() + (need - have).clamp(min=0)
    first = torch.cumsum(took, 0) - took
    mine = table[seq]
    gone = (col >= need[:, None]) & (col < have[:, None]) | (split[:, None] & (col == at[:, None]))
    fresh = (col >= have[:, None]) & (col < need[:, None]) | (split[:, None] & (col == at[:, None]))
    place = first[:, None] + torch.where(col >= have[:, None], split.int()[:, None] + col - have[:, None], 0)
    rows = torch.where(fresh, free[torch.where(fresh, place, 0)].int(), mine)
    refs.index_add_(0, mine.flatten().long(), -gone.int().flatten())
    refs.index_add_(0, rows.flatten().long(), fresh.int().flatten())
    table[seq] = rows
    kv_len[seq] = to.int()
    pick = torch.nonzero(split)[:, 0]
    new, old = rows[pick, at[pick]].long(), old[pick]
    copy = torch.arange(page, device=DEV) < (kept % page)[pick][:, None]
    if pick.numel():
        for t in (s["k"], s["v"]):
            for layer in t:
                r = _rows(layer, c["layout"])
                r[new] = torch.where(copy[:, :, None, None], r[old], r[new])


def _plain_compact(s):
    refs, table, kv_len, page = s["refs"], s["table"], s["kv_len"], s["case"]["page"]
    used = refs > 0
    total = used.sum()
    ids = torch.arange(refs.numel(), device=DEV)
    move, hole = torch.nonzero(used & (ids >= total))[:, 0], torch.nonzero(~used & (ids < total))[:, 0]
    to = ids.clone()
    to[move] = hole
    held = torch.arange(table.shape[1], device=DEV) < ((kv_len.long() + page - 1) // page)[:, None]
    table.copy_(torch.where(held, to[table.long()].int(), table))
    refs[hole] = refs[move]
    refs[move] = 0
    for t in (s["k"], s["v"]):
        for layer in t:
            layer[hole] = layer[move]
    return total.int().view(1)


def run(s):
    c = s["case"]
    if c["op"] in ("prompt", "chunk"):
        if not own:
            return _plain_attn(s)
        from rag_kv_cache_re_gb300 import qcf as Q
        scale = 1.0 / math.sqrt(c["D"])
        if c["op"] == "prompt":
            got = Q.qcf_packed_causal_attn(s["q"], s["k"], s["v"], s["row_start"], s["max_len"], scale, window=c["window"],
                                           want_lse=c["lse"], out=s["out"])
        else:
            got = Q.qcf_paged_chunk_attn(s["cache"], s["batch"], s["q"], scale, window=c["window"], want_lse=c["lse"], out=s["out"])
        return {"o": got[0], "lse": got[1]} if c["lse"] else got
    s["now"].copy_(s["start"])
    live = None
    if own:
        from rag_kv_cache_re_gb300 import qcf as Q
        if c["op"] == "fork":
            Q.qcf_pages_fork(s["pool"], s["a"], s["b"])
        elif c["op"] == "resize":
            Q.qcf_pages_resize(s["pool"], s["b"], s["a"])
        else:
            live = Q.qcf_pages_compact(s["pool"])
    elif c["op"] == "compact":
        live = _plain_compact(s)
    else:
        (_plain_fork if c["op"] == "fork" else _plain_resize)(s)
    out = {"refs": s["refs"], "table": s["table"], "kv_len": s["kv_len"], "k": s["k"], "v": s["v"]}
    return out if live is None else dict(out, live=live)


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    if case["op"] not in ("prompt", "chunk") or work(case)["flops"] > 1e12:
        return None   # pages and tables are moved, not computed
    s = prepare(case, seed)
    c, out, r = s["case"], s["out"].double(), 0
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    G = c["Hq"] // c["Hkv"]
    for b, n in enumerate(s["new"]):
        if c["op"] == "prompt":
            K, V = s["k"][r: r + n].double(), s["v"][r: r + n].double()
        else:
            where = [(p, j) for p in s["prefix_pages"].tolist() for j in range(c["page"])][: c["prefix"]]
            where += [(p, j) for p in s["page_table"][b].tolist() for j in range(c["page"])][: s["lens"][b]]
            ids, row = (torch.tensor(x, device=DEV) for x in zip(*where))
            K, V = ((t[ids, :, row] if c["layout"] == "heads" else t[ids, row]).double() for t in (s["k_pages"], s["v_pages"]))
        behind = K.shape[0] - n
        for i in range(0, n, 512):
            at = torch.arange(behind + i, behind + min(n, i + 512), device=DEV)[:, None]
            key = torch.arange(K.shape[0], device=DEV)[None]
            sees = (key <= at) & (key + c["window"] > at) if c["window"] else key <= at
            rows = slice(r + i, r + min(n, i + 512))
            for h in range(c["Hq"]):
                x = torch.einsum("nd,jd->nj", s["q"][rows, h].double(), K[:, h // G]) / math.sqrt(c["D"])
                x = torch.where(sees, x, -math.inf)
                lse[rows, h] = torch.logsumexp(x, -1)
                out[rows, h] = torch.softmax(x, -1) @ V[:, h // G]
        r += n
    return {"o": out, "lse": lse} if c["lse"] else out
