"""Cases of the rotary, paged-cache and shared-prefix attention operators: inputs, plain forms, 64-bit values.

The operators continue a batch of sequences over one retrieved context whose fused K/V is already known:
  rope    positions turned into rotations (both pair layouts, part of a head, scaled frequencies)
  table   cosine and sine tables of scaled frequencies for long contexts
  append  new keys and values of a batch written into a paged cache, the rotation applied on the way
  attn    attention of a batch whose sequences share a prefix in the cache and each have tokens of their own
"""
import math
import random

import numpy as np
import torch

own = False  # False: the plain forms below; True: the framework's operators

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _rope(name, n, heads, of, D, R, pairs, type_, scaling, max_pos, inverse=False):
    return dict(name=name, op="rope", n=n, heads=heads, of=of, D=D, R=R, pairs=pairs, type=type_, scaling=scaling,
                max_pos=max_pos, theta=1e4, inverse=inverse)


def _append(name, seqs, new_lo, new_hi, own_hi, pad, prefix, Hq, Hkv, D, R, pairs, type_, page, layout, ragged):
    return dict(name=name, op="append", seqs=seqs, new_lo=new_lo, new_hi=new_hi, own_hi=own_hi, pad=pad, prefix=prefix, Hq=Hq,
                Hkv=Hkv, D=D, R=R, pairs=pairs, type=type_, page=page, layout=layout, ragged=ragged, scaling="turns", theta=1e4)


def _attn(name, seqs, new_lo, new_hi, own_hi, pad, prefix, Hq, Hkv, D, type_, page, layout, ragged):
    return dict(name=name, op="attn", seqs=seqs, new_lo=new_lo, new_hi=new_hi, own_hi=own_hi, pad=pad, prefix=prefix, Hq=Hq,
                Hkv=Hkv, D=D, type=type_, page=page, layout=layout, ragged=ragged)


def listed():
    return [
        # the q and k heads of one decode step of 16 sequences, read out of the packed q, k, v rows
        _rope("rope_step", 16, 40, 48, 128, 128, "half", "bf16", "none", 8192),
        # a whole 35-chunk request of a 64-head layout, frequencies scaled for a longer context
        _rope("rope_request", 17984, 72, 80, 128, 128, "half", "bf16", "turns", 131072),
        # the tables of one request's positions, half of each head turned, and of a 131072-position context
        dict(name="table_request", op="table", n=8192, R=64, theta=1e4, scaling="linear", first=0),
        dict(name="table_long", op="table", n=131072, R=128, theta=1e4, scaling="index", first=0),
        # one new token of each of 16 sequences
        _append("append_step", 16, 1, 1, 512, 0, 5120, 32, 8, 128, 128, "half", "bf16", 16, "rows", 1),
        # a step that mixes single tokens with new questions of up to 64 tokens, rows padded behind the last sequence
        _append("append_mixed", 64, 1, 64, 700, 37, 5120, 32, 8, 128, 128, "half", "bf16", 16, "rows", 2),
        # a whole 35-chunk context of a 64-head layout brought into pages kept head by head, half of each head turned
        _append("append_context", 1, 17984, 17984, 17984, 0, 0, 64, 8, 128, 64, "neighbours", "f16", 64, "heads", 3),
        # a few answers over a ten-chunk context, one token each: latency
        _attn("attn_step_few", 4, 1, 1, 128, 0, 5120, 32, 8, 128, "bf16", 16, "rows", 4),
        # 64 answers over the same context, one token each, up to 512 tokens of their own
        _attn("attn_step", 64, 1, 1, 512, 0, 5120, 32, 8, 128, "bf16", 16, "rows", 5),
        # 32 answers over a 131072-token context, 64 query heads
        _attn("attn_long", 32, 1, 1, 300, 0, 131072, 64, 8, 128, "bf16", 64, "rows", 6),
        # eight new questions of up to 64 tokens over 16384 tokens, pages kept head by head, rows padded behind the last one
        _attn("attn_questions", 8, 33, 64, 96, 21, 16384, 32, 8, 128, "f16", 32, "heads", 7),
        # no shared prefix: plain paged decoding of very uneven sequences, head dim 64
        _attn("attn_own", 48, 1, 1, 4000, 0, 0, 32, 16, 64, "bf16", 16, "rows", 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "table", "append", "append", "attn", "attn", "attn"])
    type_ = rng.choice(["bf16", "f16"])
    if op == "rope":
        D = rng.choice([16, 64, 80, 128])
        R = rng.choice([D, D, D // 2, D // 4 * 2 - 2])
        kv = rng.choice([1, 4, 8])
        heads = kv * (rng.choice([1, 4, 7, 8]) + 1)
        n = _log(rng, 1, max(1, 17984 * 72 * 128 // (heads * D) // 2))
        return _rope(None, min(n, 60000), heads, heads + rng.choice([0, kv]), D, R, rng.choice(["half", "neighbours"]),
                     rng.choice(["bf16", "f16", "f32"]), rng.choice(["none", "linear", "base", "turns", "index"]), _log(rng, 4096, 131072),
                     rng.random() < 0.3)
    if op == "table":
        return dict(op="table", n=_log(rng, 100, 131072), R=rng.choice([16, 32, 64, 96, 128]), theta=rng.choice([1e4, 5e5]),
                    scaling=rng.choice(["none", "linear", "base", "turns", "index"]), first=rng.choice([0, rng.randrange(100000)]))
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 4, 8])
    Hq = Hkv * rng.choice([1, 4, 7, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    layout = rng.choice(["rows", "heads"])
    seqs = _log(rng, 1, 128)
    prefix = rng.choice([0, _log(rng, 1, 16384), _log(rng, 1, 16384)])
    pad = rng.choice([0, rng.randrange(1, 40)])
    ragged = rng.randrange(1 << 20)
    if op == "append":
        hi = _log(rng, 1, max(1, 8000 // seqs))
        R = rng.choice([D, D // 2])
        return _append(None, seqs, 1, hi, hi + rng.randrange(1, 600), pad, prefix, Hq, Hkv, D, R, rng.choice(["half", "neighbours"]),
                       type_, page, layout, ragged)
    hi = rng.choice([1, 1, _log(rng, 2, max(2, 200 // seqs))])
    return _attn(None, seqs, 1, hi, hi + _log(rng, 1, min(4000, 100000 // seqs)), pad, prefix, Hq, Hkv, D, type_, page, layout, ragged)


def _lengths(c):
    """New and own token counts of every sequence of a case."""
    r = random.Random(c["ragged"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    return new, [r.randint(q, max(q, c["own_hi"])) for q in new]


def work(c):
    if c["op"] == "rope":
        moved = c["n"] * c["heads"] * c["D"] * SIZES[c["type"]]
        return {"bytes": 2 * moved + 4 * c["n"], "flops": 3 * c["n"] * c["heads"] * c["R"]}
    if c["op"] == "table":
        return {"bytes": 4 * c["n"] * c["R"], "flops": 2 * c["n"] * c["R"]}
    new, lens = _lengths(c)
    row = c["Hkv"] * c["D"] * 2
    if c["op"] == "append":
        moved = sum(new) * (2 * row + c["Hq"] * c["D"] * 2)
        return {"bytes": 2 * moved + 4 * sum(-(-n // c["page"]) for n in new) + 8 * len(new),
                "flops": 3 * sum(new) * (c["Hq"] + c["Hkv"]) * c["R"]}
    keys = sum(q * (c["prefix"] + n) - q * (q - 1) // 2 for q, n in zip(new, lens))
    return {"bytes": 2 * sum(new) * c["Hq"] * c["D"] * 2 + 2 * row * (c["prefix"] + sum(lens)),
            "flops": 4 * c["Hq"] * c["D"] * keys}


# ------------------------------------------------------------------ inputs

_SCALING = {  # factor, original length, turns below which a frequency is divided, turns above which it is kept, amplitude
    "none": None, "linear": (8.0, 0, 0.0, 0.0, 1.0), "base": (8.0, 0, 0.0, 0.0, 1.0),
    "turns": (8.0, 8192, 1.0, 4.0, 1.0), "index": (16.0, 8192, 1.0, 32.0, 0.1 * math.log(16.0) + 1.0)}


def _scaling(c):
    from rag_kv_cache_re_gb300 import qcf as Q
    v = _SCALING[c["scaling"]]
    return None if v is None else Q.RopeScaling(c["scaling"], factor=v[0], original=v[1], low=v[2], high=v[3], amplitude=v[4])


def _randn(shape, g, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    c, g = dict(case), torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        rows = _randn((c["n"], c["of"], c["D"]), g, TYPES[c["type"]])
        s["x"] = rows[:, : c["heads"]]
        s["pos"] = torch.randint(0, c["max_pos"], (c["n"],), generator=g, device=DEV, dtype=torch.int32)
        if own:
            from rag_kv_cache_re_gb300 import qcf as Q
            s["table"] = Q.ScaledRopeTable(c["max_pos"], c["R"], c["theta"], DEV, scaling=_scaling(c))
        return s
    if c["op"] == "table":
        c["first"] += seed % 1000
        s["cos"] = torch.empty((c["n"], c["R"] // 2), dtype=torch.float32, device=DEV)
        s["sin"] = torch.empty_like(s["cos"])
        if own:
            s["scaling"] = _scaling(c)
        return s
    new, lens = _lengths(c)
    T, page, Hkv, D = TYPES[c["type"]], c["page"], c["Hkv"], c["D"]
    n_rows = sum(new) + c["pad"]
    own_pages = [-(-n // page) for n in lens]
    n_prefix = -(-c["prefix"] // page)
    n_pages = n_prefix + sum(own_pages) + 3
    shape = (n_pages, page, Hkv, D) if c["layout"] == "rows" else (n_pages, Hkv, page, D)
    s["k_pages"], s["v_pages"] = _randn(shape, g, T), _randn(shape, g, T)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["prefix_pages"] = order[:n_prefix].contiguous()
    wide = max(own_pages)
    count = torch.tensor(own_pages, device=DEV)
    first = n_prefix + torch.cumsum(count, 0) - count
    col = torch.arange(wide, device=DEV)
    s["page_table"] = torch.where(col < count[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], 0).to(torch.int32)
    s["row_start"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["kv_len"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["max_q"], s["max_len"], s["rows"] = max(new), max(lens), sum(new)
    if c["op"] == "append":  # the packed q, k, v rows of the projection before
        rows = _randn((n_rows, c["Hq"] + 2 * Hkv, D), g, T)
        s["q"], s["k"], s["v"] = rows.split([c["Hq"], Hkv, Hkv], 1)
        s["out"] = torch.zeros((n_rows, c["Hq"], D), dtype=T, device=DEV)
    else:
        s["q"] = _randn((n_rows, c["Hq"], D), g, T, 1.5)
        s["out"] = torch.zeros_like(s["q"])
    if own:
        from rag_kv_cache_re_gb300 import qcf as Q
        s["cache"] = Q.PagedKV(s["k_pages"], s["v_pages"], layout=c["layout"])
        s["batch"] = Q.PagedBatch(s["row_start"], s["kv_len"], s["page_table"], n_rows=n_rows, max_q=s["max_q"], max_len=s["max_len"],
                                  prefix_pages=s["prefix_pages"], prefix_len=c["prefix"])
        if c["op"] == "append":
            s["table"] = Q.ScaledRopeTable(c["prefix"] + s["max_len"], c["R"], c["theta"], DEV, scaling=_scaling(c))
    return s


# ------------------------------------------------------------------ plain forms

def _frequencies(c):
    """Angles per position of every pair, 64 bits, and the factor on cosine and sine."""
    k = torch.arange(c["R"] // 2, device=DEV, dtype=torch.float64)
    w = c["theta"] ** (-2.0 * k / c["R"])
    if c["scaling"] == "none":
        return w, 1.0
    factor, original, low, high, amplitude = _SCALING[c["scaling"]]
    if c["scaling"] == "linear":
        return w / factor, amplitude
    if c["scaling"] == "base":
        return (c["theta"] * factor ** (c["R"] / (c["R"] - 2))) ** (-2.0 * k / c["R"]), amplitude
    if c["scaling"] == "turns":
        keep = ((original * w / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    else:
        at = [c["R"] * math.log(original / (2 * math.pi * t)) / (2 * math.log(c["theta"])) for t in (high, low)]
        a, b = max(0, math.floor(at[0])), min(c["R"] // 2 - 1, math.ceil(at[1]))
        keep = 1 - ((k - a) / max(b - a, 1e-3)).clamp(0, 1)
    return w * (keep + (1 - keep) / factor), amplitude


def _cos_sin(c, pos):
    w, amplitude = _frequencies(c)
    angle = pos.double()[:, None] * w
    return (angle.cos() * amplitude).float(), (angle.sin() * amplitude).float()


def _turn(x, cos, sin, pairs):
    """x [n][H][D] in 32 bits, the first R entries of each head turned; cos and sin [n][R/2]."""
    R = 2 * cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = x[..., : R // 2], x[..., R // 2: R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., R:]], -1)


def _places(s):
    """Sequence and own position of every row of the batch."""
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(s["row_start"].long(), row, right=True) - 1
    return seq, s["kv_len"][seq].long() - s["row_start"][seq + 1].long() + row


def _rows(pages, layout):
    """The pages as [page][row][head][D]."""
    return pages if layout == "rows" else pages.transpose(1, 2)


def _plain_append(s):
    c, n = s["case"], s["rows"]
    seq, pos = _places(s)
    cos, sin = _cos_sin(c, c["prefix"] + pos)
    where = s["page_table"][seq, pos // c["page"]].long(), pos % c["page"]
    _rows(s["k_pages"], c["layout"])[where] = _turn(s["k"][:n].float(), cos, sin, c["pairs"]).to(s["k"].dtype)
    _rows(s["v_pages"], c["layout"])[where] = s["v"][:n]
    s["out"][:n] = _turn(s["q"][:n].float(), cos, sin, c["pairs"]).to(s["q"].dtype)
    return {"k": s["k_pages"], "v": s["v_pages"], "q": s["out"]}


def _plain_attn(s):
    c, n = s["case"], s["rows"]
    Hq, D = s["q"].shape[1:]
    Hkv, B, Q, L, scale = c["Hkv"], c["seqs"], s["max_q"], s["max_len"], 1.0 / math.sqrt(c["D"])
    G = Hq // Hkv
    q = s["q"][:n].float()
    kp, vp = _rows(s["k_pages"], c["layout"]), _rows(s["v_pages"], c["layout"])
    # the shared part: every row against the prefix
    shared = s["prefix_pages"].long()
    K, V = kp[shared].flatten(0, 1)[: c["prefix"]].float(), vp[shared].flatten(0, 1)[: c["prefix"]].float()
    rows = q.view(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
    x = scale * rows @ K.permute(1, 2, 0)                                    # [Hkv][n G][prefix]
    top = x.amax(-1) if c["prefix"] else torch.full((Hkv, n * G), -math.inf, device=DEV)
    top = top.view(Hkv, n, G).transpose(0, 1)                                # [n][Hkv][G]
    # the own part: rows laid out [B][Q], each against its sequence's own keys
    new = (s["row_start"][1:] - s["row_start"][:-1]).long()
    i = torch.arange(Q, device=DEV)
    row = torch.where(i < new[:, None], s["row_start"][:-1].long()[:, None] + i, n)   # n: a row behind the last
    j = torch.arange(L, device=DEV)
    keys = s["page_table"].long()[:, j // c["page"]], (j % c["page"]).expand(B, L)
    Ko, Vo = kp[keys].float(), vp[keys].float()                              # [B][L][Hkv][D]
    last = s["kv_len"].long()[:, None] - new[:, None] + i                    # own position of each row
    hidden = (j > last[:, :, None])[:, None, :, None]                        # [B][1][Q][1][L]
    qo = torch.cat([q, q.new_zeros(1, Hq, D)])[row].view(B, Q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, Q * G, D)
    y = (scale * qo @ Ko.permute(0, 2, 3, 1)).view(B, Hkv, Q, G, L).masked_fill(hidden, -math.inf)
    # one softmax over both
    both = torch.maximum(torch.cat([top, top.new_zeros(1, Hkv, G)])[row].transpose(1, 2), y.amax(-1))
    y = (y - both[..., None]).exp()
    acc, total = (y.view(B, Hkv, Q * G, L) @ Vo.transpose(1, 2)).view(B, Hkv, Q, G, D), y.sum(-1)

    def back(t):
        return t.new_zeros((n + 1, Hkv, G) + t.shape[4:]).index_put((row,), t.transpose(1, 2))[:n]

    acc, total, both = back(acc), back(total), back(both)                    # [n][Hkv][G]..
    x = (x - both.transpose(0, 1).reshape(Hkv, n * G, 1)).exp()
    acc = acc + (x @ V.transpose(0, 1)).view(Hkv, n, G, D).transpose(0, 1)
    total = total + x.sum(-1).view(Hkv, n, G).transpose(0, 1)
    s["out"][:n] = (acc / total[..., None]).view(n, Hq, D).to(s["q"].dtype)
    return s["out"]


def run(s):
    c = s["case"]
    if own:
        from rag_kv_cache_re_gb300 import qcf as Q
        if c["op"] == "rope":
            return Q.qcf_rope_apply(s["x"], s["pos"], s["table"], interleaved=c["pairs"] != "half", inverse=c["inverse"])
        if c["op"] == "table":
            Q.qcf_rope_table_fill(s["cos"], s["sin"], c["theta"], first_pos=c["first"], scaling=s["scaling"])
            return {"cos": s["cos"], "sin": s["sin"]}
        if c["op"] == "append":
            q = Q.qcf_paged_append(s["cache"], s["batch"], s["k"], s["v"], table=s["table"], interleaved=c["pairs"] != "half", q=s["q"],
                                   q_out=s["out"])
            return {"k": s["k_pages"], "v": s["v_pages"], "q": q}
        return Q.qcf_shared_prefix_attn(s["cache"], s["batch"], s["q"], 1.0 / math.sqrt(c["D"]), out=s["out"])
    if c["op"] == "rope":
        cos, sin = _cos_sin(c, s["pos"])
        return _turn(s["x"].float(), cos, -sin if c["inverse"] else sin, c["pairs"]).to(s["x"].dtype)
    if c["op"] == "table":
        cos, sin = _cos_sin(c, torch.arange(c["first"], c["first"] + c["n"], device=DEV))
        return {"cos": cos, "sin": sin}
    return _plain_append(s) if c["op"] == "append" else _plain_attn(s)


# ------------------------------------------------------------------ 64 bits, from the definitions

def _exact_rates(c):
    """Radians per position of pair 0, 1, .. and the amplitude, one by one."""
    R, theta = c["R"], c["theta"]
    kind = c["scaling"]
    factor, original, low, high, amplitude = _SCALING[kind] or (1.0, 1, 0.0, 0.0, 1.0)
    if kind == "base":
        theta *= math.pow(factor, R / (R - 2.0))
    rates = []
    for k in range(R // 2):
        w = math.exp(-2.0 * k / R * math.log(theta))
        if kind == "linear":
            w /= factor
        elif kind == "turns":
            turns = original * w / math.tau
            if turns < low:
                w /= factor
            elif turns <= high:
                u = (turns - low) / (high - low)
                w = (1 - u) * w / factor + u * w
        elif kind == "index":
            bound = [math.log(original / (math.tau * t), theta) * R / 2 for t in (high, low)]
            first, last = max(math.floor(bound[0]), 0), min(math.ceil(bound[1]), R // 2 - 1)
            u = min(max((k - first) / max(last - first, 1e-3), 0.0), 1.0)
            w = u * w / factor + (1 - u) * w
        rates.append(w)
    return rates, amplitude


def _exact_turn(x, pos, c, sign=1.0):
    """x [n][H][D]: its pairs as complex numbers, times amplitude * exp(i p w)."""
    rates, amplitude = _exact_rates(c)
    R = c["R"]
    angle = sign * pos.double()[:, None] * torch.tensor(rates, dtype=torch.float64, device=x.device)
    unit = torch.polar(torch.full_like(angle, amplitude), angle)[:, None]
    y = x.double().clone()
    where = (slice(0, R // 2), slice(R // 2, R)) if c["pairs"] == "half" else (slice(0, R, 2), slice(1, R, 2))
    z = torch.complex(y[..., where[0]], y[..., where[1]]) * unit
    y[..., where[0]], y[..., where[1]] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _exact_turn(s["x"], s["pos"], c, -1.0 if c["inverse"] else 1.0)
    if c["op"] == "table":
        rates, amplitude = _exact_rates(c)
        angle = np.outer(np.arange(c["first"], c["first"] + c["n"], dtype=np.float64), np.array(rates))
        return {"cos": amplitude * np.cos(angle), "sin": amplitude * np.sin(angle)}
    new, lens = _lengths(c)
    page, heads = c["page"], c["layout"] == "heads"
    table = s["page_table"].cpu().tolist()
    if c["op"] == "append":
        k, v, q = s["k_pages"].double(), s["v_pages"].double(), s["out"].double()
        r = 0
        for b in range(len(new)):
            p = torch.arange(lens[b] - new[b], lens[b], device=DEV)
            ids = torch.tensor(table[b], device=DEV)[p // page]
            kr = _exact_turn(s["k"][r: r + new[b]], p + c["prefix"], c)
            vr = s["v"][r: r + new[b]].double()
            q[r: r + new[b]] = _exact_turn(s["q"][r: r + new[b]], p + c["prefix"], c)
            if heads:
                k[ids, :, p % page], v[ids, :, p % page] = kr, vr
            else:
                k[ids, p % page], v[ids, p % page] = kr, vr
            r += new[b]
        return {"k": k, "v": v, "q": q}
    if work(c)["flops"] > 1e12:
        return None
    flat = [(t.transpose(1, 2) if heads else t).double() for t in (s["k_pages"], s["v_pages"])]
    pre = [t[s["prefix_pages"].long()].flatten(0, 1)[: c["prefix"]] for t in flat]
    out, r = s["out"].double(), 0
    for b in range(len(new)):
        mine = torch.tensor(table[b][: -(-lens[b] // page)], device=DEV)
        K, V = (torch.cat([p, t[mine].flatten(0, 1)[: lens[b]]]) for p, t in zip(pre, flat))
        limit = c["prefix"] + torch.arange(lens[b] - new[b], lens[b], device=DEV)
        hidden = torch.arange(K.shape[0], device=DEV) > limit[:, None]
        for h in range(c["Hkv"]):
            G = c["Hq"] // c["Hkv"]
            qh = s["q"][r: r + new[b], h * G: (h + 1) * G].double()
            logits = torch.einsum("ngd,jd->gnj", qh, K[:, h]) / math.sqrt(c["D"])
            p = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
            out[r: r + new[b], h * G: (h + 1) * G] = torch.einsum("gnj,jd->ngd", p, V[:, h])
        r += new[b]
    return out
