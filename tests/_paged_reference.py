"""Plain 64-bit forms of the rotary, paged-append and shared-prefix attention operators, and
the batches their tests run on."""
import math

import torch

DEV = "cuda"


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ----------------------------------------------------------------- rotation

def rates(R, theta, kind="none", factor=1.0, original=0, low=0.0, high=0.0):
    """Radians per position of each pair, as the header's formulas read."""
    if kind == "base":
        theta = theta * factor ** (R / (R - 2))
    w = [theta ** (-2.0 * k / R) for k in range(R // 2)]
    if kind == "linear":
        w = [v / factor for v in w]
    if kind == "turns":
        g = [min(1.0, max(0.0, (original * v / (2 * math.pi) - low) / (high - low))) for v in w]
        w = [v * (x + (1 - x) / factor) for v, x in zip(w, g)]
    if kind == "index":
        at = [R * math.log(original / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (high, low)]
        a, b = max(0, math.floor(at[0])), min(R // 2 - 1, math.ceil(at[1]))
        g = [1 - min(1.0, max(0.0, (k - a) / max(b - a, 1e-3))) for k in range(R // 2)]
        w = [v * (x + (1 - x) / factor) for v, x in zip(w, g)]
    return torch.tensor(w, dtype=torch.float64)


def rotate(x, pos, w, interleaved=False, amplitude=1.0):
    """(x rotated, |a| + |b| of every entry's pair) in 64 bits; x [n][H][D], pos [n], w [R/2]."""
    R = 2 * w.numel()
    angle = pos.double()[:, None, None] * w.to(x.device)
    c, s = amplitude * angle.cos(), amplitude * angle.sin()
    y, mag = x.double().clone(), x.double().abs()
    ia, ib = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def rotation_tolerance(y, mag, dtype, amplitude=1.0):
    """Cosine and sine rounded to 32 bits (2^-24 relative), one rounding per product and one of the
    sum: 3 * 2^-24 * amplitude * (|a| + |b|), taken as 4; then one rounding to dtype (half a step,
    2^-25 below fp16's normal range)."""
    return half_step(dtype) * y.abs() + 4 * 2.0 ** -24 * max(1.0, amplitude) * mag + (2.0 ** -25 if dtype == torch.float16 else 1e-40)


# ----------------------------------------------------------------- batches

class Batch:
    """A paged batch with random pages.  Slots that hold no token are filled with `junk`."""

    def __init__(self, new, lens, prefix, Hkv, D, page, layout, dtype, seed, pad=0, lead=0, junk=float("nan"), spare=3,
                 table_cols=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g, self.new, self.lens, self.prefix, self.page, self.layout, self.dtype = g, new, lens, prefix, page, layout, dtype
        self.Hkv, self.D = Hkv, D
        own = [-(-n // page) for n in lens]
        n_prefix = -(-prefix // page)
        n_pages = n_prefix + sum(own) + spare
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        cols = table_cols or max(own + [1])
        self.table = torch.zeros((len(new), cols), dtype=torch.int32, device=DEV)
        at = n_prefix
        for b, n in enumerate(own):
            self.table[b, :n] = order[at: at + n]
            at += n
        self.prefix_pages = order[:n_prefix].contiguous() if n_prefix else None
        shape = (n_pages, page, Hkv, D) if layout == "rows" else (n_pages, Hkv, page, D)
        self.k = torch.full(shape, junk, dtype=dtype, device=DEV)
        self.v = torch.full(shape, junk, dtype=dtype, device=DEV)
        self.row_start = torch.tensor([lead] + [lead + sum(new[: i + 1]) for i in range(len(new))], dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.n_rows = lead + sum(new) + pad
        self.max_q, self.max_len = max(new + [0]), max(lens + [0])

    def randn(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.g, device=DEV) * std).to(self.dtype)

    def rows(self, pages):
        return pages if self.layout == "rows" else pages.transpose(1, 2)

    def own_at(self, b, n=None):
        """(page, row) of the own tokens 0 .. n - 1 of sequence b."""
        p = torch.arange(self.lens[b] if n is None else n, device=DEV)
        return self.table[b].long()[p // self.page], p % self.page

    def prefix_at(self):
        p = torch.arange(self.prefix, device=DEV)
        return (self.prefix_pages.long()[p // self.page], p % self.page) if self.prefix else (p, p)

    def fill(self, std_k=1.0, std_v=1.0):
        """Random keys and values in every slot that holds a token."""
        for where in [self.prefix_at()] + [self.own_at(b) for b in range(len(self.new))]:
            n = where[0].numel()
            self.rows(self.k)[where] = self.randn(n, self.Hkv, self.D, std=std_k)
            self.rows(self.v)[where] = self.randn(n, self.Hkv, self.D, std=std_v)
        return self

    def bind(self, Q, **over):
        kw = dict(n_rows=self.n_rows, max_q=self.max_q, max_len=self.max_len, prefix_pages=self.prefix_pages, prefix_len=self.prefix)
        kw.update(over)
        return Q.PagedKV(self.k, self.v, self.layout), Q.PagedBatch(self.row_start, self.kv_len, self.table, **kw)

    def spans(self):
        r = int(self.row_start[0])
        for b, n in enumerate(self.new):
            yield b, r, n
            r += n


# ----------------------------------------------------------------- attention

def attention(bt, q, scale, skip_prefix=()):
    """(o, lse, tolerance of o, of lse) in 64 bits for every row of a batch; rows of no sequence stay NaN.
    skip_prefix: prefix tokens left out.

    Tolerance of one output entry, with A = sum_j p_j |V_j| over the softmax weights p:
      logits: fp32 sums of D exact products, (D + 8) 2^-24 of the sum of their magnitudes, and
        the exponent's argument and result rounded (2^-21): a relative error d of each weight,
        twice (weight and normaliser): 2 d A
      weights rounded to the cache's type before they meet the values: half a step of A, and in fp16
        2^-25 for each weight below 2^-14 of its unit, which is 2^-7 of the largest or less: 2^-32 sum_j |V_j|
      fp32 sums of the weighted values and the merging of partial sums: 2^-18 A
      the output rounded once: half a step of |o|.
    lse: the largest error of a logit, and a logarithm and a sum of it in 32 bits (2^-20 of 1 + |lse|)."""
    n, Hq, D = q.shape
    G = Hq // bt.Hkv
    o = torch.full((n, Hq, D), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), float("nan"), dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
    at = bt.prefix_at()
    Kp, Vp = bt.rows(bt.k)[at].double(), bt.rows(bt.v)[at].double()
    step = half_step(bt.dtype)
    for b, r, nq in bt.spans():
        if nq == 0:
            continue
        own = bt.own_at(b)
        K, V = torch.cat([Kp, bt.rows(bt.k)[own].double()]), torch.cat([Vp, bt.rows(bt.v)[own].double()])
        j = torch.arange(K.shape[0], device=q.device)
        hidden = j > (bt.prefix + bt.lens[b] - nq + torch.arange(nq, device=q.device))[:, None]
        for s in skip_prefix:
            hidden[:, s] = True
        K, V = torch.where(hidden.all(0)[:, None, None], 0.0, K), torch.where(hidden.all(0)[:, None, None], 0.0, V)
        for h in range(bt.Hkv):
            qh = q[r: r + nq, h * G: (h + 1) * G].double()
            x = (scale * torch.einsum("ngd,jd->gnj", qh, K[:, h])).masked_fill(hidden, -math.inf)
            top = scale * torch.einsum("ngd,jd->gnj", qh.abs(), K[:, h].abs()).masked_fill(hidden, 0.0).amax(-1)
            e = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(e.isinf(), 0.0, e)[..., None])
            oh = torch.einsum("gnj,jd->ngd", p, V[:, h])
            A = torch.einsum("gnj,jd->ngd", p, V[:, h].abs())
            small = 2.0 ** -32 * V[:, h].abs().sum(0) if bt.dtype == torch.float16 else 0.0
            d = ((D + 8) * 2.0 ** -24 * top + 2.0 ** -21).transpose(0, 1)[..., None]
            o[r: r + nq, h * G: (h + 1) * G] = oh
            lse[r: r + nq, h * G: (h + 1) * G] = e.transpose(0, 1)
            ltol[r: r + nq, h * G: (h + 1) * G] = d[..., 0] + 2.0 ** -20 * (1 + e.transpose(0, 1).abs())
            tol[r: r + nq, h * G: (h + 1) * G] = (2 * d + step + 2.0 ** -18) * A + step * oh.abs() + 2.0 ** -25 + small
    return o, lse, tol, ltol
