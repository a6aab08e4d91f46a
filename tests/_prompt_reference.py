"""Plain 64-bit form of causal attention with a window, for the prompt and chunk attention tests."""
import math

import torch

from _paged_reference import half_step


def attend(q, K, V, first, scale, window=0, gone=()):
    """(o, lse, tolerance of o, of lse) in 64 bits: q [n][Hq][D] at positions first, first + 1, ..; K, V [m][Hkv][D] at
    0, 1, ..; keys at the positions `gone` left out.

    Tolerance of one output entry, with A = sum_j p_j |V_j| over the softmax weights p:
      logits: fp32 sums of D exact products, (D + 8) 2^-24 of the sum of their magnitudes, and
        the exponent's argument and result rounded (2^-21): a relative error d of each weight,
        twice (weight and normaliser): 2 d A
      weights rounded to the type of q before they meet the values: half a step of A, and in fp16
        2^-25 for each weight below 2^-14 of its unit, which is 2^-7 of the largest or less: 2^-32 sum_j |V_j|
      fp32 sums of the weighted values and the merging of partial sums: 2^-18 A
      the output rounded once: half a step of |o|.
    lse: the largest error of a logit, and a logarithm and a sum of it in 32 bits (2^-20 of 1 + |lse|)."""
    n, Hq, D = q.shape
    Hkv, step = K.shape[1], half_step(q.dtype)
    G = Hq // Hkv
    at = first + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(K.shape[0], device=q.device)[None]
    hidden = j > at
    if window:
        hidden = hidden | (j <= at - window)
    for s in gone:
        hidden[:, s] = True
    never = hidden.all(0)[:, None, None]
    K, V = torch.where(never, 0.0, K.double()), torch.where(never, 0.0, V.double())
    o, tol = (torch.empty((n, Hq, D), dtype=torch.float64, device=q.device) for _ in range(2))
    lse, ltol = (torch.empty((n, Hq), dtype=torch.float64, device=q.device) for _ in range(2))
    for h in range(Hq):
        qh, Kh, Vh = q[:, h].double(), K[:, h // G], V[:, h // G]
        x = (scale * qh @ Kh.T).masked_fill(hidden, -math.inf)
        top = (scale * qh.abs() @ Kh.abs().T).masked_fill(hidden, 0.0).amax(-1)
        e = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(e.isinf(), 0.0, e)[:, None])
        A = p @ Vh.abs()
        small = 2.0 ** -32 * Vh.abs().sum(0) if q.dtype == torch.float16 else 0.0
        d = (D + 8) * 2.0 ** -24 * top + 2.0 ** -21
        o[:, h], lse[:, h] = p @ Vh, e
        ltol[:, h] = d + 2.0 ** -20 * (1 + torch.where(e.isinf(), 0.0, e).abs())
        tol[:, h] = (2 * d[:, None] + step + 2.0 ** -18) * A + step * o[:, h].abs() + 2.0 ** -25 + small
    return o, lse, tol, ltol


def batch_attention(bt, q, scale, window=0, gone_own=None):
    """The same for every row of a paged batch (rows of no sequence: NaN).  gone_own: {sequence: own tokens left out}."""
    n, Hq, D = q.shape
    res = [torch.full((n, Hq, D), float("nan"), dtype=torch.float64, device=q.device), None,
           torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device), None]
    res[1], res[3] = torch.full_like(res[0][..., 0], float("nan")), torch.zeros_like(res[2][..., 0])
    Kp, Vp = (bt.rows(t)[bt.prefix_at()] for t in (bt.k, bt.v))
    for b, r, nq in bt.spans():
        if nq:
            K, V = (torch.cat([x, bt.rows(t)[bt.own_at(b)]]) for x, t in ((Kp, bt.k), (Vp, bt.v)))
            gone = [bt.prefix + j for j in (gone_own or {}).get(b, ())]
            for full, part in zip(res, attend(q[r: r + nq], K, V, bt.prefix + bt.lens[b] - nq, scale, window, gone)):
                full[r: r + nq] = part
    return res
