"""Prompt attention, chunk attention and the page operators at the ends of what their documentation allows: as many sequences and
arguments as a call takes, offsets past 32 bits, keys and values of one tensor, pages of the prefix outside the cache."""
import pytest
import torch

import _paged_reference as R
import _prompt_reference as P
from test_pages_gpu import Pool, i32
from test_prompt_gpu import Q, check_packed, clean_status, within  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = "cuda"


# ----------------------------------------------------------------- many sequences, far rows

@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (2, 1, 128)])
def test_packed_8000_prompts(Q, Hq, Hkv, D):  # noqa: F811
    g = torch.Generator().manual_seed(D)
    lens = torch.randint(0, 6, (8000,), generator=g).tolist()
    lens[7000], lens[7999] = 700, 3
    check_packed(Q, lens, Hq, Hkv, D, torch.bfloat16, seed=1, max_len=700, lead=1, pad=1)


@pytest.mark.parametrize("prefix", [0, 600])
def test_chunk_8000_sequences(Q, prefix):  # noqa: F811
    """One page for each, every fifth without new rows, one with many; rows of a few of them against 64 bits, the others against
    the same sequences a hundred to a call."""
    new, lens = [0 if i % 5 == 4 else 1 for i in range(8000)], [i % 16 + 1 for i in range(8000)]
    new[4000], lens[4000] = 200, 300
    bt = R.Batch(new, lens, prefix, 2, 64, 16, "rows", torch.float16, seed=prefix + 1, pad=3).fill()
    q = bt.randn(bt.n_rows, 8, 64)
    cache, batch = bt.bind(Q)
    out, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    spans = list(bt.spans())
    Kp, Vp = (bt.rows(t)[bt.prefix_at()] for t in (bt.k, bt.v))
    for b in [0, 1, 31, 32, 2047, 2048, 3998, 4000, 4001, 7997, 7998]:
        _, r, n = spans[b]
        K, V = (torch.cat([x, bt.rows(t)[bt.own_at(b)]]) for x, t in ((Kp, bt.k), (Vp, bt.v)))
        o, e, tol, ltol = P.attend(q[r: r + n], K, V, prefix + lens[b] - n, 0.1)
        within(out[r: r + n], o, tol, f"sequence {b}")
        within(lse[r: r + n], e, ltol, f"lse of sequence {b}")
    for b in range(0, 8000, 800):
        r0, r1 = spans[b][1], spans[b + 100][1]
        few = Q.PagedBatch((bt.row_start[b: b + 101] - r0).contiguous(), bt.kv_len[b: b + 100].contiguous(), bt.table[b: b + 100].contiguous(), r1 - r0,
                           bt.max_q, bt.max_len, bt.prefix_pages, prefix)
        got = Q.qcf_paged_chunk_attn(cache, few, q[r0:r1], 0.1)
        # each is off by half a step of the weights and half a one of the output, of the largest value at most; a fifth half step
        # is for the logits: 4 ((64 + 8) 2^-24 |logit| + 2^-21) + 2^-17 is less than 2^-11 up to |logit| 25, where these end at 10
        assert (got.double() - out[r0:r1].double()).abs().max() <= 5 * R.half_step(torch.float16) * bt.rows(bt.v).nan_to_num(0).abs().max()


def test_packed_beyond_32_bit_offsets(Q):  # noqa: F811
    """Rows of q, k and v that begin more than 2^31 entries behind the first, and o as large as a call takes (2^24 heads of a row, 4 GB)."""
    n, seqs, Hq, Hkv, D = 1000, 262, 64, 8, 128
    rows = torch.empty((n * seqs, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for part in rows.split(20000):
        part.normal_(generator=g)
    q, k, v = rows.split([Hq, Hkv, Hkv], 1)
    assert rows.numel() > 1 << 31 and q.shape[0] * Hq * D * 2 > (1 << 32) - (1 << 22)
    out, lse = Q.qcf_packed_causal_attn(q, k, v, i32([n * i for i in range(seqs + 1)]), n, 0.08, want_lse=True)
    for b in (0, 130, 260, 261):
        at = slice(b * n, (b + 1) * n)
        o, e, tol, ltol = P.attend(q[at], k[at], v[at], 0, 0.08)
        within(out[at], o, tol, f"sequence {b}")
        within(lse[at], e, ltol, f"lse of sequence {b}")


# ----------------------------------------------------------------- layouts

@pytest.mark.parametrize("D,layout", [(128, "rows"), (64, "heads"), (16, "rows")])
def test_chunk_keys_and_values_of_one_tensor(Q, D, layout):  # noqa: F811
    """Keys and values side by side in each row, or in each page; the same bits as from tensors of their own."""
    bt = R.Batch([70, 1, 1, 200], [300, 90, 17, 260], 600, 2, D, 16, layout, torch.bfloat16, seed=D).fill()
    q = bt.randn(bt.n_rows, 8, D)
    cache, batch = bt.bind(Q)
    both = torch.stack([bt.k, bt.v], 2 if layout == "rows" else 1)
    k, v = both.unbind(2 if layout == "rows" else 1)
    assert not k.is_contiguous()
    assert torch.equal(Q.qcf_paged_chunk_attn(Q.PagedKV(k, v, layout), batch, q, 0.1), Q.qcf_paged_chunk_attn(cache, batch, q, 0.1))


@pytest.mark.parametrize("layout,Hkv,D,page", [("rows", 3, 16, 8), ("rows", 8, 128, 32), ("heads", 2, 64, 16), ("rows", 1, 64, 8)])
def test_pages_of_keys_and_values_of_one_tensor(Q, layout, Hkv, D, page):  # noqa: F811
    """Copies between pages whose rows have gaps: the other tensor's rows, and a head that belongs to neither."""
    n_pages, wide = 40, Hkv + 1
    shape = (n_pages, page, 2, wide, D) if layout == "rows" else (n_pages, 2, wide, page, D)
    g = torch.Generator(device=DEV).manual_seed(page)
    layers = [torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    pick = (lambda t, i: t[:, :, i, :Hkv]) if layout == "rows" else (lambda t, i: t[:, i, :Hkv])
    spare = (lambda t: t[:, :, :, Hkv]) if layout == "rows" else (lambda t: t[:, :, Hkv])
    p = Pool(Q, n_pages, 6, 10, layers=2, Hkv=Hkv, D=D, page=page, layout=layout)
    p.k, p.v = ([pick(t, i) for t in layers] for i in (0, 1))
    p.caches = [Q.PagedKV(k, v, layout) for k, v in zip(p.k, p.v)]
    p.pages = [[t.cpu().clone() for t in store] for store in (p.k, p.v)]
    p.pool = Q.PagePool.empty(p.caches, 6, 10 * page)
    before = [spare(t).clone() for t in layers]
    p.resize([3 * page + 1, 2 * page, page - 1, 0, 0, 0])
    p.fork([0, 0, 2], [3, 4, 5])
    p.check()
    p.resize([2 * page + 3, 0], [3, 1])
    p.compact()
    p.check()
    assert all(torch.equal(a, spare(t)) for a, t in zip(before, layers)), "a head of neither tensor changed"


# ----------------------------------------------------------------- many arguments

def test_thousands_of_arguments(Q):  # noqa: F811
    """More sequences than the plan has threads: growth, forks, a turnover and a bad argument behind the first thousand."""
    S = 2500
    p = Pool(Q, 9000, S, 3, layers=1, Hkv=1, page=8)
    p.resize([i % 17 for i in range(S)])
    p.check()
    src, dst = [i for i in range(S) if i % 2 == 0], [i for i in range(S) if i % 2]
    p.fork(src[::-1], dst)
    p.check()
    order = [(i * 7) % S for i in range(S)]
    p.resize([(p.lens[i] * 5 + i) % 20 for i in order], order)
    p.check()
    p.compact()
    p.check()
    for bad in ([0] * (S - 1) + [25], [0] * 1024 + [-1] + [0] * (S - 1025)):
        Q.qcf_pages_resize(p.pool, i32(bad))
        p.check(2)
    Q.qcf_pages_fork(p.pool, i32(src + [1]), i32(dst + [1]))      # the last one from itself
    p.check(2)
    Q.qcf_pages_fork(p.pool, i32(src), i32(dst[:-1] + [dst[0]]))  # a destination twice
    p.check(2)
    p.resize([0] * S)
    p.check()


# ----------------------------------------------------------------- a prefix with bad pages

@pytest.mark.parametrize("new", [[40, 1, 200], [1] * 20])
def test_bad_pages_of_the_prefix(Q, new):  # noqa: F811
    """Their keys are left out for every row, alone and in a group."""
    lens, prefix = [n + 30 * i for i, n in enumerate(new)], 700
    bt = R.Batch(new, lens, prefix, 2, 128, 16, "rows", torch.bfloat16, seed=len(new)).fill()
    q = bt.randn(bt.n_rows, 8, 128)
    cache, batch = bt.bind(Q)
    was = bt.prefix_pages.clone()
    Kp, Vp = (bt.rows(t)[bt.prefix_at()] for t in (bt.k, bt.v))
    gone = [*range(0, 16), *range(16 * 20, 16 * 21), *range(16 * 43, 700)]
    bt.prefix_pages[0], bt.prefix_pages[20], bt.prefix_pages[43] = -1, bt.k.shape[0], 1 << 30
    out, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    assert Q.qcf_query_status() == 2
    bt.prefix_pages.copy_(was)
    for b, r, n in bt.spans():
        K, V = (torch.cat([x, bt.rows(t)[bt.own_at(b)]]) for x, t in ((Kp, bt.k), (Vp, bt.v)))
        o, e, tol, ltol = P.attend(q[r: r + n], K, V, prefix + lens[b] - n, 0.1, 0, gone)
        within(out[r: r + n], o, tol, f"sequence {b}")
        within(lse[r: r + n], e, ltol, f"lse of sequence {b}")
