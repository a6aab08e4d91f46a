"""Prompts, their pages and what goes on from them, as a serving program uses the operators together: packed prompts, pages
taken and filled, chunks of further tokens, answers forked from one sequence, single tokens, sequences that end, the cache made dense."""
import pytest
import torch

import _prompt_reference as P

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def Q():
    from rag_kv_cache_re_gb300 import qcf
    return qcf


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


class Serving:
    """Two layers' caches, one pool, and on the side every sequence's keys and values as they were when they came."""

    def __init__(self, Q, n_seq, n_pages, page, layout, Hq, Hkv, D, dtype, max_len):
        self.Q, self.page, self.layout, self.Hq, self.Hkv, self.D, self.dtype = Q, page, layout, Hq, Hkv, D, dtype
        self.g = torch.Generator(device=DEV).manual_seed(D + page)
        shape = (n_pages, page, Hkv, D) if layout == "rows" else (n_pages, Hkv, page, D)
        self.caches = [Q.PagedKV(*(torch.full(shape, float("nan"), dtype=dtype, device=DEV) for _ in range(2)), layout) for _ in range(2)]
        self.pool = Q.PagePool.empty(self.caches, n_seq, max_len)
        self.table = Q.ScaledRopeTable(max_len, D, 1e4, DEV)
        self.lens = [0] * n_seq
        self.past = [[(torch.zeros((0, Hkv, D), dtype=dtype, device=DEV),) * 2 for _ in range(n_seq)] for _ in range(2)]
        self.max_len, self.scale = max_len, D ** -0.5

    def rows(self, n):
        r = (torch.randn((n, self.Hq + 2 * self.Hkv, self.D), generator=self.g, device=DEV) * 1.2).to(self.dtype)
        return r.split([self.Hq, self.Hkv, self.Hkv], 1)

    def batch(self, seqs, new):
        """The batch of these sequences: their rows of the table side by side, as the pool holds them now."""
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        at = i32(seqs).long()
        return self.Q.PagedBatch(i32(start), self.pool.kv_len[at].contiguous(), self.pool.page_table[at].contiguous(), n_rows=start[-1], max_q=max(new),
                                 max_len=self.max_len)

    def take(self, seqs, new):
        for s, n in zip(seqs, new):
            self.lens[s] += n
        self.Q.qcf_pages_resize(self.pool, i32([self.lens[s] for s in seqs]), i32(seqs))

    def step(self, seqs, new, whole=False):
        """New tokens of some sequences through both layers; with `whole`, their packed attention as prompts too."""
        Q = self.Q
        self.take(seqs, new)
        batch = self.batch(seqs, new)
        for layer, cache in enumerate(self.caches):
            q, k, v = self.rows(sum(new))
            rq = Q.qcf_paged_append(cache, batch, k, v, self.table, q=q)
            out, lse = Q.qcf_paged_chunk_attn(cache, batch, rq, self.scale, want_lse=True)
            short = Q.qcf_shared_prefix_attn(cache, batch, rq, self.scale)
            r = 0
            pages = [c if self.layout == "rows" else c.transpose(1, 2) for c in (cache.k, cache.v)]
            for s, n in zip(seqs, new):
                p = torch.arange(self.lens[s] - n, self.lens[s], device=DEV)
                where = self.pool.page_table[s].long()[p // self.page], p % self.page
                self.past[layer][s] = tuple(torch.cat([old, new[where]]) for old, new in zip(self.past[layer][s], pages))
                K, V = self.past[layer][s]
                assert torch.equal(V[-n:], v[r: r + n])
                o, e, tol, ltol = P.attend(rq[r: r + n], K, V, self.lens[s] - n, self.scale)
                for got, ref, t in ((out, o, tol), (lse, e, ltol), (short, o, tol)):
                    assert torch.all((got[r: r + n].double() - ref).abs() <= t), f"layer {layer}, sequence {s}"
                r += n
            if whole:
                pos = torch.cat([torch.arange(n, device=DEV, dtype=torch.int32) for n in new])
                rk = Q.qcf_rope_apply(k, pos, self.table)
                packed = Q.qcf_packed_causal_attn(rq, rk, v.contiguous(), batch.row_start, max(new), self.scale)
                r = 0
                for s, n in zip(seqs, new):
                    K, V = self.past[layer][s]
                    o, _, tol, _ = P.attend(rq[r: r + n], rk[r: r + n], V, 0, self.scale)
                    assert torch.all((packed[r: r + n].double() - o).abs() <= tol), f"packed, sequence {s}"
                    r += n

    def fork(self, src, dst):
        self.Q.qcf_pages_fork(self.pool, i32(src), i32(dst))
        for s, d in zip(src, dst):
            self.lens[d] = self.lens[s]
            for layer in range(2):
                self.past[layer][d] = self.past[layer][s]

    def cut(self, seqs, to):
        self.Q.qcf_pages_resize(self.pool, i32(to), i32(seqs))
        for s, n in zip(seqs, to):
            self.lens[s] = n
            for layer in range(2):
                self.past[layer][s] = tuple(t[:n] for t in self.past[layer][s])

    def settled(self):
        assert self.Q.qcf_query_status() == 0 and self.pool.kv_len.tolist() == self.lens
        count = [0] * self.pool.refs.numel()
        for s, n in enumerate(self.lens):
            for p in self.pool.page_table[s, : -(-n // self.page)].tolist():
                count[p] += 1
        assert count == self.pool.refs.tolist()


@pytest.mark.parametrize("page,layout,Hq,Hkv,D,dtype", [
    (16, "rows", 8, 2, 128, torch.bfloat16), (64, "heads", 4, 4, 64, torch.float16), (8, "heads", 7, 1, 128, torch.bfloat16), (32, "rows", 4, 2, 16, torch.float16)])
def test_a_cache_through_its_life(Q, page, layout, Hq, Hkv, D, dtype):
    Q.qcf_query_status()
    s = Serving(Q, 9, 6000 // page, page, layout, Hq, Hkv, D, dtype, 1024)
    s.step([0, 1, 2], [300, 45, 513], whole=True)       # prompts
    s.settled()
    s.step([2, 0], [200, 70])                           # chunks of further tokens
    s.fork([0, 0, 0, 2], [3, 4, 5, 6])                  # answers to the first, another way on from the third
    s.settled()
    for _ in range(3):                                  # single tokens, each sequence its own
        s.step([3, 4, 5, 6, 1, 2], [1] * 6)
    s.settled()
    s.cut([4, 5], [365, 100])                           # one answer takes back its last tokens, one goes back into the prompt
    s.step([4, 5, 3], [1, 6, 1])
    s.cut([1, 2], [0, 0])                               # two end
    s.settled()
    live = int(Q.qcf_pages_compact(s.pool))
    assert live == sum(r > 0 for r in s.pool.refs.tolist()) and s.pool.refs[live:].sum() == 0
    s.settled()
    s.step([6, 3, 0, 4, 5], [33, 1, 2, 1, 1])           # the others go on from where their pages are now
    s.step([7, 8, 6], [130, 1, 1])                      # and new ones come into the pages of those that ended
    s.settled()
