"""The page operators on the GPU against plain lists on the host."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAD_INDEX, NO_PAGES = 2, 4


@pytest.fixture(scope="module")
def Q():
    from rag_kv_cache_re_gb300 import qcf
    return qcf


@pytest.fixture(autouse=True)
def clean_status(Q):
    Q.qcf_query_status()
    yield
    assert Q.qcf_query_status() == 0, "a device-side check failed"


class Pool:
    """A pool with random pages in every layer, and the same on the host: refs, table rows, lengths, pages."""

    def __init__(self, Q, n_pages, n_seq, cols, layers=2, Hkv=2, D=16, page=8, layout="rows", dtype=torch.bfloat16, seed=0, gap=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        shape = (n_pages, page, Hkv, D) if layout == "rows" else (n_pages, Hkv, page, D)
        self.k, self.v = ([], [])
        for store in (self.k, self.v):
            for _ in range(layers):
                t = torch.randn((n_pages, page * Hkv * D + gap), generator=g, device=DEV).to(dtype)
                store.append(t[:, : page * Hkv * D].view(shape) if not gap else t.as_strided(shape, (page * Hkv * D + gap, *self._strides(shape))))
        self.caches = [Q.PagedKV(k, v, layout) for k, v in zip(self.k, self.v)]
        self.Q, self.page, self.layout, self.cols = Q, page, layout, cols
        self.refs, self.lens, self.rows = [0] * n_pages, [0] * n_seq, [[] for _ in range(n_seq)]
        self.pages = [[t.cpu().clone() for t in store] for store in (self.k, self.v)]
        self.pool = Q.PagePool.empty(self.caches, n_seq, cols * page)
        self.pool.page_table.fill_(-7)   # what is behind a row's pages has no meaning

    @staticmethod
    def _strides(shape):
        return (shape[2] * shape[3], shape[3], 1)

    def per(self, t):
        return t if self.layout == "rows" else t.transpose(1, 2)

    def held(self, n):
        return -(-n // self.page)

    def copy(self, src, dst, rows):
        for store in self.pages:
            for t in store:
                self.per(t)[dst, :rows] = self.per(t)[src, :rows]

    def fork(self, src, dst):
        free = iter([i for i, r in enumerate(self.refs) if r == 0])
        old = [list(r) for r in self.rows]
        for s, d in zip(src, dst):
            for p in old[d]:
                self.refs[p] -= 1
            rest = self.lens[s] % self.page
            row = old[s][: self.lens[s] // self.page]
            for p in row:
                self.refs[p] += 1
            if rest:
                new = next(free)
                self.copy(old[s][-1], new, rest)
                self.refs[new] = 1
                row = row + [new]
            self.rows[d], self.lens[d] = row, self.lens[s]
        self.Q.qcf_pages_fork(self.pool, i32(src), i32(dst))

    def resize(self, to, seqs=None):
        before = list(self.refs)
        free = iter([i for i, r in enumerate(self.refs) if r == 0])
        for s, n in zip(range(len(self.lens)) if seqs is None else seqs, to):
            row, now = self.rows[s], self.lens[s]
            kept = min(now, n)
            if now != n and kept % self.page and before[row[kept // self.page]] > 1:
                new = next(free)
                self.copy(row[kept // self.page], new, kept % self.page)
                self.refs[row[kept // self.page]] -= 1
                self.refs[new] += 1
                row[kept // self.page] = new
            for p in row[self.held(n):]:
                self.refs[p] -= 1
            del row[self.held(n):]
            while len(row) < self.held(n):
                row.append(next(free))
                self.refs[row[-1]] += 1
            self.lens[s] = n
        self.Q.qcf_pages_resize(self.pool, i32(to), None if seqs is None else i32(seqs))

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        move = dict(zip([i for i, r in enumerate(self.refs) if r > 0 and i >= live], [i for i, r in enumerate(self.refs) if r == 0 and i < live]))
        for a, b in move.items():
            self.copy(a, b, self.page)
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[move.get(p, p) for p in row] for row in self.rows]
        assert int(self.Q.qcf_pages_compact(self.pool)) == live

    def check(self, status=0):
        assert self.Q.qcf_query_status() == status
        assert self.pool.refs.tolist() == self.refs and self.pool.kv_len.tolist() == self.lens
        table = self.pool.page_table.tolist()
        for got, row in zip(table, self.rows):
            assert got[: len(row)] == row
        for mine, theirs in zip(self.pages, (self.k, self.v)):
            for a, b in zip(mine, theirs):
                assert torch.equal(a.contiguous().view(torch.int16), b.cpu().contiguous().view(torch.int16)), "the pages differ"
        assert all(p >= 0 for row in self.rows for p in row)


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


LAYOUTS = [dict(), dict(layout="heads", page=16, D=64), dict(page=32, Hkv=3, D=128, layers=1, dtype=torch.float16), dict(layout="heads", Hkv=5, gap=24, layers=3),
           dict(gap=8, Hkv=1, page=64), dict(page=256, D=64, layers=1, Hkv=8)]


@pytest.mark.parametrize("kw", LAYOUTS)
def test_a_life_of_a_pool(Q, kw):
    """Random calls one after the other: every count, table, length and page as on the host."""
    r = random.Random(len(str(kw)))
    p = Pool(Q, 120, 12, 9, seed=3, **kw)
    p.check()
    p.resize([r.randint(0, 3 * p.page) for _ in range(12)])
    p.check()
    for step in range(12):
        kind = r.choice(["fork", "resize", "resize", "compact"])
        if kind == "fork":
            dst = r.sample(range(12), r.randint(1, 5))
            src = [r.choice([s for s in range(12) if s not in dst]) for _ in dst]
            p.fork(src, dst)
        elif kind == "resize":
            seqs = r.sample(range(12), r.randint(1, 12))
            p.resize([r.choice([0, p.lens[s], p.lens[s] + 1 if p.lens[s] < 4 * p.page else 0, r.randint(0, 4 * p.page)]) for s in seqs], seqs)
        else:
            p.compact()
        p.check()
    p.compact()
    p.check()


def test_growth_and_forks_one_token_at_a_time(Q):
    p = Pool(Q, 40, 4, 8, page=8)
    for n in range(1, 20):
        p.resize([n, 0, 0, 0])
    p.check()
    p.fork([0, 0], [1, 2])                       # 16 tokens shared, three copied twice
    p.check()
    assert p.refs[p.rows[0][0]] == 3 and len({row[2] for row in p.rows[:3]}) == 3
    p.resize([10, 10], [1, 2])                   # both cut back into a shared page: each gets its own
    p.check()
    assert len({row[1] for row in p.rows[:3]}) == 3
    p.resize([24], [0])
    p.fork([0], [3])                             # a whole number of pages: nothing to copy
    p.check()
    p.resize([8], [3])                           # cut back to a whole page: nothing to copy either
    p.check()
    assert p.rows[3] == p.rows[0][:1]
    p.fork([1], [3])                             # onto a sequence that holds pages
    p.check()
    p.resize([0, 0, 0, 0])
    p.check()
    assert not any(p.refs)


@pytest.mark.parametrize("n_pages", [1, 15, 16, 17, 16383, 16384, 16385, 50000])
def test_pools_of_many_pages(Q, n_pages):
    """Free pages behind many passes of the search, all pages taken, moves from end to end."""
    p = Pool(Q, n_pages, 6, n_pages, layers=1, Hkv=1, page=8)
    a = n_pages // 3
    p.resize([8 * a, 8 * a, 8 * (n_pages - 2 * a), 0, 0, 0])
    p.check()
    assert all(p.refs)
    p.resize([0], [0])
    p.compact()
    p.check()
    p.resize([0, 8 * a], [1, 4])
    p.check()
    p.compact()
    p.check()


def test_too_few_pages_change_nothing(Q):
    p = Pool(Q, 20, 5, 20, page=8)
    p.resize([80, 60, 10, 0, 0])                 # 10 + 8 + 2
    p.check()
    for call in (lambda: Q.qcf_pages_resize(p.pool, i32([88, 0]), i32([0, 1])),          # what is given back serves the next call
                 lambda: Q.qcf_pages_resize(p.pool, i32([1]), i32([3])), lambda: Q.qcf_pages_fork(p.pool, i32([1]), i32([3]))):
        call()
        p.check(NO_PAGES)
    p.resize([0], [1])
    p.resize([88], [0])
    p.fork([2], [3])
    p.check()


def test_bad_arguments_change_nothing(Q):
    p = Pool(Q, 30, 5, 6, page=8)
    p.resize([20, 9, 8, 0, 0])
    p.check()
    fork, resize = Q.qcf_pages_fork, Q.qcf_pages_resize
    for call in (lambda: fork(p.pool, i32([0, 1]), i32([3, 3])), lambda: fork(p.pool, i32([0, 3]), i32([3, 4])), lambda: fork(p.pool, i32([0]), i32([0])),
                 lambda: fork(p.pool, i32([5]), i32([3])), lambda: fork(p.pool, i32([0]), i32([-1])), lambda: fork(p.pool, i32([0, 1]), i32([3, 5])),
                 lambda: resize(p.pool, i32([1, 2]), i32([3, 3])), lambda: resize(p.pool, i32([49]), i32([3])), lambda: resize(p.pool, i32([-1]), i32([0])),
                 lambda: resize(p.pool, i32([1]), i32([5])), lambda: resize(p.pool, i32([1]), i32([-2]))):
        call()
        p.check(BAD_INDEX)
    for value in (-1, 49):
        p.pool.kv_len[1] = value
        for call in (lambda: resize(p.pool, i32([1]), i32([1])), lambda: fork(p.pool, i32([1]), i32([3])), lambda: fork(p.pool, i32([0]), i32([1])),
                     lambda: Q.qcf_pages_compact(p.pool)):
            call()
            assert Q.qcf_query_status() == BAD_INDEX
        p.pool.kv_len[1] = 9
        p.check()


def test_bad_pages_are_left_out(Q):
    """A row that names a page outside the cache: flagged, and nothing outside is touched."""
    p = Pool(Q, 30, 4, 6, page=8)
    p.resize([24, 20, 0, 0])
    p.pool.page_table[0, 1] = 30
    Q.qcf_pages_fork(p.pool, i32([0]), i32([2]))
    assert Q.qcf_query_status() == BAD_INDEX
    assert p.pool.page_table[2, :3].tolist() == [p.rows[0][0], 30, p.rows[0][2]]
    Q.qcf_pages_resize(p.pool, i32([0]), i32([2]))
    assert Q.qcf_query_status() == BAD_INDEX
    p.pool.page_table[1, 2] = -5                 # the page that would be copied
    before = p.pool.refs.tolist()
    Q.qcf_pages_fork(p.pool, i32([1]), i32([3]))
    assert Q.qcf_query_status() == BAD_INDEX
    assert p.pool.refs.tolist() == before and p.pool.kv_len.tolist() == [24, 20, 0, 0]
    Q.qcf_pages_compact(p.pool)
    assert Q.qcf_query_status() == 0             # nothing to move: nothing looked at
    p.pool.page_table[0, 1], p.pool.page_table[1, 2] = p.rows[0][1], p.rows[1][2]
    p.check()


def test_captured_turnover(Q):
    """A captured resize and compact replayed with other lengths."""
    p = Pool(Q, 60, 6, 10, page=8, layers=3)
    p.resize([40, 3, 17, 0, 64, 9])
    to = i32([0] * 6)
    Q.qcf_pages_resize(p.pool, i32(p.lens))
    Q.qcf_pages_compact(p.pool)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qcf_pages_resize(p.pool, to)
        live = Q.qcf_pages_compact(p.pool)
    p.check()
    real_resize, real_compact = p.Q.qcf_pages_resize, p.Q.qcf_pages_compact

    class Quiet:   # the host's side alone: the graph does the rest
        qcf_pages_resize = staticmethod(lambda *a: None)
        qcf_pages_compact = staticmethod(lambda *a: sum(r > 0 for r in p.refs))
        qcf_query_status = staticmethod(Q.qcf_query_status)
    p.Q = Quiet
    for lens in ([8, 8, 8, 8, 8, 8], [0, 0, 70, 0, 1, 1], [50, 49, 0, 48, 0, 0], [0] * 6):
        to.copy_(i32(lens))
        graph.replay()
        p.resize(lens)
        p.compact()
        p.check()
        assert int(live) == sum(r > 0 for r in p.refs)
    assert real_resize is Q.qcf_pages_resize and real_compact is Q.qcf_pages_compact


def test_pages_far_apart(Q):
    """Pages whose entries lie more than 2^31 entries from the first."""
    n, page, D = 6, 8, 16
    stride = (1 << 29) + 8
    k = [torch.empty((n - 1) * stride + page * D, dtype=torch.bfloat16, device=DEV).as_strided((n, page, 1, D), (stride, D, D, 1)) for _ in range(2)]
    g = torch.Generator(device=DEV).manual_seed(0)
    for t in k:
        t.copy_(torch.randn(t.shape, generator=g, device=DEV).to(t.dtype))
    pool = Q.PagePool.empty([Q.PagedKV(*k)], 3, 32)
    Q.qcf_pages_resize(pool, i32([16, 16, 11]))
    Q.qcf_pages_resize(pool, i32([0, 16, 11]))
    held = [t[5, :3].clone() for t in k], [t[4].clone() for t in k]
    assert int(Q.qcf_pages_compact(pool)) == 4
    assert pool.page_table[2, :2].tolist() == [0, 1]
    assert all(torch.equal(a[1, :3], b) for a, b in zip(k, held[0])) and all(torch.equal(a[0], b) for a, b in zip(k, held[1]))


def test_no_sequences_and_empty_calls(Q):
    p = Pool(Q, 10, 3, 4)
    Q.qcf_pages_resize(p.pool, i32([]), i32([]))
    Q.qcf_pages_fork(p.pool, i32([]), i32([]))
    assert int(Q.qcf_pages_compact(p.pool)) == 0
    p.check()
    empty = Q.PagePool.empty(p.caches, 0, 8)
    assert int(Q.qcf_pages_compact(empty)) == 0
