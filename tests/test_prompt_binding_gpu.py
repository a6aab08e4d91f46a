"""What the binding of prompt attention, chunk attention and the page operators refuses, and how it keeps a pool's scratch."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = {"dtype": torch.int32, "device": DEV}


@pytest.fixture(scope="module")
def Q():
    from rag_kv_cache_re_gb300 import qcf
    return qcf


@pytest.fixture(autouse=True)
def clean_status(Q):
    Q.qcf_query_status()
    yield
    assert Q.qcf_query_status() == 0, "a device-side check failed"


def rows(n, H, D=64, dtype=torch.bfloat16, device=DEV):
    return torch.zeros((n, H, D), dtype=dtype, device=device)


PACKED = {
    "fewer keys": lambda a: a.update(k=rows(15, 2)),
    "other heads": lambda a: a.update(v=rows(16, 1)),
    "other head dim": lambda a: a.update(k=rows(16, 2, 32), v=rows(16, 2, 32)),
    "other type": lambda a: a.update(k=rows(16, 2, dtype=torch.float16)),
    "float32": lambda a: a.update(q=rows(16, 4, dtype=torch.float32), k=rows(16, 2, dtype=torch.float32), v=rows(16, 2, dtype=torch.float32)),
    "other strides": lambda a: a.update(v=rows(16, 4)[:, :2]),
    "entries apart": lambda a: a.update(q=rows(16, 4, 128)[:, :, ::2]),
    "two dimensions": lambda a: a.update(q=rows(16, 4).view(16, 256)),
    "keys on the host": lambda a: a.update(k=rows(16, 2, device="cpu")),
    "starts on the host": lambda a: a.update(row_start=torch.tensor([0, 16], dtype=torch.int32)),
    "64-bit starts": lambda a: a.update(row_start=torch.tensor([0, 16], device=DEV)),
    "no starts": lambda a: a.update(row_start=torch.zeros(0, **I32)),
    "uneven heads": lambda a: a.update(q=rows(16, 3)),
    "head dim 12": lambda a: a.update(q=rows(16, 4, 12), k=rows(16, 2, 12), v=rows(16, 2, 12)),
    "max_len beyond 32 bits": lambda a: a.update(max_len=2**32 + 16),
    "negative max_len": lambda a: a.update(max_len=-1),
    "window beyond 32 bits": lambda a: a.update(window=2**32 + 1),
    "negative window": lambda a: a.update(window=-1),
    "scale 0": lambda a: a.update(scale=0.0),
    "out of another shape": lambda a: a.update(out=rows(16, 2)),
    "out of another type": lambda a: a.update(out=rows(16, 4, dtype=torch.float16)),
    "out on the host": lambda a: a.update(out=rows(16, 4, device="cpu")),
    "out with gaps": lambda a: a.update(out=rows(16, 8)[:, :4]),
}


@pytest.mark.parametrize("what", list(PACKED))
def test_packed(Q, what):
    a = dict(q=rows(16, 4), k=rows(16, 2), v=rows(16, 2), row_start=torch.tensor([0, 16], **I32), max_len=16, scale=0.1)
    PACKED[what](a)
    with pytest.raises(Q.QcfError):
        Q.qcf_packed_causal_attn(**a)


def cache(Q, page=16, Hkv=2, D=64, n=8, dtype=torch.bfloat16):
    return Q.PagedKV(*(torch.zeros((n, page, Hkv, D), dtype=dtype, device=DEV) for _ in range(2)))


CHUNK = {
    "other rows": lambda a: a.update(q=rows(3, 4)),
    "other head dim": lambda a: a.update(q=rows(4, 4, 32)),
    "other type": lambda a: a.update(q=rows(4, 4, dtype=torch.float16)),
    "on the host": lambda a: a.update(q=rows(4, 4, device="cpu")),
    "uneven heads": lambda a: a.update(q=rows(4, 3)),
    "window beyond 32 bits": lambda a: a.update(window=2**32 + 1),
    "negative window": lambda a: a.update(window=-3),
    "scale without a number": lambda a: a.update(scale=float("nan")),
    "out with gaps": lambda a: a.update(out=rows(4, 8)[:, :4]),
    "in place over rows apart": lambda a: a.update(q=(t := rows(4, 8))[:, :4], out=t.view(-1)[: 4 * 4 * 64].view(4, 4, 64)),
}


@pytest.mark.parametrize("what", list(CHUNK))
def test_chunk(Q, what):
    kv = cache(Q)
    batch = Q.PagedBatch(torch.tensor([0, 4], **I32), torch.tensor([20], **I32), torch.tensor([[1, 2]], **I32), 4, 4, 32)
    a = dict(cache=kv, batch=batch, q=rows(4, 4), scale=0.1)
    CHUNK[what](a)
    with pytest.raises(Q.QcfError):
        Q.qcf_paged_chunk_attn(**a)


def test_pool(Q):
    kv = cache(Q)
    refs, table, lens = torch.zeros(8, **I32), torch.zeros((3, 4), **I32), torch.zeros(3, **I32)
    for caches, r, t, n in (([], refs, table, lens), ([kv], refs[:7], table, lens), ([kv], refs.long(), table, lens), ([kv], refs, table[:2], lens),
                            ([kv], refs, table.view(-1), lens), ([kv], refs, table[:, ::2], lens), ([kv], refs.cpu(), table, lens),
                            ([kv], refs, table, lens.cpu())):
        with pytest.raises(Q.QcfError):
            Q.PagePool(caches, r, t, n)
    with pytest.raises(Q.QcfError):
        Q.PagePool.empty([], 3, 64)
    one = torch.ones(1, **I32)
    for caches in ([kv, cache(Q, D=128)], [kv, cache(Q, dtype=torch.float16)], [kv, cache(Q, page=32)]):   # the library's to say, at each call
        pool = Q.PagePool(caches, refs, table, lens)
        with pytest.raises(Q.QcfError):
            Q.qcf_pages_resize(pool, one, one)
    pool = Q.PagePool([kv], refs, table, lens)
    for bad in (one.long(), one.cpu(), one.view(1, 1), torch.ones((), **I32), torch.ones(4, **I32)[::2]):
        with pytest.raises(Q.QcfError):
            Q.qcf_pages_resize(pool, bad, bad)
        with pytest.raises(Q.QcfError):
            Q.qcf_pages_fork(pool, bad, bad)
    with pytest.raises(Q.QcfError):
        Q.qcf_pages_fork(pool, one, torch.ones(2, **I32))
    with pytest.raises(Q.QcfError):
        Q.qcf_pages_resize(pool, torch.ones(4, **I32))   # more than there are sequences
    assert not refs.any() and not lens.any() and not table.any()


def test_a_pools_scratch_outlives_its_calls(Q):
    """A pool used on a stream of its own and let go of while that stream is busy: nobody else gets its scratch before."""
    kv, s = cache(Q), torch.cuda.Stream()
    pool = Q.PagePool.empty([kv], 3, 64)
    new = torch.tensor([20, 33, 0], **I32)
    table, lens = pool.page_table, pool.kv_len
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)   # a tenth of a second
        Q.qcf_pages_resize(pool, new)
    Q.qcf_pages_resize(pool, torch.tensor([20, 33, 0], **I32), stream=s)
    at, size = pool._ws.data_ptr(), pool._ws.numel()
    pool._ws_ptr = pool._ws = None
    del pool
    others = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
    busy = not s.query()
    assert not busy or at not in [t.data_ptr() for t in others]
    s.synchronize()
    assert lens.tolist() == [20, 33, 0] and table[0, :2].tolist() == [0, 1] and table[1, :3].tolist() == [2, 3, 4]
