"""Argument checks of the prompt, chunk and page entry points: errors come back before any launch, so they
need no GPU (pointers are never dereferenced)."""
import ctypes as C

import pytest

from test_paged_refusals import ALIGN, ARG, BATCH_ERRORS, CACHE_ERRORS, OK, SHAPE, WS, P, L, batch, cache, changed  # noqa: F401


def packed(L, **kw):
    a = dict(q=P, qs=4096, k=P, v=P, kvs=1024, dtype=0, start=P, n_seq=0, n_rows=64, max_len=64, Hq=32, Hkv=8, D=128, scale=0.1, window=0, o=2 * P,
             ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return L.lib().qcf_packed_causal_attn(a["q"], a["qs"], a["k"], a["v"], a["kvs"], a["dtype"], a["start"], a["n_seq"], a["n_rows"], a["max_len"],
                                          a["Hq"], a["Hkv"], a["D"], a["scale"], a["window"], a["o"], None, a["ws"], a["ws_bytes"], None)


SHARED = [(dict(q=None), ARG), (dict(o=None), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=3e38), ARG),
          (dict(window=-1), ARG), (dict(window=2 ** 31 - 1), OK), (dict(Hq=0), SHAPE), (dict(Hq=12), SHAPE), (dict(Hq=8 * 129, qs=1 << 20), SHAPE),
          (dict(qs=4088), SHAPE), (dict(qs=4100), ALIGN), (dict(q=P + 8), ALIGN), (dict(o=P + 4), ALIGN), (dict(ws=P + 128), ALIGN), (dict(o=P, qs=4104), SHAPE), (dict(o=P), OK)]


@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(), OK), (dict(k=None), ARG), (dict(v=None), ARG), (dict(start=None), ARG), (dict(dtype=2), ARG), (dict(dtype=-1), ARG), (dict(n_seq=-1), SHAPE),
    (dict(n_seq=8001), SHAPE), (dict(n_rows=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(n_rows=1 << 20), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=0), SHAPE),
    (dict(D=12), SHAPE), (dict(D=136, qs=8192, kvs=8192), SHAPE), (dict(D=80), OK), (dict(D=8), OK), (dict(kvs=1016), SHAPE), (dict(kvs=1028), ALIGN), (dict(k=P + 8), ALIGN),
    (dict(v=P + 8), ALIGN)])
def test_packed_arguments(L, kw, expect):  # noqa: F811
    assert packed(L, **kw) == expect


def chunk(L, c, b, **kw):
    a = dict(q=P, qs=4096, Hq=32, scale=0.1, window=0, o=2 * P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return L.lib().qcf_paged_chunk_attn(C.byref(c) if c else None, C.byref(b) if b else None, a["q"], a["qs"], a["Hq"], a["scale"], a["window"], a["o"], None,
                                        a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", CACHE_ERRORS)
def test_chunk_cache(L, kw, expect):  # noqa: F811
    assert chunk(L, cache(L, **kw), batch(L)) == expect


@pytest.mark.parametrize("kw,expect", BATCH_ERRORS)
def test_chunk_batch(L, kw, expect):  # noqa: F811
    assert chunk(L, cache(L), batch(L, **kw)) == expect


@pytest.mark.parametrize("kw,expect", SHARED)
def test_chunk_arguments(L, kw, expect):  # noqa: F811
    assert chunk(L, cache(L), batch(L), **kw) == expect


def test_chunk_sizes(L):  # noqa: F811
    assert chunk(L, None, batch(L)) == ARG and chunk(L, cache(L), None) == ARG
    assert chunk(L, cache(L), batch(L, n_seq=8001)) == SHAPE
    assert chunk(L, cache(L), batch(L, n_rows=1 << 20)) == SHAPE


def test_injected_faults(L):  # noqa: F811
    lib = L.lib()
    pages = lambda: lib.qcf_pages_compact(C.byref(pool(L)), P, P, 1 << 40, None)  # noqa: E731
    for kind, expect in ((1, ARG), (2, WS), (4, ALIGN)):
        for call in (lambda: packed(L), lambda: chunk(L, cache(L), batch(L)), pages):
            lib.qcf_debug_set_fault(kind)
            assert call() == expect
            lib.qcf_debug_set_fault(0)


def pool(L, caches=None, **kw):
    caches = caches or [cache(L), cache(L)]
    keep = (L.PagedKV * len(caches))(*caches)
    s = changed(L.PagePool(keep, len(caches), P, P, 4, P, 4), **kw)
    s.keep = keep
    return s


@pytest.mark.parametrize("kw,n,expect", [
    (dict(), 0, OK), (dict(refs=None), 0, ARG), (dict(page_table=None), 0, ARG), (dict(kv_len=None), 0, ARG), (dict(page_table=None, kv_len=None, n_seq=0), 0, OK),
    (dict(n_caches=0), 0, SHAPE), (dict(n_caches=257), 0, SHAPE), (dict(n_seq=-1), 0, SHAPE), (dict(n_seq=65536), 0, SHAPE), (dict(table_stride=0), 0, SHAPE),
    (dict(table_stride=(1 << 20) + 1), 0, SHAPE), (dict(), -1, SHAPE), (dict(), 5, SHAPE), (dict(refs=P + 4), 0, ALIGN), (dict(page_table=P + 2), 0, ALIGN), (dict(page_table=P + 4, kv_len=P + 4), 0, OK)])
def test_pool_arguments(L, kw, n, expect):  # noqa: F811
    lib, p = L.lib(), pool(L, **kw)
    assert lib.qcf_pages_fork(C.byref(p), P, P, n, P, 1 << 40, None) == expect
    assert lib.qcf_pages_resize(C.byref(p), None, P, n, P, 1 << 40, None) == expect
    assert (lib.qcf_pages_workspace_size(C.byref(p), n) > 0) == (expect == OK)


def test_pool_caches_and_pointers(L):  # noqa: F811
    lib = L.lib()
    for kw, expect in CACHE_ERRORS:
        assert lib.qcf_pages_fork(C.byref(pool(L, [cache(L), cache(L, **kw)])), P, P, 0, P, 1 << 40, None) == expect
    for kw in (dict(n_pages=99), dict(Hkv=4), dict(dtype=1), dict(row_stride=1032), dict(page_size=8)):
        assert lib.qcf_pages_fork(C.byref(pool(L, [cache(L), cache(L, **kw)])), P, P, 0, P, 1 << 40, None) == SHAPE
    p = pool(L)
    assert lib.qcf_pages_fork(None, P, P, 0, P, 1 << 40, None) == ARG and lib.qcf_pages_fork(C.byref(p), None, P, 0, P, 1 << 40, None) == ARG
    assert lib.qcf_pages_fork(C.byref(p), P, None, 0, P, 1 << 40, None) == ARG and lib.qcf_pages_resize(C.byref(p), P, None, 0, P, 1 << 40, None) == ARG
    assert lib.qcf_pages_compact(C.byref(p), None, P, 1 << 40, None) == ARG
    need = lib.qcf_pages_workspace_size(C.byref(p), 3)
    assert lib.qcf_pages_fork(C.byref(p), P, P, 3, P, need - 1, None) == WS and lib.qcf_pages_resize(C.byref(p), P, P, 3, None, need, None) == WS
    assert lib.qcf_pages_compact(C.byref(p), P, P + 64, 1 << 40, None) == ALIGN
