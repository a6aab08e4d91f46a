"""Argument checks of the rotary, paged-append and shared-prefix attention entry points: errors come
back before any launch, so they need no GPU (pointers are never dereferenced)."""
import ctypes as C
import os

import pytest

OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
P = 0x100000


@pytest.fixture(scope="module")
def L():
    from rag_kv_cache_re_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    _lib.lib()
    return _lib


def changed(s, **kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def cache(L, **kw):
    return changed(L.PagedKV(P, P, L.QCF_BF16, 100, 16, 8, 128, 16 * 8 * 128, 8 * 128, 128), **kw)


def batch(L, **kw):
    return changed(L.PagedBatch(4, 0, 1, 64, P, P, P, 4, 100, P), **kw)


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(kind=9), ARG), (dict(kind=-1), ARG), (dict(factor=0.5), ARG), (dict(factor=float("nan")), ARG),
    (dict(original=0), ARG), (dict(low=4.0), ARG), (dict(low=-1.0), ARG), (dict(kind=4, low=0.0), ARG), (dict(amplitude=float("inf")), ARG),
    (dict(kind=2), SHAPE)])
def test_table_scaling(L, kw, expect):
    sc = changed(L.RopeScaling(3, 8192, 8.0, 1.0, 4.0, 1.0), **kw)
    R = 2 if kw.get("kind") == 2 else 64
    assert L.lib().qcf_rope_table_fill(P, P, 0, 0, R, 1e4, C.byref(sc), None) == expect


@pytest.mark.parametrize("cos,sin,first,n,R,theta,expect", [
    (None, P, 0, 0, 64, 1e4, ARG), (P, None, 0, 0, 64, 1e4, ARG), (P, P, 0, 0, 64, 1.0, ARG), (P, P, 0, 0, 64, float("inf"), ARG),
    (P, P, -1, 0, 64, 1e4, SHAPE), (P, P, 0, -1, 64, 1e4, SHAPE), (P, P, 2 ** 31 - 5, 6, 64, 1e4, SHAPE), (P, P, 0, 0, 63, 1e4, SHAPE),
    (P, P, 0, 0, 0, 1e4, SHAPE), (P, P, 0, 0, 514, 1e4, SHAPE), (P + 4, P, 0, 0, 64, 1e4, ALIGN), (P, P, 0, 0, 512, 1e4, OK)])
def test_table_arguments(L, cos, sin, first, n, R, theta, expect):
    assert L.lib().qcf_rope_table_fill(cos, sin, first, n, R, theta, None, None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(x=None), ARG), (dict(y=None), ARG), (dict(pos=None), ARG), (dict(cos=None), ARG), (dict(dtype=3), ARG),
    (dict(dtype=-1), ARG), (dict(mode=4), ARG), (dict(mode=3), OK), (dict(n=-1), SHAPE), (dict(H=0), SHAPE), (dict(D=127, xs=4096), SHAPE),
    (dict(D=514, xs=8192), SHAPE), (dict(R=130), SHAPE), (dict(R=5), SHAPE), (dict(R=0), SHAPE), (dict(xs=1016), SHAPE), (dict(ys=1016), SHAPE),
    (dict(y=P, ys=1032), SHAPE), (dict(xs=1028), OK), (dict(dtype=2, xs=1025), OK), (dict(x=P + 8), ALIGN),
    (dict(n=2 ** 31 - 1, H=60000, xs=60000 * 128, ys=60000 * 128), SHAPE)])
def test_rope_apply_arguments(L, kw, expect):
    a = dict(x=P, xs=1024, y=2 * P, ys=1024, n=0, H=8, D=128, dtype=0, pos=P, cos=P, R=128, mode=0)
    a.update(kw)
    t = L.RopeTable(a["cos"], P, 100, a["R"])
    assert L.lib().qcf_rope_apply(a["x"], a["xs"], a["y"], a["ys"], a["n"], a["H"], a["D"], a["dtype"], a["pos"], C.byref(t), a["mode"],
                                  None) == expect


CACHE_ERRORS = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(dtype=2), ARG), (dict(n_pages=0), SHAPE), (dict(page_size=4), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=512), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=32), SHAPE), (dict(row_stride=64), SHAPE), (dict(head_stride=0), SHAPE),
    (dict(page_stride=-8), SHAPE), (dict(row_stride=1028), ALIGN), (dict(k=P + 2), ALIGN)]
BATCH_ERRORS = [
    (dict(row_start=None), ARG), (dict(kv_len=None), ARG), (dict(page_table=None), ARG), (dict(prefix_pages=None), ARG), (dict(n_seq=-1), SHAPE),
    (dict(n_seq=65536), SHAPE), (dict(n_rows=-1), SHAPE), (dict(max_q=-1), SHAPE), (dict(max_len=65), SHAPE), (dict(table_stride=0), SHAPE),
    (dict(prefix_len=-1), SHAPE), (dict(prefix_len=2 ** 31 - 100), SHAPE), (dict(prefix_pages=None, prefix_len=0), OK), (dict(n_seq=0), OK)]


def append(L, c, b, k=P, v=P, kvs=1024, R=128, cos=P, mode=0, q=P, qs=4096, qo=2 * P, qos=4096, Hq=32, table=True):
    t = L.RopeTable(cos, P, 1000, R)
    return L.lib().qcf_paged_append(C.byref(c) if c else None, C.byref(b) if b else None, k, v, kvs, C.byref(t) if table else None, mode, q, qs, qo,
                                    qos, Hq, None)


def attend(L, c, b, q=P, qs=4096, Hq=32, scale=0.1, o=P, ws=P, ws_bytes=1 << 40):
    return L.lib().qcf_shared_prefix_attn(C.byref(c) if c else None, C.byref(b) if b else None, q, qs, Hq, scale, o, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", CACHE_ERRORS)
def test_cache_arguments(L, kw, expect):
    assert append(L, cache(L, **kw), batch(L)) == expect
    assert attend(L, cache(L, **kw), batch(L)) == expect


@pytest.mark.parametrize("kw,expect", BATCH_ERRORS)
def test_batch_arguments(L, kw, expect):
    assert append(L, cache(L), batch(L, **kw)) == expect
    assert attend(L, cache(L), batch(L, **kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(k=None), ARG), (dict(v=None), ARG), (dict(q=None), ARG), (dict(qo=None), ARG), (dict(q=None, qo=None), OK), (dict(cos=None), ARG),
    (dict(mode=2), ARG), (dict(mode=1), OK), (dict(R=130), SHAPE), (dict(R=7), SHAPE), (dict(Hq=0), SHAPE), (dict(kvs=1016), SHAPE), (dict(qs=4088), SHAPE),
    (dict(qos=4088), SHAPE), (dict(qo=P, qos=4104), SHAPE), (dict(kvs=1028), ALIGN), (dict(q=P + 2), ALIGN), (dict(k=P + 8), ALIGN), (dict(table=False), OK)])
def test_append_arguments(L, kw, expect):
    assert append(L, cache(L), batch(L), **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(q=None), ARG), (dict(o=None), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(Hq=20), SHAPE), (dict(Hq=136, qs=17408), SHAPE), (dict(qs=4088), SHAPE), (dict(qs=4100), ALIGN), (dict(o=P + 8), ALIGN), (dict(ws=P + 16), ALIGN)])
def test_attention_arguments(L, kw, expect):
    assert attend(L, cache(L), batch(L), **kw) == expect


def test_null_descriptors_and_injected_faults(L):
    assert append(L, None, batch(L)) == ARG and append(L, cache(L), None) == ARG
    assert attend(L, None, batch(L)) == ARG and attend(L, cache(L), None) == ARG
    assert L.lib().qcf_rope_apply(P, 1024, 2 * P, 1024, 0, 8, 128, 0, P, None, 0, None) == ARG
    for call in (append, attend):
        for kind, expect in ((1, ARG), (4, ALIGN)):
            assert L.lib().qcf_debug_set_fault(kind) == OK
            assert call(L, cache(L), batch(L)) == expect
            assert call(L, cache(L), batch(L)) == OK
    assert L.lib().qcf_debug_set_fault(2) == OK
    assert attend(L, cache(L), batch(L)) == WS


def test_workspace_of_malformed_arguments_is_zero(L):
    size = L.lib().qcf_shared_prefix_attn_workspace_size
    assert size(C.byref(cache(L, D=32)), C.byref(batch(L)), 32) == 0
    assert size(C.byref(cache(L)), C.byref(batch(L)), 30) == 0
    assert size(None, C.byref(batch(L)), 32) == 0


def test_binding_refuses_host_tensors(L):
    torch = pytest.importorskip("torch")
    from rag_kv_cache_re_gb300 import qcf as Q
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(L.QcfError):
        Q.PagedKV(k, k.clone())
    with pytest.raises(L.QcfError):
        Q.RopeScaling("sideways")
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(L.QcfError):
        Q.PagedBatch(i, i, torch.zeros((3, 2), dtype=torch.int32), 3, 1, 32)       # row_start of n_seq + 1 entries
    with pytest.raises(L.QcfError):
        Q.PagedBatch(torch.zeros(4, dtype=torch.int64), i, torch.zeros((3, 2), dtype=torch.int32), 3, 1, 32)
    with pytest.raises(L.QcfError):
        Q.PagedBatch(torch.zeros(4, dtype=torch.int32), i, torch.zeros((2, 2), dtype=torch.int32), 3, 1, 32)


def test_a_refused_layout_leaves_no_workspace_size_behind(L):
    """The size that one batch keeps for a layout is asked for again after a cache of that layout was refused."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    from rag_kv_cache_re_gb300 import qcf as Q
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    bt = Q.PagedBatch(i32(0, 1, 2), i32(5, 9), torch.zeros((2, 4), dtype=torch.int32), 2, 1, 64)

    def layout(**kw):
        struct = cache(L, **kw)
        return SimpleNamespace(struct=struct, ref=C.byref(struct), page_size=16, Hkv=8, D=128)
    for wrong in (dict(row_stride=1028), dict(k=P + 2), dict(n_pages=0)):
        assert bt.workspace_size(layout(**wrong), 32) == 0
    good = bt.workspace_size(layout(), 32)
    assert good > 0 and bt.workspace_size(layout(), 32) == good


@pytest.mark.parametrize("kw,expect", [
    (dict(q=P, o=P, qs=4096), OK), (dict(q=P, o=P, qs=4104), SHAPE), (dict(q=P, o=P, qs=6144), SHAPE), (dict(q=P, o=2 * P, qs=6144), OK),
    (dict(q=P, o=P, qs=6144, Hq=48), OK)])
def test_attention_writes_over_its_queries_only_row_for_row(L, kw, expect):
    """o may be q only where the rows of both lie Hq D entries apart."""
    assert attend(L, cache(L), batch(L), **kw) == expect
    assert attend(L, cache(L), batch(L, prefix_len=0, prefix_pages=None), **kw) == expect
