"""Packed prompt attention and chunk attention over pages, on the GPU, against the plain 64-bit form of
_prompt_reference."""
import pytest
import torch

import _paged_reference as R
import _prompt_reference as P

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def Q():
    from rag_kv_cache_re_gb300 import qcf
    return qcf


@pytest.fixture(autouse=True)
def clean_status(Q):
    Q.qcf_query_status()
    yield
    assert Q.qcf_query_status() == 0, "a device-side check failed"


def within(got, ref, tol, what):
    assert got.shape == ref.shape
    bad = ~(((got.double() - ref).abs() <= tol) | (got.double() == ref))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {ref[bad][0].item()} +- {tol[bad][0].item():.3g}")


# ----------------------------------------------------------------- packed prompts

def packed(lens, Hq, Hkv, D, dtype, seed, lead=0, pad=0, junk=float("nan"), std=1.2):
    """Packed q, k, v rows; rows of no prompt hold junk."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lead + sum(lens) + pad
    rows = (torch.randn((n, Hq + 2 * Hkv, D), generator=g, device=DEV) * std).to(dtype)
    rows[:lead] = junk
    rows[n - pad:] = junk
    start = torch.tensor([lead + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    return (*rows.split([Hq, Hkv, Hkv], 1), start)


def check_packed(Q, lens, Hq, Hkv, D, dtype, seed=0, lead=0, pad=0, window=0, scale=None, max_len=None, std=1.2):
    scale = D ** -0.5 if scale is None else scale
    q, k, v, start = packed(lens, Hq, Hkv, D, dtype, seed, lead, pad, std=std)
    out = torch.full((q.shape[0], Hq, D), 7.0, dtype=dtype, device=DEV)
    kept = q.clone(), k.clone(), v.clone()
    got, lse = Q.qcf_packed_causal_attn(q, k, v, start, max_len or max(lens + [1]), scale, window=window, want_lse=True, out=out)
    assert got is out
    r = lead
    for b, n in enumerate(lens):
        if n:
            o, e, tol, ltol = P.attend(q[r: r + n], k[r: r + n], v[r: r + n], 0, scale, window)
            within(out[r: r + n], o, tol, f"sequence {b}")
            within(lse[r: r + n], e, ltol, f"lse of sequence {b}")
        r += n
    assert torch.all(out[:lead] == 7.0) and torch.all(out[r:] == 7.0), "a row of no prompt changed"
    assert all(torch.equal(a.view(torch.int16), b.contiguous().view(torch.int16)) for a, b in zip(kept, (q.contiguous(), k.contiguous(), v.contiguous())))
    again, lse2 = Q.qcf_packed_causal_attn(q, k, v, start, max_len or max(lens + [1]), scale, window=window, want_lse=True)
    assert torch.equal(again[lead: r], out[lead: r]) and torch.equal(lse2[lead: r], lse[lead: r]), "a repeat gives other bits"
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 8, 64), (6, 2, 128), (4, 1, 16), (14, 2, 80), (16, 1, 64), (3, 1, 8), (40, 1, 128)])
@pytest.mark.parametrize("lens", [[1], [130], [0, 1, 63, 0, 64, 65, 129, 0], [257, 2, 511]])
def test_packed(Q, dtype, Hq, Hkv, D, lens):
    check_packed(Q, lens, Hq, Hkv, D, TYPES[dtype], seed=sum(lens), lead=3, pad=5)


@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 129, 1000])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (2, 2, 64)])
def test_packed_window(Q, Hq, Hkv, D, window):
    check_packed(Q, [700, 1, 130, 40], Hq, Hkv, D, torch.bfloat16, seed=window, window=window, pad=1)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([3000], 8, 2, 128), ([1500, 2100], 2, 2, 128), ([5001], 7, 1, 64), ([2500, 1, 1, 1900], 16, 2, 64)])
def test_packed_long(Q, lens, Hq, Hkv, D):
    check_packed(Q, lens, Hq, Hkv, D, torch.bfloat16, seed=9)
    check_packed(Q, lens, Hq, Hkv, D, torch.float16, seed=10, window=777)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_packed_sharp_and_flat(Q, dtype):
    """Logits of hundreds (nearly one-hot weights, a maximum that keeps growing) and of nearly nothing."""
    check_packed(Q, [600, 300], 8, 2, 128, TYPES[dtype], seed=4, std=6.0)
    check_packed(Q, [600, 300], 8, 2, 128, TYPES[dtype], seed=5, scale=1e-6)


def test_packed_many_short(Q):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (1000,), generator=g).tolist()
    check_packed(Q, lens, 4, 2, 64, torch.bfloat16, seed=1, max_len=64)


def test_packed_rows_apart_and_in_place(Q):
    """q with a stride of its own, and o over q."""
    lens, Hq, Hkv, D = [200, 90], 8, 2, 128
    q, k, v, start = packed(lens, Hq, Hkv, D, torch.bfloat16, 6)
    ref = Q.qcf_packed_causal_attn(q, k, v, start, 200, 0.1)
    wide = torch.full((290, Hq + 3, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :Hq] = q
    assert torch.equal(Q.qcf_packed_causal_attn(wide[:, :Hq], k, v, start, 200, 0.1), ref)
    mine = q.contiguous()
    assert Q.qcf_packed_causal_attn(mine, k, v, start, 200, 0.1, out=mine) is mine
    assert torch.equal(mine, ref)


def test_packed_nan_stays_in_its_place(Q):
    """A NaN query stays in its row and head; a NaN key or value in its own sequence."""
    lens, Hq, Hkv, D = [150, 170, 130], 8, 2, 128
    q, k, v, start = packed(lens, Hq, Hkv, D, torch.bfloat16, 8)
    ref = Q.qcf_packed_causal_attn(q, k, v, start, 170, 0.1)
    q2 = q.contiguous()
    q2[200, 3] = float("nan")
    got = Q.qcf_packed_causal_attn(q2, k, v, start, 170, 0.1)
    assert torch.isnan(got[200, 3]).all()
    got[200, 3] = ref[200, 3]
    assert torch.equal(got, ref)
    k2, v2 = k.clone(), v.clone()
    k2[319], v2[150] = float("nan"), float("inf")
    got = Q.qcf_packed_causal_attn(q, k2, v2, start, 170, 0.1)
    assert torch.equal(got[:150], ref[:150]) and torch.equal(got[320:], ref[320:])
    assert not torch.isfinite(got[150:320]).all()


def test_packed_leaves_out_bad_sequences(Q):
    lens, Hq, Hkv, D = [50, 60, 70], 4, 2, 64
    q, k, v, start = packed(lens, Hq, Hkv, D, torch.float16, 2)
    ref = Q.qcf_packed_causal_attn(q, k, v, start, 70, 0.1)

    def run(at, bound):
        out = torch.full_like(ref, 7.0)
        Q.qcf_packed_causal_attn(q, k, v, torch.tensor(at, dtype=torch.int32, device=DEV), bound, 0.1, out=out)
        assert Q.qcf_query_status() == 2
        return out
    out = run([0, 50, 110, 180], 65)                       # the last is longer than the bound
    assert torch.equal(out[:110], ref[:110]) and torch.all(out[110:] == 7.0)
    out = run([0, 50, 110, 181], 100)                      # ends behind the rows
    assert torch.equal(out[:110], ref[:110]) and torch.all(out[110:] == 7.0)
    out = run([-1, 50, 110, 180], 100)                     # begins before them
    assert torch.all(out[:50] == 7.0) and torch.equal(out[50:], ref[50:])
    out = run([0, 110, 50, 180], 200)                      # descends
    assert torch.all(out[110 + 70:] == 7.0)
    run([0, 50, 110, 180], 0)


def test_packed_captured_step_follows_the_lengths(Q):
    Hq, Hkv, D = 8, 2, 128
    q, k, v, start = packed([400, 300], Hq, Hkv, D, torch.bfloat16, 12)
    out = torch.zeros_like(q.contiguous())
    Q.qcf_packed_causal_attn(q, k, v, start, 700, 0.09, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qcf_packed_causal_attn(q, k, v, start, 700, 0.09, out=out)
    for lens in ([400, 300], [700, 0], [1, 699], [0, 5]):
        start.copy_(torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        r = 0
        for n in lens:
            if n:
                o, _, tol, _ = P.attend(q[r: r + n], k[r: r + n], v[r: r + n], 0, 0.09)
                within(out[r: r + n], o, tol, str(lens))
            r += n
        assert torch.all(out[r:] == 7.0)


def test_packed_on_another_stream(Q):
    q, k, v, start = packed([300, 200], 8, 2, 128, torch.bfloat16, 13)
    ref = Q.qcf_packed_causal_attn(q, k, v, start, 300, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [Q.qcf_packed_causal_attn(q, k, v, start, 300, 0.1, stream=side) for _ in range(8)]
    mine = [Q.qcf_packed_causal_attn(q, k, v, start, 300, 0.1) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref) for g in got + mine)


# ----------------------------------------------------------------- chunks over pages

def check_chunk(Q, bt, Hq, window=0, scale=None, gone_own=None, status=0, **over):
    scale = bt.D ** -0.5 if scale is None else scale
    q = bt.randn(bt.n_rows, Hq, bt.D, std=1.3)
    cache, batch = bt.bind(Q, **over)
    out = torch.full_like(q, 7.0)
    got, lse = Q.qcf_paged_chunk_attn(cache, batch, q, scale, window=window, want_lse=True, out=out)
    assert got is out and Q.qcf_query_status() == status
    o, e, tol, ltol = P.batch_attention(bt, q, scale, window, gone_own)
    rows = ~torch.isnan(e[:, 0])
    within(out[rows], o[rows], tol[rows], "o")
    within(lse[rows], e[rows], ltol[rows], "lse")
    assert torch.all(out[~rows] == 7.0), "a padding row changed"
    again, lse2 = Q.qcf_paged_chunk_attn(cache, batch, q, scale, window=window, want_lse=True)
    assert torch.equal(again[rows], out[rows]) and torch.equal(lse2[rows], lse[rows]), "a repeat gives other bits"
    Q.qcf_query_status()
    return out


BATCHES = [  # new, own lengths, prefix
    ([1], [1], 0), ([64], [700], 0), ([200], [200], 0), ([5, 0, 130, 1], [90, 10, 131, 2000], 0), ([40, 3], [60, 300], 129), ([300, 1, 1], [1000, 77, 128], 640),
    ([1, 1, 1, 1, 1], [1, 127, 128, 129, 600], 0), ([17], [17], 1000)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("Hq,Hkv,D,page,layout", [
    (32, 8, 128, 16, "rows"), (8, 8, 64, 8, "heads"), (6, 2, 128, 256, "heads"), (4, 2, 16, 32, "rows"), (16, 1, 64, 128, "rows"), (7, 1, 128, 64, "heads")])
@pytest.mark.parametrize("new,lens,prefix", BATCHES)
def test_chunk(Q, dtype, Hq, Hkv, D, page, layout, new, lens, prefix):
    bt = R.Batch(new, lens, prefix, Hkv, D, page, layout, TYPES[dtype], seed=sum(lens) + D, pad=4, lead=2).fill()
    check_chunk(Q, bt, Hq)


@pytest.mark.parametrize("window", [1, 63, 64, 128, 200, 1000, 100000])
@pytest.mark.parametrize("page", [8, 64])
def test_chunk_window(Q, window, page):
    """Windows that end inside the own tokens, inside the prefix and before its first token."""
    bt = R.Batch([70, 1, 300, 5], [90, 500, 900, 5], 333, 2, 128, page, "rows", torch.bfloat16, seed=window, pad=1).fill()
    check_chunk(Q, bt, 8, window=window)


@pytest.mark.parametrize("new,lens,prefix,Hq,Hkv,D", [
    ([512], [9000], 0, 8, 2, 128), ([1, 1], [12000, 3], 0, 8, 2, 128), ([1000, 30], [1000, 4000], 3000, 4, 4, 64), ([64], [20000], 0, 32, 8, 128),
    ([1] * 40, [(i * 37) % 1500 + 1 for i in range(40)], 700, 16, 4, 128)])
def test_chunk_long(Q, new, lens, prefix, Hq, Hkv, D):
    bt = R.Batch(new, lens, prefix, Hkv, D, 32, "rows", torch.bfloat16, seed=7).fill()
    check_chunk(Q, bt, Hq)
    bt = R.Batch(new, lens, prefix, Hkv, D, 16, "heads", torch.float16, seed=8).fill(std_k=3.0)
    check_chunk(Q, bt, Hq, window=2500)


GROUPS = [  # runs of short sequences before, between and behind longer ones, some without rows, over a prefix of several tiles
    ([1] * 40, [(i * 53) % 700 + 1 for i in range(40)]),
    ([1, 0, 1, 300, 1, 1, 0, 0, 2, 1, 50, 1], [200, 7, 129, 400, 1, 128, 5, 900, 256, 384, 90, 33]),
    ([2, 1, 3, 4] * 20, [(i * 37) % 300 + 4 for i in range(80)]), ([0, 0, 1, 0], [9, 0, 300, 4]), ([1, 0, 0, 1] + [0] * 60 + [1, 1], [60 + i for i in range(66)])]


@pytest.mark.parametrize("Hq,Hkv,D,page,layout,dtype", [
    (32, 8, 128, 16, "rows", "bf16"), (16, 1, 64, 64, "heads", "f16"), (7, 1, 128, 8, "heads", "bf16"), (4, 4, 128, 128, "rows", "f16"), (24, 1, 16, 32, "rows", "bf16")])
@pytest.mark.parametrize("prefix", [512, 1301])
@pytest.mark.parametrize("new,lens", GROUPS)
def test_chunk_groups_of_short_sequences(Q, Hq, Hkv, D, page, layout, dtype, prefix, new, lens):
    bt = R.Batch(new, lens, prefix, Hkv, D, page, layout, TYPES[dtype], seed=len(new) + D, pad=3, lead=1).fill()
    check_chunk(Q, bt, Hq)
    check_chunk(Q, bt, Hq, window=prefix)


def test_chunk_groups_leave_out_bad_sequences_and_pages(Q):
    new, lens = [1] * 12 + [40] + [1] * 3, [100 + 9 * i for i in range(16)]
    bt = R.Batch(new, lens, 700, 2, 128, 16, "rows", torch.bfloat16, seed=2).fill()
    q = bt.randn(bt.n_rows, 8, 128)
    cache, batch = bt.bind(Q)
    ref, rlse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    bt.kv_len[5] = 0                               # fewer tokens than new rows
    out = torch.full_like(ref, 7.0)
    Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, out=out)
    assert Q.qcf_query_status() == 2
    assert torch.all(out[5] == 7.0)
    bt.kv_len[5] = lens[5]
    o, e, tol, ltol = P.batch_attention(bt, q, 0.1)
    keep = [i for i in range(bt.n_rows) if i != 5]
    within(out[keep], o[keep], tol[keep], "beside a bad sequence")
    was = int(bt.table[7, 1])
    bt.table[7, 1] = -3                            # tokens 16 .. 31 of one of them
    got, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    assert Q.qcf_query_status() == 2
    bt.table[7, 1] = was
    o, e, tol, ltol = P.batch_attention(bt, q, 0.1, 0, {7: range(16, 32)})
    within(got, o, tol, "with a bad page")
    within(lse, e, ltol, "lse with a bad page")
    assert torch.equal(Q.qcf_paged_chunk_attn(cache, batch, q, 0.1), ref) and rlse.shape == lse.shape


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (16, 1, 64), (7, 1, 128)])
def test_chunk_groups_keep_one_sequences_nan_to_itself(Q, Hq, Hkv, D):
    """NaN and infinity in keys and values of some sequences of a group: the others' rows have the bits they have without."""
    new, lens = [1, 1, 2, 1, 1, 0, 1, 3, 1, 1], [300, 5, 129, 640, 1, 9, 128, 77, 200, 256]
    bt = R.Batch(new, lens, 900, Hkv, D, 16, "rows", torch.bfloat16, seed=4).fill()
    q = bt.randn(bt.n_rows, Hq, D)
    cache, batch = bt.bind(Q)
    ref, rlse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    o, _, tol, _ = P.batch_attention(bt, q, 0.1)
    within(ref, o, tol, "before")
    for b, j, what, value in ((0, 299, bt.v, float("nan")), (3, 0, bt.v, float("inf")), (6, 127, bt.k, float("nan")), (7, 10, bt.v, float("-inf"))):
        page, row = (int(t[j]) for t in bt.own_at(b))
        bt.rows(what)[page, row] = value
    got, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    hurt = {0, 3, 6, 7}
    for b, r, n in bt.spans():
        same = torch.equal(got[r: r + n], ref[r: r + n]) and torch.equal(lse[r: r + n], rlse[r: r + n])
        assert same != (b in hurt) or n == 0, f"sequence {b}"


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("at", range(112, 145, 8))
def test_chunk_groups_with_rows_before_and_behind_a_tile(Q, D, dtype, at):
    """New rows of a group's sequence on both sides of a key tile's border, in more than one warp: the rows before it see
    none of the tile's keys."""
    bt = R.Batch([16, 8, 16, 16, 1, 16], [40, 8, at, at + 3, 300, 16 + at], 700, 4, D, 16, "rows", TYPES[dtype], seed=at).fill()
    q = bt.randn(bt.n_rows, 4, D)
    cache, batch = bt.bind(Q)
    got, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    o, e, tol, ltol = P.batch_attention(bt, q, 0.1)
    within(got, o, tol, "o")
    within(lse, e, ltol, "lse")


def test_chunk_groups_of_many(Q):
    """Hundreds of single tokens, a cache that changes under a captured call."""
    lens = [(i * 29) % 260 + 1 for i in range(300)]
    bt = R.Batch([1] * 300, lens, 2000, 4, 64, 32, "rows", torch.float16, seed=5, pad=2, table_cols=9).fill()
    check_chunk(Q, bt, 16, max_len=288)
    q = bt.randn(bt.n_rows, 16, 64)
    cache, batch = bt.bind(Q, max_len=288)
    out = torch.zeros_like(q)
    Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, out=out)
    for step in (1, 40, 100):
        bt.lens = [max(1, n - step) for n in lens]
        bt.kv_len.copy_(torch.tensor(bt.lens, dtype=torch.int32))
        graph.replay()
        o, _, tol, _ = P.batch_attention(bt, q, 0.1)
        within(out[:300], o[:300], tol[:300], f"{step} fewer")


def test_chunk_agrees_with_the_shared_prefix_call(Q):
    """Two ways through the same batch: each within its tolerance of the same values."""
    bt = R.Batch([30, 1, 64], [200, 90, 64], 1500, 8, 128, 16, "rows", torch.bfloat16, seed=3).fill()
    q = bt.randn(bt.n_rows, 32, 128)
    cache, batch = bt.bind(Q)
    o, _, tol, _ = P.batch_attention(bt, q, 0.09)
    within(Q.qcf_paged_chunk_attn(cache, batch, q, 0.09), o, tol, "chunk")
    within(Q.qcf_shared_prefix_attn(cache, batch, q, 0.09), o, tol, "shared prefix")


def test_chunk_leaves_out_bad_pages(Q):
    """Keys of pages outside the cache are left out; a row without any key gets 0 and -infinity."""
    bt = R.Batch([40, 3], [200, 3], 0, 2, 128, 16, "rows", torch.bfloat16, seed=5).fill()
    gone = {0: list(range(32, 48)) + list(range(160, 176)), 1: [0, 1, 2]}
    keep = bt.table.clone()
    bt.table[0, 2], bt.table[0, 10], bt.table[1, 0] = -1, 10 ** 6, bt.k.shape[0]
    bad = bt.table.clone()
    q = bt.randn(bt.n_rows, 8, 128)
    cache, batch = bt.bind(Q)
    got, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    assert Q.qcf_query_status() == 2
    bt.table.copy_(keep)
    o, e, tol, ltol = P.batch_attention(bt, q, 0.1, 0, gone)
    within(got[:40], o[:40], tol[:40], "o")
    within(lse[:40], e[:40], ltol[:40], "lse")
    assert torch.all(got[40:] == 0) and torch.all(lse[40:] == -float("inf"))
    bt.table.copy_(bad)


def test_chunk_leaves_out_bad_sequences(Q):
    bt = R.Batch([10, 200, 30], [50, 300, 30], 100, 2, 64, 16, "rows", torch.float16, seed=6).fill()
    q = bt.randn(bt.n_rows, 4, 64)
    cache, batch = bt.bind(Q)
    ref = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1)
    for where, value, lost in (("kv_len", (0, 9), (0, 10)), ("kv_len", (1, 301), (10, 210)), ("kv_len", (2, -1), (210, 240))):
        t = getattr(bt, where)
        old = int(t[value[0]])
        t[value[0]] = value[1]
        out = torch.full_like(ref, 7.0)
        Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, out=out)
        assert Q.qcf_query_status() == 2
        t[value[0]] = old
        assert torch.all(out[lost[0]: lost[1]] == 7.0)
        assert torch.equal(out[: lost[0]], ref[: lost[0]]) and torch.equal(out[lost[1]:], ref[lost[1]:])


def test_chunk_beyond_32_bit_offsets(Q):
    """Pages whose entries lie more than 2^31 entries from the first."""
    bt = R.Batch([40, 1], [150, 70], 50, 1, 128, 16, "rows", torch.bfloat16, seed=4).fill()
    ref = check_chunk(Q, bt, 4)
    n = bt.k.shape[0]
    stride = (1 << 31) // (n // 2)      # entries from page to page: the last pages lie beyond 2^31
    stride -= stride % 8
    far = []
    for t in (bt.k, bt.v):
        flat = torch.empty((n - 1) * stride + 16 * 128, dtype=torch.bfloat16, device=DEV)
        far.append(flat.as_strided(t.shape, (stride, 128, 128, 1)))
        far[-1].copy_(t)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(bt.n_rows, 4, 128, generator=g, device=DEV).to(torch.bfloat16)
    cache, batch = bt.bind(Q)
    assert torch.equal(Q.qcf_paged_chunk_attn(Q.PagedKV(*far), batch, q, 0.1), Q.qcf_paged_chunk_attn(cache, batch, q, 0.1))
    assert ref.shape == q.shape


def test_chunk_in_place_and_captured(Q):
    bt = R.Batch([100, 1, 30], [400, 900, 30], 200, 8, 128, 16, "rows", torch.bfloat16, seed=11, pad=2).fill()
    q = bt.randn(bt.n_rows, 32, 128)
    cache, batch = bt.bind(Q)
    ref, lse = Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, want_lse=True)
    mine = q.clone()
    assert Q.qcf_paged_chunk_attn(cache, batch, mine, 0.1, out=mine) is mine
    assert torch.equal(mine[:131], ref[:131]) and torch.equal(mine[131:], q[131:])
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        Q.qcf_paged_chunk_attn(cache, batch, q, 0.1, out=out)
    for lens in ([400, 900, 30], [100, 1, 30], [333, 256, 30]):
        bt.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        bt.lens = lens
        graph.replay()
        o, _, tol, _ = P.batch_attention(bt, q, 0.1)
        within(out[:131], o[:131], tol[:131], str(lens))


def test_calls_side_by_side(Q):
    """Captured calls replayed on streams of their own beside eager ones, nothing waiting in between."""
    runs, seen = [], []
    for seed in (1, 2, 3):
        bt = R.Batch([64, 1, 1, 200], [3000, 900, 4000, 260], 500, 8, 128, 16, "rows", torch.bfloat16, seed=seed).fill()
        q = bt.randn(bt.n_rows, 32, 128)
        cache, batch = bt.bind(Q)
        a, k, v, start = packed([700, 300], 8, 2, 128, torch.bfloat16, seed)

        def run(cache=cache, batch=batch, q=q, a=a, k=k, v=v, start=start, keep=bt):
            return Q.qcf_paged_chunk_attn(cache, batch, q, 0.1), Q.qcf_packed_causal_attn(a, k, v, start, 700, 0.1)
        runs.append(run)
        seen.append([t.clone() for t in run()])
    torch.cuda.synchronize()
    held, graphs = [], []
    for run in runs[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(run())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for _ in range(6):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
            with torch.cuda.stream(streams[2]):
                got.append(runs[2]())
        torch.cuda.synchronize()
        for out, ref in [(h, r) for h, r in zip(held, seen)] + [(g, seen[2]) for g in got]:
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), "a call gives other bits beside the others"
