"""Rotary positions, the paged cache and attention over a shared prefix, on the GPU, against the
plain 64-bit forms of _paged_reference."""
import math

import pytest
import torch

import _paged_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALINGS = {
    "none": None, "linear": dict(factor=8.0), "base": dict(factor=4.0),
    "turns": dict(factor=8.0, original=8192, low=1.0, high=4.0), "index": dict(factor=16.0, original=4096, low=1.0, high=32.0)}


@pytest.fixture(scope="module")
def Q():
    from rag_kv_cache_re_gb300 import qcf
    return qcf


@pytest.fixture(autouse=True)
def clean_status(Q):
    Q.qcf_query_status()
    yield
    assert Q.qcf_query_status() == 0, "a device-side check failed"


def scaling(Q, kind, amplitude=1.0):
    return None if kind == "none" else Q.RopeScaling(kind, amplitude=amplitude, **SCALINGS[kind])


def randn(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


def within(got, ref, tol, what):
    assert got.shape == ref.shape
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {ref[bad][0].item()} +- {tol[bad][0].item():.3g}")


# ----------------------------------------------------------------- tables

@pytest.mark.parametrize("kind", list(SCALINGS))
@pytest.mark.parametrize("n,first,half,theta,amplitude", [
    (1, 0, 1, 1e4, 1.0), (3, 131070, 64, 1e4, 1.0), (1000, 7, 32, 5e5, 1.25), (257, 2 ** 30, 3, 1e4, 1.0), (4097, 0, 8, 1e4, 0.5),
    (700, 65530, 256, 1e4, 1.0)])
def test_rope_table_fill(Q, kind, n, first, half, theta, amplitude):
    if kind == "base" and half == 1:
        pytest.skip("base scaling needs more than one pair")
    if kind == "none":
        amplitude = 1.0
    cos = torch.full((n + 1, half), 9.0, device=DEV)   # one row more than filled: it stays
    sin = torch.full((n + 1, half), 9.0, device=DEV)
    Q.qcf_rope_table_fill(cos[:n], sin[:n], theta, first, scaling(Q, kind, amplitude))
    w = R.rates(2 * half, theta, kind, **(SCALINGS[kind] or {}))
    angle = (first + torch.arange(n, dtype=torch.float64))[:, None] * w
    # the angle's rate, product and argument reduction in 64 bits: a few 2^-53 of the angle; then
    # one rounding to 32 bits (half a step of the result)
    tol = amplitude * 8 * 2.0 ** -53 * (1 + angle.abs())
    for got, ref in ((cos, amplitude * angle.cos()), (sin, amplitude * angle.sin())):
        within(got[:n].cpu(), ref, tol + 2.0 ** -24 * ref.abs() * (1 + 2.0 ** -20) + 1e-40, kind)
        assert torch.all(got[n] == 9.0)


def test_rope_table_fill_continues_a_table(Q):
    whole = Q.ScaledRopeTable(3000, 128, 1e4, DEV, scaling(Q, "turns"))
    cos, sin = torch.empty_like(whole.cos), torch.empty_like(whole.sin)
    for a, b in ((0, 1), (1, 1024), (1024, 2999), (2999, 3000)):
        c, s = torch.empty((b - a, 64), device=DEV), torch.empty((b - a, 64), device=DEV)
        Q.qcf_rope_table_fill(c, s, 1e4, a, scaling(Q, "turns"))
        cos[a:b], sin[a:b] = c, s
    assert torch.equal(cos, whole.cos) and torch.equal(sin, whole.sin)


def test_rope_table_fill_agrees_with_the_host_tables(Q):
    host = Q.RopeTable(5000, 128, 1e4, DEV)
    dev = Q.ScaledRopeTable(5000, 128, 1e4, DEV)
    # both round a 64-bit value once; the values may differ in their last places, so by a step at most
    for a, b in ((host.cos, dev.cos), (host.sin, dev.sin)):
        assert torch.all((a.double() - b.double()).abs() <= 2.0 ** -23 * b.double().abs() + 1e-15)


# ----------------------------------------------------------------- rotation

ROPE_CASES = [  # n, H, D, R, row padding in heads
    (1, 1, 16, 16, 0), (16, 40, 128, 128, 8), (33, 5, 128, 64, 0), (7, 3, 64, 30, 1), (130, 2, 80, 80, 0), (50, 9, 80, 38, 2),
    (5, 72, 128, 128, 8), (257, 1, 2, 2, 7), (3, 4, 96, 48, 0), (9, 6, 512, 512, 0), (1000, 4, 128, 32, 4)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,H,D,rot,more", ROPE_CASES)
def test_rope_apply(Q, dtype, interleaved, n, H, D, rot, more):
    T = TYPES[dtype]
    rows = randn(n + D, n, H + more, D, dtype=T)
    x = rows[:, :H]
    before = rows.clone()
    table = Q.ScaledRopeTable(9000, rot, 1e4, DEV, scaling(Q, "turns"))
    pos = torch.randint(0, 9000, (n,), device=DEV, dtype=torch.int32)
    pos[0], pos[-1] = 8999, 0
    w = R.rates(rot, 1e4, "turns", **SCALINGS["turns"])
    ref, mag = R.rotate(x, pos, w, interleaved)
    tol = R.rotation_tolerance(ref, mag, T)
    got = Q.qcf_rope_apply(x, pos, table, interleaved)
    within(got, ref, tol, "out of place")
    assert torch.equal(rows, before), "the input changed"
    back = Q.qcf_rope_apply(got.contiguous(), pos, table, interleaved, inverse=True)
    iref, imag = R.rotate(got, -pos, w, interleaved)
    within(back, iref, R.rotation_tolerance(iref, imag, T), "inverse")
    assert Q.qcf_rope_apply(x, pos, table, interleaved, out=x) is x
    assert torch.equal(x, got), "in place differs"
    assert torch.equal(rows[:, H:], before[:, H:]), "entries between rows changed"


def test_rope_apply_is_the_reposition_of_whole_heads(Q):
    K = randn(5, 600, 8, 128)
    table = Q.RopeTable(4096, 128, 1e4, DEV)
    moved = Q.qcf_rope_reposition(K, torch.empty_like(K), [0, 100, 600], [37, 4000], table)
    pos = torch.tensor([37] * 100 + [4000] * 500, dtype=torch.int32, device=DEV)
    assert torch.equal(Q.qcf_rope_apply(K, pos, table), moved)


def test_rope_apply_gradient_is_the_inverse_rotation(Q):
    """d(sum g . y)/dx = R(-p) g: against 64-bit differences of the formula, fp32 in and out."""
    n, H, D, rot = 4, 2, 16, 12
    for interleaved in (False, True):
        x, g = randn(1, n, H, D, dtype=torch.float32), randn(2, n, H, D, dtype=torch.float32)
        pos = torch.tensor([0, 3, 77, 500], dtype=torch.int32, device=DEV)
        w = R.rates(rot, 1e4)
        dx = Q.qcf_rope_apply(g, pos, Q.ScaledRopeTable(512, rot, 1e4, DEV), interleaved, inverse=True)
        h = 2.0 ** -10   # the map is linear: differences are exact up to 64-bit rounding
        num = torch.empty(n, H, D, dtype=torch.float64, device=DEV)
        for d in range(D):
            e = torch.zeros(n, H, D, dtype=torch.float64, device=DEV)
            e[..., d] = h
            up = R.rotate(x.double() + e, pos, w, interleaved)[0] - R.rotate(x.double() - e, pos, w, interleaved)[0]
            num[..., d] = (up * g.double()).sum(-1) / (2 * h)
        formula, mag = R.rotate(g, -pos, w, interleaved)
        within(dx, formula, R.rotation_tolerance(formula, mag, torch.float32), "gradient")
        within(dx, num, R.rotation_tolerance(formula, mag, torch.float32) + 1e-11, "gradient against differences")


def test_rope_apply_leaves_padding_and_bad_rows(Q):
    x = randn(3, 6, 4, 64)
    table = Q.ScaledRopeTable(100, 64, 1e4, DEV)
    out = torch.full_like(x, 7.0)
    Q.qcf_rope_apply(x, torch.tensor([5, -1, 99, -1, 0, 1], dtype=torch.int32, device=DEV), table, out=out)
    assert torch.all(out[[1, 3]] == 7.0) and torch.equal(out[4], x[4]) and Q.qcf_query_status() == 0
    out.fill_(7.0)
    Q.qcf_rope_apply(x, torch.tensor([5, 100, 99, -2, 0, 1 << 30], dtype=torch.int32, device=DEV), table, out=out)
    assert Q.qcf_query_status() == 2
    assert torch.all(out[[1, 3, 5]] == 7.0) and not torch.any(out[[0, 2, 4]] == 7.0)


def test_rope_apply_beyond_32_bit_offsets(Q):
    """Rows whose first entries lie more than 2^31 entries apart."""
    n, stride = 3, (1 << 30) + 8
    flat = torch.empty((n - 1) * stride + 128, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((n, 1, 128), (stride, 128, 1))
    x.copy_(randn(9, n, 1, 128))
    table = Q.ScaledRopeTable(64, 128, 1e4, DEV)
    pos = torch.tensor([1, 2, 63], dtype=torch.int32, device=DEV)
    ref, mag = R.rotate(x, pos, R.rates(128, 1e4))
    Q.qcf_rope_apply(x, pos, table, out=x)
    within(x, ref, R.rotation_tolerance(ref, mag, torch.bfloat16), "far rows")


# ----------------------------------------------------------------- append

def check_append(Q, bt, Hq, rot, interleaved, rotate=True, in_place=False, max_pos=None):
    n, D, T = bt.n_rows, bt.D, bt.dtype
    rows = bt.randn(n, Hq + 2 * bt.Hkv, D)
    q, k, v = rows.split([Hq, bt.Hkv, bt.Hkv], 1)
    k0, v0, q0 = bt.k.clone(), bt.v.clone(), q.clone()
    cache, batch = bt.bind(Q)
    table = Q.ScaledRopeTable(max_pos or bt.prefix + bt.max_len + 1, rot, 1e4, DEV) if rotate else None
    out = q if in_place else torch.full((n, Hq, D), 7.0, dtype=T, device=DEV)
    got = Q.qcf_paged_append(cache, batch, k, v, table, interleaved, q=q, q_out=out)
    assert got is out
    kr, vr, qr = bt.rows(k0).clone(), bt.rows(v0).clone(), q0.clone() if in_place else torch.full_like(out, 7.0)
    w = R.rates(rot, 1e4)
    for b, r, nq in bt.spans():
        where = tuple(t[bt.lens[b] - nq:] for t in bt.own_at(b))
        pos = bt.prefix + torch.arange(bt.lens[b] - nq, bt.lens[b], device=DEV)
        vr[where] = v[r: r + nq]
        if not rotate:
            kr[where], qr[r: r + nq] = k[r: r + nq], q0[r: r + nq]
            continue
        for src, dst in ((k[r: r + nq], bt.rows(bt.k)[where]), (q0[r: r + nq], out[r: r + nq])):
            ref, mag = R.rotate(src, pos, w, interleaved)
            within(dst, ref, R.rotation_tolerance(ref, mag, T), f"sequence {b}")
        kr[where], qr[r: r + nq] = bt.rows(bt.k)[where], out[r: r + nq]
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    assert same(bt.rows(bt.k), kr) and same(bt.rows(bt.v), vr), "a slot outside the new rows changed, or a value"
    assert same(out, qr), "a query row outside the batch changed"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["rows", "heads"])
@pytest.mark.parametrize("new,lens,prefix,Hq,Hkv,D,rot,page", [
    ([1], [1], 0, 1, 1, 16, 16, 8),
    ([1] * 16, [3, 500, 16, 17, 1, 2, 9, 64, 65, 33, 15, 100, 7, 8, 31, 32], 5120, 32, 8, 128, 128, 16),
    ([5, 0, 1, 33, 0], [5, 9, 70, 33, 0], 13, 8, 2, 64, 64, 8),
    ([40, 1, 100], [300, 1, 100], 1, 28, 4, 128, 64, 256),
    ([3, 17], [3, 20], 2, 6, 3, 64, 30, 32),
    ([2] * 70, [2 + i for i in range(70)], 0, 4, 4, 16, 12, 16),
    ([1] * 1100, [1 + i % 40 for i in range(1100)], 100, 2, 1, 64, 64, 64)])
def test_paged_append(Q, dtype, layout, new, lens, prefix, Hq, Hkv, D, rot, page):
    for i, interleaved in enumerate((False, True)):
        bt = R.Batch(new, lens, prefix, Hkv, D, page, layout, TYPES[dtype], seed=17 + i, pad=3 * i, lead=2 * i)
        check_append(Q, bt, Hq, rot, interleaved)


def test_paged_append_without_rotation_and_in_place(Q):
    args = ([4, 1, 9], [20, 1, 9], 30, 2, 64, 16, "rows", torch.bfloat16)
    check_append(Q, R.Batch(*args, seed=1, pad=2), 8, 64, False, rotate=False)
    check_append(Q, R.Batch(*args, seed=2, pad=2, lead=1), 8, 64, False, in_place=True)
    bt = R.Batch(*args, seed=3)
    cache, batch = bt.bind(Q)
    k, v = bt.randn(14, 2, 64), bt.randn(14, 2, 64)
    assert Q.qcf_paged_append(cache, batch, k, v) is None
    assert torch.equal(bt.rows(bt.k)[bt.own_at(2)], k[5:]) and torch.equal(bt.rows(bt.v)[bt.own_at(0)][16:], v[:4])


def test_paged_append_refuses_bad_pages_positions_and_lengths(Q):
    bt = R.Batch([2, 2, 2, 2], [2, 10, 9, 40], 10, 2, 64, 8, "rows", torch.bfloat16, seed=4, junk=0.0)
    bt.table[1, 1] = bt.k.shape[0]      # a page behind the cache: that sequence's rows 8 and 9
    bt.table[2, 1] = -5                 # row 8 of the third
    k, v, q = bt.randn(8, 2, 64), bt.randn(8, 2, 64), bt.randn(8, 4, 64)
    cache, batch = bt.bind(Q)
    out = torch.full_like(q, 7.0)
    Q.qcf_paged_append(cache, batch, k, v, Q.ScaledRopeTable(10 + 39, 64, 1e4, DEV), q=q, q_out=out)  # position 49 is outside
    assert Q.qcf_query_status() == 2
    used = (bt.rows(bt.k).abs().sum((2, 3)) > 0).sum()
    assert used == 2 + 0 + 1 + 1
    assert torch.all(out[7] == 7.0) and not torch.any(out[:7] == 7.0)
    # a length below the new rows, above the bound, rows behind n_rows: nothing of the sequence is written
    for change in (lambda: bt.kv_len.__setitem__(0, 1), lambda: bt.kv_len.__setitem__(0, 41),
                   lambda: bt.row_start.copy_(torch.tensor([0, 3, 4, 6, 8], dtype=torch.int32)),
                   lambda: bt.row_start.copy_(torch.tensor([0, 2, 4, 6, 9], dtype=torch.int32))):
        bt = R.Batch([2, 2, 2, 2], [2, 10, 9, 40], 10, 2, 64, 8, "rows", torch.bfloat16, seed=4, junk=0.0)
        change()
        cache, batch = bt.bind(Q)
        out.fill_(7.0)
        Q.qcf_paged_append(cache, batch, k, v, Q.ScaledRopeTable(100, 64, 1e4, DEV), q=q, q_out=out)
        assert Q.qcf_query_status() == 2
        assert torch.any(out == 7.0) and not torch.all(out == 7.0)


# ----------------------------------------------------------------- attention

def check_attention(Q, bt, Hq, q_more=0, std=1.0, want_lse=True, scale=None, **over):
    n, D = bt.n_rows, bt.D
    rows = bt.randn(n, Hq + q_more, D, std=std)
    q = rows[:, :Hq]
    scale = scale or 1.0 / math.sqrt(D)
    o, lse, tol, ltol = R.attention(bt, q, scale)
    cache, batch = bt.bind(Q, **over)
    out = torch.full((n, Hq, D), 7.0, dtype=bt.dtype, device=DEV)
    got = Q.qcf_shared_prefix_attn(cache, batch, q, scale, want_lse=want_lse, out=out)
    if want_lse:
        out, glse = got
    real = torch.zeros(n, dtype=torch.bool, device=DEV)
    for b, r, nq in bt.spans():
        real[r: r + nq] = True
    assert torch.all(out[~real] == 7.0), "a row of no sequence was written"
    within(out[real], o[real], tol[real], "attention")
    if want_lse:
        within(glse[real], lse[real], ltol[real], "lse")
    again = Q.qcf_shared_prefix_attn(cache, batch, q, scale)
    assert torch.equal(again[real], out[real]), "a second call gives other bits"


ATTN_CASES = [  # new, lens, prefix, Hq, Hkv, D, page
    ([1], [1], 0, 1, 1, 16, 8),
    ([1], [1], 1, 4, 4, 16, 16),
    ([1, 1, 1], [1, 64, 65], 127, 32, 8, 128, 16),
    ([1, 1], [129, 1], 128, 32, 8, 128, 128),
    ([1] * 5, [1, 2, 300, 16, 1000], 129, 28, 4, 128, 8),
    ([1] * 64, [1 + 7 * i for i in range(64)], 2049, 32, 8, 128, 16),
    ([7, 0, 1, 64, 0], [7, 5, 200, 80, 0], 1000, 16, 4, 128, 32),
    ([33, 64, 48], [33, 70, 500], 700, 32, 8, 128, 64),
    ([130], [1000], 0, 8, 8, 128, 256),
    ([1, 3], [5000, 700], 0, 16, 1, 128, 64),
    ([1] * 33, [40] * 33, 3333, 16, 1, 128, 32),
    ([2, 5, 1], [90, 5, 33], 77, 4, 4, 16, 8),
    ([1, 40], [260, 100], 515, 7, 1, 64, 16),
    ([20, 1, 1], [20, 3000, 1], 260, 32, 16, 64, 64),
    ([1] * 200, [1 + i % 5 for i in range(200)], 6000, 8, 2, 64, 16),
    ([97] * 8, [100 + 29 * i for i in range(8)], 1000, 32, 8, 128, 16),     # units of the prefix dealt out, the last row block half empty
    ([61, 3, 70], [61, 900, 70], 2000, 48, 3, 64, 32),                      # 16 heads a KV head
    ([5] * 9, [5 + 40 * i for i in range(9)], 400, 15, 5, 128, 8),          # 3 heads a KV head: rows left over in every tile
    ([1] * 700, [1 + (37 * i) % 90 for i in range(700)], 131, 2, 1, 128, 8),
    ([1, 6, 9], [300, 6, 40], 1500, 32, 4, 128, 256),
    ([300], [300], 64, 4, 1, 128, 64),                                      # a long question: early rows see few of its keys
    ([1] * 40, [1 + 11 * i for i in range(40)], 90, 8, 8, 16, 16),          # head dim 16 with more rows than a tile
    # prefixes long enough for their own kernel, with 7, 3, 8, 2 and 4 heads a KV head and last pages cut short
    ([1, 2, 3, 4], [30, 2, 300, 16], 9000, 28, 4, 128, 8),
    ([5] * 9, [5 + 40 * i for i in range(9)], 3003, 15, 5, 128, 8),
    ([1, 6, 9], [300, 6, 40], 9000, 32, 4, 128, 256),
    ([20, 1, 1], [20, 3000, 1], 4000, 32, 16, 64, 64),
    ([1, 40], [260, 100], 12000, 7, 1, 64, 16),
    ([7, 0, 1, 64, 0], [7, 5, 200, 80, 0], 3001, 16, 4, 128, 32),
]
LONG_CASES = [   # either side of the border between the two kernels: 3 tiles of 32 keys to each of 152 x 6 (D = 64: x 12) warps
    ([1] * 8, [3] * 8, 2736 * 32 // 16, 32, 8, 128, 16), ([1] * 8, [3] * 8, 2736 * 32 // 16 + 1, 32, 8, 128, 16),
    ([1] * 8, [3] * 8, 5472 * 32 // 16, 32, 8, 64, 16), ([1] * 8, [3] * 8, 5472 * 32 // 16 + 1, 32, 8, 64, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["rows", "heads"])
@pytest.mark.parametrize("new,lens,prefix,Hq,Hkv,D,page", ATTN_CASES + LONG_CASES)
def test_shared_prefix_attn(Q, dtype, layout, new, lens, prefix, Hq, Hkv, D, page):
    other = layout == "heads"
    bt = R.Batch(new, lens, prefix, Hkv, D, page, layout, TYPES[dtype], seed=len(new) + prefix, pad=5 * other, lead=3 * other).fill()
    check_attention(Q, bt, Hq, q_more=2 * other, want_lse=not other)


@pytest.mark.parametrize("std,scale", [(8.0, None), (1.0, 4.0), (0.01, None)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [1500, 10000])
def test_shared_prefix_attn_sharp_and_flat(Q, prefix, D, std, scale):
    bt = R.Batch([1, 2, 1, 30], [40, 9, 700, 64], prefix, 2, D, 16, "rows", torch.bfloat16, seed=3).fill()
    check_attention(Q, bt, 8, std=std, scale=scale)


def test_shared_prefix_attn_growing_logits(Q):
    """Keys whose logits grow along the prefix: the running maximum moves in every tile."""
    for D, prefix in ((64, 2000), (128, 2000), (64, 18000), (128, 18000)):
        bt = R.Batch([1, 1, 16], [300, 2, 60], prefix, 2, D, 32, "rows", torch.bfloat16, seed=6).fill()
        ramp = torch.linspace(0.05, 6.0, prefix, device=DEV)[:, None, None]
        bt.rows(bt.k)[bt.prefix_at()] = (ramp * torch.ones(prefix, 2, D, device=DEV)).to(torch.bfloat16)
        check_attention(Q, bt, 8)


@pytest.mark.parametrize("dtype", list(TYPES)[:2])
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("prefix", [0, 2000, 18000])
def test_shared_prefix_attn_small_weights_count(Q, prefix, D, dtype):
    """One key far above thousands whose weights are 2^-20.4 of its own: below fp16's normal range beside a
    largest weight of 1, and more than a hundredth of the sum."""
    bt = R.Batch([1, 1, 16], [18000 if prefix == 0 else 300, 2, 60], prefix, 2, D, 32, "rows", TYPES[dtype], seed=16).fill()
    q = torch.zeros(bt.n_rows, 8, D, dtype=TYPES[dtype], device=DEV)
    q[..., 0] = 8.0
    bt.k.zero_()
    for at in [bt.prefix_at()] + [bt.own_at(b) for b in range(3)]:
        bt.rows(bt.v)[at] = (1.0 + 0.25 * torch.rand(at[0].numel(), 2, D, generator=bt.g, device=DEV)).to(TYPES[dtype])
    for at in [bt.prefix_at()] if prefix else [bt.own_at(b) for b in range(3)]:
        bt.rows(bt.k)[at[0][1], at[1][1], :, 0] = 1.7675
        bt.rows(bt.v)[at[0][1], at[1][1]] = 0.0
    o, _, tol, _ = R.attention(bt, q, 1.0)
    cache, batch = bt.bind(Q)
    within(Q.qcf_shared_prefix_attn(cache, batch, q, 1.0), o, tol, "small weights")


def test_shared_prefix_attn_many_sequences(Q):
    """As many sequences as a call takes; most of one token, some empty."""
    n = 2048
    new = [0 if i % 7 == 3 else 1 for i in range(n)]
    lens = [q + (i * 13) % 5 for i, q in enumerate(new)]
    bt = R.Batch(new, lens, 40, 1, 64, 8, "rows", torch.bfloat16, seed=21).fill()
    q = bt.randn(bt.n_rows, 2, 64)
    cache, batch = bt.bind(Q)
    got = Q.qcf_shared_prefix_attn(cache, batch, q, 0.125)
    # every sequence alone is too many calls of the reference: gather all keys and mask
    at = bt.prefix_at()
    K, V = bt.rows(bt.k)[at][:, 0].double(), bt.rows(bt.v)[at][:, 0].double()
    seq = torch.tensor([i for i, x in enumerate(new) if x], device=DEV)
    pos = torch.arange(8, device=DEV)
    page = bt.table.long()[seq][:, pos // 8]
    live = pos < bt.kv_len[seq][:, None]
    Ko = torch.where(live[..., None], bt.rows(bt.k)[page, pos % 8][:, :, 0].double(), 0.0)
    Vo = torch.where(live[..., None], bt.rows(bt.v)[page, pos % 8][:, :, 0].double(), 0.0)
    x = torch.cat([torch.einsum("nhd,jd->nhj", q.double(), K), torch.einsum("nhd,njd->nhj", q.double(), Ko).masked_fill(~live[:, None], -math.inf)], -1) * 0.125
    p = torch.softmax(x, -1)
    ref = torch.einsum("nhj,jd->nhd", p[..., :40], V) + torch.einsum("nhj,njd->nhd", p[..., 40:], Vo)
    A = torch.einsum("nhj,jd->nhd", p[..., :40], V.abs()) + torch.einsum("nhj,njd->nhd", p[..., 40:], Vo.abs())
    # half a step of the weights and of the output; the 32-bit errors of _paged_reference.attention stay below 2^-13 here
    # (magnitudes of a logit's sum below 64 * 4 * 4 * 0.125)
    within(got, ref, (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -8 * ref.abs(), "many sequences")


def test_shared_prefix_attn_refuses_what_it_cannot_take(Q):
    from rag_kv_cache_re_gb300 import QcfError
    bt = R.Batch([1] * 3, [4] * 3, 10, 2, 64, 16, "rows", torch.bfloat16, seed=1).fill()
    cache, batch = bt.bind(Q)
    q = bt.randn(3, 8, 64)
    for bad in (lambda: Q.qcf_shared_prefix_attn(cache, batch, q.cpu(), 0.1), lambda: Q.qcf_shared_prefix_attn(cache, batch, q[:2], 0.1),
                lambda: Q.qcf_shared_prefix_attn(cache, batch, q.half(), 0.1), lambda: Q.qcf_shared_prefix_attn(cache, batch, q[:, :3].contiguous(), 0.1),
                lambda: Q.qcf_shared_prefix_attn(cache, batch, q, 0.0), lambda: Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, out=q[:, :4]),
                lambda: Q.qcf_shared_prefix_attn(cache, batch, q.transpose(1, 2).contiguous().transpose(1, 2), 0.1),
                lambda: Q.qcf_shared_prefix_attn(cache, bt.bind(Q, prefix_len=33)[1], q, 0.1),
                lambda: Q.qcf_shared_prefix_attn(cache, bt.bind(Q, max_len=17)[1], q, 0.1),
                lambda: bt.bind(Q, max_len=1 << 32), lambda: bt.bind(Q, max_q=-1),
                lambda: Q.qcf_paged_append(cache, batch, q[:, :2], q[:, 2:5]), lambda: Q.qcf_paged_append(cache, batch, q[:, :2], q[:, 2:4], q_out=q),
                lambda: Q.qcf_paged_append(cache, batch, q[:, :1], q[:, 1:2]),
                lambda: Q.qcf_rope_apply(q, torch.zeros(2, dtype=torch.int32, device=DEV), Q.ScaledRopeTable(8, 64, 1e4, DEV)),
                lambda: Q.qcf_rope_apply(q, torch.zeros(3, dtype=torch.int64, device=DEV), Q.ScaledRopeTable(8, 64, 1e4, DEV)),
                lambda: Q.qcf_rope_apply(q, torch.zeros(3, dtype=torch.int32, device=DEV), Q.ScaledRopeTable(8, 128, 1e4, DEV))):
        with pytest.raises(QcfError):
            bad()
    many = torch.zeros(2050, dtype=torch.int32, device=DEV)
    batch = Q.PagedBatch(many, many[1:].clone(), torch.zeros((2049, 1), dtype=torch.int32, device=DEV), 3, 1, 16)
    with pytest.raises(QcfError):
        Q.qcf_shared_prefix_attn(cache, batch, q, 0.1)


def test_shared_prefix_attn_loose_bounds(Q):
    """Bounds far above the batch: max_q, max_len and table columns nothing reaches."""
    for D in (16, 64, 128):
        bt = R.Batch([1, 4, 1], [70, 5, 1], 200, 2, D, 16, "rows", torch.bfloat16, seed=8, table_cols=200).fill()
        check_attention(Q, bt, 8, max_q=100, max_len=3200)


def test_shared_prefix_attn_leaves_bad_pages_out(Q):
    for D, prefix, Hq, Hkv in ((64, 300, 8, 2), (128, 300, 8, 2), (128, 2000, 8, 2), (64, 8000, 64, 8), (128, 8000, 64, 8)):
        bt = R.Batch([1] * 6, [5, 40, 9, 1, 17, 300], prefix, Hkv, D, 16, "rows", torch.bfloat16, seed=5, spare=0).fill()
        bt.prefix_pages[3] = bt.k.shape[0] + 4
        bt.prefix_pages[7] = -1
        q = bt.randn(6, Hq, D)
        good = bt.prefix_pages.clone()
        good[3], good[7] = 0, 0
        cache, batch = bt.bind(Q)
        got, lse = Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, want_lse=True)
        assert Q.qcf_query_status() == 2
        bt.prefix_pages.copy_(good)
        o, _, tol, _ = R.attention(bt, q, 0.1, skip_prefix=[*range(48, 64), *range(112, 128)])
        within(got, o, tol, "prefix pages")
        # own pages: the fifth sequence loses all of its two pages and has no prefix
        bt = R.Batch([1] * 6, [5, 40, 9, 1, 17, 300], 0, Hkv, D, 16, "rows", torch.bfloat16, seed=5).fill()
        bt.table[4, :2] = torch.tensor([1 << 30, -7], dtype=torch.int32)
        cache, batch = bt.bind(Q)
        got, lse = Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, want_lse=True)
        assert Q.qcf_query_status() == 2
        assert torch.all(got[4] == 0) and torch.all(lse[4] == -math.inf), "a row that sees no key"
        bt.table[4, :2] = 0
        o, _, tol, _ = R.attention(bt, q, 0.1)
        keep = torch.tensor([0, 1, 2, 3, 5], device=DEV)
        within(got[keep], o[keep], tol[keep], "other sequences")


def test_shared_prefix_attn_leaves_bad_sequences_out(Q):
    for D, prefix in ((64, 150), (128, 150), (128, 24000)):
        for change in ("short", "long", "rows"):
            bt = R.Batch([2, 3, 1], [40, 20, 7], prefix, 2, D, 16, "rows", torch.bfloat16, seed=9).fill()
            q = bt.randn(6, 8, D)
            o, _, tol, _ = R.attention(bt, q, 0.1)
            cache, batch = bt.bind(Q)
            if change == "short":
                bt.kv_len[1] = 2
            elif change == "long":
                bt.kv_len[1] = 41
            else:
                bt.row_start[3] = 8   # the last sequence reaches behind n_rows
            out = torch.full_like(q, 7.0)
            Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, out=out)
            assert Q.qcf_query_status() == 2
            bad = slice(5, 6) if change == "rows" else slice(2, 5)
            assert torch.all(out[bad] == 7.0)
            keep = [r for r in range(6) if not bad.start <= r < bad.stop]
            within(out[keep], o[keep], tol[keep], change)


def test_shared_prefix_attn_nan_queries_and_output_over_q(Q):
    """A NaN in one head's query makes that head's row NaN, joined or not, and nothing else; the output may be q."""
    for new, lens, prefix, Hq, D in (([1, 1, 9], [300, 2, 60], 0, 8, 128), ([1, 1, 1], [300, 2, 60], 900, 8, 64), ([3, 1, 30], [300, 2, 60], 900, 8, 128),
                                     ([3, 1, 30], [300, 2, 60], 6000, 8, 128), ([1, 1, 9], [300, 2, 60], 50, 8, 16)):
        bt = R.Batch(new, lens, prefix, 2, D, 16, "rows", torch.bfloat16, seed=12).fill()
        q = bt.randn(bt.n_rows, Hq, D)
        o, _, tol, _ = R.attention(bt, q, 0.1)
        cache, batch = bt.bind(Q)
        q[1, 3, 5] = math.nan
        got, lse = Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, want_lse=True)
        gone = torch.zeros(bt.n_rows, Hq, dtype=torch.bool, device=DEV)
        gone[1, 3] = True
        assert torch.equal(lse.isnan(), gone) and torch.equal(got.isnan(), gone[..., None].expand_as(got))
        within(got[~gone], o[~gone], tol[~gone], "other rows")
        assert Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, out=q) is q
        assert torch.equal(q.view(torch.int16), got.view(torch.int16))


def test_shared_prefix_attn_wide_bounds_of_many_sequences(Q):
    """Each of 256 sequences may be long and may bring many rows, but all rows together are few."""
    bt = R.Batch([1] * 255 + [40], [1 + i % 30 for i in range(255)] + [70], 90, 8, 128, 16, "rows", torch.bfloat16, seed=14, table_cols=8192).fill()
    check_attention(Q, bt, 64, max_q=512, max_len=131072)


def test_shared_prefix_attn_overlapping_sequences_are_not_run(Q):
    """Row ranges that go back make more work than the bounds allow: flagged, nothing written, nothing hangs."""
    n, rows = 2048, 512
    for prefix in (0, 100):
        cache = Q.PagedKV(*(torch.zeros(4, 256, 8, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
        start = torch.tensor([0, rows] * (n // 2) + [0], dtype=torch.int32, device=DEV)   # every second range runs backwards
        lens = torch.full((n,), 131072, dtype=torch.int32, device=DEV)
        table = torch.zeros(n, 512, dtype=torch.int32, device=DEV)
        pages = torch.zeros(1, dtype=torch.int32, device=DEV) if prefix else None
        batch = Q.PagedBatch(start, lens, table, rows, rows, 131072, pages, prefix)
        out = torch.full((rows, 64, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        Q.qcf_shared_prefix_attn(cache, batch, torch.ones_like(out), 0.1, out=out)
        assert Q.qcf_query_status() == 2
        assert torch.all(out == 7.0)


def test_empty_batches_write_nothing(Q):
    for new, lens in (([], []), ([0, 0], [0, 5])):
        bt = R.Batch(new, lens, 40, 2, 64, 16, "rows", torch.bfloat16, seed=2, pad=4, junk=0.0, table_cols=1)
        cache, batch = bt.bind(Q)
        q, out = bt.randn(4, 4, 64), torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, out=out)
        Q.qcf_paged_append(cache, batch, bt.randn(4, 2, 64), bt.randn(4, 2, 64), Q.ScaledRopeTable(64, 64, 1e4, DEV), q=q, q_out=out)
        assert torch.all(out == 7.0) and torch.all(bt.k == 0)
    bt = R.Batch([], [], 0, 2, 64, 16, "rows", torch.bfloat16, seed=2, table_cols=1)
    cache, batch = bt.bind(Q)
    assert Q.qcf_shared_prefix_attn(cache, batch, bt.randn(0, 4, 64), 0.1).shape == (0, 4, 64)


def test_cache_beyond_32_bit_offsets(Q):
    """Pages more than 2^31 entries from the base, in both layouts."""
    for layout in ("rows", "heads"):
        page, Hkv, D = 16, 8, 128
        n_pages = (1 << 31) // (page * Hkv * D) + 64
        bt = R.Batch([1, 2], [20, 33], 50, Hkv, D, page, layout, torch.bfloat16, seed=4)
        shape = (n_pages, page, Hkv, D) if layout == "rows" else (n_pages, Hkv, page, D)
        bt.k, bt.v = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        far = n_pages - 1 - torch.arange(bt.table.numel() + bt.prefix_pages.numel(), device=DEV, dtype=torch.int32)
        bt.prefix_pages.copy_(far[:4])
        bt.table.copy_(far[4:].view_as(bt.table))
        bt.fill()
        check_attention(Q, bt, 32)
        k, v = bt.randn(3, Hkv, D), bt.randn(3, Hkv, D)
        cache, batch = bt.bind(Q)
        Q.qcf_paged_append(cache, batch, k, v)
        assert torch.equal(bt.rows(bt.k)[bt.own_at(1)][31:], k[1:]) and torch.equal(bt.rows(bt.v)[bt.own_at(0)][19:], v[:1])


# ----------------------------------------------------------------- streams, graphs, the way they are used

@pytest.mark.parametrize("Hkv,prefix", [(8, 700), (4, 700), (4, 12000)])   # the prefix in the stream (one block of rows, two), and on its own kernel
def test_captured_steps_replay_with_other_lengths(Q, Hkv, prefix):
    """Append and attention captured once; replayed after tokens and lengths changed, two graphs and
    an eager call side by side on different streams."""
    made = []
    for seed in (1, 2):
        bt = R.Batch([1, 1, 1], [5, 60, 200], prefix, Hkv, 128, 16, "rows", torch.bfloat16, seed=seed, table_cols=40, spare=30).fill()
        bt.table[:, 13:] = 0
        order = torch.randperm(bt.k.shape[0], device=DEV)
        used = set(bt.prefix_pages.tolist()) | {int(p) for b in range(3) for p in bt.table[b, : -(-bt.lens[b] // 16)]}
        spare = [int(p) for p in order if int(p) not in used]
        for b in range(3):
            n = -(-bt.lens[b] // 16)
            bt.table[b, n: n + 3] = torch.tensor([spare.pop() for _ in range(3)], dtype=torch.int32)
        table = Q.ScaledRopeTable(prefix + 1300, 128, 1e4, DEV)
        rows = bt.randn(3, 32 + 2 * Hkv, 128)
        cache, batch = bt.bind(Q, max_len=640)
        qo, out = torch.empty(3, 32, 128, dtype=torch.bfloat16, device=DEV), torch.empty(3, 32, 128, dtype=torch.bfloat16, device=DEV)

        def step(rows=rows, cache=cache, batch=batch, table=table, qo=qo, out=out):
            q, k, v = rows.split([32, Hkv, Hkv], 1)
            Q.qcf_paged_append(cache, batch, k, v, table, q=q, q_out=qo)
            Q.qcf_shared_prefix_attn(cache, batch, qo, 0.09, out=out)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        made.append((bt, rows, graph, step, qo, out, torch.cuda.Stream()))
    for turn in range(20):
        torch.cuda.synchronize()
        for bt, rows, *_ in made:
            bt.kv_len += 1
            bt.lens = [n + 1 for n in bt.lens]
            rows.copy_(bt.randn(3, 32 + 2 * Hkv, 128))
        torch.cuda.synchronize()
        for bt, rows, graph, step, qo, out, stream in made:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for bt, rows, graph, step, qo, out, stream in made:
            got, gq = out.clone(), qo.clone()
            o, _, tol, _ = R.attention(bt, gq, 0.09)
            within(got, o, tol, f"replay {turn}")
            step()
            assert torch.equal(got, out) and torch.equal(gq, qo), "replay and eager call differ"


def test_other_streams(Q):
    bt = R.Batch([1, 4], [50, 9], 300, 2, 128, 16, "rows", torch.bfloat16, seed=8).fill()
    q = bt.randn(5, 8, 128)
    o, _, tol, _ = R.attention(bt, q, 0.1)
    cache, batch = bt.bind(Q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [Q.qcf_shared_prefix_attn(cache, batch, q, 0.1, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    for x in outs:
        within(x, o, tol, "stream")
        assert torch.equal(x, outs[0])


def test_answers_go_on_from_one_context(Q):
    """A tiny decoder: a context prefilled once and brought into pages, then three sequences that share it
    take several tokens each, through the library's norms, GEMMs, append and attention; the logits of every
    step are those of a full prefill of context and tokens (bf16 arithmetic both ways: the decoder's stated
    bound for hidden states, 2e-2 of the logits' scale)."""
    import qcfdata as qd
    from rag_kv_cache_re_gb300 import model as M
    spec = qd.TINY
    m = M.DeviceModel(qd.ModelWeights(spec), DEV, max_pos=256)
    Hq, Hkv, D, d = spec.n_heads, spec.n_kv_heads, spec.head_dim, spec.d_model
    ctx = torch.randint(0, spec.vocab, (77,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    Kc, Vc, _, _ = Q.qcf_full_prefill(m, ctx)
    page, B = 8, 3
    prefix_pages = torch.randperm(40, device=DEV)[:10].to(torch.int32)
    rest = torch.tensor([p for p in range(40) if p not in set(prefix_pages.tolist())], dtype=torch.int32, device=DEV)
    table = rest[: B * 4].view(B, 4).contiguous()
    caches = []
    for l in range(spec.n_layers):   # the context's rows, already rotated, into the prefix pages
        cache = Q.PagedKV(*(torch.full((40, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)))
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        Q.qcf_paged_append(cache, Q.PagedBatch(i32(0, 77), i32(77), prefix_pages[None].contiguous(), 77, 77, 77), Kc[l], Vc[l])
        caches.append(cache)
    seqs = [[], [], []]
    kv_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    gen = torch.Generator().manual_seed(5)
    for counts in ([5, 1, 3], [1, 1, 1], [1, 2, 0], [1, 1, 9]):   # a question each, then single tokens and more questions
        new = [torch.randint(0, spec.vocab, (c,), generator=gen).tolist() for c in counts]
        for s, t in zip(seqs, new):
            s.extend(t)
        ids = torch.tensor(sum(new, []) + [0, 0], dtype=torch.int32, device=DEV)   # two padding rows
        n = ids.numel()
        row_start = torch.tensor([0] + counts, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
        kv_len += torch.tensor(counts, dtype=torch.int32, device=DEV)
        batch = Q.PagedBatch(row_start, kv_len, table, n, 16, 32, prefix_pages, 77)
        x = Q.qcf_embed_rows(m, ids, None, n)
        for l in range(spec.n_layers):
            t = m.layer_tensors[l]
            qkv = Q.qcf_linear(Q.qcf_rmsnorm(x, t["g_attn"], spec.eps), t["w_qkv"]).view(n, Hq + 2 * Hkv, D)
            q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
            Q.qcf_paged_append(caches[l], batch, k, v, m.rope, q=q, q_out=q)
            o = Q.qcf_shared_prefix_attn(caches[l], batch, q, 1.0 / math.sqrt(D), out=torch.zeros((n, Hq, D), dtype=torch.bfloat16, device=DEV))
            Q.qcf_linear(o.view(n, Hq * D), t["w_o"], out=x, add=True)
            gu = Q.qcf_linear(Q.qcf_rmsnorm(x, t["g_mlp"], spec.eps), t["w_gu"]).float().view(n, -1, 2, 64)
            act = (torch.nn.functional.silu(gu[:, :, 0]) * gu[:, :, 1]).reshape(n, -1).to(torch.bfloat16)
            Q.qcf_linear(act, t["w_down"], out=x, add=True)
        for b in range(B):
            if counts[b] == 0:
                continue
            logits, _ = Q.qcf_lm_head(m, x[int(row_start[b + 1]) - 1].contiguous())
            whole = torch.cat([ctx, torch.tensor(seqs[b], dtype=torch.int32, device=DEV)])
            ref = Q.qcf_full_prefill(m, whole)[2]
            scale = max(1.0, float(ref.double().square().mean().sqrt()))
            assert torch.all((logits - ref).abs() <= 2e-2 * scale + 2e-2 * ref.abs())
