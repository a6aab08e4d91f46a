"""Calls of the rotary and paged operators at the far end of what their documentation allows, and side by side."""
import pytest
import torch

import _paged_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def Q():
    from rag_kv_cache_re_gb300 import qcf
    return qcf


@pytest.fixture(autouse=True)
def clean_status(Q):
    Q.qcf_query_status()
    yield
    assert Q.qcf_query_status() == 0, "a device-side check failed"


def test_rope_apply_of_more_than_32_bits_of_pairs(Q):
    """2^32 + 2^17 pairs of entries in one call, eight to a thread: every row as in a call of its own."""
    n, D, block = (1 << 24) + 512, 512, 1 << 12
    x = torch.empty((n, 1, D), dtype=torch.bfloat16, device=DEV)   # 17 GB
    g = torch.Generator(device=DEV).manual_seed(11)
    some = torch.randn((block, 1, D), generator=g, device=DEV).to(torch.bfloat16)
    some_pos = torch.randint(0, 4096, (block,), generator=g, device=DEV, dtype=torch.int32)
    whole = n // block * block
    x[:whole].view(-1, block, 1, D).copy_(some.expand(whole // block, block, 1, D))
    x[whole:] = some[: n - whole]
    pos = torch.cat([some_pos.repeat(whole // block), some_pos[: n - whole]])
    table = Q.ScaledRopeTable(4096, D, 1e4, DEV)
    ref, mag = R.rotate(some, some_pos, R.rates(D, 1e4))
    turned = Q.qcf_rope_apply(some, some_pos, table)
    assert torch.all((turned.double() - ref).abs() <= R.rotation_tolerance(ref, mag, torch.bfloat16))
    assert Q.qcf_rope_apply(x, pos, table, out=x) is x
    bits = turned.view(torch.int16)
    assert all(torch.equal(part.view(torch.int16), bits[: part.shape[0]]) for part in x.split(block))


@pytest.mark.parametrize("Hkv,prefix,D", [(8, 700, 128), (4, 12000, 128), (2, 9000, 64)])
def test_eager_calls_run_beside_replayed_graphs(Q, Hkv, prefix, D):
    """Two captured steps replayed on streams of their own while the same kind of step is called eagerly on a
    third, nothing waiting in between: the bits of each alone."""
    Hq = 32
    steps, graphs, held, seen = [], [], [], []
    for seed in (1, 2, 3):
        bt = R.Batch([1, 5, 1, 1], [5, 60, 200, 1], prefix, Hkv, D, 16, "rows", torch.bfloat16, seed=seed).fill()
        table = Q.ScaledRopeTable(prefix + bt.max_len, D, 1e4, DEV)
        rows = bt.randn(bt.n_rows, Hq + 2 * Hkv, D)
        cache, batch = bt.bind(Q)

        def step(rows=rows, cache=cache, batch=batch, table=table):
            q, k, v = rows.split([Hq, Hkv, Hkv], 1)
            qo = Q.qcf_paged_append(cache, batch, k, v, table, q=q)
            return (qo, *Q.qcf_shared_prefix_attn(cache, batch, qo, 0.09, want_lse=True))
        steps.append(step)
        seen.append([t.clone() for t in step()])
        q = seen[-1][0]
        o, _, tol, _ = R.attention(bt, q, 0.09)
        assert torch.all((seen[-1][1].double() - o).abs() <= tol)
    torch.cuda.synchronize()
    for step in steps[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(step())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for _ in range(8):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
            with torch.cuda.stream(streams[2]):
                got.append(steps[2]())
        torch.cuda.synchronize()
        for out, ref in [(h, r) for h, r in zip(held, seen)] + [(g, seen[2]) for g in got]:
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), "a step gives other bits beside the others"
