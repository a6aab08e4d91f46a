"""What a refused compaction of a pool leaves and returns."""
import pytest
import torch

from test_pages_gpu import BAD_INDEX, Pool, Q, clean_status, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [-1, 49])
def test_refused_compact_returns_no_count(Q, value):  # noqa: F811
    """A length out of range: no page moves, so no count may say which pages are free."""
    p = Pool(Q, 30, 5, 6, page=8)
    p.resize([20, 9, 8, 0, 0])
    p.resize([0], [0])                           # holes below the others' pages
    p.check()
    p.pool.kv_len[1] = value
    live = Q.qcf_pages_compact(p.pool)
    assert Q.qcf_query_status() == BAD_INDEX
    assert live.tolist() == [-1]
    p.pool.kv_len[1] = 9
    p.check()
    p.compact()
    p.check()


def test_replayed_compact_says_each_time(Q):  # noqa: F811
    """A captured compaction replayed over a good, a bad and again a good length."""
    p = Pool(Q, 30, 5, 6, page=8)
    p.resize([20, 9, 8, 0, 0])
    Q.qcf_pages_compact(p.pool)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        live = Q.qcf_pages_compact(p.pool)
    for length, status, count in ((9, 0, 6), (49, BAD_INDEX, -1), (9, 0, 6)):
        p.pool.kv_len[1] = length
        graph.replay()
        assert Q.qcf_query_status() == status and live.tolist() == [count]
    p.check()
