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
