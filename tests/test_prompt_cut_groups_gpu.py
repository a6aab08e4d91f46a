"""Chunk attention of groups of short sequences whose own tokens are so many that units are cut among them: parts that begin
with keys of one sequence, which most warps see nothing of and which leave the other rows' sums as they were cleared."""
import pytest
import torch

import _paged_reference as R
from test_prompt_gpu import TYPES, Q, check_chunk, clean_status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(32, 2, 128, "bf16"), (16, 1, 64, "f16"), (32, 8, 128, "f16"), (7, 1, 64, "bf16")])
@pytest.mark.parametrize("own", [300, 1500])
def test_parts_that_begin_among_own_tokens(Q, Hq, Hkv, D, dtype, own):  # noqa: F811
    """Rows in both row tiles of a CTA (16 heads a KV head), and in one of them, whose tiles go by turns."""
    lens = [own + 131 * (i % 5) for i in range(64)]
    bt = R.Batch([1] * 64, lens, 512, Hkv, D, 16, "rows", TYPES[dtype], seed=own + D).fill()
    check_chunk(Q, bt, Hq)
