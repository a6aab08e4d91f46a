"""Prompt and chunk attention of every kind of head group up to 128 query heads to a KV head: with one, two or a few tokens to a
row tile of 128 score rows, and row tiles that leave 1 to 64 of them unused."""
import pytest
import torch

import _paged_reference as R
from test_prompt_gpu import TYPES, Q, check_chunk, check_packed, clean_status  # noqa: F401

pytestmark = pytest.mark.gpu

GROUPS = [17, 32, 33, 42, 43, 48, 49, 64, 65, 71, 96, 97, 128]


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("G", GROUPS)
def test_packed(Q, G, D):  # noqa: F811
    """A row tile in part and whole, one and two of them to a CTA, several units."""
    per = 128 // G
    check_packed(Q, [1, per, 2 * per, 2 * per + 1, 4 * per, 9 * per + 1, 130], G, 1, D, torch.bfloat16, seed=G, lead=2, pad=3)


@pytest.mark.parametrize("Hkv,D,dtype", [(1, 128, "bf16"), (2, 64, "f16")])
@pytest.mark.parametrize("G", GROUPS)
def test_packed_long(Q, G, Hkv, D, dtype):  # noqa: F811
    """Units of many key tiles, whole and cut between them."""
    check_packed(Q, [900, 1, 301], G * Hkv, Hkv, D, TYPES[dtype], seed=G + 1)
    check_packed(Q, [900, 1, 301], G * Hkv, Hkv, D, TYPES[dtype], seed=G + 2, window=200)


@pytest.mark.parametrize("Hkv,D,page,layout,dtype", [(1, 128, 16, "rows", "f16"), (2, 128, 64, "heads", "bf16"), (2, 64, 8, "rows", "bf16")])
@pytest.mark.parametrize("G", GROUPS)
def test_chunk(Q, G, Hkv, D, page, layout, dtype):  # noqa: F811
    """Single tokens, tokens of a few row tiles and a long chunk, behind a prefix and cached tokens."""
    per = 128 // G
    bt = R.Batch([1, 4 * per, 2 * per, 0, 1, 70, 3], [2000, 300, 2 * per, 9, 1, 500, 129], 700, Hkv, D, page, layout, TYPES[dtype], seed=G, pad=2, lead=1).fill()
    check_chunk(Q, bt, G * Hkv)
    check_chunk(Q, bt, G * Hkv, window=300)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", GROUPS)
def test_chunk_of_one_token(Q, G, D):  # noqa: F811
    """One token over a long cache: its unit cut into many parts."""
    bt = R.Batch([1], [9001], 0, 1, D, 32, "rows", torch.bfloat16, seed=G).fill()
    check_chunk(Q, bt, G)
