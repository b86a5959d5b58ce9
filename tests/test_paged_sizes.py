"""Sizes past those for which every index of the paged calls stays inside its type: refused before anything touches a GPU."""
from __future__ import annotations

import pytest

from test_paged import A, GOOD, INVALID, call, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("keep", [(1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1])
def test_evict_to_more_than_a_sequence_can_have(lib, keep):  # noqa: F811
    assert call(lib, "evict", B=1, Hkv=1, keep=keep, new_width=1 << 27) == INVALID


FAR = dict(lengths=20 * A, starts=24 * A, new_lengths=30 * A, kept=40 * A)  # where long rows of numbers meet nothing


@pytest.mark.parametrize("B", [(1 << 30) + 1, (1 << 31) - 1])
@pytest.mark.parametrize("op", sorted(GOOD))
def test_more_sequences_than_an_index_and_a_warp_s_step_hold(lib, op, B):  # noqa: F811
    strides = GOOD[op]["strides"]
    strides = strides[:-2] + (0, 0) if op == "evict" else strides[:-1] + (0,)  # one row of the table for all
    assert call(lib, op, B=B, Hkv=1, Hq=1, strides=strides, **FAR) == INVALID


# key heads a D apart in what is read, so that nothing meets anything
@pytest.mark.parametrize("Hkv", [(1 << 24) + 1, 1 << 28])
@pytest.mark.parametrize("op", sorted(GOOD))
def test_more_key_heads_than_a_block_of_rows_can_index(lib, op, Hkv):  # noqa: F811
    cache, tokens = (8, 8, 64), (64, 8)
    strides = {"append": (*tokens, *tokens, *cache, *cache, 10), "fwd": (*tokens, *cache, *cache, 10),
               "weights": (*tokens, *cache, 10), "evict": (*cache, *cache, 10, 4)}[op]
    far = dict(K=A, V=20 * A, Q=A, kc=40 * A, vc=60 * A, w=80 * A if op != "append" else None, table=400 * A, lengths=401 * A,
               starts=402 * A, O=410 * A, LSE=500 * A, ws=600 * A, out=700 * A, new=403 * A, new_lengths=404 * A, kept=410 * A)
    assert call(lib, op, B=1, T=1, pages=1, keep=16, recent=0, Hkv=Hkv, Hq=Hkv, strides=strides, **far) == INVALID
