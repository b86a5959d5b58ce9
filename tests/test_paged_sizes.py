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
