"""Sizes past those for which every index of the paged calls stays inside its type: refused before anything touches a GPU."""
from __future__ import annotations

import pytest

from test_paged import INVALID, call, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("keep", [(1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1])
def test_evict_to_more_than_a_sequence_can_have(lib, keep):  # noqa: F811
    assert call(lib, "evict", B=1, Hkv=1, keep=keep, new_width=1 << 27) == INVALID
