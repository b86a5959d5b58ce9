"""What a paged call writes overlaps nothing that it reads besides: refused before anything touches a GPU."""
from __future__ import annotations

import pytest

from test_paged import A, INVALID, call, lib  # noqa: F401  (a fixture)

# In the calls of test_paged the caches reach over 1,638,400 bytes each, the weights over 51,200, the tables over 160 and 64.
EVICT = [
    dict(w=3 * A), dict(w=4 * A + 1024), dict(w=3 * A - 64), dict(kc=11 * A + 4096),  # weights and a cache
    dict(table=3 * A + 64), dict(table=4 * A + 1024), dict(table=11 * A + 128), dict(vc=5 * A),
    dict(new=3 * A + 64), dict(new=4 * A + 1024), dict(new=11 * A + 128),
    dict(lengths=3 * A + 64), dict(lengths=4 * A + 1024), dict(lengths=11 * A + 128),
]


@pytest.mark.parametrize("over", EVICT, ids=str)
def test_evict(lib, over):  # noqa: F811
    assert call(lib, "evict", **over) == INVALID


# the weights beside the caches that the same call writes
APPEND = [dict(w=3 * A), dict(w=3 * A + 4096), dict(w=4 * A + 64), dict(w=4 * A - 64), dict(w=11 * A, kc=11 * A + 1024)]


@pytest.mark.parametrize("over", APPEND, ids=str)
def test_append(lib, over):  # noqa: F811
    assert call(lib, "append", **over) == INVALID
