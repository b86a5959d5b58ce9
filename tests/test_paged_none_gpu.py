"""A page number that is none, through all of the paged calls: NaN rows, NaN weights at whatever those rows see, and an
eviction that keeps these first and the positions without a page last."""
from __future__ import annotations

import pytest
import torch

from paged_batches import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype,count", [(64, torch.float16, 100), (128, torch.bfloat16, 3)])
def test_what_follows_from_it(D, dtype, count):
    import attention_forward_03_gb300 as fa2
    b = Batch([100, 90], [count, 2], 2, D, 16, dtype, seed=D, spare=8)
    b.table[0, 2] = b.pages  # positions 32 to 47 of the first sequence
    q = b.tokens(4)
    o, lse = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch)
    sees = torch.arange(100 - count, 100, device="cuda") >= 32
    assert torch.equal(lse[:count].isnan().all(-1), sees) and torch.equal(o[:count].isnan().all(-1).all(-1), sees)
    assert not lse[count:].isnan().any() and not o[count:].isnan().any()
    w = fa2.paged_key_weights(q, lse, b.kc, *b.batch)
    at = [i for i in range(7) if i != 2]
    of = w[b.table[0, at].long()].transpose(1, 2).reshape(6 * 16, 2)[:84]  # the last row sees every position
    assert of.isnan().all()
    assert not w[b.table[1].long()[:6]].isnan().any()
    new = b.free[:4].reshape(2, 2)
    n, kept = fa2.paged_cache_evict(b.kc, b.vc, w, b.table, b.lens, new, 20, 4)
    assert kept[0].tolist() == [list(range(16)) + list(range(96, 100))] * 2 and n.tolist() == [20, 20]
