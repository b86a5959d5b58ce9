"""max_query_length chooses the kernels of the paged calls: whatever it is they are right to the same bounds, and the same
call gives the same bits again."""
from __future__ import annotations

import math

import pytest
import torch

from bounds import check_key_weights, check_paged_attention
from paged_batches import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    from attention_forward_03_gb300 import binding
    yield binding
    assert binding.fa2_device_status(clear=True) == 0


@pytest.mark.parametrize("lengths,counts,Hq,Hkv,D,page,dtype", [
    ([1500, 700, 40], [300, 1, 5], 8, 2, 64, 16, F16),
    ([2000] * 6, [40, 1, 1, 7, 200, 33], 24, 8, 128, 32, BF16),
    ([500, 400], [17, 17], 16, 1, 96, 64, BF16),
])
def test_any_number_is_right_and_repeats(lengths, counts, Hq, Hkv, D, page, dtype):
    import attention_forward_03_gb300 as fa2
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=Hq)
    q = b.tokens(Hq, 1.5)
    scale = 1 / math.sqrt(D)
    for most in (0, 1, 2, 16, max(counts), b.T, 1 << 30, None):
        o, lse = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch, max_query_length=most)
        w = fa2.paged_key_weights(q, lse, b.kc, *b.batch, max_query_length=most)
        check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, scale)
        check_key_weights(w, q, lse, b.kc, None, b.batch, scale)
        for _ in range(3):
            again = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch, max_query_length=most)
            assert torch.equal(again[0], o) and torch.equal(again[1], lse)
            assert torch.equal(fa2.paged_key_weights(q, lse, b.kc, *b.batch, max_query_length=most), w)
