"""The device watchdog in the paged calls, without any GPU fault: a launch whose first tile is withheld ends by its own
limit and says so, and the next launch on the same workspace is right."""
from __future__ import annotations

import pytest
import torch

from bounds import check_key_weights, check_paged_attention
from paged_batches import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    m.fa2_device_status(clear=True)
    return m


@pytest.mark.parametrize("counts", [[1, 1], [300, 200], [300, 1], [2600, 2600]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("op", ["attention", "weights"])
def test_a_withheld_tile_times_out(fa2, counts, D, op):
    b = Batch([6000, 2600], counts, 4, D, 16, torch.bfloat16, seed=2)
    q = b.tokens(8)
    o, lse = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch)

    def call():
        return fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch) if op == "attention" else \
            fa2.paged_key_weights(q, lse, b.kc, *b.batch)

    call()
    torch.cuda.synchronize()
    try:
        fa2.fa2_set_watchdog_ns(20_000_000)  # 20 ms
        assert fa2.library().fa2_test_withhold_next_load(1) == fa2.FA2_OK
        call()
        torch.cuda.synchronize()  # returns: every wait is bounded
        assert fa2.fa2_device_status(clear=True) > 0
    finally:
        fa2.library().fa2_test_withhold_next_load(0)
        fa2.fa2_set_watchdog_ns(0)
    got = call()
    torch.cuda.synchronize()
    assert fa2.fa2_device_status(clear=True) == 0
    if op == "attention":
        check_paged_attention(*got, q, b.kc, b.vc, b.batch, D ** -0.5)
    else:
        check_key_weights(got, q, lse, b.kc, None, b.batch, D ** -0.5)
