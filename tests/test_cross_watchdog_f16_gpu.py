"""The device watchdog in cross attention's fp16 backward, whose compute warps wait for the K/V tile and for one another
before a unit's first step: a launch whose first tile is withheld ends by its own limit, and the next one is right."""
from __future__ import annotations

import pytest
import torch

from bounds import check_cross_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Nq,Nk,D,lengths", [(300, 900, 64, [900, 500]), (300, 900, 128, [900, 500]), (300, 77, 96, None),
                                             (3000, 100, 64, [100, 1])])
def test_a_withheld_tile_times_out(Nq, Nk, D, lengths):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as fa2
    fa2.fa2_device_status(clear=True)
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(2, 4, n, D, generator=g).half().cuda() for n in (Nq, Nk, Nk))
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    o, lse = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    call = lambda: fa2.cross_attention_backward(q, k, v, o, lse, q, key_lengths=n)  # noqa: E731
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
    check_cross_bwd(got, q, k, v, o, lse, q, D ** -0.5, n)
