"""The device watchdog in cross attention, without any GPU fault: a launch whose first K/V tile is withheld ends by its
own limit and says so, and the next launch on the same workspace is right."""
from __future__ import annotations

import pytest
import torch

from bounds import check_cross_bwd, check_cross_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    m.fa2_device_status(clear=True)
    return m


@pytest.mark.parametrize("Nq,D", [(1, 128), (1, 64), (300, 128), (300, 64)])
def test_a_withheld_tile_times_out(fa2, Nq, D):
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(2, 4, n, D, generator=g).bfloat16().cuda() for n in (Nq, 900, 900))
    n = torch.tensor([900, 500], dtype=torch.int32).cuda()
    o, lse = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    calls = [lambda: fa2.cross_attention_forward(q, k, v, key_lengths=n)]
    if Nq > 1:
        calls.append(lambda: fa2.cross_attention_backward(q, k, v, o, lse, q, key_lengths=n))
    for call in calls:
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
        if len(got) == 2:
            check_cross_fwd(*got, q, k, v, D ** -0.5, n)
        else:
            check_cross_bwd(got, q, k, v, o, lse, q, D ** -0.5, n)


def test_a_withheld_tile_of_a_cut_unit_times_out(fa2):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(1, 2, n, 64, generator=g).bfloat16().cuda() for n in (300, 6000, 6000))
    fa2.cross_attention_forward(q, k, v)
    torch.cuda.synchronize()
    try:
        fa2.fa2_set_watchdog_ns(20_000_000)  # 20 ms
        assert fa2.library().fa2_test_withhold_next_load(1) == fa2.FA2_OK
        fa2.cross_attention_forward(q, k, v)
        torch.cuda.synchronize()  # the holders of the units' first tiles give up waiting for the others, too
        assert fa2.fa2_device_status(clear=True) > 0
    finally:
        fa2.library().fa2_test_withhold_next_load(0)
        fa2.fa2_set_watchdog_ns(0)
    o, lse = fa2.cross_attention_forward(q, k, v)
    torch.cuda.synchronize()
    assert fa2.fa2_device_status(clear=True) == 0
    check_cross_fwd(o, lse, q, k, v, 0.125, None)


@pytest.mark.parametrize("Nk", [900, 6000])  # whole units and cut ones
def test_a_withheld_tile_times_out_with_key_tiles_in_turn(fa2, Nk):
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(2, 4, n, 64, generator=g).bfloat16().cuda() for n in (100, Nk, Nk))
    fa2.cross_attention_forward(q, k, v)
    torch.cuda.synchronize()
    try:
        fa2.fa2_set_watchdog_ns(20_000_000)  # 20 ms
        assert fa2.library().fa2_test_withhold_next_load(1) == fa2.FA2_OK
        fa2.cross_attention_forward(q, k, v)
        torch.cuda.synchronize()
        assert fa2.fa2_device_status(clear=True) > 0
    finally:
        fa2.library().fa2_test_withhold_next_load(0)
        fa2.fa2_set_watchdog_ns(0)
    o, lse = fa2.cross_attention_forward(q, k, v)
    torch.cuda.synchronize()
    assert fa2.fa2_device_status(clear=True) == 0
    check_cross_fwd(o, lse, q, k, v, 0.125, None)
