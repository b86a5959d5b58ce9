"""The gradient from keys given in parts: each part with the O and LSE of the softmax over all of them."""
from __future__ import annotations

import pytest
import torch

from bounds import check_cross_bwd

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    yield m
    assert m.fa2_device_status(clear=True) == 0


def make(Hq, Hkv, Nq, Nk, D, dtype):
    g = torch.Generator().manual_seed(Nq + D)
    q, do = (torch.randn(2, Hq, Nq, D, generator=g).to(dtype).cuda() for _ in range(2))
    k, v = (torch.randn(2, Hkv, Nk, D, generator=g).to(dtype).cuda() for _ in range(2))
    return q, k, v, do


@pytest.mark.parametrize("D,dtype", [(32, F16), (64, BF16), (96, BF16), (128, F16)])
@pytest.mark.parametrize("cuts", [[1], [1, 2, 3], [129, 130], [40, 200]], ids=str)
def test_each_part_with_the_whole_softmax(fa2, D, dtype, cuts):
    Nk = 203
    q, k, v, do = make(4, 2, 150, Nk, D, dtype)
    o, lse = fa2.cross_attention_forward(q, k, v)
    for a, b in zip([0] + cuts, cuts + [Nk]):
        kk, vv = k[:, :, a:b].contiguous(), v[:, :, a:b].contiguous()
        grads = fa2.cross_attention_backward(q, kk, vv, o, lse, do)
        check_cross_bwd(grads, q, kk, vv, o, lse, do, D ** -0.5, None)
        if b - a == 1:  # the part's gradient is not zero: its weight is below 1
            assert float(grads[0].abs().max()) > 0 and float(grads[1].abs().max()) > 0


@pytest.mark.parametrize("Nk", [100, 300])
def test_parts_by_key_lengths(fa2, Nk):
    # the first key alone of one batch entry, all of the other
    q, k, v, do = make(2, 2, 70, Nk, 64, F16)
    o, lse = fa2.cross_attention_forward(q, k, v)
    n = torch.tensor([1, Nk], dtype=torch.int32).cuda()
    k[0, :, 1:], v[0, :, 1:] = float("nan"), float("nan")
    grads = fa2.cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    check_cross_bwd(grads, q, k, v, o, lse, do, 0.125, n)
    assert float(grads[0][0].abs().max()) > 0


def test_a_part_that_was_the_whole(fa2):
    # rows whose weight is all on one key: with that key alone, O is V and dS exactly zero
    q, k, v, do = make(2, 1, 40, 2, 64, BF16)
    o, lse = fa2.cross_attention_forward(q, k, v, key_lengths=torch.ones(2, dtype=torch.int32).cuda())
    k1, v1 = k[:, :, :1].contiguous(), v[:, :, :1].contiguous()
    assert torch.equal(o, v1.expand_as(o))
    dq, dk, _ = fa2.cross_attention_backward(q, k1, v1, o, lse, do)
    assert bool((dq == 0).all()) and bool((dk == 0).all())
