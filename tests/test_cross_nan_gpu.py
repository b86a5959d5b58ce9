"""NaN and infinities in cross attention's inputs, in each of its kernels: where they show, and where they must not."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    yield m
    assert m.fa2_device_status(clear=True) == 0


CASES = [  # Nq, Nk, lengths, D: few rows, whole and cut; few keys; tcgen05, whole, keys in turn, cut
    (1, 77, None, 64), (1, 150, None, 64), (3, 4000, [4000, 3500], 128),
    (40, 77, None, 64), (300, 100, [77, 100], 128), (300, 150, None, 64), (300, 150, [150, 130], 128),
    (100, 700, None, 32), (100, 5000, [4900, 5000], 64), (200, 6000, None, 128),
]


def make(c, dtype):
    Nq, Nk, lengths, D = c
    g = torch.Generator().manual_seed(Nq + Nk)
    q, do = (torch.randn(2, 4, Nq, D, generator=g).to(dtype).cuda() for _ in range(2))
    k, v = (torch.randn(2, 2, Nk, D, generator=g).to(dtype).cuda() for _ in range(2))
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    return q, k, v, do, n


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_a_query_row_keeps_it_to_itself(fa2, c, value):
    q, k, v, _, n = make(c, BF16)
    want = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    q[0, 1, 0, 3] = value  # an infinity: scores of +inf and -inf, by the signs of its keys' elements
    o, lse = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    assert bool(o[0, 1, 0].isnan().all()) and bool(lse[0, 1, 0].isnan())
    o[0, 1, 0], lse[0, 1, 0] = want[0][0, 1, 0], want[1][0, 1, 0]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("c", CASES, ids=str)
def test_a_key_shows_in_every_row_of_its_head(fa2, c):
    q, k, v, _, n = make(c, F16)
    want = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    k[1, 0, 60, 5] = NAN
    o, lse = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    assert bool(o[1, :2].isnan().all()) and bool(lse[1, :2].isnan().all())
    assert torch.equal(o[0], want[0][0]) and torch.equal(o[1, 2:], want[0][1, 2:]) and torch.equal(lse[1, 2:], want[1][1, 2:])


@pytest.mark.parametrize("c", CASES, ids=str)
def test_the_gradient_of_a_nan_row(fa2, c):
    # P of the row is NaN: its dQ, and dK and dV of every key that its head has, not only dK
    q, k, v, do, n = make(c, F16)
    clean = fa2.cross_attention_backward(q, k, v, *fa2.cross_attention_forward(q, k, v, key_lengths=n), do, key_lengths=n)
    q[0, 1, 0, 3] = NAN
    dq, dk, dv = fa2.cross_attention_backward(q, k, v, *fa2.cross_attention_forward(q, k, v, key_lengths=n), do, key_lengths=n)
    keys = c[1] if n is None else c[2][0]
    assert bool(dq[0, 1, 0].isnan().all()) and int(dq.isnan().any(-1).sum()) == 1
    assert bool(dk[0, 0, :keys].isnan().all()) and bool(dv[0, 0, :keys].isnan().all())
    for t, w in ((dk, clean[1]), (dv, clean[2])):
        assert torch.equal(t[0, 0, keys:], w[0, 0, keys:]) and torch.equal(t[0, 1], w[0, 1]) and torch.equal(t[1], w[1])
