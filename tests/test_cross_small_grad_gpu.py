"""Cross attention's fp16 gradient for upstream gradients of any size: P and dS are rounded to 16 bits, and must not be
lost among fp16's subnormals when dO is small or the keys are many.

The bound is that of bounds.py without its allowance for subnormals (2^-25 of the other factor for every weight, which
a gradient from small dO would disappear in). The kernels take P and dS 2^e times as large, e per tile of 128 keys: the
largest up to 14 with 2^e (D max |dO_id| max |V_jd| + max |Delta_i|) <= 2^15, so what is left of it is 2^-25 * 2^-e.
Here e is that of all the head's keys, which is no larger, less 1 for the 32-bit rounding of the sum at a power of two.
The result's own half step among the subnormals is 2^-25.
"""
from __future__ import annotations

import math

import pytest
import torch

from bounds import E32, sizes_of
from oracle import cross as ref

pytestmark = pytest.mark.gpu

F16 = torch.float16
U = torch.finfo(F16).eps / 2


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    yield m
    assert m.fa2_device_status(clear=True) == 0


def make(B, Hq, Hkv, Nq, Nk, D, lengths, size, v_size=1.0):
    g = torch.Generator().manual_seed(Nq + Nk + D)
    q, do = (torch.randn(B, Hq, Nq, D, generator=g) for _ in range(2))
    k, v = (torch.randn(B, Hkv, Nk, D, generator=g) for _ in range(2))
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    return q.half().cuda(), k.half().cuda(), (v * v_size).half().cuda(), (do * size).half().cuda(), n


def shift(do, o, v, lengths):
    """At most the e of every key head's tiles, [B, Hkv]."""
    B, Hq = do.shape[:2]
    H, Nk = v.shape[1:3]
    if lengths is not None:
        v = v.masked_fill((torch.arange(Nk, device=v.device)[None] >= lengths[:, None])[:, None, :, None], 0)
    most = lambda t: t.amax(-1)  # noqa: E731
    delta = (do.double() * o.double()).sum(-1).abs()
    size = do.shape[3] * most(do.abs().reshape(B, H, -1)).double() * most(v.abs().reshape(B, H, -1)).double() + \
        most(delta.reshape(B, H, -1))
    return [[min(14, max(0, math.floor(math.log2(2 ** 15 / max(x, 1e-30))))) - 1 for x in row] for row in size.tolist()]


def check(grads, q, k, v, o, lse, do, scale, n):
    want = ref.backward(q, k, v, o, lse, do, scale, n)
    s32 = (16 * sizes_of(q, k, scale, n) + 4 * float(lse[~lse.isinf()].abs().max()) + 64) * E32
    B, group = q.shape[0], q.shape[1] // k.shape[1]
    left = 2.0 ** -25 * torch.tensor([[2.0 ** -e for e in row] for row in shift(do, o, v, n)], dtype=torch.float64)
    for name, got in zip(("dq", "dk", "dv"), grads):
        x, rounded, summed = want[name]
        if name == "dq":
            other = k.double().abs().sum(2, keepdim=True).cpu() * scale * left[:, :, None, None]
            other = other.repeat_interleave(group, 1)
        else:
            other = (q.double() * scale if name == "dk" else do.double()).abs().sum(2, keepdim=True).cpu()
            other = other.unflatten(1, (k.shape[1], group)).sum(2) * left[:, :, None, None]
        tol = U * (rounded + x.abs()) * (1 + U) + s32 * rounded + 2.0 ** -20 * summed + 2.0 ** -25 + other
        got = got.cpu().double()
        assert bool(got.isfinite().all()), name
        bad = (got - x).abs() > tol
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, worst {float(((got - x).abs() / tol).max())} tolerances"


CASES = [  # B, Hq, Hkv, Nq, Nk, D, lengths: one key tile (dQ straight out), many (dQ added up), cut units
    (2, 4, 2, 200, 100, 64, None), (1, 2, 2, 300, 77, 128, None), (2, 2, 1, 130, 128, 32, [128, 1]),
    (1, 4, 2, 300, 8192, 64, None), (2, 2, 2, 200, 6000, 128, [6000, 1500]), (1, 2, 2, 700, 1500, 96, None),
    (1, 2, 1, 100, 20000, 32, None), (3, 4, 4, 90, 900, 64, [0, 900, 300]),
]


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4, 1e-6])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_gradient(fa2, c, size):
    q, k, v, do, n = make(*c, size)
    o, lse = fa2.cross_attention_forward(q, k, v, key_lengths=n)
    grads = fa2.cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    check(grads, q, k, v, o, lse, do, c[5] ** -0.5, n)


@pytest.mark.parametrize("size,v_size", [(1e-4, 1000.0), (300.0, 1.0), (5.0, 5000.0), (1e-6, 1e-4)])
def test_sizes_of_the_two_factors(fa2, size, v_size):
    # P (dP - Delta) has room for large values, and none of them overflows in 16 bits
    q, k, v, do, n = make(2, 4, 2, 150, 700, 64, None, size, v_size)
    o, lse = fa2.cross_attention_forward(q, k, v)
    grads = [t.clone() for t in fa2.cross_attention_backward(q, k, v, o, lse, do)]
    want = ref.backward(q, k, v, o, lse, do, 0.125)
    for t, (x, _, _) in zip(grads, want.values()):  # what fp16 cannot hold at all is not asked for
        t[(x.abs() > 60000).cuda()] = 0
        x[x.abs() > 60000] = 0
    assert all(bool(t.isfinite().all()) for t in grads)
    if max(float(x.abs().max()) for x, _, _ in want.values()) < 60000:
        check(grads, q, k, v, o, lse, do, 0.125, n)


def test_heads_of_different_sizes(fa2):
    q, k, v, do, _ = make(2, 4, 2, 150, 2000, 64, None, 1.0)
    do *= torch.tensor([[1e-4, 1e-4, 10.0, 10.0], [1e-2, 1e-3, 1e-5, 1.0]]).half().cuda()[:, :, None, None]
    o, lse = fa2.cross_attention_forward(q, k, v)
    check(fa2.cross_attention_backward(q, k, v, o, lse, do), q, k, v, o, lse, do, 0.125, None)


def test_many_heads(fa2):
    B, H, Nq, Nk, D, scale = 3, 3000, 3, 40, 32, 32 ** -0.5
    q, k, v, do, _ = make(B, H, H, Nq, Nk, D, None, 1e-4)
    o, lse = fa2.cross_attention_forward(q, k, v)
    dq, dk, dv = fa2.cross_attention_backward(q, k, v, o, lse, do)
    Q, K, V, G, O = (t.double() for t in (q, k, v, do, o))
    p = torch.exp(Q @ K.transpose(2, 3) * scale - lse.double()[..., None])
    ds = p * (G @ V.transpose(2, 3) - (G * O).sum(-1, keepdim=True))
    big = p * (G.abs() @ V.abs().transpose(2, 3) + (G * O).abs().sum(-1, keepdim=True))
    s32 = (16 * float((Q.abs() @ K.abs().transpose(2, 3)).max()) * scale + 4 * float(lse.abs().max()) + 64) * E32
    left = 2.0 ** -25 * 2.0 ** -(min(min(row) for row in shift(do, o, v, None)))
    for got, x, r, s, f in (
            (dq, ds @ K * scale, ds.abs() @ K.abs() * scale, big @ K.abs() * scale, K.abs().sum(2, keepdim=True) * scale),
            (dk, ds.transpose(2, 3) @ Q * scale, ds.abs().transpose(2, 3) @ Q.abs() * scale,
             big.transpose(2, 3) @ Q.abs() * scale, Q.abs().sum(2, keepdim=True) * scale),
            (dv, p.transpose(2, 3) @ G, p.transpose(2, 3) @ G.abs(), p.transpose(2, 3) @ G.abs(), G.abs().sum(2, keepdim=True))):
        tol = U * (r + x.abs()) * (1 + U) + s32 * r + 2.0 ** -20 * s + 2.0 ** -25 + left * f
        assert bool(((got.double() - x).abs() <= tol).all())


def test_captured_and_replayed_with_another_size(fa2):
    q, k, v, do, _ = make(2, 4, 2, 300, 900, 64, None, 1.0)
    o, lse = fa2.cross_attention_forward(q, k, v)
    fa2.cross_attention_backward(q, k, v, o, lse, do)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = fa2.cross_attention_backward(q, k, v, o, lse, do)
    for size in (1e-4, 0.1, 50.0):
        do.copy_(make(2, 4, 2, 300, 900, 64, None, size)[3])
        graph.replay()
        torch.cuda.synchronize()
        check(grads, q, k, v, o, lse, do, 0.125, None)
        want = fa2.cross_attention_backward(q, k, v, o, lse, do)
        assert torch.equal(grads[1], want[1]) and torch.equal(grads[2], want[2])


def test_infinities_do_not_reach_other_heads(fa2):
    q, k, v, do, _ = make(1, 4, 4, 70, 300, 64, None, 1e-3)
    o, lse = fa2.cross_attention_forward(q, k, v)
    want = fa2.cross_attention_backward(q, k, v, o, lse, do)
    do[0, 2, 7, 1] = float("inf")
    got = fa2.cross_attention_backward(q, k, v, o, lse, do)
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[0, [0, 1, 3]], b[0, [0, 1, 3]])
    assert not bool(got[1][0, 2].isfinite().all())
