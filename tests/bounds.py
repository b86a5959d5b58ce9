"""How far a kernel's result may be from its definition in 64 bits, derived from the arithmetic.

Head norm with position rotation (near). For a result y that is a sum of terms of total size m (the oracle's
magnitude): half a step of the 16-bit type, |y| * eps16 / 2, for the one
rounding; and 32 steps of 2^-24 * m for the arithmetic in 32 bits: the mean
of squares (at most 32 + 5 + 1 additions, each a relative half step, halved
by the root), rsqrtf (2 steps), and up to 5 products and sums after it,
below 30 half steps together. The backward's mean adds as many again: 64. The
gain gradient is one such product per row, added up in at most 8 + 5 + 8 rows,
warps and threads of a block and 1280 / 8 + 8 blocks, below 256 + 64 half steps.

Cross attention. For O, per element, with A = sum_j p_ij |v_j| (u = half a step of the
16-bit type relative to the value): the weights are rounded once (u * A), the
result once (u * |O|). The 32-bit part: a score is a sum of D products in
32 bits, off by at most 16 steps of 2^-24 of s = scale * sum_d |q_d k_d| (16
accumulation steps at D = 128), which the exponential turns into a relative
error of its weight; ex2 and the sums add less than 32 such steps. In fp16 a
weight below 2^-14 (of a sum that is at least 1) is off by 2^-25 instead. LSE:
the same 32-bit part, and 4 steps of its own size for the logarithm and the
product with ln 2.

Bounds for the gradients, from O and LSE as the call got them: P and dS are
rounded once each (u * `rounded`, the oracle's sum of the terms' sizes), the
result once (u * |x|). The 32-bit part: weights off by 16 steps of s and 4 of
|LSE| (relative to `rounded`), dP and Delta by 16 steps of 2^-24 of the
products they are sums of (2^-20 * `summed`), and 64 steps for the sums. fp16:
P or dS below 2^-14 is off by 2^-25 of the other factor instead.
"""
from __future__ import annotations

import torch

from oracle import cross as ref

E32 = 2.0 ** -24
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half a step of the smallest fp16 subnormals


def near(got, want, mag, steps, dtype=None):
    dtype = dtype or got.dtype
    half = torch.finfo(dtype).eps / 2
    tol = half * want.abs() + steps * E32 * mag * (1 + half) + TINY.get(dtype, 0.0)
    got = got.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol).nan_to_num(0).max())} tolerances"


def sizes_of(q, k, scale, n):
    """max over all rows of scale * sum_d |q_d k_d|."""
    most = 0.0
    for b, h, g, m in ref._heads(q, k, n):
        if m:
            most = max(most, float((q[b, h].float().abs() @ k[b, g, :m].float().abs().T).max()) * scale)
    return most


def check_cross_fwd(o, lse, q, k, v, scale, n):
    want_o, want_l, a = ref.forward(q, k, v, scale, n)
    u = torch.finfo(q.dtype).eps / 2
    s32 = (16 * sizes_of(q, k, scale, n) + 32) * E32
    tol = u * (a + want_o.abs()) * (1 + u) + s32 * a
    if q.dtype == torch.float16:
        vs = v.float().nan_to_num(0.0).abs().sum(2).repeat_interleave(q.shape[1] // v.shape[1], 1)
        tol = tol + 2.0 ** -25 * (vs.cpu().double()[:, :, None] + 1)
    o, lse = o.cpu().double(), lse.cpu().double()
    empty = want_l.isinf()
    assert torch.equal(lse.isinf(), empty) and bool((lse[empty] > 0).all())
    assert bool((o[empty] == 0).all())
    assert not o.isnan().any() and not lse.isnan().any()
    bad = (o - want_o).abs() > tol
    assert not bad.any(), f"O: {int(bad.sum())} of {bad.numel()}, worst {float(((o - want_o).abs() / tol.clamp(min=1e-30)).max())} tolerances"
    dl = (lse - want_l)[~empty].abs()
    tl = s32 + 4 * E32 * want_l[~empty].abs()
    assert bool((dl <= tl).all()), f"LSE off by {float((dl / tl).max())} tolerances"


def check_cross_bwd(grads, q, k, v, o, lse, do, scale, n):
    want = ref.backward(q, k, v, o, lse, do, scale, n)
    u = torch.finfo(q.dtype).eps / 2
    fin = lse[~lse.isinf()]
    s32 = (16 * sizes_of(q, k, scale, n) + 4 * (float(fin.abs().max()) if fin.numel() else 0) + 64) * E32
    group = q.shape[1] // k.shape[1]
    for name, got in zip(("dq", "dk", "dv"), grads):
        x, rounded, summed = want[name]
        tol = u * (rounded + x.abs()) * (1 + u) + s32 * rounded + 2.0 ** -20 * summed
        if q.dtype == torch.float16:
            if name == "dq":
                other = k.float().nan_to_num(0.0, 0.0, 0.0).abs().sum(2, keepdim=True).repeat_interleave(group, 1) * scale
            else:
                other = (q.float() * scale if name == "dk" else do.float()).abs().sum(2, keepdim=True)
                other = other.unflatten(1, (k.shape[1], group)).sum(2)
            tol = tol + 2.0 ** -25 * (other.cpu().double() + 1)
        got = got.cpu().double()
        assert not got.isnan().any(), name
        bad = (got - x).abs() > tol
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, worst {float(((got - x).abs() / tol.clamp(min=1e-30)).max())} tolerances"
        if n is not None and name != "dq":  # zeros behind the keys, exactly
            for b in range(k.shape[0]):
                assert bool((got[b, :, min(max(int(n[b]), 0), k.shape[2]):] == 0).all()), name
