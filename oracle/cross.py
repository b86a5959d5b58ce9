"""Cross attention and its gradient in 64 bits (torch tensors in, torch float64 on the CPU out), head by head from the
definition. Shares no code with the GPU path.

The 64-bit products run on the device the tensors are on (plain torch
operations), only the loop and the results are on the host.
"""
from __future__ import annotations

import torch


def _heads(q, k, lengths):
    B, Hq = q.shape[:2]
    for b in range(B):
        n = k.shape[2] if lengths is None else min(max(int(lengths[b]), 0), k.shape[2])
        for h in range(Hq):
            yield b, h, h // (Hq // k.shape[1]), n


def forward(q, k, v, scale, lengths=None):
    """(O, LSE, A): A[b, h, i, :] = sum_j p_ij |v_j|, the size of the terms O is summed from."""
    o = torch.zeros(q.shape, dtype=torch.float64)
    a = torch.zeros_like(o)
    lse = torch.full(q.shape[:3], float("inf"), dtype=torch.float64)
    for b, h, g, n in _heads(q, k, lengths):
        if n == 0:
            continue
        kk, vv = k[b, g, :n].double(), v[b, g, :n].double()
        x = (q[b, h].double() @ kk.T) * scale
        l = torch.logsumexp(x, -1)
        p = torch.exp(x - l[:, None])
        lse[b, h], o[b, h], a[b, h] = l.cpu(), (p @ vv).cpu(), (p @ vv.abs()).cpu()
    return o, lse, a


def backward(q, k, v, o, lse, do, scale, lengths=None):
    """{"dq": (value, rounded, summed), "dk": ..., "dv": ...}, with P from `lse` and Delta from `o` as given.

    `rounded` is what the rounding of P and dS to 16 bits is relative to (sum of |dS| |k| and so on), `summed` the size
    of the products dP - Delta is the difference of, carried through the same sums.
    """
    out = {n: [torch.zeros(t.shape, dtype=torch.float64) for _ in range(3)] for n, t in
           (("dq", q), ("dk", k), ("dv", v))}
    for b, h, g, n in _heads(q, k, lengths):
        if n == 0:
            continue
        qq, kk, vv, gg, oo = (t.double() for t in (q[b, h], k[b, g, :n], v[b, g, :n], do[b, h], o[b, h]))
        p = torch.exp((qq @ kk.T) * scale - lse[b, h].double().to(q.device)[:, None])
        ds = p * (gg @ vv.T - (gg * oo).sum(-1, keepdim=True))
        big = p * (gg.abs() @ vv.abs().T + (gg * oo).abs().sum(-1, keepdim=True))
        for name, at, vals in (
                ("dq", (b, h, slice(None)), (ds @ kk * scale, ds.abs() @ kk.abs() * scale, big @ kk.abs() * scale)),
                ("dk", (b, g, slice(0, n)), (ds.T @ qq * scale, ds.abs().T @ qq.abs() * scale, big.T @ qq.abs() * scale)),
                ("dv", (b, g, slice(0, n)), (p.T @ gg, p.T @ gg.abs(), p.T @ gg.abs()))):
            for t, x in zip(out[name], vals):
                t[at] += x.cpu()
    return out
