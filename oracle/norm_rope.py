"""Head norm with position rotation and its gradient, in 64 bits on the CPU (torch tensors in, torch float64 out).

Row by row from the definition: y = x / sqrt(mean(x^2) + eps) * gain, then the
leading 2 * half elements rotated in pairs. Shares no code with the GPU path.
"""
from __future__ import annotations

import torch


def _pairs(rot: int, interleaved: bool):
    """Element indices (first, second) of the rotated pairs."""
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _angles(cos, sin, positions, B, N):
    if cos is None:
        return None, None
    pos = torch.arange(N).expand(B, N) if positions is None else positions.cpu().long().expand(B, N)
    out = []
    for t in (cos, sin):
        t = t.cpu().double()
        inside = (pos >= 0) & (pos < t.shape[0])
        a = t[pos.clamp(0, t.shape[0] - 1)]
        a[~inside] = float("nan")
        out.append(a[:, None])  # [B, 1, N, rot/2]
    return out[0], out[1]


def forward(x, gain, cos, sin, positions=None, eps=1e-6, interleaved=False):
    """(y, magnitude): the result and the size of the terms it is summed from, both like x."""
    x = x.cpu().double()
    B, _, N, D = x.shape
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps)
    if gain is not None:
        y = y * gain.cpu().double()
    c, s = _angles(cos, sin, positions, B, N)
    mag = y.abs()
    if c is not None:
        a, b = _pairs(2 * c.shape[-1], interleaved)
        out, m = y.clone(), mag.clone()
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        m[..., a] = m[..., b] = mag[..., a] + mag[..., b]
        y, mag = out, m
    return y, mag


def backward(g, x, gain, cos, sin, positions=None, eps=1e-6, interleaved=False):
    """(dx, magnitude of its terms, d gain, magnitude of its terms)."""
    x, g = x.cpu().double(), g.cpu().double()
    B, _, N, D = x.shape
    c, s = _angles(cos, sin, positions, B, N)
    h, hm = g.clone(), g.abs()
    if c is not None:
        a, b = _pairs(2 * c.shape[-1], interleaved)
        h[..., a], h[..., b] = g[..., a] * c + g[..., b] * s, g[..., b] * c - g[..., a] * s
        m = hm.clone()
        m[..., a] = m[..., b] = hm[..., a] + hm[..., b]
        hm = m
    r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps)
    n = x * r
    w = torch.ones(D, dtype=torch.float64) if gain is None else gain.cpu().double()
    dx = r * (h * w - n * (h * w * n).mean(-1, keepdim=True))
    dx_mag = r * (hm * w.abs() + n.abs() * (hm * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, dx_mag, (h * n).sum((0, 1, 2)), (hm * n.abs()).sum((0, 1, 2))
