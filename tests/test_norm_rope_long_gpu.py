"""The gains' gradients of the head norm over many tokens, with a bound that follows the size.

A gain's gradient is a sum of one product per row in 32 bits: each thread adds up the rows it walks, the row groups of a
warp meet in shuffles and the 8 warps of a block in shared memory, and the blocks' partial sums are added in 32 runs,
then the runs. The depth of that tree, in half steps of 2^-24 of the terms' sum, and 64 half steps for a product itself
(r and the mean of squares, the rotation, the product with the gain's factor) bound the error; the rounding to the
gain's type comes on top.
"""
from __future__ import annotations

import pytest
import torch

from bounds import near
from oracle import norm_rope as ref

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    return m


def depth(tokens, heads, other_heads, D):
    """Additions on the way of a row's product into the sum over `heads` heads, beside `other_heads` of the other side."""
    lanes = {32: 2, 64: 4, 96: 8, 128: 8, 256: 16, 512: 32, 1024: 32}[D]
    groups = 256 // lanes  # rows a block works on at once
    cap = min(2 * torch.cuda.get_device_properties(0).multi_processor_count, 1280)
    mine, other = -(-heads // 8), -(-other_heads // 8)  # items of a token: up to 8 heads each
    blocks = cap * mine // (mine + other) - 1  # at least, with as many items as fill the device
    rows = -(-tokens * mine // (blocks * groups)) * 8
    return rows + 32 // lanes + 8 + -(-cap // 32) + 32


@pytest.mark.parametrize("B,N,Hq,Hkv,D,dtype,gain", [
    (4, 4096, 8, 2, 128, BF16, torch.float32), (1, 40000, 4, 4, 64, F16, torch.float32),
    (3, 7001, 8, 1, 96, BF16, BF16), (2, 16411, 2, 1, 256, F16, F16),
])
def test_gain_gradients_over_many_tokens(fa2, B, N, Hq, Hkv, D, dtype, gain):
    g = torch.Generator().manual_seed(N)
    packed = (torch.randn(B, N, Hq + Hkv, D, generator=g) * 2).to(dtype).cuda()
    q, k = packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq:].transpose(1, 2)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(gain).cuda() for _ in range(2))
    gq, gk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    a = torch.arange(N, dtype=torch.float64)[:, None] * f[None]
    cos, sin = a.cos().float().cuda(), a.sin().float().cuda()
    dq, dk, dqw, dkw = fa2.qk_norm_rope_backward(gq, gk, q, k, qw, kw, cos, sin)
    for got, gw, up, x, w, other in ((dq, dqw, gq, q, qw, Hkv), (dk, dkw, gk, k, kw, Hq)):
        dx, dx_mag, dw, dw_mag = ref.backward(up, x, w, cos, sin, None, 1e-6, False)
        near(got, dx, dx_mag, 64)
        near(gw, dw, dw_mag, depth(B * N, x.shape[1], other, D) + 64)
    again = fa2.qk_norm_rope_backward(gq, gk, q, k, qw, kw, cos, sin)
    assert torch.equal(dqw, again[2]) and torch.equal(dkw, again[3])  # a fixed order
