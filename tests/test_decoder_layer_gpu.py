"""The attention part of a decoder layer, as a program runs it: the head norm and rotation out of the packed projection,
causal self-attention, the norm of the cross queries, cross attention over padded encoder states, and all of it
backward into the packed projection's gradient. Every stage is checked against its definition in 64 bits on the values
the stage before it gave."""
from __future__ import annotations

import pytest
import torch

from bounds import check_cross_bwd, check_cross_fwd, near
from oracle import norm_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    yield m
    assert m.fa2_device_status(clear=True) == 0


def tables(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f[None]
    return a.cos().float().cuda(), a.sin().float().cuda()


class Layer:
    def __init__(self, fa2, B=2, H=6, Hkv=2, N=150, Ne=333, D=64, dtype=torch.float16, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.fa2, self.shape = fa2, (B, H, Hkv, N, Ne, D)
        self.packed = (r(B, N, 3 * H, D) * 2).to(dtype).cuda()
        self.enc_k, self.enc_v = (r(B, Hkv, Ne, D).to(dtype).cuda() for _ in range(2))
        self.lengths = torch.tensor([Ne, Ne // 3], dtype=torch.int32).cuda()
        self.gains = [(1 + 0.2 * r(D)).cuda() for _ in range(3)]
        self.cos, self.sin = tables(512, D)
        self.up = r(B, H, N, D).to(dtype).cuda()

    def split(self, t):
        H = self.shape[1]
        return [t[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3)]

    def forward(self):
        f = self.fa2
        q, k, v = self.split(self.packed)
        self.q, self.k = f.qk_norm_rope_forward(q, k, *self.gains[:2], self.cos, self.sin)
        self.v = v.contiguous()
        self.o, self.lse = f.attention_forward(self.q, self.k, self.v, is_causal=True)
        self.cq, _ = f.qk_norm_rope_forward(self.o, None, self.gains[2])
        self.co, self.clse = f.cross_attention_forward(self.cq, self.enc_k, self.enc_v, key_lengths=self.lengths)
        return self.co

    def backward(self):
        f = self.fa2
        self.dcq, self.dek, self.dev = f.cross_attention_backward(self.cq, self.enc_k, self.enc_v, self.co, self.clse,
                                                                  self.up, key_lengths=self.lengths)
        self.do, _, self.dg2, _ = f.qk_norm_rope_backward(self.dcq, None, self.o, None, self.gains[2])
        self.dq, self.dk, dv = f.attention_backward(self.q, self.k, self.v, self.o, self.lse, self.do, is_causal=True)
        self.dpacked = torch.empty_like(self.packed)
        q, k, _ = self.split(self.packed)
        gq, gk, gv = self.split(self.dpacked)
        gv.copy_(dv)
        _, _, self.dg0, self.dg1 = f.qk_norm_rope_backward(self.dq, self.dk, q, k, *self.gains[:2], self.cos, self.sin,
                                                           dq=gq, dk=gk)
        return [self.dpacked, self.dek, self.dev, self.dg0, self.dg1, self.dg2]


@pytest.mark.parametrize("dtype,D", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_stage_by_stage(fa2, dtype, D):
    m = Layer(fa2, dtype=dtype, D=D)
    m.forward()
    m.backward()
    scale = D ** -0.5
    q, k, _ = m.split(m.packed)
    near(m.q, *norm_rope.forward(q, m.gains[0], m.cos, m.sin), 32)
    near(m.k, *norm_rope.forward(k, m.gains[1], m.cos, m.sin), 32)
    near(m.cq, *norm_rope.forward(m.o, m.gains[2], None, None), 32)
    check_cross_fwd(m.co, m.clse, m.cq, m.enc_k, m.enc_v, scale, m.lengths)
    check_cross_bwd((m.dcq, m.dek, m.dev), m.cq, m.enc_k, m.enc_v, m.co, m.clse, m.up, scale, m.lengths)
    dx, mag, dw, dw_mag = norm_rope.backward(m.dcq, m.o, m.gains[2], None, None)
    near(m.do, dx, mag, 64)
    near(m.dg2, dw, dw_mag, 320)
    for x, g, got, gain, dgain in ((q, m.dq, m.split(m.dpacked)[0], m.gains[0], m.dg0),
                                   (k, m.dk, m.split(m.dpacked)[1], m.gains[1], m.dg1)):
        dx, mag, dw, dw_mag = norm_rope.backward(g, x, gain, m.cos, m.sin)
        near(got, dx, mag, 64)
        near(dgain, dw, dw_mag, 320)


def test_captured_as_one_graph(fa2):
    m = Layer(fa2)
    m.forward()
    m.backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [m.forward()] + m.backward()
    other = Layer(fa2, seed=5)
    m.packed.copy_(other.packed)
    m.enc_k.copy_(other.enc_k)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    cq, o = m.cq.clone(), m.o.clone()
    # the eager run on the same values: everything but the two dQ sums (atomic adds in no fixed order) and what
    # comes after them is the same bit for bit
    again = [m.forward()] + m.backward()
    assert torch.equal(got[0], again[0]) and torch.equal(got[2], again[2]) and torch.equal(got[3], again[3])
    assert torch.equal(cq, m.cq) and torch.equal(o, m.o)
    for a, b in zip(got, again):
        assert bool(a.isfinite().all()) and float((a.double() - b.double()).norm()) <= 2e-3 * float(b.double().norm())


@pytest.mark.parametrize("dtype,D", [(torch.float16, 64), (torch.bfloat16, 128)])
def test_a_single_token_gives_the_prompts_last_row(fa2, dtype, D):
    # serving: the last token alone, at its position, through the same calls
    m = Layer(fa2, dtype=dtype, D=D)
    co = m.forward()
    B, H, _, N, _, _ = m.shape
    pos = torch.full((B, 1), N - 1).cuda()
    q, k, _ = m.split(m.packed[:, -1:])
    cache = torch.zeros_like(m.k)
    cache[:, :, :N - 1] = m.k[:, :, :N - 1]
    q1, _ = fa2.qk_norm_rope_forward(q, k, *m.gains[:2], m.cos, m.sin, positions=pos, k_out=cache[:, :, N - 1:])
    assert torch.equal(cache, m.k) and torch.equal(q1, m.q[:, :, -1:])
    cq, _ = fa2.qk_norm_rope_forward(m.o[:, :, -1:], None, m.gains[2])
    assert torch.equal(cq, m.cq[:, :, -1:])
    one, lse = fa2.cross_attention_forward(cq, m.enc_k, m.enc_v, key_lengths=m.lengths)
    check_cross_fwd(one, lse, cq, m.enc_k, m.enc_v, D ** -0.5, m.lengths)
    # both are within the bound of the same row, so within two of each other: u (A + |O|), A <= max |v|
    u = torch.finfo(dtype).eps / 2
    assert float((one - co[:, :, -1:]).abs().max()) <= 2 * 2.1 * u * float(m.enc_v.abs().max())
