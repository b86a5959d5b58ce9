"""The head norm with position rotation on the GPU against its definition in 64 bits (the bounds: bounds.py)."""
from __future__ import annotations

import pytest
import torch

from bounds import near
from oracle import norm_rope as ref

pytestmark = pytest.mark.gpu

@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()


def ops():
    import attention_forward_03_gb300 as fa2
    return fa2


def tables(rows, rot):
    if not rot:
        return None, None
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f[None]
    return a.cos().float().cuda(), a.sin().float().cuda()


def packed(B, N, Hq, Hkv, D, dtype, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(B, N, Hq + 2 * Hkv, D, generator=g) * scale).to(dtype).cuda()
    return t[:, :, :Hq].transpose(1, 2), t[:, :, Hq:Hq + Hkv].transpose(1, 2)


def gains(D, kind, dtype, seed=1):
    if kind == "none":
        return None, None
    g = torch.Generator().manual_seed(seed)
    t = torch.float32 if kind == "f32" else dtype
    return tuple((1 + 0.3 * torch.randn(D, generator=g)).to(t).cuda() for _ in range(2))


CASES = [  # B, N, Hq, Hkv, D, rot, interleaved, gain, dtype, gathered positions
    (1, 1, 1, 1, 64, 64, False, "f32", torch.float16, False),
    (2, 1, 32, 8, 128, 128, False, "f32", torch.bfloat16, True),
    (3, 17, 5, 1, 32, 32, False, "16", torch.float16, True),
    (2, 33, 3, 3, 32, 16, True, "none", torch.bfloat16, False),
    (1, 100, 7, 2, 96, 96, False, "f32", torch.bfloat16, False),
    (2, 31, 4, 2, 96, 32, False, "16", torch.float16, True),
    (1, 65, 9, 3, 96, 96, True, "f32", torch.float16, False),
    (1, 257, 12, 12, 64, 32, True, "f32", torch.float16, False),
    (2, 129, 6, 2, 128, 64, False, "none", torch.bfloat16, True),
    (1, 500, 16, 4, 128, 128, True, "16", torch.bfloat16, False),
    (2, 9, 3, 1, 256, 256, False, "f32", torch.float16, True),
    (1, 40, 2, 2, 256, 16, True, "16", torch.bfloat16, False),
    (1, 7, 3, 2, 512, 512, False, "f32", torch.bfloat16, False),
    (2, 5, 2, 1, 512, 128, True, "f32", torch.float16, True),
    (1, 6, 3, 1, 1024, 1024, False, "f32", torch.float16, False),
    (2, 3, 2, 2, 1024, 512, False, "16", torch.bfloat16, True),
    (1, 4, 2, 1, 1024, 1024, True, "f32", torch.bfloat16, False),
    (2, 50, 8, 2, 128, 0, False, "f32", torch.bfloat16, False),
    (1, 3000, 10, 3, 64, 64, False, "f32", torch.bfloat16, False),
]


def make(c, seed=0):
    B, N, Hq, Hkv, D, rot, inter, gain, dtype, gather = c
    q, k = packed(B, N, Hq, Hkv, D, dtype, seed)
    qw, kw = gains(D, gain, dtype, seed + 1)
    cos, sin = tables(N + 50, rot)
    pos = None
    if gather and rot:
        g = torch.Generator().manual_seed(seed + 2)
        pos = torch.randint(0, N + 50, (B, N), generator=g).cuda()
    return q, k, qw, kw, cos, sin, pos


@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(c):
    q, k, qw, kw, cos, sin, pos = make(c)
    qo, ko = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin, positions=pos, eps=1e-5, interleaved=c[6])
    assert qo.is_contiguous() and ko.is_contiguous() and qo.dtype == q.dtype
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        near(got, *ref.forward(x, w, cos, sin, pos, 1e-5, c[6]), 32)


@pytest.mark.parametrize("c", CASES, ids=str)
def test_backward(c):
    q, k, qw, kw, cos, sin, pos = make(c, 5)
    g = torch.Generator().manual_seed(9)
    gq, gk = ((torch.randn(*t.shape, generator=g)).to(t.dtype).cuda() for t in (q, k))
    dq, dk, dqw, dkw = ops().qk_norm_rope_backward(gq, gk, q, k, qw, kw, cos, sin, positions=pos, eps=1e-5,
                                                   interleaved=c[6])
    for got, gw, up, x, w in ((dq, dqw, gq, q, qw), (dk, dkw, gk, k, kw)):
        dx, dx_mag, dw, dw_mag = ref.backward(up, x, w, cos, sin, pos, 1e-5, c[6])
        near(got, dx, dx_mag, 64)
        if w is None:
            assert gw is None
        else:
            assert gw.dtype == w.dtype
            near(gw, dw, dw_mag, 320)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences_of_the_forward(inter):
    # <dx, d> of the kernel against (L(x + e d) - L(x - e d)) / 2e in 64 bits
    c = (2, 5, 3, 2, 64, 32, inter, "f32", torch.float16, True)
    q, k, qw, kw, cos, sin, pos = make(c, 3)
    g = torch.Generator().manual_seed(4)
    up = torch.randn(*q.shape, generator=g).half().cuda()
    dq, _, dqw, _ = ops().qk_norm_rope_backward(up, torch.zeros_like(k), q, k, qw, kw, cos, sin, positions=pos,
                                                interleaved=inter)
    x, w, u = q.cpu().double(), qw.cpu().double(), up.cpu().double()
    loss = lambda x, w: float((ref.forward(x, w, cos, sin, pos, 1e-6, inter)[0] * u).sum())  # noqa: E731
    d, dg, e = torch.randn(*x.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64), 1e-5
    num = (loss(x + e * d, w + e * dg) - loss(x - e * d, w - e * dg)) / (2 * e)
    ana = float((dq.cpu().double() * d).sum() + (dqw.cpu().double() * dg).sum())
    # each dq is off by half an fp16 step at most, and the differences by e^2 of the terms
    tol = float((dq.cpu().double().abs() * d.abs()).sum()) * 2.0 ** -10 + 1e-6 * float(u.abs().sum())
    assert abs(num - ana) <= tol


def test_one_side_alone():
    q, k, qw, kw, cos, sin, _ = make((2, 12, 4, 2, 64, 64, False, "f32", torch.bfloat16, False))
    both = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin)
    only_q, none = ops().qk_norm_rope_forward(q, None, qw, None, cos, sin)
    assert none is None and torch.equal(only_q, both[0])
    none, only_k = ops().qk_norm_rope_forward(None, k, None, kw, cos, sin)
    assert none is None and torch.equal(only_k, both[1])
    gk = torch.randn_like(k)
    r = ops().qk_norm_rope_backward(None, gk, None, k, None, kw, cos, sin)
    assert r[0] is None and r[2] is None
    dx, mag, dw, dw_mag = ref.backward(gk, k, kw, cos, sin)
    near(r[1], dx, mag, 64)
    near(r[3], dw, dw_mag, 320)


def test_empty_shapes():
    z = torch.empty(0, 2, 5, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, device="cuda")
    qo, ko = ops().qk_norm_rope_forward(z, z, w, w)
    assert qo.shape == z.shape
    r = ops().qk_norm_rope_backward(z, z, z, z, w, w)
    assert torch.equal(r[2], torch.zeros(64, device="cuda")) and torch.equal(r[3], torch.zeros(64, device="cuda"))


@pytest.mark.parametrize("kind", ["i64", "i32", "row", "strided"])
def test_positions(kind):
    q, k, qw, kw, cos, sin, _ = make((3, 20, 2, 1, 64, 64, False, "f32", torch.float16, False))
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(0, 70, (3, 20), generator=g)
    if kind == "i32":
        pos = pos.int()
    elif kind == "row":
        pos = pos[0].contiguous()
    pos = pos.cuda()
    if kind == "strided":
        pos = pos.t().contiguous().t()
        assert not pos.is_contiguous()
    qo, ko = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin, positions=pos)
    near(qo, *ref.forward(q, qw, cos, sin, pos), 32)
    near(ko, *ref.forward(k, kw, cos, sin, pos), 32)


def test_positions_outside_the_tables_show_as_nan():
    q, k, qw, kw, cos, sin, _ = make((1, 6, 2, 2, 64, 32, False, "f32", torch.float16, False))
    pos = torch.tensor([[0, -1, 55, 56, 2 ** 40, 3]]).cuda()  # the tables have 56 rows
    qo, _ = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin, positions=pos)
    near(qo, *ref.forward(q, qw, cos, sin, pos), 32)
    assert qo[0, 0].isnan().any(-1).tolist() == [False, True, False, True, True, False]
    assert not qo[..., 32:].isnan().any()


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_on_a_packed_projection(inter):
    c = (2, 37, 5, 2, 96, 32, inter, "f32", torch.bfloat16, False)
    q, k, qw, kw, cos, sin, _ = make(c)
    want = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin, interleaved=inter)
    whole = q._base.clone()
    v_before = whole[:, :, 7:].clone()
    q2, k2 = whole[:, :, :5].transpose(1, 2), whole[:, :, 5:7].transpose(1, 2)
    got = ops().qk_norm_rope_forward(q2, k2, qw, kw, cos, sin, interleaved=inter, q_out=q2, k_out=k2)
    assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert torch.equal(whole[:, :, 7:], v_before)
    # backward into the packed gradient, over its own upstream gradients
    gq, gk = torch.randn_like(want[0]), torch.randn_like(want[1])
    ref_out = ops().qk_norm_rope_backward(gq, gk, q, k, qw, kw, cos, sin, interleaved=inter)
    d = torch.full_like(whole, 7.0)
    d[:, :, :5], d[:, :, 5:7] = gq.transpose(1, 2), gk.transpose(1, 2)
    dq, dk = d[:, :, :5].transpose(1, 2), d[:, :, 5:7].transpose(1, 2)
    got = ops().qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, interleaved=inter, dq=dq, dk=dk)
    for a, b in zip(got, ref_out):
        assert torch.equal(a, b)
    assert bool((d[:, :, 7:] == 7.0).all())


def test_into_a_cache_slot():
    # a decoding step writes its one key row into position 11 of the cache
    q, k, qw, kw, cos, sin, _ = make((3, 1, 8, 2, 128, 128, False, "f32", torch.bfloat16, False))
    pos = torch.full((3, 1), 11).cuda()
    cache = torch.full((3, 2, 64, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin, positions=pos, k_out=cache[:, :, 11:12])
    near(cache[:, :, 11:12], *ref.forward(k, kw, cos, sin, pos), 32)
    cache[:, :, 11] = 5.0
    assert bool((cache == 5.0).all())


def test_special_values():
    # an all-zero row stays zero (eps > 0); inf and NaN stay in their own row
    q, k, qw, kw, cos, sin, _ = make((1, 8, 2, 1, 64, 64, False, "f32", torch.float16, False))
    q = q.contiguous()
    q[0, 0, 1] = 0
    q[0, 0, 2, 5] = float("inf")
    q[0, 1, 3, 63] = float("nan")
    q[0, 1, 4] = 65504.0
    qo, _ = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin)
    assert bool((qo[0, 0, 1] == 0).all())
    rows = qo.isnan().any(-1)[0]
    assert rows.nonzero().tolist() == [[0, 2], [1, 3]]
    want, mag = ref.forward(q, qw, cos, sin)
    near(qo[0, 1, 4], want[0, 1, 4], mag[0, 1, 4], 32)


def test_offsets_past_32_bits():
    # the second batch lies more than 2^31 elements behind the first
    far = 2 ** 31 + 4096
    big = torch.empty(far + 4 * 6 * 64, dtype=torch.float16, device="cuda")
    q = big.as_strided((2, 4, 6, 64), (far, 6 * 64, 64, 1))
    q.copy_(torch.randn(2, 4, 6, 64, generator=torch.Generator().manual_seed(0)).half().cuda())
    cos, sin = tables(6, 64)
    want, mag = ref.forward(q, None, cos, sin)
    qo, _ = ops().qk_norm_rope_forward(q, None, None, None, cos, sin, q_out=q)
    near(qo, want, mag, 32)


def test_another_stream_and_two_at_once():
    c = (2, 400, 8, 2, 128, 128, False, "f32", torch.bfloat16, False)
    sets = [make(c, s) for s in (0, 1)]
    ups = [[torch.randn_like(t.contiguous()) for t in s[:2]] for s in sets]
    want = [(ops().qk_norm_rope_forward(*s[:6]), ops().qk_norm_rope_backward(*u, *s[:6])) for s, u in zip(sets, ups)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = [(ops().qk_norm_rope_forward(*s[:6], stream=st), ops().qk_norm_rope_backward(*u, *s[:6], stream=st))
               for s, u, st in zip(sets, ups, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert all(torch.equal(i, j) for i, j in zip(x, y))  # gain sums too: their order is fixed


def test_captured_and_replayed_on_new_inputs():
    c = (2, 100, 4, 2, 64, 64, False, "f32", torch.bfloat16, False)
    q, k, qw, kw, cos, sin, _ = make(c, 0)
    up = [torch.randn_like(t.contiguous()) for t in (q, k)]
    ops().qk_norm_rope_backward(*up, q, k, qw, kw, cos, sin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin) + ops().qk_norm_rope_backward(*up, q, k, qw, kw, cos, sin)
    for seed in (7, 8):
        q2, k2 = make(c, seed)[:2]
        q.copy_(q2)
        k.copy_(k2)
        graph.replay()
        torch.cuda.synchronize()
        want = ops().qk_norm_rope_forward(q, k, qw, kw, cos, sin) + ops().qk_norm_rope_backward(*up, q, k, qw, kw, cos, sin)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_binding_refusals():
    q, k, qw, kw, cos, sin, _ = make((2, 10, 4, 2, 64, 64, False, "f32", torch.float16, False))
    f, Err = ops().qk_norm_rope_forward, ops().Fa2Error
    bad = [
        lambda: f(q, k.bfloat16(), qw, kw, cos, sin),
        lambda: f(q, k[:, :, :5], qw, kw, cos, sin),
        lambda: f(q.float(), k.float(), qw, kw, cos, sin),
        lambda: f(q, k, qw.half(), kw, cos, sin),
        lambda: f(q, k, qw[:32], kw, cos, sin),
        lambda: f(q, k, qw, kw, cos, None),
        lambda: f(q, k, qw, kw, cos.double(), sin.double()),
        lambda: f(q, k, qw, kw, cos[:9], sin[:9]),
        lambda: f(q, k, qw, kw, cos, sin, positions=torch.zeros(2, 9, dtype=torch.long, device="cuda")),
        lambda: f(q, k, qw, kw, cos, sin, positions=torch.zeros(2, 10, device="cuda")),
        lambda: f(q, k, qw, kw, positions=torch.zeros(2, 10, dtype=torch.long, device="cuda")),
        lambda: f(q, k, qw, kw, cos, sin, q_out=torch.empty(2, 4, 10, 32, dtype=torch.float16, device="cuda")),
        lambda: f(q.transpose(2, 3), k.transpose(2, 3)),
        lambda: ops().qk_norm_rope_backward(None, k, q, k, qw, kw, cos, sin),
        lambda: ops().qk_norm_rope_backward(q, k, q, k, qw, kw, cos, sin, workspace=torch.empty(64, device="cuda")),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: f(q, k, qw, kw, cos[:, :12].contiguous(), sin[:, :12].contiguous()),  # rot 24
                 lambda: f(q, k, qw, kw, cos, sin, q_out=q.clone()[:, :1].expand(2, 4, 10, 64)),  # rows overlap
                 lambda: f(q, q, k_out=q)):  # k_out is exactly k, but q reads it too
        with pytest.raises(Err):
            call()
