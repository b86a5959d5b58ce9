"""Cross attention on the GPU against its definition in 64 bits (the bounds: bounds.py)."""
from __future__ import annotations

import math

import pytest
import torch

from bounds import check_cross_bwd as check_bwd, check_cross_fwd as check_fwd
from oracle import cross as ref

pytestmark = pytest.mark.gpu

@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    from attention_forward_03_gb300 import binding
    yield binding
    assert binding.fa2_device_status(clear=True) == 0


def ops():
    import attention_forward_03_gb300 as fa2
    return fa2


def inputs(B, Hq, Hkv, Nq, Nk, D, dtype, lengths=None, seed=0, garbage=float("nan"), sq=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = (r(B, Hq, Nq, D) * sq).to(dtype).cuda(), r(B, Hkv, Nk, D).to(dtype).cuda(), r(B, Hkv, Nk, D).to(dtype).cuda()
    n = None
    if lengths is not None:
        n = torch.tensor(lengths, dtype=torch.int32).cuda()
        behind = torch.arange(Nk).cuda()[None] >= n[:, None]
        k.masked_fill_(behind[:, None, :, None], garbage)
        v.masked_fill_(behind[:, None, :, None], garbage)
    return q, k, v, n


F16, BF16 = torch.float16, torch.bfloat16
SHAPES = [  # B, Hq, Hkv, Nq, Nk, D, dtype, lengths
    (1, 1, 1, 1, 1, 64, F16, None),
    (1, 2, 2, 1, 17, 32, BF16, None),
    (2, 4, 4, 1, 1500, 64, F16, None),
    (3, 8, 2, 1, 300, 128, BF16, [300, 0, 129]),
    (2, 6, 2, 3, 130, 96, F16, [1, 130]),
    (4, 16, 2, 1, 65, 64, BF16, [0, 64, 65, 63]),
    (1, 7, 1, 2, 5000, 128, F16, [4999]),
    (1, 32, 4, 2, 777, 32, F16, None),
    (2, 2, 1, 40, 200, 64, BF16, [200, 3]),
    (1, 3, 3, 77, 77, 64, F16, None),
    (2, 4, 4, 128, 128, 128, BF16, [128, 127]),
    (2, 2, 2, 129, 256, 96, F16, [255, 0]),
    (1, 4, 2, 100, 1, 128, F16, None),
    (1, 2, 2, 256, 16, 64, BF16, None),
    (1, 2, 2, 257, 1000, 32, F16, [993]),
    (1, 4, 2, 63, 128, 128, BF16, [127]),
    (3, 2, 2, 65, 127, 96, F16, [0, 16, 127]),
    (2, 6, 2, 700, 33, 32, BF16, [33, 17]),
    (1, 2, 2, 3000, 77, 64, F16, None),
    (1, 2, 1, 100, 129, 64, F16, [129]),
    (5, 4, 4, 300, 513, 64, F16, [0, 1, 512, 513, 400]),
    (3, 6, 2, 200, 700, 128, BF16, [700, 16, 450]),
    (2, 5, 5, 513, 640, 96, BF16, None),
    (1, 16, 2, 1000, 1500, 64, BF16, [1200]),
    (1, 1, 1, 1, 20000, 128, BF16, None),
    (1, 16, 1, 1, 3001, 64, F16, None),
    (2, 8, 8, 16, 1000, 96, BF16, [1000, 513]),
    (2, 17, 1, 1, 700, 128, F16, [700, 64]),
    (1, 8, 2, 4, 190, 128, BF16, None),
    (300, 4, 2, 1, 256, 64, BF16, [(37 * i) % 257 for i in range(300)]),
    (70, 1, 1, 3, 90, 32, BF16, [(7 * i) % 91 for i in range(70)]),
    (40, 2, 2, 130, 260, 64, F16, [(13 * i) % 261 for i in range(40)]),
]


@pytest.mark.parametrize("c", SHAPES, ids=str)
def test_forward(lib, c):
    B, Hq, Hkv, Nq, Nk, D, dtype, lengths = c
    q, k, v, n = inputs(*c)
    scale = 1 / math.sqrt(D)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    check_fwd(o, lse, q, k, v, scale, n)
    again = ops().cross_attention_forward(q, k, v, key_lengths=n)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # no order of its own
    # whole units per SM (no workspace)
    o2, l2 = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
    rc = lib.library().fa2_cross_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), l2.data_ptr(),
                                     None if n is None else n.data_ptr(), B, Hq, Hkv, Nq, Nk, D, scale,
                                     lib._dtype_code_of(dtype), None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0, lib.error_text(rc)
    check_fwd(o2, l2, q, k, v, scale, n)


def upstream(q, seed=11):
    return torch.randn(*q.shape, generator=torch.Generator().manual_seed(seed)).to(q.dtype).cuda()


@pytest.mark.parametrize("c", SHAPES, ids=str)
def test_backward(c):
    q, k, v, n = inputs(*c, seed=2)
    scale = 1 / math.sqrt(c[5])
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    do = upstream(q)
    outs = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    grads = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n, dq=outs[0], dk=outs[1], dv=outs[2])
    assert all(a is b for a, b in zip(grads, outs))
    check_bwd(grads, q, k, v, o, lse, do, scale, n)
    again = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])  # dK, dV: a fixed order
    if c[4] <= 128:
        assert torch.equal(grads[0], again[0])  # dQ: one term per row


def test_gradient_against_differences_of_the_forward():
    # <dx, d> against (L(x + e d) - L(x - e d)) / 2e in 64 bits, with O and LSE of the definition
    q, k, v, n = inputs(2, 4, 2, 5, 40, 64, F16, [37, 0], sq=1.0)
    k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
    do = upstream(q)
    o, lse, _ = ref.forward(q, k, v, 0.125, n)
    g = ops().cross_attention_backward(q, k, v, o.half().cuda(), lse.float().cuda(), do, key_lengths=n)
    rnd = torch.Generator().manual_seed(5)
    d = [torch.randn(*t.shape, generator=rnd, dtype=torch.float64).cuda() for t in (q, k, v)]
    loss = lambda *t: float((ref.forward(*t, 0.125, n)[0] * do.cpu().double()).sum())  # noqa: E731
    e = 1e-5
    num = (loss(*(t.double() + e * x for t, x in zip((q, k, v), d))) - loss(*(t.double() - e * x for t, x in zip((q, k, v), d)))) / (2 * e)
    ana = sum(float((a.double() * x).sum()) for a, x in zip(g, d))
    want = ref.backward(q, k, v, o.half().cuda(), lse.float().cuda(), do, 0.125, n)
    # half an fp16 step of P, dS, O (in Delta) and the result each, of the terms' sizes
    tol = sum(float(((w[1] + w[2] / 2) * x.cpu().abs()).sum()) for w, x in zip(want.values(), d)) * 2.0 ** -10
    assert abs(num - ana) <= tol


@pytest.mark.parametrize("c", [(2, 4, 2, 130, 300, 128, BF16, [300, 130]), (2, 2, 2, 150, 300, 64, F16, [90, 150])], ids=str)
@pytest.mark.parametrize("garbage", [float("inf"), 65504.0])
def test_backward_does_not_use_what_lies_behind_the_keys(c, garbage):
    q, k, v, n = inputs(*c, garbage=garbage)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    do = upstream(q)
    grads = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    check_bwd(grads, q, k, v, o, lse, do, c[5] ** -0.5, n)


@pytest.mark.parametrize("shape", [(2, 4, 2, 0, 9), (2, 4, 2, 9, 0), (0, 4, 2, 3, 3), (1, 0, 2, 3, 3)])
def test_backward_of_nothing(shape):
    B, Hq, Hkv, Nq, Nk = shape
    q, k, v, _ = inputs(B, Hq, Hkv, Nq, Nk, 64, F16)
    lse = torch.zeros(B, Hq, Nq, device="cuda")
    g = ops().cross_attention_backward(q, k, v, q, lse, q)
    for a, b in zip(g, (q, k, v)):
        assert a.shape == b.shape and bool((a == 0).all())


@pytest.mark.parametrize("lengths,Nk,D", [([0, 0], 200, 64), ([0, 200], 200, 64), ([0, 0], 100, 64), ([0, 100], 100, 64),
                                          ([33, 0], 128, 128), ([0, 5], 90, 96)])
def test_backward_with_empty_batch_entries(lengths, Nk, D):
    q, k, v, n = inputs(2, 4, 2, 70, Nk, D, BF16, lengths)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    do = upstream(q)
    outs = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n, dq=outs[0], dk=outs[1], dv=outs[2])
    check_bwd(outs, q, k, v, o, lse, do, D ** -0.5, n)
    assert all(bool((outs[0][b] == 0).all()) for b in range(2) if lengths[b] == 0)


@pytest.mark.parametrize("c", [(2, 4, 2, 260, 700, 128, BF16, [700, 310]), (2, 2, 2, 300, 900, 64, F16, [333, 900]),
                               (2, 2, 2, 5000, 100, 64, F16, [100, 90]), (1, 2, 2, 4000, 128, 128, BF16, [128])], ids=str)
def test_backward_captured_and_replayed_on_new_inputs(c):
    q, k, v, n = inputs(*c, garbage=0.0)
    do = upstream(q)
    ops().cross_attention_backward(q, k, v, *ops().cross_attention_forward(q, k, v, key_lengths=n), do, key_lengths=n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
        grads = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    for seed in (5, 6, 7):
        q2, k2, v2, _ = inputs(*c[:-1], seed=seed)
        for a, b in ((q, q2), (k, k2), (v, v2)):
            a.copy_(b)
        n.copy_(torch.tensor([max(0, int(x) - c[4] // 5 * (seed - 4)) for x in c[-1]], dtype=torch.int32))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        check_bwd(grads, q, k, v, o, lse, do, c[5] ** -0.5, n)
        want = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
        assert torch.equal(grads[1], want[1]) and torch.equal(grads[2], want[2])


@pytest.mark.parametrize("c", [(1, 8, 1, 4, 900, 128, BF16, [801]), (2, 2, 2, 150, 300, 64, F16, [300, 150])], ids=str)
@pytest.mark.parametrize("garbage", [float("inf"), 65504.0])
def test_what_lies_behind_the_keys_is_not_used(c, garbage):
    q, k, v, n = inputs(*c, garbage=garbage)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    check_fwd(o, lse, q, k, v, c[5] ** -0.5, n)
    clean = ops().cross_attention_forward(q, k.masked_fill(k.abs() >= 65504, 0), v.masked_fill(v.abs() >= 65504, 0),
                                          key_lengths=n)
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("Nq", [1, 200])
def test_lengths_outside_the_range_count_as_the_nearer_end(Nq):
    q, k, v, _ = inputs(3, 4, 2, Nq, 100, 64, F16)
    n = torch.tensor([-5, 1000, 2 ** 31 - 1], dtype=torch.int32).cuda()
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    check_fwd(o, lse, q, k, v, 0.125, n)


@pytest.mark.parametrize("Nq,Hq", [(1, 4), (90, 2)])
def test_no_keys_at_all(Nq, Hq):
    q, k, v, _ = inputs(2, Hq, 2, Nq, 5, 64, F16)
    o, lse = ops().cross_attention_forward(q, k[:, :, :0].contiguous(), v[:, :, :0].contiguous())
    assert bool((o == 0).all()) and bool((lse == float("inf")).all())
    e = ops().cross_attention_forward(q[:, :, :0].contiguous(), k, v)
    assert e[0].shape == (2, Hq, 0, 64) and e[1].shape == (2, Hq, 0)


@pytest.mark.parametrize("Nq", [1, 300])
def test_extreme_scores(Nq):
    # one dominant key late in a ragged row; all scores far below zero; scores of +-3e4 (fp16 inputs)
    for D in (64, 128):
        q, k, v, _ = inputs(1, 2, 2, Nq, 700, D, F16, seed=3)
        k[0, 0, 690] = q[0, 0, 0] * 4
        k[0, 1] = -q[0, 1, :1].abs() * 2
        n = torch.tensor([695], dtype=torch.int32).cuda()
        o, lse = ops().cross_attention_forward(q, k, v, scale=1.0, key_lengths=n)
        check_fwd(o, lse, q, k, v, 1.0, n)


@pytest.mark.parametrize("Nq", [1, 300])
def test_nan_and_inf_stay_in_their_rows(Nq):
    q, k, v, _ = inputs(2, 2, 2, Nq, 150, 64, BF16)
    want = ops().cross_attention_forward(q, k, v)
    q[0, 1, 0, 3] = float("nan")
    o, lse = ops().cross_attention_forward(q, k, v)
    assert bool(o[0, 1, 0].isnan().all())
    o[0, 1, 0], lse[0, 1, 0] = want[0][0, 1, 0], want[1][0, 1, 0]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_rows_behind_the_outputs_are_left_alone():
    for Nq, Hq in ((1, 6), (130, 2)):
        q, k, v, n = inputs(2, Hq, 2, Nq, 333, 96, BF16, [333, 20])
        big = torch.full((2 * Hq * Nq * 96 + 4096,), 7.0, dtype=BF16, device="cuda")
        lbig = torch.full((2 * Hq * Nq + 1024,), 7.0, device="cuda")
        out, lse = big[:2 * Hq * Nq * 96].view(q.shape), lbig[:2 * Hq * Nq].view(2, Hq, Nq)
        ops().cross_attention_forward(q, k, v, key_lengths=n, out=out, lse=lse)
        check_fwd(out, lse, q, k, v, 96 ** -0.5, n)
        assert bool((big[2 * Hq * Nq * 96:] == 7).all()) and bool((lbig[2 * Hq * Nq:] == 7).all())


@pytest.mark.parametrize("c", [(2, 8, 2, 1, 4000, 128, BF16, [4000, 1700]), (1, 2, 2, 300, 4000, 64, F16, [3333])], ids=str)
def test_captured_and_replayed_on_new_inputs(c):
    # a replay runs over the workspace the one before it left behind
    q, k, v, n = inputs(*c)
    ops().cross_attention_forward(q, k, v, key_lengths=n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    for seed in (5, 6, 7):
        q2, k2, v2, _ = inputs(*c[:-1], seed=seed)
        for a, b in ((q, q2), (k, k2), (v, v2)):
            a.copy_(b)
        n.copy_(torch.tensor([int(x) - 100 * (seed - 4) for x in c[-1]], dtype=torch.int32))
        for _ in range(3):
            o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        want = ops().cross_attention_forward(q, k, v, key_lengths=n)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        check_fwd(o, lse, q, k, v, c[5] ** -0.5, n)


CUT = [  # fewer heads than SMs, keys long enough to cut each head's unit between several
    (1, 32, 8, 8, 1700, 64, BF16, None),
    (1, 8, 8, 150, 4500, 32, F16, None),
    (2, 8, 4, 150, 4500, 128, BF16, [4500, 0]),
    (4, 2, 2, 300, 2300, 96, F16, [1, 2300, 129, 1024]),
    (1, 1, 1, 40, 30000, 64, F16, [29999]),
    (1, 1, 1, 257, 30000, 128, BF16, None),
]


@pytest.mark.parametrize("c", CUT, ids=str)
def test_units_cut_between_many_sms(c):
    q, k, v, n = inputs(*c)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    check_fwd(o, lse, q, k, v, c[5] ** -0.5, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, glse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    for _ in range(5):  # over the workspace and the flags that the replay before left
        go.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(go, o) and torch.equal(glse, lse)


SPLIT_KEYS = [  # at most 128 rows per key head, D <= 64: the key tiles go to the two sub-tiles in turn
    (3, 8, 8, 128, 700, 64, BF16, None),           # whole units, an even number of tiles
    (40, 8, 4, 50, 600, 64, F16, None),            # more units than SMs, an odd number
    (20, 16, 8, 40, 1000, 32, BF16, [(97 * i) % 1001 for i in range(20)]),  # 0 to 8 tiles each
    (2, 2, 2, 17, 650, 64, BF16, [513, 1]),
    (1, 8, 8, 100, 3000, 64, F16, [2945]),         # cut units
    (30, 8, 8, 20, 9000, 32, F16, [300 * i for i in range(30)]),  # cut units among whole ones
]


@pytest.mark.parametrize("c", SPLIT_KEYS, ids=str)
def test_key_tiles_in_turn(c):
    q, k, v, n = inputs(*c)
    if n is not None:  # a dominant key in one sub-tile only, and scores far below zero in a head
        k[0, 0, : int(c[-1][0])] *= 0.1
        k[1 % c[0], -1, min(200, max(int(c[-1][1 % c[0]]) - 1, 0))] = 4 * q[1 % c[0], -1, 0]
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    check_fwd(o, lse, q, k, v, c[5] ** -0.5, n)
    again = ops().cross_attention_forward(q, k, v, key_lengths=n)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


CUT_ROWS = [  # the backward's units are key tiles, cut along the query rows
    (1, 8, 2, 1024, 77, 64, BF16, None),
    (2, 4, 4, 2100, 200, 128, F16, [200, 0]),
    (2, 2, 1, 2000, 300, 32, BF16, [129, 300]),
    (1, 1, 1, 9000, 128, 96, F16, [100]),
    (1, 1, 1, 20000, 40, 128, BF16, None),
]


@pytest.mark.parametrize("c", CUT_ROWS, ids=str)
def test_backward_units_cut_between_many_sms(c):
    q, k, v, n = inputs(*c)
    do = upstream(q)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    grads = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    check_bwd(grads, q, k, v, o, lse, do, c[5] ** -0.5, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    for _ in range(5):  # over the workspace and the flags that the replay before left
        for t in again:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[1], grads[1]) and torch.equal(again[2], grads[2])  # a fixed order


@pytest.mark.parametrize("c", [(2, 4, 2, 70, 1, 64, BF16, None), (3, 4, 2, 130, 200, 128, F16, [1, 200, 1]),
                               (2, 2, 2, 300, 90, 96, BF16, [90, 1])], ids=str)
def test_gradient_over_one_key(c):
    # the softmax is constant: dQ and dK are zero, not dP - Delta's rounding; a NaN is not lost in it
    q, k, v, n = inputs(*c)
    do = upstream(q)
    o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
    grads = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    check_bwd(grads, q, k, v, o, lse, do, c[5] ** -0.5, n)
    one = [b for b in range(c[0]) if n is None or c[-1][b] == 1]
    for b in one:
        assert bool((grads[0][b] == 0).all()) and bool((grads[1][b] == 0).all())
    do[one[0], 0, 5, 7] = float("nan")
    dq, dk, dv = ops().cross_attention_backward(q, k, v, o, lse, do, key_lengths=n)
    assert bool(dq[one[0], 0, 5].isnan().all()) and bool((dq[one[0], 1] == 0).all())
    assert bool(dk[one[0], 0, 0].isnan().any()) and bool(dv[one[0], 0, 0, 7].isnan())


def test_two_streams_at_once():
    cs = [(2, 8, 2, 1, 6000, 128, BF16, [6000, 2000]), (1, 4, 4, 400, 6000, 64, F16, [5001])]
    sets = [inputs(*c) for c in cs]
    want = [ops().cross_attention_forward(q, k, v, key_lengths=n) for q, k, v, n in sets]
    streams = [torch.cuda.Stream() for _ in cs * 2]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [ops().cross_attention_forward(q, k, v, key_lengths=n, stream=s) for (q, k, v, n), s in zip(sets * 2, streams)]
        grads = [ops().cross_attention_backward(q, k, v, *w, q, key_lengths=n, stream=s)
                 for (q, k, v, n), w, s in zip(sets * 2, want * 2, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want * 2):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for (q, k, v, n), w, g in zip(sets * 2, want * 2, grads):
        check_bwd(g, q, k, v, *w, q, q.shape[3] ** -0.5, n)


def test_offsets_past_32_bits():
    # K and V of 2^31 + elements each: the last batch entry's keys lie past 2^32 bytes
    B, Hkv, Nk, D = 5, 2, 2 ** 22 - 7, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.zeros(B, Hkv, Nk, D, dtype=BF16, device="cuda")
    v = torch.zeros(B, Hkv, Nk, D, dtype=BF16, device="cuda")
    for t in (k, v):
        t[-1, :, -2000:].normal_(generator=g)
    n = torch.tensor([0, 0, 3, 0, Nk], dtype=torch.int32).cuda()
    for Nq in (1, 200):
        q = torch.randn(B, Hkv, Nq, D, generator=torch.Generator().manual_seed(1)).to(BF16).cuda() * 8
        o, lse = ops().cross_attention_forward(q, k, v, key_lengths=n)
        check_fwd(o, lse, q, k, v, 0.125, n)


def test_binding_refusals():
    q, k, v, n = inputs(2, 4, 2, 3, 50, 64, F16, [50, 50])
    f = ops().cross_attention_forward
    for call in (
        lambda: f(q, k, v[:, :, :40].contiguous()), lambda: f(q, k.bfloat16(), v), lambda: f(q[:, :3].contiguous(), k, v),
        lambda: f(q.transpose(1, 2), k, v), lambda: f(q, k[..., :32].contiguous(), v[..., :32].contiguous()),
        lambda: f(q[:1].contiguous(), k, v), lambda: f(q, k, v, key_lengths=n.long()), lambda: f(q, k, v, key_lengths=n[:1]),
        lambda: f(q, k, v, key_lengths=n.cpu()), lambda: f(q, k, v, out=q[:, :2]), lambda: f(q, k, v, lse=torch.empty(2, 4, 4, device="cuda")),
        lambda: f(q, k, v, workspace=torch.empty(16, device="cuda")), lambda: f(q.cpu(), k, v),
    ):
        with pytest.raises((ValueError, TypeError)):
            call()
    b = ops().cross_attention_backward
    o, lse = f(q, k, v, key_lengths=n)
    for call in (lambda: b(q, k, v, o[:, :2], lse, o), lambda: b(q, k, v, o, lse[:, :2], o), lambda: b(q, k, v, o, lse.half(), o),
                 lambda: b(q, k, v, o, lse, o.transpose(2, 3)), lambda: b(q, k, v, o, lse, o, dk=q),
                 lambda: b(q, k, v, o, lse, o, workspace=torch.empty(256, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ops().Fa2Error):
        b(q, k, v, o, lse, o, dk=k)
    for call in (lambda: f(q, k, v, scale=0.0), lambda: f(q, k, v, scale=float("nan")), lambda: f(q, k, v, out=q),
                 lambda: f(*(torch.zeros(1, 1, 2, 80, dtype=F16, device="cuda") for _ in range(3)))):
        with pytest.raises(ops().Fa2Error):
            call()
