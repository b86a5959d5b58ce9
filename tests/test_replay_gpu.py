"""Captured self-attention replayed on inputs that change before every replay, with units cut between SMs: a replay
carries its launch's tag again, and must not take the partial results that the replay before left behind."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
REPLAYS = 8


@pytest.fixture(scope="module")
def fa2():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as m
    m.fa2_device_status(clear=True)
    yield m
    assert m.fa2_device_status(clear=True) == 0


def fill(tensors, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in tensors:
        t.normal_(generator=g)


def new(c):
    B, H, N, D, dtype, _ = c
    return [torch.empty(B, H, N, D, dtype=dtype, device="cuda") for _ in range(4)]


FORWARD = [  # B, H, N, D, dtype, causal: no multiple of the SMs' count
    (1, 5, 2100, 128, BF16, False),
    (1, 8, 8192, 128, BF16, False),
    (1, 7, 3000, 128, F16, True),
    (2, 5, 2500, 96, F16, False),
    (1, 9, 4000, 64, F16, False),
    (1, 9, 4000, 64, BF16, True),
    (3, 3, 1900, 32, BF16, False),
    (1, 5, 3100, 256, BF16, False),
    (1, 6, 2300, 256, F16, True),
]


@pytest.mark.parametrize("c", FORWARD, ids=str)
def test_forward(fa2, c):
    q, k, v, _ = new(c)
    fill((q, k, v), 0)
    call = lambda: fa2.attention_forward(q, k, v, is_causal=c[5], schedule="balanced")  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call()
    for seed in range(1, 1 + REPLAYS):
        fill((q, k, v), seed)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), seed


BACKWARD = [
    (1, 5, 2100, 128, BF16, False),
    (1, 8, 8192, 128, BF16, False),
    (1, 7, 3000, 128, F16, True),
    (2, 5, 2500, 96, BF16, False),
    (1, 9, 4000, 64, F16, False),
    (1, 9, 4000, 64, BF16, True),
    (3, 3, 1900, 32, F16, True),
]


@pytest.mark.parametrize("c", BACKWARD, ids=str)
def test_backward(fa2, c):
    q, k, v, do = new(c)
    fill((q, k, v, do), 0)

    def call():
        o, lse = fa2.attention_forward(q, k, v, is_causal=c[5], schedule="balanced")
        return fa2.attention_backward(q, k, v, o, lse, do, is_causal=c[5], schedule="balanced")

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = call()
    for seed in range(1, 1 + REPLAYS):
        fill((q, k, v, do), seed)
        for t in grads:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        # dK and dV are summed in a fixed order; dQ is not
        assert torch.equal(grads[1], want[1]) and torch.equal(grads[2], want[2]), seed
        assert float((grads[0].double() - want[0].double()).norm()) <= 2e-3 * float(want[0].double().norm()), seed


@pytest.mark.parametrize("schedule", ["auto", "balanced"])
@pytest.mark.parametrize("on_a_stream", [False, True])
def test_two_graphs_replayed_at_once(fa2, schedule, on_a_stream):
    # each graph's cut units have partial results of their own
    sets = [new((1, 8, 8192, 128, BF16, False))[:3] for _ in range(2)]
    graphs, outs = [], []
    for i, s in enumerate(sets):
        fill(s, i)
        fa2.attention_forward(*s, schedule=schedule)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            arg = {"stream": torch.cuda.current_stream()} if on_a_stream else {}
            outs.append(fa2.attention_forward(*s, schedule=schedule, **arg))
        graphs.append(g)
    want = [fa2.attention_forward(*s, schedule=schedule) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
