"""Few new tokens over long keys: one attention unit held by many CTAs, all of which join its rows. Against the definition in
64 bits; captured and replayed; in a workspace with anything in it; its waits bounded."""
from __future__ import annotations

import math

import pytest
import torch

from bounds import check_paged_attention
from paged_batches import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


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


CASES = [  # lengths, new tokens, Hq, Hkv, D, page, dtype, causal
    ([4000], [40], 32, 8, 128, 16, BF16, True),      # 19 parts, rows of one sub-tile and a part of the other
    ([5000], [17], 40, 8, 64, 16, F16, True),        # groups of 5
    ([3001], [33], 24, 8, 96, 32, F16, True),        # one sub-tile, 99 rows
    ([2000], [50], 7, 1, 64, 64, BF16, True),        # parts for every tile: 16
    ([1030], [1030], 1, 1, 128, 128, F16, True),     # a unit per 256 tokens, up to 9 tiles, some without a part
    ([9000], [100], 12, 4, 32, 256, BF16, False),
    ([900, 880, 890], [50, 50, 45], 14, 2, 128, 16, BF16, True),   # sequences of 7 and 8 tiles
    ([2500, 2500], [129, 128], 2, 2, 128, 16, F16, True),          # two units to a sequence, one of a single token
    ([2600], [3], 96, 1, 64, 16, BF16, True),        # a token's 96 rows
    ([2048], [300], 4, 1, 96, 16, BF16, True),       # groups of five CTAs and of more
    ([3, 8000], [40, 40], 8, 2, 64, 16, F16, True),  # more tokens than positions beside a long sequence
]


def run(b, Hq, D, causal, **more):
    q = b.tokens(Hq, 1.5)
    out = torch.full((b.T, Hq, D), 7.0, dtype=b.dtype, device="cuda")
    lse = torch.full((b.T, Hq), 7.0, device="cuda")
    got = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, is_causal=causal, out=out, lse=lse, **more)
    return q, got


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(i):
    lengths, counts, Hq, Hkv, D, page, dtype, causal = CASES[i]
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=700 + i, layout=["heads", "slots", "packed"][i % 3], before=i % 2,
              behind=i % 3)
    more = {}
    if i % 2:  # anything in the workspace
        more["workspace"] = torch.randint(0, 256, (ops().fa2_paged_fwd_workspace_bytes(D),), dtype=torch.uint8, device="cuda")
    q, (o, lse) = run(b, Hq, D, causal, **more)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1 / math.sqrt(D), causal=causal)
    # the same bits again
    o2, lse2 = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, is_causal=causal, out=torch.full_like(o, 7.0),
                                             lse=torch.full_like(lse, 7.0))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_replayed():
    b = Batch([6000], [40], 8, 64, 16, F16, seed=21)
    q = b.tokens(32)
    fa2 = ops()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            o, lse = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    for length in (6000, 3000, 45, 5999, 20, 6000):  # other lengths: other parts
        b.lens.fill_(length)
        q.copy_(torch.randn(q.shape, generator=b.g).to(q.dtype))
        want = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
        for _ in range(3):
            o.fill_(7.0)
            lse.fill_(7.0)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_rows_that_are_nan_or_see_nothing():
    b = Batch([4000, 4000], [24, 24], 2, 128, 16, BF16, seed=5)
    q = b.tokens(8)
    q[3, 1, 5] = float("nan")
    q[30, 7, 0] = float("inf")
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    bad = torch.zeros(48, 8, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[30, 7] = True
    assert lse[bad].isnan().all() and o[bad].isnan().all()
    assert not lse[~bad].isnan().any() and not o[~bad].isnan().any()
    clean = q.clone()
    clean[bad] = 0
    o2, lse2 = ops().paged_attention_forward(clean, b.kc, b.vc, b.table, b.lens, b.starts)
    assert torch.equal(o[~bad], o2[~bad]) and torch.equal(lse[~bad], lse2[~bad])
    b.lens.zero_()
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    assert (o == 0).all() and (lse == float("inf")).all()


def test_a_wait_that_runs_out(lib):
    b = Batch([6000], [40], 8, 64, 16, F16, seed=22)
    q = b.tokens(32)
    fa2 = ops()
    want = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    torch.cuda.synchronize()
    lib.fa2_set_watchdog_ns(20_000_000)
    try:
        assert lib.library().fa2_test_withhold_next_load(1) == 0
        fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
        torch.cuda.synchronize()
        assert lib.fa2_device_status(clear=True) > 0
    finally:
        lib.library().fa2_test_withhold_next_load(0)
        lib.fa2_set_watchdog_ns(0)
    got = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert lib.fa2_device_status(clear=False) == 0
