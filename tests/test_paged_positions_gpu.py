"""Where attention over a long paged cache takes V from: with queries of zeros every seen position weighs the same, and every
column of V is zero but at one position, so a tile or page that is left out, read twice or from elsewhere shows as a whole
value, however long the cache is.

The bound: every score is 0 and every weight 1, exactly, in 16 bits too; l and O are sums of whole numbers below 2^24 and of
one number and zeros; so what is off is the reciprocal and its product, a step of 2^-24 each, and O's own rounding."""
from __future__ import annotations

import pytest
import torch

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


CASES = [  # lengths, new tokens, Hq, Hkv, D, page, dtype
    ([70000], [1], 8, 1, 64, 64, F16),
    ([70001], [1], 8, 2, 128, 16, F16),
    ([32000, 100, 50003], [1, 1, 1], 4, 4, 96, 128, BF16),
    ([65537], [7], 2, 1, 32, 32, F16),
    ([70000], [40], 8, 2, 128, 16, F16),         # units that all of their CTAs join
    ([40000, 30001], [600, 300], 8, 2, 64, 256, F16),
    ([20000, 35000], [129, 64], 6, 2, 96, 32, F16),
    ([5000], [5000], 4, 1, 128, 64, BF16),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("causal", [True, False])
def test_attention_takes_every_position_s_own_row(i, causal):
    import attention_forward_03_gb300 as fa2
    lengths, counts, Hq, Hkv, D, page, dtype = CASES[i]
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=900 + i, layout=["heads", "slots", "packed"][i % 3])
    q = torch.zeros(b.T, Hq, D, dtype=dtype, device="cuda")
    tol = torch.finfo(dtype).eps / 2 + 3 * 2.0 ** -24
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        b.vc.copy_(torch.zeros_like(b.vc).masked_fill_(~b.used[:, None, :, None], float("nan")))
        want = torch.zeros(b.T, Hkv, D, dtype=torch.float64, device="cuda")
        t0 = 0
        for s, (length, count) in enumerate(zip(lengths, counts)):
            at = torch.stack([torch.randperm(length, generator=g)[:D] for _ in range(Hkv)])  # [Hkv, D]
            edges = [x for x in (0, 15, 16, 127, 128, 255, length - 129, length - count, length - 2, length - 1) if 0 <= x < length]
            for k, x in enumerate(edges):
                at[(k + seed) % Hkv, k] = x
            value = (torch.rand(Hkv, D, generator=g) * 30000 + 2000).to(dtype)
            at, value = at.cuda(), value.cuda()
            h, d = (x.cuda() for x in torch.meshgrid(torch.arange(Hkv), torch.arange(D), indexing="ij"))
            b.vc[b.table[s].long()[at // page], h, at % page, d] = value
            sees = torch.arange(length - count, length, device="cuda") + 1 if causal else torch.full((count,), length, device="cuda")
            want[t0:t0 + count] = (value.double() / sees[:, None, None]) * (at < sees[:, None, None])
            t0 += count
        o = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, is_causal=causal)[0].double()
        want = want.repeat_interleave(Hq // Hkv, 1)
        bad = (o - want).abs() > tol * want
        assert not bad.any() and not o.isnan().any(), f"{int(bad.sum())} of {bad.numel()}"
