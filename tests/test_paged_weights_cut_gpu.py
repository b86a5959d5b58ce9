"""Key weights whose shares end one cut unit and begin the next with two steps, so that one warpgroup leaves a partial sum,
then joins others, a step apart: the same bits however often, in a workspace that holds large numbers wherever no sum of the
call's own has been written yet."""
from __future__ import annotations

import math

import pytest
import torch

from bounds import check_key_weights
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


@pytest.mark.parametrize("length,count,D,dtype", [  # of 152 CTAs 24, 120, 56 and 32 have such a share
    (3576, 512, 128, BF16), (4448, 128, 64, F16), (2304, 200, 128, F16), (2184, 300, 64, BF16)])
def test_the_same_bits_again(length, count, D, dtype):
    import attention_forward_03_gb300 as fa2
    b = Batch([length], [count], 8, D, 64, dtype, seed=length)
    q = b.tokens(32, 1.5)
    lse = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch)[1]
    workspace = torch.empty(fa2.fa2_paged_key_weights_workspace_bytes(), dtype=torch.uint8, device="cuda")
    out, want = (torch.zeros_like(b.weights) for _ in range(2))

    def call(out):
        workspace.fill_(0x7f)  # 3.4e38 as a float
        return fa2.paged_key_weights(q, lse, b.kc, *b.batch, out=out, workspace=workspace)

    call(want)
    check_key_weights(want, q, lse, b.kc, None, b.batch, 1 / math.sqrt(D))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1000):
        wrong += (call(out) != want).sum()
    assert int(wrong) == 0
