"""The paged key/value cache on the GPU against its definitions in 64 bits (the bounds: bounds.py)."""
from __future__ import annotations

import math

import pytest
import torch

from bounds import check_key_weights, check_paged_attention
from oracle import paged as ref
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


CASES = [  # lengths, new tokens, Hq, Hkv, D, page, dtype
    ([1], [1], 1, 1, 64, 16, F16),
    ([1, 0, 17], [1, 0, 1], 4, 2, 32, 16, BF16),
    ([15, 16, 17, 33], [1, 1, 1, 1], 8, 8, 64, 16, F16),
    ([300, 129, 128, 5], [1, 1, 1, 1], 8, 2, 128, 32, BF16),
    ([1000, 1, 0, 64], [1, 1, 0, 1], 12, 12, 96, 64, F16),
    ([5000], [1], 7, 1, 128, 16, F16),
    ([700, 3], [2, 3], 8, 1, 64, 128, BF16),
    ([777, 130], [5, 1], 6, 2, 96, 16, BF16),
    ([200, 0, 90], [40, 0, 90], 2, 2, 64, 16, F16),
    ([128], [128], 4, 1, 128, 128, BF16),
    ([129, 257], [129, 130], 2, 2, 96, 64, F16),
    ([500], [17], 16, 1, 128, 32, F16),
    ([400, 33, 1, 256], [100, 33, 1, 7], 28, 4, 64, 32, F16),
    ([260], [260], 3, 3, 32, 256, BF16),
    ([640, 300], [300, 300], 5, 1, 128, 16, BF16),
    ([1500], [37], 40, 1, 64, 16, F16),
    ([900, 5, 0, 77, 513], [256, 2, 0, 1, 64], 24, 8, 128, 64, BF16),
    ([3, 20], [5, 20], 4, 2, 64, 16, BF16),  # more tokens than positions
    ([0, 40], [4, 2], 4, 4, 128, 16, F16),
    ([(37 * i) % 257 for i in range(150)], [1 if i % 5 else 0 for i in range(150)], 4, 2, 64, 16, BF16),
    ([(13 * i) % 301 + 20 for i in range(40)], [(7 * i) % 20 for i in range(40)], 8, 2, 128, 32, F16),
    ([2000, 1800, 1], [700, 1, 1], 8, 2, 128, 64, BF16),
    ([1000] * 3, [500, 20, 3], 14, 2, 96, 16, F16),
    ([2100], [1030], 2, 1, 32, 64, F16),
    ([70, 64], [3, 2], 256, 1, 64, 16, BF16),
    ([70, 10], [3, 2], 150, 1, 128, 16, F16),
]
LAYOUTS = ["heads", "slots", "packed"]


def name_of(c):
    return "-".join(str(x)[:24].replace(" ", "") for x in c)


@pytest.mark.parametrize("i", range(len(CASES)), ids=[name_of(c) for c in CASES])
def test_attention(i):
    lengths, counts, Hq, Hkv, D, page, dtype = CASES[i]
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=i, layout=LAYOUTS[i % 3], before=i % 2, behind=i % 3)
    q = b.tokens(Hq, 1.5)
    scale = 1 / math.sqrt(D)
    out = torch.full((b.T, Hq, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((b.T, Hq), 7.0, device="cuda")
    got = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check_paged_attention(out, lse, q, b.kc, b.vc, b.batch, scale)
    first, last = int(b.starts[0]), int(b.starts[-1])
    for t in (out, lse):  # rows of no sequence
        assert bool((t[:first] == 7).all()) and bool((t[last:] == 7).all())
    # no order of its own, also where every kernel is told of the longest sequence or of a wrong one
    for most in (None, max(counts), 1):
        again = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, max_query_length=most)
        if most is None:
            assert torch.equal(again[0][first:last], out[first:last]) and torch.equal(again[1][first:last], lse[first:last])
        check_paged_attention(*again, q, b.kc, b.vc, b.batch, scale)


@pytest.mark.parametrize("i", range(len(CASES)), ids=[name_of(c) for c in CASES])
def test_attention_of_all_positions(i):
    lengths, counts, Hq, Hkv, D, page, dtype = CASES[i]
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=50 + i)
    q = b.tokens(Hq, 2.0)
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, scale=0.2, is_causal=False)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 0.2, False)


@pytest.mark.parametrize("n", [1, 2, 5, 40])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
def test_attention_without_starts(n, D, dtype):
    b = Batch([n, 300, 64, 111], [n] * 4, 2, D, 16, dtype, seed=n, uniform=True)
    q = b.tokens(8, 1.5)
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1 / math.sqrt(D))


@pytest.mark.parametrize("count", [1, 50])
def test_attention_of_a_strided_q_and_a_wide_table(count):
    b = Batch([500, 90], [count] * 2, 4, 64, 32, BF16, seed=3, width=40)
    packed = (torch.randn(12, b.T, 2 * b.D, generator=b.g)).to(BF16).cuda()
    q = packed[2:10, :, b.D:].transpose(0, 1)  # heads outside, half of longer rows
    wide = torch.full((2, 80), -1, dtype=torch.int32, device="cuda")
    wide[:, 10:50] = b.table
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, wide[:, 10:50], b.lens, b.starts)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1 / 8)


@pytest.mark.parametrize("counts", [[1, 1, 1], [1, 30, 200]])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_that_are_none(counts, D):
    # sequence 0: its second page; 1: one that only its last tokens see; 2: none of those in use
    b = Batch([100, 260, 250], counts, 2, D, 16, BF16, seed=9, spare=4)
    b.table[0, 1] = b.pages
    b.table[1, 15] = -1
    q = b.tokens(4)
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1 / math.sqrt(D))
    assert bool(o[0].isnan().all()) and not o[-1].isnan().any()
    lse = torch.full((b.T, 4), 3.0, device="cuda")
    w = ops().paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts, weights=b.weights.clone())
    check_key_weights(w, q, lse, b.kc, b.weights, b.batch, 1 / math.sqrt(D))


def test_lengths_and_starts_out_of_range_are_bounded():
    b = Batch([64, 64], [8, 8], 2, 64, 16, F16, seed=4)
    q = b.tokens(4)
    want = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
    lens = torch.tensor([2 ** 30, -5], dtype=torch.int32, device="cuda")
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, lens, b.starts)
    assert torch.equal(o[:8], want[0][:8]) and torch.equal(lse[:8], want[1][:8])
    assert bool((o[8:] == 0).all()) and bool((lse[8:] == float("inf")).all())
    starts = torch.tensor([-3, 8, 2 ** 30], dtype=torch.int32, device="cuda")
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, starts)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("count", [1, 64])
def test_scores_far_apart_and_infinite(count):
    # rising scores across tiles, a dominant last key, -inf scores; a NaN key behind the row is not seen
    b = Batch([1000], [count], 1, 64, 16, F16, seed=6)
    q = torch.ones(count, 2, 64, dtype=F16, device="cuda")
    for i in range(1000):
        pg = int(b.table[0, i // 16])
        b.kc[pg, 0, i % 16] = i / 200 - 2.5
    b.kc[int(b.table[0, 0]), 0, :8, 0] = float("-inf")
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, scale=1.0)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1.0)
    if count > 1:
        b.kc[int(b.table[0, 999 // 16]), 0, 999 % 16] = float("nan")
        o, lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts, scale=1.0)
        assert bool(lse[-1].isnan().all()) and not lse[:-1].isnan().any()


@pytest.mark.parametrize("i", range(len(CASES)), ids=[name_of(c) for c in CASES])
@pytest.mark.parametrize("causal", [True, False])
def test_key_weights(i, causal):
    lengths, counts, Hq, Hkv, D, page, dtype = CASES[i]
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=100 + i, layout=LAYOUTS[(i + 1) % 3], before=i % 2, behind=i % 3)
    q = b.tokens(Hq, 1.5)
    scale = 1 / math.sqrt(D)
    lse = ref.attention(q, b.kc, b.vc, *b.batch, scale, causal)[1].float().cuda()
    out = torch.full_like(b.weights, -1.0)
    before = b.weights.clone()
    got = ops().paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts, is_causal=causal, weights=b.weights, out=out)
    assert got is out and torch.equal(before, b.weights)
    check_key_weights(out, q, lse, b.kc, b.weights, b.batch, scale, causal)
    assert bool((out.transpose(1, 2)[~b.used] == -1).all())  # slots of no sequence
    for most in (None, max(counts), 1):
        again = b.weights.clone()
        got = ops().paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts, is_causal=causal, weights=again,
                                      max_query_length=most)
        assert got is again
        check_key_weights(again, q, lse, b.kc, b.weights, b.batch, scale, causal)
        if most is None:
            assert torch.equal(again.transpose(1, 2)[b.used], out.transpose(1, 2)[b.used])
    fresh = ops().paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts, is_causal=causal)
    check_key_weights(fresh, q, lse, b.kc, None, b.batch, scale, causal)
    assert bool((fresh.transpose(1, 2)[~b.used] == 0).all())


def test_key_weights_of_a_step_add_up_to_its_rows():
    b = Batch([500, 31, 1], [3, 1, 1], 2, 64, 16, BF16, seed=8)
    q = b.tokens(6)
    lse = ops().paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)[1]
    w = ops().paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts)
    # every softmax row sums to one: 3 query heads to a key head. A row's 500 terms: 16 * 20 + 4 * 8 + 32 steps, summed
    # in 64 bits here
    assert abs(float(w.double().sum()) - 5 * 6) < 30 * 400 * 2.0 ** -24


@pytest.mark.parametrize("i", range(len(CASES)), ids=[name_of(c) for c in CASES])
def test_append(i):
    lengths, counts, Hq, Hkv, D, page, dtype = CASES[i]
    b = Batch(lengths, counts, Hkv, D, page, dtype, seed=200 + i, layout=LAYOUTS[i % 3], before=i % 2, behind=i % 3)
    packed = b.tokens(3 * Hkv)
    k, v = packed[:, Hkv:2 * Hkv], packed[:, 2 * Hkv:]
    want = ref.append(k, v, b.kc, b.vc, b.weights if i % 4 else None, *b.batch)
    got = ops().paged_cache_append(k, v, b.kc, b.vc, b.table, b.lens, b.starts, weights=b.weights if i % 4 else None)
    assert got[0] is b.kc and got[1] is b.vc
    for a, w in zip((b.kc, b.vc, b.weights), want):
        if w is not None:
            assert torch.equal(a.cpu().nan_to_num(99.0), w.nan_to_num(99.0))


def test_append_leaves_pages_that_are_none():
    b = Batch([40, 40], [20, 20], 2, 64, 16, F16, seed=2)
    b.table[0, 1], b.table[1, 2] = b.pages + 5, -1
    k, v = b.tokens(2), b.tokens(2)
    want = ref.append(k, v, b.kc, b.vc, b.weights, *b.batch)
    ops().paged_cache_append(k, v, b.kc, b.vc, b.table, b.lens, b.starts, weights=b.weights)
    for a, w in zip((b.kc, b.vc, b.weights), want):
        assert torch.equal(a.cpu().nan_to_num(99.0), w.nan_to_num(99.0))


EVICTIONS = [  # lengths, Hkv, D, page, dtype, keep, recent
    ([1], 1, 64, 16, F16, 1, 0),
    ([2], 1, 32, 16, BF16, 1, 1),
    ([100, 3, 0, 50], 2, 64, 16, F16, 50, 8),
    ([1000, 257, 258, 31], 3, 128, 32, BF16, 257, 257),
    ([777, 512], 2, 96, 64, F16, 300, 0),
    ([5000], 1, 64, 128, BF16, 4999, 1),
    ([5000, 4000], 2, 128, 16, F16, 1, 0),
    ([64, 65, 66], 4, 64, 256, BF16, 64, 10),
    ([60000], 1, 32, 16, F16, 50000, 100),
    ([90, 20], 2, 64, 16, F16, 0, 0),
]


@pytest.mark.parametrize("i", range(len(EVICTIONS)), ids=[name_of(c) for c in EVICTIONS])
@pytest.mark.parametrize("values", ["spread", "equal", "ties", "special"])
def test_evict(i, values):
    lengths, Hkv, D, page, dtype, keep, recent = EVICTIONS[i]
    width = -(-keep // page)
    b = Batch(lengths, [0] * len(lengths), Hkv, D, page, dtype, seed=300 + i, layout=LAYOUTS[i % 3],
              spare=len(lengths) * width + 1)
    if values == "equal":
        b.weights.fill_(0.25)
    elif values == "ties":
        b.weights = (b.weights * 7).floor()
    elif values == "special":
        w = b.weights.flatten()
        w -= 0.5
        for k, x in enumerate((float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-45, -1e-45)):
            w[k::31] = x
    new = b.free[:len(lengths) * width].reshape(len(lengths), width)
    want = ref.evict(b.kc, b.vc, b.weights, b.table, b.lens, new, keep, recent)
    got = ops().paged_cache_evict(b.kc, b.vc, b.weights, b.table, b.lens, new, keep, recent)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    for a, w in zip((b.kc, b.vc, b.weights), want[2:]):
        assert torch.equal(a.cpu().nan_to_num(99.0), w.nan_to_num(99.0))


def test_evict_with_pages_that_are_none():
    b = Batch([100, 70], [0, 0], 2, 64, 16, F16, seed=5, spare=9)
    b.table[0, 2], b.table[1, 0] = -1, b.pages
    new = b.free[:6].reshape(2, 3).clone()
    new[1, 1] = -4
    want = ref.evict(b.kc, b.vc, b.weights, b.table, b.lens, new, 40, 4)
    got = ops().paged_cache_evict(b.kc, b.vc, b.weights, b.table, b.lens, new, 40, 4)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    for a, w in zip((b.kc, b.vc, b.weights), want[2:]):
        assert torch.equal(a.cpu().nan_to_num(99.0), w.nan_to_num(99.0))


def test_refusals():
    b = Batch([64, 64], [1, 1], 2, 64, 16, F16, spare=9)
    q, k = b.tokens(4), b.tokens(2)
    fa2 = ops()
    lse = torch.zeros(2, 4, device="cuda")
    new = b.free[:4].reshape(2, 2)

    def attend(**over):
        a = dict(q=q, k_cache=b.kc, v_cache=b.vc, block_table=b.table, key_lengths=b.lens, query_starts=b.starts)
        return fa2.paged_attention_forward(**{**a, **over})

    attend()
    for over in (dict(q=q[0]), dict(q=q.bfloat16()), dict(q=q.float()), dict(q=b.tokens(3)), dict(q=q[..., :32]),
                 dict(q=q.cpu()), dict(k_cache=b.kc[:3]), dict(v_cache=b.vc.transpose(2, 3)), dict(v_cache=b.vc[..., :32]),
                 dict(block_table=b.table.long()), dict(block_table=b.table[0]), dict(block_table=b.table.T.contiguous().T),
                 dict(block_table=b.table.cpu()), dict(key_lengths=b.lens[:1]), dict(key_lengths=b.lens.long()),
                 dict(query_starts=b.starts[:2]), dict(query_starts=b.starts.float()), dict(q=b.tokens(4)[:1], query_starts=None),
                 dict(out=q[:1]), dict(lse=lse.half()), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            attend(**over)
    for over in (dict(scale=0.0), dict(scale=float("nan")), dict(max_query_length=-1), dict(out=q),
                 dict(k_cache=b.kc[:, :, :8], v_cache=b.vc[:, :, :8]),
                 dict(q=torch.zeros(2 * 4 * 64 + 4, dtype=F16, device="cuda")[4:].view(2, 4, 64))):
        with pytest.raises(fa2.Fa2Error):
            attend(**over)
    with pytest.raises(ValueError):
        fa2.paged_cache_append(k, k[:1], b.kc, b.vc, b.table, b.lens, b.starts)
    with pytest.raises(ValueError):
        fa2.paged_cache_append(k, k, b.kc, b.vc, b.table, b.lens, b.starts, weights=b.weights.half())
    with pytest.raises(fa2.Fa2Error):
        fa2.paged_cache_append(b.kc[0].transpose(0, 1)[:2], k, b.kc, b.vc, b.table, b.lens, b.starts)
    with pytest.raises(ValueError):
        fa2.paged_key_weights(q, lse[:1], b.kc, b.table, b.lens, b.starts)
    with pytest.raises(ValueError):
        fa2.paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts, weights=b.weights[:2])
    with pytest.raises(fa2.Fa2Error):
        fa2.paged_key_weights(q, lse, b.kc, b.table, b.lens, b.starts, scale=-1.0)
    for keep, recent in ((33, 0), (8, 9), (-1, -1), (8, -1)):
        with pytest.raises(ValueError):
            fa2.paged_cache_evict(b.kc, b.vc, b.weights, b.table, b.lens, new, keep, recent)
    with pytest.raises(ValueError):
        fa2.paged_cache_evict(b.kc, b.vc, b.weights, b.table, b.lens, new[:1], 8)
    with pytest.raises(fa2.Fa2Error):
        fa2.paged_cache_evict(b.kc, b.vc, b.weights, b.table, b.lens, b.table, 8)
    with pytest.raises(TypeError):
        fa2.paged_cache_evict(b.kc.float(), b.vc.float(), b.weights, b.table, b.lens, new, 8)


def test_no_tokens_and_no_sequences():
    fa2 = ops()
    b = Batch([20, 5], [0, 0], 2, 64, 16, F16, seed=1)
    q, lse = b.tokens(4), torch.zeros(0, 4, device="cuda")
    o, l = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)
    w = fa2.paged_key_weights(q, lse, b.kc, b.table, b.lens, weights=b.weights, out=torch.zeros_like(b.weights))
    assert torch.equal(w.transpose(1, 2)[b.used], b.weights.transpose(1, 2)[b.used])
    fa2.paged_cache_append(q[:, :2], q[:, :2], b.kc, b.vc, b.table, b.lens)
    none = (b.table[:0], b.lens[:0])
    assert fa2.paged_attention_forward(q, b.kc, b.vc, *none)[0].shape == (0, 4, 64)
    n, kept = fa2.paged_cache_evict(b.kc, b.vc, b.weights, *none, b.table[:0], 4)
    assert n.shape == (0,) and kept.shape == (0, 2, 4)


@pytest.mark.parametrize("D", [64, 128])
def test_key_weights_where_many_units_lack_their_second_tile(D):
    # lengths around 128 and 256, in runs: warpgroups and loads of the one tile go on without those of the other
    lengths = [90] * 40 + [200] * 9 + [128] * 25 + [256, 257, 129, 1] * 20 + [300] * 30 + [60] * 60
    for counts in ([1] * len(lengths), [1 + (i % 4) * 29 for i in range(len(lengths))]):
        counts = [min(n, length) for n, length in zip(counts, lengths)]
        b = Batch(lengths, counts, 4, D, 16, BF16, seed=21)
        q = b.tokens(8)
        lse = torch.full((b.T, 8), 5.0, device="cuda")
        for most in (None, max(counts)):
            w = ops().paged_key_weights(q, lse, b.kc, *b.batch, max_query_length=most)
            check_key_weights(w, q, lse, b.kc, None, b.batch, D ** -0.5)
