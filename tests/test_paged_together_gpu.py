"""The paged cache as a serving program uses it: prompts in chunks, single tokens, evictions, one after another; captured
and replayed; on other streams and in several threads; on long caches."""
from __future__ import annotations

import math
import threading

import pytest
import torch

from bounds import check_key_weights, check_paged_attention
from oracle import norm_rope as rope_ref  # noqa: F401  (the definitions that the calls below stand beside)
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


class Server:
    """A pool of pages and the sequences in it (tables on the host, as a scheduler keeps them)."""

    def __init__(self, B, Hq, Hkv, D, page, pages, dtype, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.D, self.page, self.dtype = B, Hq, Hkv, D, page, dtype
        self.kc, self.vc = (torch.full((pages, Hkv, page, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.weights = torch.full((pages, Hkv, page), float("nan"), device="cuda")
        self.free = torch.randperm(pages, generator=self.g).tolist()
        self.tables, self.lengths = [[] for _ in range(B)], [0] * B
        self.keys, self.values = [[] for _ in range(B)], [[] for _ in range(B)]  # what each sequence was given

    def device(self, counts):
        width = max(1, max(len(t) for t in self.tables))
        table = torch.tensor([t + [-1] * (width - len(t)) for t in self.tables], dtype=torch.int32, device="cuda")
        at = [0]
        for n in counts:
            at.append(at[-1] + n)
        to = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return table, to(self.lengths), to(at)

    def step(self, counts):
        """Norm and rotation, append, attention, key weights of `counts` new tokens; checked; returns nothing."""
        fa2, T = ops(), sum(counts)
        for b, n in enumerate(counts):
            self.lengths[b] += n
            while len(self.tables[b]) * self.page < self.lengths[b]:
                self.tables[b].append(self.free.pop())
        batch = self.device(counts)
        heads = self.Hq + 2 * self.Hkv
        packed = torch.randn(1, T, heads, self.D, generator=self.g).to(self.dtype).cuda()
        q, k, v = packed[:, :, :self.Hq], packed[:, :, self.Hq:self.Hq + self.Hkv], packed[0, :, self.Hq + self.Hkv:]
        where = torch.cat([torch.arange(self.lengths[b] - n, self.lengths[b]) for b, n in enumerate(counts)]).cuda()[None]
        angle = torch.arange(4096, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, self.D, 2) / self.D)
        # the norm writes tokens first, the layout that the cache's calls take
        qn, kn = torch.empty(1, T, self.Hq, self.D, dtype=self.dtype, device="cuda"), torch.empty(
            1, T, self.Hkv, self.D, dtype=self.dtype, device="cuda")
        fa2.qk_norm_rope_forward(q.transpose(1, 2), k.transpose(1, 2), cos=angle.cos().float().cuda(),
                                 sin=angle.sin().float().cuda(), positions=where, q_out=qn.transpose(1, 2),
                                 k_out=kn.transpose(1, 2))
        qn, kn = qn[0], kn[0]
        fa2.paged_cache_append(kn, v, self.kc, self.vc, batch[0], batch[1], batch[2], weights=self.weights)
        o, lse = fa2.paged_attention_forward(qn, self.kc, self.vc, *batch)
        before = self.weights.clone()
        fa2.paged_key_weights(qn, lse, self.kc, *batch, weights=self.weights)
        scale = 1 / math.sqrt(self.D)
        check_paged_attention(o, lse, qn, self.kc, self.vc, batch, scale)
        check_key_weights(self.weights, qn, lse, self.kc, before, batch, scale)
        # what lies in the cache is what each sequence was given, in order
        t = 0
        for b, n in enumerate(counts):
            self.keys[b].append(kn[t:t + n].cpu())
            self.values[b].append(v[t:t + n].cpu())
            t += n
        self.look()

    def look(self):
        for b in range(self.B):
            if not self.lengths[b]:
                continue
            for cache, given in ((self.kc, self.keys[b]), (self.vc, self.values[b])):
                got = cache[self.tables[b]].transpose(1, 2).flatten(0, 1)[:self.lengths[b]].cpu()
                assert torch.equal(got, torch.cat(given))

    def evict(self, keep, recent):
        fa2 = ops()
        table, lens, _ = self.device([0] * self.B)
        width = -(-keep // self.page)
        new = [[self.free.pop() for _ in range(width)] for _ in range(self.B)]
        new_table = torch.tensor(new, dtype=torch.int32, device="cuda")
        want = ref.evict(self.kc, self.vc, self.weights, table, lens, new_table, keep, recent)
        n, kept = fa2.paged_cache_evict(self.kc, self.vc, self.weights, table, lens, new_table, keep, recent)
        for got, w in zip((n, kept, self.kc, self.vc, self.weights), want):
            assert torch.equal(got.cpu().nan_to_num(99) if got.is_floating_point() else got.cpu(),
                               w.nan_to_num(99) if w.is_floating_point() else w)
        self.lengths = n.tolist()
        for b in range(self.B):
            used = -(-self.lengths[b] // self.page)
            self.free += self.tables[b] + new[b][used:]
            self.tables[b] = new[b][:used]
            rows = kept[b, :, :self.lengths[b]].cpu().long()  # [Hkv, kept]
            for given in (self.keys, self.values):
                if given[b]:
                    x = torch.cat(given[b])
                    given[b] = [torch.stack([x[rows[h], h] for h in range(self.Hkv)], 1)]
        self.look()


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, BF16), (12, 12, 64, 32, F16), (7, 1, 96, 64, BF16)])
def test_prompts_tokens_and_evictions(Hq, Hkv, D, page, dtype):
    s = Server(3, Hq, Hkv, D, page, 2200 // page + 40, dtype, seed=Hq)
    s.step([300, 1, 40])       # two prompts and a first token
    s.step([200, 1, 1])        # the next chunk among single tokens
    s.step([1, 1, 1])
    s.evict(100, 10)
    s.step([1, 1, 1])
    s.step([33, 0, 150])       # new chunks behind what was kept; one sequence waits
    s.evict(64, 64)
    s.step([1, 1, 1])
    s.evict(64, 0)


@pytest.mark.parametrize("counts", [[1, 1, 1], [200, 1, 90], [5, 3, 2]])
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
def test_captured_and_replayed(counts, D, dtype):
    # the same buffers with other contents: tables, lengths, queries; a replay repeats its launches' tags
    fa2 = ops()
    lengths = [2500, 40, 1700]
    sets = [Batch(lengths if i != 1 else [1300, 90, 2600], counts, 2, D, 16, dtype, seed=i, width=170, spare=20) for i in range(3)]
    pages = max(b.pages for b in sets)
    kc, vc = (torch.zeros(pages, 2, 16, D, dtype=dtype, device="cuda") for _ in range(2))
    weights = torch.zeros(pages, 2, 16, device="cuda")
    table, lens, starts = sets[0].table.clone(), sets[0].lens.clone(), sets[0].starts.clone()
    q = torch.empty(sum(counts), 8, D, dtype=dtype, device="cuda")
    new = torch.zeros(3, 4, dtype=torch.int32, device="cuda")

    def fill(b):
        for t, x in ((kc, b.kc), (vc, b.vc), (weights, b.weights)):
            t[:b.pages] = x
        table.copy_(b.table)
        lens.copy_(b.lens)
        new.copy_(b.free[:12].reshape(3, 4))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(7)).to(dtype))

    def calls():
        fa2.paged_cache_append(q[:, :2], q[:, 2:4], kc, vc, table, lens, starts, weights=weights)
        o, lse = fa2.paged_attention_forward(q, kc, vc, table, lens, starts)
        fa2.paged_key_weights(q, lse, kc, table, lens, starts, weights=weights)
        n, kept = fa2.paged_cache_evict(kc, vc, weights, table, lens, new, 50, 5)
        return o, lse, n, kept

    def state(outs):
        return [t.clone() for t in (*outs, kc, vc, weights)]

    fill(sets[0])
    calls()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = calls()
        graphs.append((graph, outs))
    for k in range(6):
        b = sets[k % 3]
        fill(b)
        want = state(calls())
        for graph, outs in graphs:
            fill(b)
            graph.replay()
            torch.cuda.synchronize()
            for got, w in zip(state(outs), want):
                assert torch.equal(got.nan_to_num(99), w.nan_to_num(99))


def test_two_graphs_replayed_at_once():
    fa2 = ops()
    runs = []
    for seed in range(2):
        b = Batch([4000, 600, 2500], [1, 300, 2], 2, 128, 32, BF16, seed=seed)
        q = b.tokens(8)
        stream = torch.cuda.Stream()
        want = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
        w = fa2.paged_key_weights(q, want[1], b.kc, b.table, b.lens, b.starts)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = fa2.paged_attention_forward(q, b.kc, b.vc, b.table, b.lens, b.starts)
            got_w = fa2.paged_key_weights(q, got[1], b.kc, b.table, b.lens, b.starts)
        runs.append((graph, stream, (*got, got_w), (*want, w), b, q))
    for _ in range(5):
        for _, _, got, _, _, _ in runs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, got, want, _, _ in runs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_stream_of_its_own():
    fa2 = ops()
    b = Batch([700, 20], [40, 1], 2, 64, 16, F16, seed=1, spare=12)
    q, k = b.tokens(6), b.tokens(2)
    caches = b.kc.clone(), b.vc.clone(), b.weights.clone()
    want_cache = ref.append(k, k, *caches, *b.batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa2.paged_cache_append(k, k, b.kc, b.vc, *b.batch, weights=b.weights, stream=side)
    o, lse = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch, stream=side)
    w = fa2.paged_key_weights(q, lse, b.kc, *b.batch, weights=b.weights, out=torch.zeros_like(b.weights), stream=side)
    fresh = fa2.paged_key_weights(q, lse, b.kc, *b.batch, stream=side)
    new = b.free[:6].reshape(2, 3)
    n, kept = fa2.paged_cache_evict(b.kc, b.vc, b.weights, b.table, b.lens, new, 40, 3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    scale = 1 / 8
    old = [t.cuda() for t in want_cache]
    check_paged_attention(o, lse, q, old[0], old[1], b.batch, scale)
    check_key_weights(w, q, lse, old[0], old[2], b.batch, scale)
    check_key_weights(fresh, q, lse, old[0], None, b.batch, scale)
    want = ref.evict(*want_cache, b.table, b.lens, new, 40, 3)
    assert torch.equal(n.cpu(), want[0]) and torch.equal(kept.cpu(), want[1]) and torch.equal(
        b.kc.cpu().nan_to_num(9), want[2].nan_to_num(9))


def test_two_threads_on_one_stream():
    fa2 = ops()
    sets = []
    for seed in range(2):
        b = Batch([3000, 9, 800], [60, 1, 3], 2, 64, 16, F16, seed=seed)
        sets.append((b, b.tokens(8)))

    def calls(b, q):
        o, lse = fa2.paged_attention_forward(q, b.kc, b.vc, *b.batch)
        return o, lse, fa2.paged_key_weights(q, lse, b.kc, *b.batch)

    want = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    wrong, both = [], threading.Barrier(2)

    def work(i):
        both.wait()
        for _ in range(40):
            got = [calls(*sets[i]) for _ in range(3)]
            torch.cuda.current_stream().synchronize()
            wrong.extend(i for g in got if not all(torch.equal(a, b) for a, b in zip(g, want[i])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("counts", [[1, 1], [100, 40]])
def test_offsets_past_32_bits(counts):
    # two sequences in the first and last pages of caches of 2^31 + elements (5 GB each)
    fa2 = ops()
    pages, Hkv, page, D = 20600, 8, 128, 128
    assert pages * Hkv * page * D > 2 ** 31
    kc, vc = (torch.zeros(pages, Hkv, page, D, dtype=BF16, device="cuda") for _ in range(2))
    weights = torch.zeros(pages, Hkv, page, device="cuda")
    lens = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2], [pages - 3, pages // 2, 5]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(0)
    for row in table.tolist():
        for i in row:
            kc[i], vc[i] = (torch.randn(Hkv, page, D, generator=g).to(BF16).cuda() for _ in range(2))
            weights[i] = torch.rand(Hkv, page, generator=g).cuda()
    q, k = (torch.randn(sum(counts), h, D, generator=g).to(BF16).cuda() for h in (16, 8))
    small = torch.arange(6, dtype=torch.int32).reshape(2, 3)  # the same pages in a small pool
    ids = table.flatten().long()
    parts = [t[ids] for t in (kc, vc, weights)]
    want_parts = ref.append(k, k, *parts, small, lens, starts)
    fa2.paged_cache_append(k, k, kc, vc, table, lens, starts, weights=weights)
    for t, want in zip((kc, vc, weights), want_parts):
        assert torch.equal(t[ids].cpu(), want)
    parts = [t[ids] for t in (kc, vc, weights)]
    batch = (small, lens, starts)
    o, lse = fa2.paged_attention_forward(q, kc, vc, table, lens, starts)
    check_paged_attention(o, lse, q, parts[0], parts[1], batch, D ** -0.5)
    w = fa2.paged_key_weights(q, lse, kc, table, lens, starts, weights=weights, out=torch.empty_like(weights))
    check_key_weights(w[ids], q, lse, parts[0], parts[2], batch, D ** -0.5)
    new = torch.tensor([[pages - 10], [7]], dtype=torch.int32, device="cuda")
    n, kept = fa2.paged_cache_evict(kc, vc, weights, table, lens, new, 128, 16)
    want = ref.evict(*(torch.cat([t, t[:2] * 0]) for t in parts), small, lens, torch.tensor([[6], [7]]), 128, 16)
    assert torch.equal(kept.cpu(), want[1])
    for t, x in zip((kc, vc, weights), want[2:]):
        assert torch.equal(t[new[:, 0].long()].cpu(), x[6:])


def test_many_sequences():
    B = 1000
    lengths = [(97 * i) % 400 for i in range(B)]
    counts = [0 if i % 7 == 0 else 1 + (i % 5) * (i % 11 == 3) * 20 for i in range(B)]
    b = Batch(lengths, counts, 1, 64, 16, BF16, seed=12)
    q = b.tokens(2)
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, *b.batch)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1 / 8)
    w = ops().paged_key_weights(q, lse, b.kc, *b.batch)
    check_key_weights(w, q, lse, b.kc, None, b.batch, 1 / 8)
    k = b.tokens(1)
    want = ref.append(k, k, b.kc, b.vc, None, *b.batch)
    ops().paged_cache_append(k, k, b.kc, b.vc, *b.batch)
    assert torch.equal(b.kc.cpu().nan_to_num(9), want[0].nan_to_num(9))


def test_one_long_sequence_and_its_last_token():
    # more positions than a selection keeps in shared memory, and one token's keys over all SMs
    b = Batch([70000], [1], 1, 64, 64, F16, seed=3, spare=900)
    q = b.tokens(8, 2.0)
    o, lse = ops().paged_attention_forward(q, b.kc, b.vc, *b.batch)
    check_paged_attention(o, lse, q, b.kc, b.vc, b.batch, 1 / 8)
    w = ops().paged_key_weights(q, lse, b.kc, *b.batch)
    check_key_weights(w, q, lse, b.kc, None, b.batch, 1 / 8)
    new = b.free[:800].reshape(1, 800)
    want = ref.evict(b.kc, b.vc, w, b.table, b.lens, new, 50000, 20)
    n, kept = ops().paged_cache_evict(b.kc, b.vc, w, b.table, b.lens, new, 50000, 20)
    assert torch.equal(kept.cpu(), want[1]) and torch.equal(b.vc.cpu().nan_to_num(9), want[3].nan_to_num(9))
