"""The paged key/value cache in 64 bits (torch float64 on the CPU out), sequence by sequence from the definitions. Shares
no code with the GPU path.

A batch is (table, lengths, starts): lists, or tensors on any device. starts None: equally many tokens each.
"""
from __future__ import annotations

import torch


def sequences(table, lengths, starts, T, page):
    """(first token, tokens, positions, pages) of each sequence."""
    B = len(lengths)
    at = [T // B * b for b in range(B + 1)] if starts is None else [int(x) for x in starts]
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        yield b, at[b], at[b + 1] - at[b], n, [int(x) for x in table[b, :-(-n // page)]]


def flat(cache, ids, h, n, fill=0.0):
    """Positions [0, n) of key head h; `fill` where the page number is not one."""
    parts = [cache[i, h].double().cpu() if 0 <= i < cache.shape[0] else
             torch.full(cache.shape[2:], fill, dtype=torch.float64) for i in ids]
    return torch.cat(parts)[:n] if parts else cache.new_zeros((0,) + tuple(cache.shape[3:])).double().cpu()


def scores(q, keys, scale, n, t0, count, j, causal):
    x = q[t0:t0 + count, j].double().cpu() @ keys.T * scale
    if causal:
        x = x.masked_fill(torch.ones(count, n, dtype=torch.bool).triu(n - count + 1), float("-inf"))
    return x


def attention(q, kc, vc, table, lengths, starts, scale, causal=True):
    """(O, LSE, A, size): A is what the rounding of the weights is relative to, sum p |v|; size the largest scale * sum |q k|."""
    T, Hq, D = q.shape
    Hkv, page = kc.shape[1:3]
    group = Hq // Hkv
    o = torch.full(q.shape, float("nan"), dtype=torch.float64)
    a, lse = o.clone(), torch.full((T, Hq), float("nan"), dtype=torch.float64)
    size = 0.0
    for b, t0, count, n, ids in sequences(table, lengths, starts, T, page):
        rows = slice(t0, t0 + count)
        o[rows], a[rows], lse[rows] = 0.0, 0.0, float("inf")
        if n == 0 or count == 0:
            continue
        for h in range(Hkv):
            keys, vals = flat(kc, ids, h, n, float("nan")), flat(vc, ids, h, n)
            for j in range(h * group, (h + 1) * group):
                x = scores(q, keys, scale, n, t0, count, j, causal)
                size = max(size, float((q[rows, j].double().cpu().abs() @ keys.nan_to_num(0).abs().T).max()) * scale)
                seen = ~(x == float("-inf")).all(-1)
                if not seen.any():
                    continue
                l = torch.logsumexp(x[seen], -1)
                p = torch.exp(x[seen] - l[:, None])
                at = torch.arange(t0, t0 + count)[seen]
                lse[at, j], o[at, j], a[at, j] = l, p @ vals, p @ vals.abs()
    return o, lse, a, size


def key_weights(q, lse, kc, weights, table, lengths, starts, scale, causal=True):
    """(out, rows, size): the written slots' new weights (NaN elsewhere), the most rows that a sum has, as above."""
    T, Hq, D = q.shape
    Hkv, page = kc.shape[1:3]
    group = Hq // Hkv
    out = torch.full(kc.shape[:3], float("nan"), dtype=torch.float64)
    size, rows = 0.0, 0
    for b, t0, count, n, ids in sequences(table, lengths, starts, T, page):
        rows = max(rows, count * group)
        for h in range(Hkv):
            keys = flat(kc, ids, h, n, float("nan"))
            w = torch.zeros(n, dtype=torch.float64)
            for j in range(h * group, (h + 1) * group):
                if n == 0 or count == 0:
                    continue
                x = scores(q, keys, scale, n, t0, count, j, causal)
                size = max(size, float((q[t0:t0 + count, j].double().cpu().abs() @ keys.nan_to_num(0).abs().T).max()) * scale)
                x = torch.exp(x - lse[t0:t0 + count, j].double().cpu()[:, None])
                if causal:  # a row without positions has an LSE of +inf
                    x = x.masked_fill(torch.ones(count, n, dtype=torch.bool).triu(n - count + 1), 0.0)
                w += x.sum(0)
            for i, pg in enumerate(ids):
                if 0 <= pg < kc.shape[0]:
                    m = min(page, n - i * page)
                    old = 0.0 if weights is None else weights[pg, h, :m].double().cpu()
                    out[pg, h, :m] = old + w[i * page:i * page + m]
    return out, rows, size


def append(k, v, kc, vc, weights, table, lengths, starts):
    """The caches and weights (CPU, their own types) after the write."""
    kc, vc, weights = kc.cpu().clone(), vc.cpu().clone(), None if weights is None else weights.cpu().clone()
    page = kc.shape[2]
    for b, t0, count, n, ids in sequences(table, lengths, starts, k.shape[0], page):
        for i in range(count):
            pos = n - count + i
            if pos < 0 or not 0 <= ids[pos // page] < kc.shape[0]:
                continue
            at = (ids[pos // page], slice(None), pos % page)
            kc[at], vc[at] = k[t0 + i].cpu(), v[t0 + i].cpu()
            if weights is not None:
                weights[at] = 0.0
    return kc, vc, weights


def evict(kc, vc, weights, table, lengths, new_table, keep, recent):
    """(new lengths, kept, k cache, v cache, weights), on the CPU in their own types."""
    kc, vc, weights = (t.cpu().clone() for t in (kc, vc, weights))
    B, Hkv, page = len(lengths), kc.shape[1], kc.shape[2]
    new_lengths = torch.zeros(B, dtype=torch.int32)
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    moved = []
    for b, _, _, n, ids in sequences(table, lengths, [0] * (B + 1), 0, page):
        new_lengths[b] = min(n, keep)
        for h in range(Hkv):
            def rank(p):
                pg = ids[p // page]
                if not 0 <= pg < kc.shape[0]:
                    return (2, 0.0, p)  # the least
                w = float(weights[pg, h, p % page])
                return (0, 0.0, p) if w != w else (1, -w, p)
            chosen = list(range(n))
            if n > keep:
                chosen = sorted(sorted(range(n - recent), key=rank)[:keep - recent]) + list(range(n - recent, n))
            kept[b, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            moved += [(b, h, j, p, ids[p // page]) for j, p in enumerate(chosen)]
    old = kc.clone(), vc.clone(), weights.clone()
    for b, h, j, p, pg in moved:
        to = int(new_table[b, j // page])
        if 0 <= to < kc.shape[0]:
            for new, was in zip((kc, vc, weights), old):
                new[to, h, j % page] = was[pg, h, p % page] if 0 <= pg < kc.shape[0] else 0.0
    return new_lengths, kept, kc, vc, weights
