"""Batches over a paged cache for the tests: pages in no order, NaN wherever no position is."""
from __future__ import annotations

import torch


class Batch:
    """k_cache, v_cache, table, lens, starts (or None), weights; `T` tokens."""

    def __init__(self, lengths, counts, Hkv, D, page, dtype, seed=0, layout="heads", before=0, behind=0, spare=2,
                 uniform=False, width=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dtype, self.Hkv, self.D, self.page = g, dtype, Hkv, D, page
        need = [-(-n // page) for n in lengths]
        self.pages = sum(need) + spare
        ids = torch.randperm(self.pages, generator=g).to(torch.int32)
        width = width or max(1, max(need, default=1))
        table = torch.full((len(lengths), width), -7, dtype=torch.int32)
        used = torch.zeros(self.pages, page, dtype=torch.bool)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = ids[at:at + k]
            used[ids[at:at + k].long()] = (torch.arange(k * page) < lengths[b]).reshape(-1, page)
            at += k
        self.free = ids[at:].cuda()
        self.used, self.table = used.cuda(), table.cuda()
        self.lens = torch.tensor(lengths, dtype=torch.int32).cuda()
        starts = [before]
        for c in counts:
            starts.append(starts[-1] + c)
        self.T = starts[-1] + behind
        self.starts = None if uniform else torch.tensor(starts, dtype=torch.int32).cuda()
        shape = (self.pages, Hkv, page, D)
        k, v = (torch.randn(shape, generator=g).to(dtype).cuda().masked_fill_(~self.used[:, None, :, None], float("nan"))
                for _ in range(2))
        if layout == "slots":  # [pages, page size, Hkv, D]
            self.kc, self.vc = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        elif layout == "packed":  # one buffer, keys and values of a page together, rows longer than D
            both = torch.full((self.pages, 2, Hkv, page, D + 8), float("nan"), dtype=dtype).cuda()
            both[:, 0, ..., :D], both[:, 1, ..., :D] = k, v
            self.kc, self.vc = both[:, 0, ..., :D], both[:, 1, ..., :D]
        else:
            self.kc, self.vc = k, v
        self.weights = torch.rand(shape[:3], generator=g).cuda()

    def tokens(self, heads, scale=1.0):
        return (torch.randn(self.T, heads, self.D, generator=self.g) * scale).to(self.dtype).cuda()

    @property
    def batch(self):
        return self.table, self.lens, self.starts
