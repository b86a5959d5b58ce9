"""Cases and plain forms of the paged key/value cache: what a serving program calls beside `attention_forward`.

Keys and values live in pages, [pages, Hkv, page size, D]; sequence b's position p is slot p % page size of page
table[b, p // page size]. The batch's new tokens are packed, [T, heads, D]: sequence b's are rows starts[b] ..
starts[b + 1], and they are the last of its lengths[b] positions (so a step's single tokens, a chunk of a prompt and
whole prompts mix in one call). Four operators:

  append   the new tokens' keys and values into their slots; the slots' attention weights set to zero
  attend   O = softmax(scale Q K^T) V of the new tokens over their sequence's positions, each seeing its own and the
           earlier ones, Hq / Hkv query heads to each key head; and the rows' log-sum-exp (a row without keys: O = 0,
           LSE = +inf)
  weigh    out[slot] = weights[slot] + the weights that the slot's key gets in the softmax rows of the new tokens of all
           Hq / Hkv query heads
  evict    of a sequence's positions `keep` stay per key head (all, where there are no more): the last `recent`, and
           those of the greatest weight among the others (of equal ones the first); keys, values and weights go in
           order to the positions 0, 1, .. of new pages; returned are the new lengths, the kept positions (-1 behind
           them) and the caches

The plain forms use elementary torch operations in 32 bits and round once at the end. They take the sequences with
equally many new tokens together.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of each of 64 sequences into its slot: a decoding step's write, latency
        {"name": "append_step", "op": "append", "B": 64, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16, "L": 4096,
         "spread": "ragged", "n": 1, "chunks": 64, "empty": False},
        # the prompts of a batch out of their packed projection into the cache
        {"name": "append_prompt", "op": "append", "B": 4, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "L": 8192,
         "spread": "ragged", "n": 8192, "chunks": 4, "empty": False},
        # single tokens of a few short sequences: the smallest call, latency
        {"name": "attend_step", "op": "attend", "B": 4, "Hq": 12, "Hkv": 12, "D": 64, "dtype": "f16", "page": 16,
         "L": 1000, "spread": "ragged", "n": 1, "chunks": 4, "empty": False},
        # a serving batch of single tokens over long, different contexts, a slot of the batch unused: the cache's bytes
        {"name": "attend_step_batch", "op": "attend", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 16, "L": 4096, "spread": "ragged", "n": 1, "chunks": 64, "empty": True},
        # one chunk of a long prompt, its earlier chunks in the cache: few units, long keys
        {"name": "attend_chunk", "op": "attend", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64,
         "L": 8192, "spread": "full", "n": 512, "chunks": 1, "empty": False},
        # two prompts' chunks among single tokens, seven query heads to a key head
        {"name": "attend_mixed", "op": "attend", "B": 16, "Hq": 28, "Hkv": 4, "D": 64, "dtype": "f16", "page": 32,
         "L": 3000, "spread": "ragged", "n": 1000, "chunks": 2, "empty": False},
        # whole prompts of the benchmark's causal shape, grouped heads: the tensor cores' rate
        {"name": "attend_prompt", "op": "attend", "B": 4, "Hq": 16, "Hkv": 4, "D": 128, "dtype": "bf16", "page": 128,
         "L": 4096, "spread": "full", "n": 4096, "chunks": 4, "empty": False},
        # a decoding step adds to the weights of everything cached: the keys' bytes
        {"name": "weigh_step_batch", "op": "weigh", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16,
         "L": 4096, "spread": "ragged", "n": 1, "chunks": 64, "empty": True},
        # a chunk of a prompt as the window that says which keys matter: products and exponentials
        {"name": "weigh_chunk", "op": "weigh", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64,
         "L": 8192, "spread": "full", "n": 512, "chunks": 1, "empty": False},
        # the last rows of ragged prompts, odd sizes
        {"name": "weigh_ragged", "op": "weigh", "B": 5, "Hq": 12, "Hkv": 4, "D": 64, "dtype": "f16", "page": 16,
         "L": 1000, "spread": "ragged", "n": 33, "chunks": 5, "empty": False},
        # small budgets of short ragged sequences, one of them within its budget
        {"name": "evict_small", "op": "evict", "B": 5, "Hkv": 4, "D": 64, "dtype": "f16", "page": 16, "L": 1000,
         "spread": "ragged", "keep": 257, "recent": 32, "empty": False},
        # a batch of long prompts cut down after they have been read
        {"name": "evict_prompt", "op": "evict", "B": 8, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "L": 8192,
         "spread": "full", "keep": 2048, "recent": 128, "empty": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        most[c["op"]] = {t: max(m[t], w[t]) for t in m}
    op = rng.choice(["append", "attend", "attend", "attend", "attend", "weigh", "weigh", "evict"])
    while True:
        c = {"op": op, "B": _log_int(rng, 1, 64), "Hkv": rng.choice([1, 2, 3, 4, 8, 12]),
             "D": rng.choice([32, 64, 64, 96, 128, 128]), "dtype": rng.choice(["f16", "bf16"]),
             "page": rng.choice([16, 16, 32, 64, 128]), "L": _log_int(rng, 1, 8192),
             "spread": rng.choice(["full", "ragged"])}
        if op in ("attend", "weigh"):
            c["Hq"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4, 7, 8])
        if op == "evict":
            c["keep"] = _log_int(rng, 1, max(c["L"], 2))
            c["recent"] = rng.randint(0, c["keep"])
        else:
            c["n"] = 1 if rng.random() < 0.35 else _log_int(rng, 1, c["L"])
            c["chunks"] = rng.choice([c["B"], c["B"], rng.randint(0, c["B"])])
        c["empty"] = c["B"] > 1 and rng.random() < 0.3
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"] and _scores(c) <= 1.1e9:
            return c


def _scores(c):
    """Score entries that the plain form holds at once."""
    if c["op"] not in ("attend", "weigh"):
        return 0
    return max(c["chunks"] * c["n"], c["B"]) * c["Hq"] * c["L"]


def _lengths(c):
    """Positions of each sequence: the same, or evenly spread over (0, L]; the last sequence's 0 where `empty`."""
    full = c["spread"] == "full"
    n = [c["L"] if full else max(1, c["L"] * (c["B"] - b) // c["B"]) for b in range(c["B"])]
    if c["empty"]:
        n[-1] = 0
    return n


def _counts(c):
    """New tokens of each sequence: `n` of the first `chunks` ones (as many as they have positions), one of the others."""
    return [min(c["n"] if b < c["chunks"] else 1, length) for b, length in enumerate(_lengths(c))]


def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _pages(g, lengths, page, free):
    """A table of pages in no order, -1 behind each sequence's last one, with `free` pages over; and the pool's size."""
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + free
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, pool, ids[at:]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    lengths = _lengths(c)
    s = {"case": c, "lens": torch.tensor(lengths, dtype=torch.int32, device="cuda"), "lengths": lengths}
    new_pages = -(-c["keep"] // page) if c["op"] == "evict" else 0
    s["table"], pool, left = _pages(g, lengths, page, 3 + B * new_pages)
    s["kc"] = _randn(g, pool, Hkv, page, D, dtype=dt)
    s["vc"] = _randn(g, pool, Hkv, page, D, dtype=dt)
    if c["op"] == "evict":
        # long tails, some keys that nothing has looked at yet, and equal weights
        w = torch.randn(pool, Hkv, page, generator=g, device="cuda").mul(2.0).exp()
        w = (w * 64).round() / 64
        s["weights"] = w.masked_fill(torch.rand(pool, Hkv, page, generator=g, device="cuda") < 0.1, 0.0)
        s["new_table"] = left[:B * new_pages].reshape(B, new_pages).contiguous()
        return s
    counts = _counts(c)
    s["counts"] = counts
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    s["starts_at"], T = at, at[-1]
    # single tokens of every sequence need no table of where each begins
    s["starts"] = None if all(n == 1 for n in counts) else torch.tensor(at, dtype=torch.int32, device="cuda")
    s["longest"] = max(counts)
    if c["op"] == "append":
        # one projection's output, four query heads to each key head; k and v are views of it
        packed = _randn(g, T, 6 * Hkv, D, dtype=dt)
        s["k"], s["v"] = packed[:, 4 * Hkv:5 * Hkv], packed[:, 5 * Hkv:]
        s["weights"] = torch.rand(pool, Hkv, page, generator=g, device="cuda")
        return s
    s["q"] = _randn(g, T, c["Hq"], D, dtype=dt, scale=1.5)
    s["scale"] = 1.0 / math.sqrt(D)
    # what a cache holds where no position is, is anything
    used = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        if n:
            ids = s["table"][b, :-(-n // page)].long()
            used[ids] = (torch.arange(len(ids) * page, device="cuda") < n).reshape(-1, page)
    s["kc"].masked_fill_(~used[:, None, :, None], float("nan"))
    s["vc"].masked_fill_(~used[:, None, :, None], float("nan"))
    if c["op"] == "weigh":
        s["lse"] = _attend(s)[1]
        s["weights"] = torch.rand(pool, Hkv, page, generator=g, device="cuda").masked_fill(~used[:, None, :], 0.0)
        s["out"] = torch.zeros_like(s["weights"])
    return s


def _slots(s, b, lo, hi):
    """(page, slot) of sequence b's positions [lo, hi)."""
    page = s["case"]["page"]
    p = torch.arange(lo, hi, device="cuda")
    return s["table"][b].long()[p // page], p % page


def _groups(s):
    """The sequences with new tokens by how many they have: (count, sequences, longest, token rows [sequences, count])."""
    by = {}
    for b, n in enumerate(s["counts"]):
        if n:
            by.setdefault(n, []).append(b)
    for n, bs in by.items():
        first = torch.tensor([s["starts_at"][b] for b in bs], device="cuda")
        rows = first[:, None] + torch.arange(n, device="cuda")[None]
        yield n, bs, max(s["lengths"][b] for b in bs), rows


def _gather(s, cache, bs, most):
    """The positions [0, most) of the sequences `bs`, [sequences, Hkv, most, D] in 32 bits; zeros where there are none."""
    page = s["case"]["page"]
    p = torch.arange(most, device="cuda")
    at = s["table"][bs].long()[:, p // page].clamp(min=0)  # [sequences, most]
    x = cache[at, :, p % page].float().transpose(1, 2)
    behind = p[None] >= s["lens"][bs][:, None]
    return x.masked_fill(behind[:, None, :, None], 0.0), at, p % page


def _scored(s, n, bs, most, rows):
    """q [sequences, Hkv, group * n, D], scores and keys of a group of sequences; -inf where a token does not see a key."""
    k, at, slot = _gather(s, s["kc"], bs, most)
    Hkv, D = k.shape[1], k.shape[3]
    group = s["case"]["Hq"] // Hkv
    q = s["q"][rows].float().reshape(len(bs), n, Hkv, group, D).permute(0, 2, 3, 1, 4)  # [sequences, Hkv, group, n, D]
    x = (q.reshape(len(bs), Hkv, group * n, D) @ k.transpose(2, 3)) * s["scale"]
    last = s["lens"][bs].long()[:, None] - n + torch.arange(n, device="cuda")[None]  # a token's own position
    hidden = torch.arange(most, device="cuda")[None, None] > last[:, :, None]  # [sequences, n, most]
    hidden = hidden[:, None, None].expand(-1, 1, group, -1, -1).reshape(len(bs), 1, group * n, most)
    return x.masked_fill(hidden, float("-inf")), at, slot


def _attend(s):
    c = s["case"]
    o, lse = torch.zeros_like(s["q"]), torch.full(s["q"].shape[:2], float("inf"), device="cuda")
    for n, bs, most, rows in _groups(s):
        x = _scored(s, n, bs, most, rows)[0]
        v = _gather(s, s["vc"], bs, most)[0]
        m = x.amax(-1, keepdim=True)  # a new token sees itself at least
        p = torch.exp(x - m)
        z = p.sum(-1, keepdim=True)
        back = lambda t: t.reshape(len(bs), c["Hkv"], -1, n, t.shape[-1]).permute(0, 3, 1, 2, 4).reshape(  # noqa: E731
            len(bs), n, c["Hq"], -1)
        o[rows] = back((p @ v) / z).to(o.dtype)
        lse[rows] = back(m + torch.log(z))[..., 0]
    return o, lse


def _weigh(s):
    c, out = s["case"], s["out"]
    for b, n in enumerate(s["lengths"]):
        if n and not s["counts"][b]:
            page, slot = _slots(s, b, 0, n)
            out[page, :, slot] = s["weights"][page, :, slot]
    for n, bs, most, rows in _groups(s):
        x, at, slot = _scored(s, n, bs, most, rows)
        group = c["Hq"] // c["Hkv"]
        lse = s["lse"][rows].reshape(len(bs), n, c["Hkv"], group).permute(0, 2, 3, 1).reshape(len(bs), c["Hkv"], -1, 1)
        w = torch.exp(x - lse).sum(2)  # [sequences, Hkv, most]
        here = torch.arange(most, device="cuda")[None] < s["lens"][bs][:, None]
        i = here.nonzero()
        page, slot = at[i[:, 0], i[:, 1]], slot[i[:, 1]]
        out[page, :, slot] = s["weights"][page, :, slot] + w.transpose(1, 2)[here]
    return out


def _append(s):
    lens, page = s["lens"].long(), s["case"]["page"]
    n = torch.tensor(s["counts"], device="cuda")
    b = torch.repeat_interleave(torch.arange(len(s["counts"]), device="cuda"), n)
    first = torch.tensor(s["starts_at"][:-1], device="cuda")
    p = lens[b] - n[b] + torch.arange(s["starts_at"][-1], device="cuda") - first[b]
    at, slot = s["table"].long()[b, p // page], p % page
    s["kc"][at, :, slot] = s["k"]
    s["vc"][at, :, slot] = s["v"]
    s["weights"][at, :, slot] = 0.0
    return s["kc"], s["vc"], s["weights"]


def _evict(s):
    c = s["case"]
    B, Hkv, page, keep, most = c["B"], c["Hkv"], c["page"], c["keep"], max(1, max(s["lengths"]))
    p = torch.arange(most, device="cuda")
    at = s["table"].long()[:, p // page].clamp(min=0)
    w = s["weights"][at, :, p % page].transpose(1, 2)  # [B, Hkv, most]
    lens = s["lens"].long()[:, None]
    rank = w.masked_fill((p[None] >= (lens - c["recent"]).clamp(min=0))[:, None], float("inf"))
    rank = rank.masked_fill((p[None] >= lens)[:, None], float("-inf"))
    order = rank.argsort(dim=-1, descending=True, stable=True)
    new_lens = lens.clamp(max=keep)
    order = order.masked_fill((p[None] >= new_lens)[:, None], most)[..., :keep].sort(-1).values  # kept positions in order
    k = order.shape[-1]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    kept[..., :k] = order.masked_fill(order == most, -1).to(torch.int32)
    b, h, j = (order < most).nonzero(as_tuple=True)
    src = order[b, h, j]
    page_from, slot_from = s["table"].long()[b, src // page], src % page
    page_to, slot_to = s["new_table"].long()[b, j // page], j % page
    for t in (s["kc"], s["vc"], s["weights"]):
        t[page_to, h, slot_to] = t[page_from, h, slot_from]
    return new_lens[:, 0].to(torch.int32), kept, s["kc"], s["vc"], s["weights"]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import attention_forward_03_gb300 as fa2
        if op == "append":
            fa2.paged_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], query_starts=s["starts"],
                                   weights=s["weights"])
            return s["kc"], s["vc"], s["weights"]
        if op == "attend":
            return fa2.paged_attention_forward(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                               query_starts=s["starts"], max_query_length=s["longest"],
                                               scale=s["scale"])
        if op == "weigh":
            return fa2.paged_key_weights(s["q"], s["lse"], s["kc"], s["table"], s["lens"], query_starts=s["starts"],
                                         max_query_length=s["longest"], scale=s["scale"], weights=s["weights"],
                                         out=s["out"])
        new_lens, kept = fa2.paged_cache_evict(s["kc"], s["vc"], s["weights"], s["table"], s["lens"], s["new_table"],
                                               s["case"]["keep"], recent=s["case"]["recent"])
        return new_lens, kept, s["kc"], s["vc"], s["weights"]
    return {"append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[op](s)


def work(case):
    c = case
    lengths, row = _lengths(c), c["D"] * 2
    table = 4 * sum(-(-n // c["page"]) for n in lengths) + 4 * c["B"]
    if c["op"] == "evict":
        # every weight is read; what is kept is read and written
        kept = sum(min(n, c["keep"]) for n in lengths) * c["Hkv"]
        return {"bytes": 4 * sum(lengths) * c["Hkv"] + kept * (2 * 2 * row + 4 + 4) + table,
                "flops": sum(lengths) * c["Hkv"]}
    counts = _counts(c)
    T = sum(counts)
    if c["op"] == "append":
        return {"bytes": T * c["Hkv"] * (2 * 2 * row + 4) + table, "flops": 0}
    keys = sum(n for n, q in zip(lengths, counts) if q) * c["Hkv"]
    # token i of q sees n - q + i + 1 positions
    pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(lengths, counts)) * c["Hq"]
    if c["op"] == "attend":
        return {"bytes": 2 * T * c["Hq"] * row + 2 * keys * row + 4 * T * c["Hq"] + table,
                "flops": 4 * pairs * c["D"]}
    return {"bytes": T * c["Hq"] * (row + 4) + keys * row + 8 * sum(lengths) * c["Hkv"] + table,
            "flops": 2 * pairs * c["D"]}


def exact(case, seed):
    s = prepare(case, seed)
    c, page = case, case["page"]
    table, lengths = s["table"].tolist(), s["lengths"]
    if c["op"] == "append":
        k, v, w = s["kc"].double(), s["vc"].double(), s["weights"].double()
        t = 0
        for b, n in enumerate(s["counts"]):
            p = lengths[b] - n
            while p < lengths[b]:  # a page at a time
                m = min(page - p % page, lengths[b] - p)
                at, r = table[b][p // page], slice(p % page, p % page + m)
                k[at, :, r] = s["k"][t:t + m].double().transpose(0, 1)
                v[at, :, r] = s["v"][t:t + m].double().transpose(0, 1)
                w[at, :, r] = 0.0
                p, t = p + m, t + m
        return k, v, w
    if c["op"] == "evict":
        return _exact_evict(s, table, lengths)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(o.shape[:2], float("inf"), dtype=torch.float64, device="cuda")
    out = s["out"].double() if c["op"] == "weigh" else None
    group = c["Hq"] // c["Hkv"]
    t = 0
    for b, (n, q) in enumerate(zip(lengths, s["counts"])):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        flat = lambda x, h: x[ids, h].flatten(0, 1)[:n].double()  # noqa: E731
        late = torch.ones(q, n, dtype=torch.bool, device="cuda").triu(n - q + 1)
        for h in range(c["Hkv"]):
            keys = flat(s["kc"], h)
            w = torch.zeros(n, dtype=torch.float64, device="cuda")
            for j in range(h * group, (h + 1) * group):
                x = torch.einsum("id,jd->ij", s["q"][t:t + q, j].double(), keys) * s["scale"]
                x[late] = float("-inf")
                if out is None:
                    lse[t:t + q, j] = torch.logsumexp(x, -1)
                    o[t:t + q, j] = torch.softmax(x, -1) @ flat(s["vc"], h)
                else:
                    w += torch.exp(x - s["lse"][t:t + q, j].double()[:, None]).sum(0)
            if out is not None:
                w = torch.nn.functional.pad(w, (0, len(ids) * page - n)).reshape(-1, page)
                here = (torch.arange(len(ids) * page, device="cuda") < n).reshape(-1, page)
                out[ids, h] = torch.where(here, s["weights"][ids, h].double() + w, out[ids, h])
        t += q
    return (o, lse) if out is None else out


def _exact_evict(s, table, lengths):
    c = s["case"]
    keep, page = c["keep"], c["page"]
    weights = s["weights"].cpu()
    kept = torch.full((c["B"], c["Hkv"], keep), -1, dtype=torch.int32)
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        of = weights[table[b][:-(-n // page)]].transpose(0, 1).flatten(1)[:, :n].double().numpy()
        for h in range(c["Hkv"]):
            old = max(n - c["recent"], 0) if n > keep else 0
            # by weight, then by position
            best = sorted(range(old), key=lambda p: (-of[h, p], p))[:keep - c["recent"]] if n > keep else []
            chosen = sorted(best) + list(range(old, n))
            kept[b, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    caches = [s[t].double() for t in ("kc", "vc", "weights")]
    for b, n in enumerate(lengths):
        m = min(n, keep)
        for h in range(c["Hkv"]):
            p = kept[b, h, :m].long().cuda()
            i = torch.arange(m, device="cuda")
            for old, new in zip(("kc", "vc", "weights"), caches):
                new[s["new_table"][b, i // page].long(), h, i % page] = s[old][s["table"][b, p // page].long(), h, p % page].double()
    return torch.tensor([min(n, keep) for n in lengths], dtype=torch.int32), kept, *caches
