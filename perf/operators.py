"""Cases and plain forms of the query/key norm with position rotation and of cross attention.

Four paths, each a call that a program makes beside `attention_forward`:

  rope        q' = R(pos) (g_q * q / rms(q)), k' likewise, for every head in one pass
              (rotated pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved)
  rope_grad   the gradients of q, k and of both gains for upstream gradients of q', k'
  cross       O = softmax(scale Q K^T) V over another sequence's keys, its first `lengths[b]`
              keys where lengths are given, Hq / Hkv query heads to each key head; and the
              rows' log-sum-exp (a row without keys: O = 0, LSE = +inf)
  cross_grad  dQ, dK, dV from O, LSE and an upstream gradient of O

The plain forms use elementary torch operations in 32 bits and round once at the end.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of each of 8 sequences, at far and different positions: what a decoding step calls per layer
        {"name": "rope_step", "op": "rope", "B": 8, "N": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "dtype": "bf16",
         "interleaved": False, "gain": "f32", "table": 8192, "gather": True},
        # a whole prompt of the length the benchmark uses, grouped heads out of one packed projection
        {"name": "rope_prompt", "op": "rope", "B": 1, "N": 8192, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "gain": "bf16", "table": 8192, "gather": False},
        # the ragged length of the tests; half of each head rotated, in neighbouring pairs
        {"name": "rope_partial", "op": "rope", "B": 2, "N": 1000, "Hq": 12, "Hkv": 12, "D": 64, "rot": 32,
         "dtype": "f16", "interleaved": True, "gain": "f32", "table": 1024, "gather": False},
        # the training step of the benchmark's B = 4, N = 4096 batch
        {"name": "rope_grad", "op": "rope_grad", "B": 4, "N": 4096, "Hq": 16, "Hkv": 4, "D": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "gain": "f32", "table": 4096, "gather": False},
        # a small ragged training batch, packed documents (positions start again inside a row)
        {"name": "rope_grad_ragged", "op": "rope_grad", "B": 2, "N": 1000, "Hq": 12, "Hkv": 12, "D": 64, "rot": 64,
         "dtype": "f16", "interleaved": False, "gain": "f32", "table": 1024, "gather": True},
        # one decoder token against a 1500-frame encoder: latency
        {"name": "cross_step", "op": "cross", "B": 4, "Hq": 12, "Hkv": 12, "Nq": 1, "Nk": 1500, "D": 64,
         "dtype": "f16", "lengths": "full", "empty": False, "pad_nan": False},
        # a serving batch of single tokens over long, differently padded sources: the cache's bytes
        {"name": "cross_step_batch", "op": "cross", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "Nk": 4096, "D": 128,
         "dtype": "bf16", "lengths": "ragged", "empty": True, "pad_nan": True},
        # a few latent rows that read a long input
        {"name": "cross_latents", "op": "cross", "B": 2, "Hq": 16, "Hkv": 16, "Nq": 256, "Nk": 16384, "D": 64,
         "dtype": "bf16", "lengths": "full", "empty": False, "pad_nan": False},
        # many image rows against a short caption
        {"name": "cross_short", "op": "cross", "B": 2, "Hq": 16, "Hkv": 16, "Nq": 4096, "Nk": 77, "D": 64,
         "dtype": "f16", "lengths": "full", "empty": False, "pad_nan": False},
        # long targets over long padded sources, grouped heads: the tensor cores' rate
        {"name": "cross_long", "op": "cross", "B": 4, "Hq": 16, "Hkv": 4, "Nq": 2048, "Nk": 8192, "D": 128,
         "dtype": "bf16", "lengths": "ragged", "empty": False, "pad_nan": True},
        # a training batch of padded sources, one of them empty
        {"name": "cross_grad", "op": "cross_grad", "B": 4, "Hq": 16, "Hkv": 16, "Nq": 1000, "Nk": 1500, "D": 64,
         "dtype": "f16", "lengths": "ragged", "empty": True, "pad_nan": True},
        # long rows both ways at the benchmark's head count
        {"name": "cross_grad_long", "op": "cross_grad", "B": 1, "Hq": 8, "Hkv": 8, "Nq": 4096, "Nk": 8192, "D": 128,
         "dtype": "bf16", "lengths": "full", "empty": False, "pad_nan": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        most[c["op"]] = {t: max(m[t], w[t]) for t in m}
    op = rng.choice(["rope", "rope_grad", "cross", "cross", "cross", "cross_grad", "cross_grad"])
    while True:
        hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
        group = rng.choice([1, 1, 2, 3, 4, 7, 8])
        d = rng.choice([32, 64, 64, 96, 128, 128])
        c = {"op": op, "B": _log_int(rng, 1, 64), "Hq": hkv * group, "Hkv": hkv, "D": d,
             "dtype": rng.choice(["f16", "bf16"])}
        if op in ("rope", "rope_grad"):
            c["N"] = _log_int(rng, 1, 8192)
            c["D"] = rng.choice([32, 64, 96, 128, 128, 256])
            c["rot"] = rng.choice([c["D"], c["D"], c["D"] // 2, 16, 0])
            c["interleaved"] = rng.random() < 0.3
            c["gain"] = rng.choice(["f32", c["dtype"], "none"] if op == "rope" else ["f32", c["dtype"]])
            c["gather"] = rng.random() < 0.5
            c["table"] = max(c["N"], _log_int(rng, 64, 16384))
        else:
            c["Nq"] = 1 if op == "cross" and rng.random() < 0.35 else _log_int(rng, 1, 4096)
            c["Nk"] = _log_int(rng, 1, 16384)
            c["lengths"] = rng.choice(["full", "ragged"])
            c["empty"] = c["lengths"] == "ragged" and rng.random() < 0.5
            c["pad_nan"] = c["lengths"] == "ragged" and rng.random() < 0.5
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"] and _scores(c) <= 1.1e9:
            return c


def _scores(c):
    """Score entries that the plain form of cross attention holds."""
    return c["B"] * c["Hq"] * c["Nq"] * c["Nk"] if c["op"].startswith("cross") else 0


def _lengths(c):
    """The batch's key counts, in a fixed order: evenly spread over (0, Nk], the first one 0 where `empty`."""
    if c["lengths"] == "full":
        return None
    n = [max(1, c["Nk"] * (b + 1) // c["B"]) for b in range(c["B"])]
    if c["empty"]:
        n[0] = 0
    return n


def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("rope", "rope_grad"):
        B, N, Hq, Hkv, D, rot = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["rot"]
        # one projection's output, [B, N, heads of q, k, v, D]; q and k are views of it
        packed = _randn(g, B, N, Hq + 2 * Hkv, D, dtype=dt, scale=2.0)
        s["q"] = packed[:, :, :Hq].transpose(1, 2)
        s["k"] = packed[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["qw"] = s["kw"] = None
        if c["gain"] != "none":
            wt = torch.float32 if c["gain"] == "f32" else dt
            s["qw"] = (1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wt)
            s["kw"] = (1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wt)
        s["cos"] = s["sin"] = s["pos"] = None
        if rot:
            at = torch.arange(c["table"], device="cuda", dtype=torch.float64)
            f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
            a = at[:, None] * f[None, :]
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
            if c["gather"]:
                # each row starts at a position of its own and goes on from there
                first = torch.randint(0, c["table"] - N + 1, (B, 1), generator=g, device="cuda")
                s["pos"] = first + torch.arange(N, device="cuda")[None, :]
        s["eps"] = 1e-6
        if c["op"] == "rope_grad":
            s["dq_out"] = _randn(g, B, Hq, N, D, dtype=dt)
            s["dk_out"] = _randn(g, B, Hkv, N, D, dtype=dt)
            # the packed projection's gradient: q's and k's parts are written in place
            d_packed = torch.zeros(B, N, Hq + 2 * Hkv, D, dtype=dt, device="cuda")
            s["dq"] = d_packed[:, :, :Hq].transpose(1, 2)
            s["dk"] = d_packed[:, :, Hq:Hq + Hkv].transpose(1, 2)
        return s
    B, Hq, Hkv, Nq, Nk, D = c["B"], c["Hq"], c["Hkv"], c["Nq"], c["Nk"], c["D"]
    s["q"] = _randn(g, B, Hq, Nq, D, dtype=dt, scale=1.5)
    s["k"] = _randn(g, B, Hkv, Nk, D, dtype=dt)
    s["v"] = _randn(g, B, Hkv, Nk, D, dtype=dt)
    s["scale"] = 1.0 / math.sqrt(D)
    s["lens"] = None
    n = _lengths(c)
    if n is not None:
        order = torch.randperm(B, generator=g, device="cuda")
        s["lens"] = torch.tensor(n, device="cuda", dtype=torch.int32)[order].contiguous()
        if c["pad_nan"]:  # what a cache holds behind a short source is anything
            behind = torch.arange(Nk, device="cuda")[None, :] >= s["lens"][:, None]
            s["k"].masked_fill_(behind[:, None, :, None], float("nan"))
            s["v"].masked_fill_(behind[:, None, :, None], float("nan"))
    if c["op"] == "cross_grad":
        s["do"] = _randn(g, B, Hq, Nq, D, dtype=dt)
        s["o"], s["lse"] = _cross(s)
    return s


def _norm_rotate(x, w, cos, sin, eps, interleaved):
    """x [B, H, N, D] in 32 bits -> (normed and rotated, normed without gain, 1 / rms)."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    xn = x * r
    y = xn if w is None else xn * w
    return _rotate(y, cos, sin, interleaved), xn, r


def _rotate(y, cos, sin, interleaved):
    if cos is None:
        return y
    half = cos.shape[-1]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1)


def _tables(s):
    """cos and sin of every token, [B or 1, 1, N, rot/2]."""
    if s["cos"] is None:
        return None, None
    n = s["q"].shape[2]
    if s["pos"] is None:
        return s["cos"][None, None, :n], s["sin"][None, None, :n]
    return s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]


def _rope(s):
    cos, sin = _tables(s)
    i = s["case"]["interleaved"]
    w = [None if t is None else t.float() for t in (s["qw"], s["kw"])]
    q = _norm_rotate(s["q"].float(), w[0], cos, sin, s["eps"], i)[0]
    k = _norm_rotate(s["k"].float(), w[1], cos, sin, s["eps"], i)[0]
    return q.to(s["q"].dtype), k.to(s["k"].dtype)


def _rope_grad_one(x, w, g, cos, sin, eps, interleaved):
    _, xn, r = _norm_rotate(x.float(), None, None, None, eps, interleaved)
    back = _rotate(g.float(), cos, None if sin is None else -sin, interleaved)  # the rotation's transpose
    dw = (back * xn).sum((0, 1, 2))
    h = back if w is None else back * w.float()
    dx = r * (h - xn * (h * xn).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw.to(w.dtype)


def _rope_grad(s):
    cos, sin = _tables(s)
    i = s["case"]["interleaved"]
    dq, dqw = _rope_grad_one(s["q"], s["qw"], s["dq_out"], cos, sin, s["eps"], i)
    dk, dkw = _rope_grad_one(s["k"], s["kw"], s["dk_out"], cos, sin, s["eps"], i)
    return dq, dk, dqw, dkw


def _grouped(s):
    """q [B, Hkv, group * Nq, D], k, v [B, Hkv, Nk, D] in 32 bits and the keys' mask (or None)."""
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    q, k, v = q.reshape(B, Hkv, Hq // Hkv * Nq, D).float(), k.float(), v.float()
    if s["lens"] is None:
        return q, k, v, None
    behind = (torch.arange(Nk, device=q.device)[None, :] >= s["lens"][:, None])[:, None, :, None]
    return q, k.masked_fill(behind, 0.0), v.masked_fill(behind, 0.0), behind.transpose(2, 3)


def _cross(s):
    q, k, v, behind = _grouped(s)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    if behind is not None:
        x = x.masked_fill(behind, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)  # a row without keys stays at exp(-inf) = 0
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.where(z > 0, m + torch.log(z), torch.full_like(z, float("inf")))
    return o.to(s["q"].dtype).reshape(s["q"].shape), lse.reshape(s["q"].shape[:3])


def _cross_grad(s):
    q, k, v, behind = _grouped(s)
    do, o = (s[t].float().reshape(q.shape) for t in ("do", "o"))
    lse = s["lse"].reshape(q.shape[:3])[..., None]
    x = (q @ k.transpose(2, 3)) * s["scale"]
    if behind is not None:
        x = x.masked_fill(behind, float("-inf"))
    p = torch.exp(x - lse)
    ds = p * (do @ v.transpose(2, 3) - (do * o).sum(-1, keepdim=True))
    dq = (ds @ k) * s["scale"]
    dk = (ds.transpose(2, 3) @ q) * s["scale"]
    dv = p.transpose(2, 3) @ do
    dt = s["q"].dtype
    return dq.to(dt).reshape(s["q"].shape), dk.to(dt), dv.to(dt)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import attention_forward_03_gb300 as fa2
        if op == "rope":
            return fa2.qk_norm_rope_forward(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], positions=s["pos"],
                                            eps=s["eps"], interleaved=s["case"]["interleaved"])
        if op == "rope_grad":
            return fa2.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["qw"], s["kw"], s["cos"],
                                             s["sin"], positions=s["pos"], eps=s["eps"],
                                             interleaved=s["case"]["interleaved"], dq=s["dq"], dk=s["dk"])
        if op == "cross":
            return fa2.cross_attention_forward(s["q"], s["k"], s["v"], scale=s["scale"], key_lengths=s["lens"])
        return fa2.cross_attention_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], scale=s["scale"],
                                            key_lengths=s["lens"])
    return {"rope": _rope, "rope_grad": _rope_grad, "cross": _cross, "cross_grad": _cross_grad}[op](s)


def work(case):
    c = case
    if c["op"] in ("rope", "rope_grad"):
        rows = c["B"] * c["N"] * (c["Hq"] + c["Hkv"])
        tensors = 2 if c["op"] == "rope" else 3
        angles = min(c["table"], c["B"] * c["N"] if c["gather"] else c["N"]) * c["rot"] * 4
        where = c["B"] * c["N"] * 8 if c["gather"] and c["rot"] else 0
        gains = 0 if c["gain"] == "none" else 2 * c["D"] * (4 if c["gain"] == "f32" else 2)
        return {"bytes": rows * c["D"] * 2 * tensors + angles + where + gains * (tensors - 1),
                "flops": rows * c["D"] * (7 if c["op"] == "rope" else 14)}
    n = _lengths(c) or [c["Nk"]] * c["B"]
    keys = sum(n)
    q_bytes = c["B"] * c["Hq"] * c["Nq"] * c["D"] * 2
    kv_bytes = keys * c["Hkv"] * c["D"] * 2
    lse = c["B"] * c["Hq"] * c["Nq"] * 4
    lens = 0 if c["lengths"] == "full" else 4 * c["B"]
    pairs = keys * c["Hq"] * c["Nq"]
    if c["op"] == "cross":
        return {"bytes": 2 * q_bytes + 2 * kv_bytes + lse + lens, "flops": 4 * pairs * c["D"]}
    # dK, dV are written whole, with zeros behind the lengths
    return {"bytes": 4 * q_bytes + 2 * kv_bytes + 2 * c["B"] * c["Hkv"] * c["Nk"] * c["D"] * 2 + lse + lens,
            "flops": 10 * pairs * c["D"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "rope_grad"):
        return _exact_rope(s)
    q, k, v = (s[t].double() for t in "qkv")
    B, Hq, Nq, D = q.shape
    group = Hq // k.shape[1]
    grad = case["op"] == "cross_grad"
    o, lse = torch.zeros_like(q), torch.full(q.shape[:3], float("inf"), dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    counts = [k.shape[2]] * B if s["lens"] is None else s["lens"].tolist()
    for b in range(B):
        n = counts[b]
        if n == 0:
            continue
        for h in range(Hq):
            kk, vv = k[b, h // group, :n], v[b, h // group, :n]
            x = torch.einsum("id,jd->ij", q[b, h], kk) * s["scale"]
            lse[b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b, h][:, None])
            o[b, h] = torch.einsum("ij,jd->id", p, vv)
            if grad:
                do = s["do"][b, h].double()
                dp = torch.einsum("id,jd->ij", do, vv)
                ds = p * (dp - (dp * p).sum(-1, keepdim=True)) * s["scale"]
                dq[b, h] = torch.einsum("ij,jd->id", ds, kk)
                dk[b, h // group, :n] += torch.einsum("ij,id->jd", ds, q[b, h])
                dv[b, h // group, :n] += torch.einsum("ij,id->jd", p, do)
    return (dq, dk, dv) if grad else (o, lse)


def _exact_rope(s):
    c = s["case"]
    n, rot = c["N"], c["rot"]
    outs, gains = [], []
    for x, w, g in ((s["q"], s["qw"], s.get("dq_out")), (s["k"], s["kw"], s.get("dk_out"))):
        x = x.double()
        ms = x.square().sum(-1) / c["D"] + s["eps"]
        # the rotation as complex products of the pairs
        turn = None
        if rot:
            rows = torch.arange(n, device=x.device).expand(c["B"], n) if s["pos"] is None else s["pos"]
            turn = torch.complex(s["cos"].double()[rows], s["sin"].double()[rows])[:, None]

        def turned(y, by):
            if by is None:
                return y
            head = y[..., :rot]
            pairs = head.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat((z, y[..., rot:]), -1)

        gain = 1.0 if w is None else w.double()
        if g is None:
            outs.append(turned(x * gain / ms.sqrt()[..., None], turn))
            continue
        u = turned(g.double(), None if turn is None else turn.conj())
        dot = (u * gain * x).sum(-1) / c["D"]
        outs.append(u * gain / ms.sqrt()[..., None] - x * (dot / ms.pow(1.5))[..., None])
        gains.append((u * x / ms.sqrt()[..., None]).sum((0, 1, 2)))
    return tuple(outs + gains)
