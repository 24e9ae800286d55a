"""Cases for the masked attention, cache and paged attention operators, with their plain forms.

Three families, each the call a user makes (``own``) beside the same operator in elementary torch operations:

* ``span_fwd`` / ``span_bwd``: sigmoid attention of a padded batch whose query rows each see one interval of keys (causal,
  prefix, documents, windows), with a tanh cap on the scores, a bias that falls with distance and heads that share keys;
* ``append``: new keys and values written into a paged cache, rotated to their positions on the way, with the queries;
* ``paged``: the queries of a decoding batch against a paged cache, whose samples may share one long prefix.

Lengths, masks and page layouts of a case are plain functions of the case; the numbers in the tensors come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
_SCORES_MOST = 2 ** 31      # Z H L^2 of a drawn training case


# ------------------------------------------------------------------------------------------------ cases

def _span(name, direction, dtype, Z, L, H, Hk, D, mask, cap, slopes, ragged):
    return {"name": name, "op": "span_" + direction, "dtype": dtype, "Z": Z, "L": L, "H": H, "Hk": Hk, "D": D, "mask": mask,
            "cap": cap, "slopes": slopes, "ragged": ragged, "layout": 1}


def _append(name, dtype, Z, L, H, Hk, D, rot, interleaved, page, cached, prefix, ragged):
    return {"name": name, "op": "append", "dtype": dtype, "Z": Z, "L": L, "H": H, "Hk": Hk, "D": D, "rot": rot,
            "interleaved": interleaved, "page": page, "cached": cached, "prefix": prefix, "ragged": ragged, "layout": 1}


def _paged(name, dtype, Z, L, H, Hk, D, page, prefix, suffix, cap, slopes):
    return {"name": name, "op": "paged", "dtype": dtype, "Z": Z, "L": L, "H": H, "Hk": Hk, "D": D, "page": page, "prefix": prefix,
            "suffix": suffix, "cap": cap, "slopes": slopes, "layout": 1}


def listed():
    return [
        # a layer over rows packed with several short cells each, no cell seeing another (the 2K single-cell layer)
        _span("fwd packed cells D64", "fwd", "bf16", 4, 2048, 12, 12, 64, "docs", 0.0, False, False),
        # prompts read in both directions and continuations read causally, capped scores, distance bias, four heads to a key head
        _span("fwd prefix cap grouped", "fwd", "bf16", 2, 4001, 16, 4, 128, "prefix", 30.0, True, True),
        # the 16K layer in its causal form, the largest forward
        _span("fwd causal 16K", "fwd", "bf16", 1, 16384, 16, 16, 128, "causal", 0.0, False, False),
        # a training step's backward over long causal rows, the largest case
        _span("bwd causal 8K", "bwd", "bf16", 2, 8192, 16, 16, 128, "causal", 0.0, False, False),
        # the backward of packed causal documents of uneven padded rows, capped, with distance bias and shared key heads
        _span("bwd packed cap grouped D64", "bwd", "bf16", 8, 2048, 12, 4, 64, "docs_causal", 30.0, True, True),
        # the accuracy path at the tiny parity shape: latency
        _span("bwd tiny fp32", "bwd", "fp32", 2, 128, 2, 2, 64, "prefix", 0.0, True, True),
        # one decoding step of a batch: one token a sample, latency
        _append("append decode", "bf16", 64, 1, 16, 4, 128, 128, False, 64, 400, 16384, False),
        # prompts going into the cache
        _append("append prompts", "bf16", 4, 4096, 16, 4, 128, 128, False, 64, 0, 0, True),
        # partly rotated heads with adjacent pairs, odd lengths, small pages, 32 bits
        _append("append partial fp32", "fp32", 7, 333, 12, 12, 64, 32, True, 16, 1000, 100, True),
        # few samples behind a short prompt: latency
        _paged("paged few short", "bf16", 4, 1, 16, 4, 128, 16, 1000, 100, 0.0, False),
        # a decoding batch that shares a 16K prefix
        _paged("paged shared 16K", "bf16", 64, 1, 16, 4, 128, 64, 16384, 500, 0.0, False),
        # several drafted tokens a sample, own long contexts, no sharing, capped with distance bias
        _paged("paged drafts D64", "bf16", 32, 4, 12, 12, 64, 32, 0, 4000, 30.0, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice([64, 128])
    H, Hk = rng.choice([(16, 16), (16, 8), (16, 4), (16, 2), (12, 12), (12, 4), (12, 2), (2, 2), (2, 1)])
    op = rng.choice(["span_fwd", "span_bwd", "span_bwd", "append", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    lay = rng.randrange(1, 1 << 20)
    if op.startswith("span"):
        L = _log(rng, 1, 200 if dtype == "fp32" else 8192)
        most = max(1, _SCORES_MOST // (H * L * L))
        Z = rng.randint(1, min(4 if dtype == "fp32" else 8, most))
        c = _span("", op[5:], dtype, Z, L, H, Hk, D, rng.choice(["full", "causal", "prefix", "docs", "docs_causal", "window"]),
                  rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]), rng.random() < 0.4, rng.random() < 0.6)
    elif op == "append":
        L = rng.choice([1, rng.randint(1, 8), _log(rng, 1, 4096)])
        Z = _log(rng, 1, max(1, min(128, 16384 // L)))
        rot = rng.choice([D, D, D // 2, D // 4])
        c = _append("", dtype, Z, L, H, Hk, D, rot, rng.random() < 0.5, rng.choice([16, 32, 64, 128]), _log(rng, 1, 8192) - 1,
                    rng.choice([0, _log(rng, 1, 65536)]), rng.random() < 0.5)
    else:
        L = rng.choice([1, 1, 1, 2, 4, 8])
        if dtype == "fp32":
            Z, prefix, suffix = _log(rng, 1, 8), rng.choice([0, _log(rng, 1, 1000)]), _log(rng, 8, 300)
        else:
            Z, prefix, suffix = _log(rng, 1, 64), rng.choice([0, _log(rng, 1, 16384)]), _log(rng, 8, 4000)
        c = _paged("", dtype, Z, L, H, Hk, D, rng.choice([16, 32, 64, 128]), prefix, suffix, rng.choice([0.0, 0.0, 30.0]),
                   rng.random() < 0.4)
    c["layout"] = lay
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ layouts: functions of the case

def _lengths(case):
    """Tokens of each sample of a padded batch; the first sample fills it."""
    rng = random.Random(case["layout"] * 7919 + 1)
    Z, L = case["Z"], case["L"]
    n = [rng.randint((L + 2) // 3, L) if case["ragged"] else L for _ in range(Z)]
    return np.asarray([L] + n[1:], np.int32)


def _spans(case, n):
    """[lo, hi) of the keys that each row sees, int32 [Z, L, 2]; rows of padding see none."""
    rng = np.random.default_rng(case["layout"] * 7919 + 2)
    Z, L, mask = case["Z"], case["L"], case["mask"]
    i = np.arange(L)
    out = np.zeros((Z, L, 2), np.int32)
    for z in range(Z):
        m = int(n[z])
        lo, hi = np.zeros(L, np.int64), np.full(L, m)
        if mask.startswith("docs"):
            mean = max(1, min(L // 4, 300))
            cuts = np.flatnonzero(rng.random(L) < 1.0 / mean)
            at = np.searchsorted(cuts, i, side="right")
            edges = np.concatenate([[0], cuts, [m]])
            lo, hi = edges[at], np.minimum(np.concatenate([cuts, [m]])[at], m)
        if mask in ("causal", "prefix", "docs_causal", "window"):
            hi = np.minimum(hi, i + 1)
        if mask == "prefix":
            hi = np.minimum(np.maximum(hi, int(rng.integers(1, m + 1))), m)
        if mask == "window":
            lo = np.maximum(lo, i + 1 - max(1, L // 6))
        lo, hi = np.where(i < m, lo, 0), np.where(i < m, hi, 0)
        out[z, :, 0], out[z, :, 1] = lo, hi
    return out


def _cached(case):
    """Tokens that each sample has in the cache before the call, and new tokens of each sample."""
    rng = random.Random(case["layout"] * 7919 + 3)
    if case["op"] == "append":
        have = [rng.randint(case["cached"] // 2, case["cached"]) for _ in range(case["Z"])]
        return np.asarray(have, np.int32), _lengths(case)
    L = case["L"]
    new = [rng.randint(1, L) for _ in range(case["Z"])]
    have = [rng.randint(max(1, case["suffix"] // 4), case["suffix"]) for _ in range(case["Z"])]
    return np.asarray([max(0, h - m) for h, m in zip(have, new)], np.int32), np.asarray(new, np.int32)


def _pages(case, total):
    """Pages of the prefix [P0] and of each sample [Z, most] (-1 behind the last), and how many there are: a shuffled pool."""
    rng = np.random.default_rng(case["layout"] * 7919 + 4)
    page = case["page"]
    ahead = -(-case["prefix"] // page) if case["op"] == "paged" else 0
    need = [-(-int(t) // page) for t in total]
    pool = rng.permutation(ahead + sum(need) + 3).astype(np.int32)
    table = np.full((len(need), max(1, max(need))), -1, np.int32)
    at = ahead
    for z, m in enumerate(need):
        table[z, :m] = pool[at:at + m]
        at += m
    return pool[:ahead], table, len(pool)


def _slopes(case, device):
    return torch.as_tensor([2.0 ** (-8.0 * (h + 1) / case["H"]) for h in range(case["H"])], dtype=torch.float32, device=device)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    t = _TYPES[case["dtype"]]
    Z, L, H, Hk, D = (case[k] for k in ("Z", "L", "H", "Hk", "D"))

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(t)

    def ints(a):
        return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)

    st = {"case": case, "alpha": 1.0 / math.sqrt(D), "q": normal(Z, L, H, D, scale=2.0 if case.get("cap") else 1.0)}
    if case["op"].startswith("span"):
        n = _lengths(case)
        st |= {"k": normal(Z, L, Hk, D, scale=2.0 if case["cap"] else 1.0), "v": normal(Z, L, Hk, D), "seqlens": ints(n),
               "spans": ints(_spans(case, n)), "bias": -math.log(L), "slopes": _slopes(case, dev) if case["slopes"] else None}
        if case["op"] == "span_bwd":
            st["dout"] = normal(Z, L, H, D)
        return st
    have, new = _cached(case)
    ahead, table, count = _pages(case, have + new)
    st |= {"k_pages": normal(count, case["page"], Hk, D), "v_pages": normal(count, case["page"], Hk, D), "page_table": ints(table),
           "seqlens_new": ints(new), "prefix_len": ints([case["prefix"]]) if case["prefix"] else None}
    if case["op"] == "append":
        half = case["rot"] // 2
        st |= {"k": normal(Z, L, Hk, D), "v": normal(Z, L, Hk, D), "cache_lens": ints(have),
               "inv_freq": torch.as_tensor(10000.0 ** (-np.arange(half) / half), dtype=torch.float32, device=dev)}
    else:
        st |= {"seqlens_k": ints(have + new), "prefix_table": ints(ahead) if case["prefix"] else None,
               "bias": -math.log(case["prefix"] + case["suffix"]), "slopes": _slopes(case, dev) if case["slopes"] else None}
    return st


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    return {"span_fwd": _span_fwd, "span_bwd": _span_bwd, "append": _append_run, "paged": _paged_run}[op](st)


def _span_fwd(st):
    if own:
        import padding_aware_sigmoid_b200 as sa
        return sa.fwd_span(st["q"], st["k"], st["v"], st["seqlens"], st["alpha"], st["bias"], spans=st["spans"],
                           cap=st["case"]["cap"], slopes=st["slopes"])
    q, k, v = (_heads(st[x], st["case"]) for x in "qkv")
    p, _ = _weights(st, q, k, False)
    return _rows(p @ v, st["case"]).to(st["q"].dtype)


def _span_bwd(st):
    if own:
        import padding_aware_sigmoid_b200 as sa
        return sa.bwd_span(st["q"], st["k"], st["v"], st["dout"], st["seqlens"], st["alpha"], st["bias"], spans=st["spans"],
                           cap=st["case"]["cap"], slopes=st["slopes"])
    q, k, v, do = (_heads(st[x], st["case"]) for x in ("q", "k", "v", "dout"))
    p, dx = _weights(st, q, k, True)
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    del p
    ds = dx.mul_(do @ v.transpose(-1, -2)).mul_(st["alpha"])
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    return tuple(_rows(x, st["case"]).to(st["q"].dtype) for x in (dq, dk, dv))


def _heads(x, case):
    """[Z, L, heads, D] as fp32 [Z, Hk, heads / Hk, L, D]."""
    Z, L, h, D = x.shape
    return x.float().reshape(Z, L, case["Hk"], h // case["Hk"], D).permute(0, 2, 3, 1, 4)


def _rows(x, case):
    Z, Hk, g, L, D = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(Z, L, Hk * g, D)


def _weights(st, q, k, slope):
    """sigma(x) where a row sees a key and 0 elsewhere, and with `slope` its derivative with respect to the product's scaled score."""
    case, n = st["case"], st["seqlens"]
    L, cap = case["L"], case["cap"]
    s = (q @ k.transpose(-1, -2)).mul_(st["alpha"])
    t = None
    if cap:
        t = s.div_(cap).tanh_()
        s = t * cap
    i = torch.arange(L, device=n.device)
    if st["slopes"] is not None:
        far = (i[:, None] - i[None, :]).abs().float()
        s = s - st["slopes"].view(1, case["Hk"], -1, 1, 1) * far
    p = torch.sigmoid(s + st["bias"])
    lo, hi = st["spans"][..., 0, None], st["spans"][..., 1, None]
    sees = (i >= lo) & (i < hi) & (i < n[:, None, None]) & (i[:, None] < n[:, None, None])
    p = p * sees[:, None, None]
    if not slope:
        return p, None
    dx = p * (1 - p)
    return p, dx if t is None else dx.mul_(1 - t * t)


def _turn(x, cos, sin, case):
    """The first `rot` entries of x's rows rotated, pair by pair."""
    rot = case["rot"]
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _append_run(st):
    case = st["case"]
    if own:
        import padding_aware_sigmoid_b200 as sa
        q, lens = sa.cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_table"], st["cache_lens"], st["seqlens_new"],
                                  inv_freq=st["inv_freq"], interleaved=case["interleaved"], q=st["q"], prefix_len=st["prefix_len"])
        return {"q": q, "lens": lens, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    L, page, new = case["L"], case["page"], st["seqlens_new"].long()[:, None]
    i = torch.arange(L, device=new.device)
    # rows of padding write the last token once more: the same values into the same place
    row = torch.minimum(i[None, :], new - 1)
    at = st["cache_lens"].long()[:, None] + row
    where = st["page_table"].long().gather(1, at // page) * page + at % page
    pos = at if st["prefix_len"] is None else at + st["prefix_len"]
    angle = pos.double()[..., None] * st["inv_freq"].double()
    cos, sin = (f(angle).float()[:, :, None] for f in (torch.cos, torch.sin))
    z = torch.arange(case["Z"], device=new.device)[:, None]
    flat = where.reshape(-1)
    for_k = _turn(st["k"][z, row].float(), cos, sin, case).to(st["k"].dtype)
    st["k_pages"].view(-1, case["Hk"], case["D"]).index_copy_(0, flat, for_k.reshape(-1, case["Hk"], case["D"]))
    st["v_pages"].view(-1, case["Hk"], case["D"]).index_copy_(0, flat, st["v"][z, row].reshape(-1, case["Hk"], case["D"]))
    live = (i[None, :] < new)[..., None, None]
    q = (_turn(st["q"].float(), cos, sin, case) * live).to(st["q"].dtype)
    return {"q": q, "lens": st["cache_lens"] + st["seqlens_new"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _paged_run(st):
    case = st["case"]
    if own:
        import padding_aware_sigmoid_b200 as sa
        return sa.fwd_paged(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["seqlens_k"], st["seqlens_new"], st["alpha"],
                            st["bias"], prefix_table=st["prefix_table"], prefix_len=st["prefix_len"], cap=case["cap"],
                            slopes=st["slopes"])
    Z, L, Hk, D = (case[x] for x in ("Z", "L", "Hk", "D"))
    G = case["H"] // Hk
    n, new = st["seqlens_k"].long(), st["seqlens_new"].long()
    i = torch.arange(L, device=n.device)
    at = (n - new)[:, None] + i                                   # place of each query among its sample's own keys
    live = i < new[:, None]
    q = st["q"].float().reshape(Z, L, Hk, G, D).permute(0, 2, 1, 3, 4)      # [Z, Hk, L, G, D]
    table = st["page_table"].long().clamp(min=0)
    k, v = (st[x][table].float().flatten(1, 2).transpose(1, 2) for x in ("k_pages", "v_pages"))      # [Z, Hk, keys, D]
    j = torch.arange(k.shape[2], device=n.device)
    sees = (j <= at[..., None]) & (j < n[:, None, None])          # [Z, L, keys]
    s = q.flatten(2, 3) @ k.transpose(-1, -2)                     # [Z, Hk, L G, keys]
    p = _paged_weights(st, s.view(Z, Hk, L, G, -1), at[..., None] - j)
    p = p * sees[:, None, :, None]
    o = p.flatten(2, 3) @ v
    if case["prefix"]:
        pre = st["prefix_table"].long()
        kp, vp = (st[x][pre].float().flatten(0, 1)[:case["prefix"]].transpose(0, 1) for x in ("k_pages", "v_pages"))  # [Hk, P, D]
        flat = q.transpose(0, 1).reshape(Hk, Z * L * G, D)
        s = (flat @ kp.transpose(-1, -2)).view(Hk, Z, L, G, -1).transpose(0, 1)
        back = at[..., None] + case["prefix"] - torch.arange(case["prefix"], device=n.device)
        p = _paged_weights(st, s, back)
        op = p.transpose(0, 1).reshape(Hk, Z * L * G, -1) @ vp
        o = o + op.view(Hk, Z, L * G, D).transpose(0, 1)
    o = o.view(Z, Hk, L, G, D).permute(0, 2, 1, 3, 4).reshape(Z, L, Hk * G, D)
    return (o * live[..., None, None]).to(st["q"].dtype)


def _paged_weights(st, s, far):
    """sigma of scores [Z, Hk, L, G, keys]; `far` [Z, L, keys]: how far each key lies behind its query."""
    case = st["case"]
    s = s * st["alpha"]
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, case["Hk"], 1, -1, 1) * far[:, None, :, None].abs().float()
    return torch.sigmoid(s + st["bias"])


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e, Z, L, H, Hk, D = _SIZE[case["dtype"]], *(case[k] for k in ("Z", "L", "H", "Hk", "D"))
    if case["op"].startswith("span"):
        n = _lengths(case)
        sp = _spans(case, n).astype(np.int64)
        pairs = H * int(np.maximum(sp[..., 1] - sp[..., 0], 0).sum())
        qs, ks = Z * L * H * D * e, Z * L * Hk * D * e
        if case["op"] == "span_fwd":
            return {"bytes": 2 * qs + 2 * ks + 8 * Z * L, "flops": 4 * D * pairs}
        return {"bytes": 3 * qs + 4 * ks + 8 * Z * L, "flops": 10 * D * pairs}
    have, new = (a.astype(np.int64) for a in _cached(case))
    tokens = int(new.sum())
    if case["op"] == "append":
        # keys, values and queries read; the cache's rows and the whole rotated queries written
        return {"bytes": e * D * (4 * tokens * Hk + tokens * H + Z * L * H) + 16 * Z, "flops": 6 * tokens * (H + Hk) * case["rot"] // 2}
    seen = int(sum(sum(int(h) + l + 1 for l in range(int(m))) for h, m in zip(have, new))) + tokens * case["prefix"]
    keys = int((have + new).sum()) + case["prefix"]
    return {"bytes": e * D * (2 * keys * Hk + tokens * H + Z * L * H), "flops": 4 * D * H * seen}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits

def _logistic(x):
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1.0, e) / (1.0 + e)


def _exact_scores(q, k, st, head, rows, cols):
    """Bias-free to biased argument of sigma, and the cap's own derivative, for one head: rows and cols are positions."""
    y = st["alpha"] * (q @ k.mT)
    d = torch.ones_like(y)
    if st["case"]["cap"]:
        c = st["case"]["cap"]
        r = torch.tanh(y / c)
        y, d = c * r, 1 - r * r
    if st["slopes"] is not None:
        y = y - st["slopes"][head].double() * (rows[:, None] - cols[None, :]).abs().double()
    return y + st["bias"], d


def exact(case, seed):
    st = prepare(case, seed)
    return {"span_fwd": _exact_span, "span_bwd": _exact_span, "append": _exact_append, "paged": _exact_paged}[case["op"]](st)


def _exact_span(st):
    case = st["case"]
    Z, L, H, Hk = (case[x] for x in ("Z", "L", "H", "Hk"))
    lens, spans, back = _lengths(case), st["spans"].long(), case["op"] == "span_bwd"
    zero = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)     # noqa: E731
    o, dq, dk, dv = zero(st["q"]), zero(st["q"]), zero(st["k"]), zero(st["k"])
    step = 4096
    for z in range(Z):
        n = int(lens[z])
        j = torch.arange(n, device=o.device)
        for h in range(H):
            kv = h * Hk // H
            K, V = st["k"][z, :n, kv].double(), st["v"][z, :n, kv].double()
            for a in range(0, n, step):
                b = min(n, a + step)
                Q = st["q"][z, a:b, h].double()
                x, d = _exact_scores(Q, K, st, h, j[a:b], j)
                hidden = (j[None] < spans[z, a:b, :1]) | (j[None] >= spans[z, a:b, 1:])
                p = _logistic(x).masked_fill_(hidden, 0.0)
                if not back:
                    o[z, a:b, h] = p @ V
                    continue
                dO = st["dout"][z, a:b, h].double()
                dv[z, :n, kv] += p.mT @ dO
                g = p * _logistic(-x) * (dO @ V.mT) * d * st["alpha"]
                dq[z, a:b, h] = g @ K
                dk[z, :n, kv] += g.mT @ Q
    return (dq, dk, dv) if back else o


def _exact_append(st):
    case = st["case"]
    have, new = _cached(case)
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    q = torch.zeros(st["q"].shape, dtype=torch.float64, device=kp.device)
    f = st["inv_freq"].double()
    table = st["page_table"].long()
    rot, page = case["rot"], case["page"]

    def turned(x, w):
        x = x.double().clone()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        c = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * w[:, None]
        x[..., a], x[..., b] = c.real, c.imag
        return x

    for z in range(case["Z"]):
        m = int(new[z])
        at = torch.arange(int(have[z]), int(have[z]) + m, device=kp.device)
        w = torch.polar(torch.ones(m, len(f), dtype=torch.float64, device=kp.device), (at + case["prefix"]).double()[:, None] * f)
        pg, slot = table[z][at // page], at % page
        kp[pg, slot], vp[pg, slot] = turned(st["k"][z, :m], w), st["v"][z, :m].double()
        q[z, :m] = turned(st["q"][z, :m], w)
    return {"q": q, "lens": None, "k_pages": kp, "v_pages": vp}


def _exact_paged(st):
    case = st["case"]
    have, new = _cached(case)
    H, Hk, page, P = case["H"], case["Hk"], case["page"], case["prefix"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    table = st["page_table"].long()

    def tokens(name, pages, count):
        return st[name][pages].double().reshape(-1, Hk, case["D"])[:count]

    for z in range(case["Z"]):
        n, m = int(have[z]) + int(new[z]), int(new[z])
        pages = table[z, :-(-n // page)]
        k, v = tokens("k_pages", pages, n), tokens("v_pages", pages, n)
        if P:
            k = torch.cat([tokens("k_pages", st["prefix_table"].long(), P), k])
            v = torch.cat([tokens("v_pages", st["prefix_table"].long(), P), v])
        j = torch.arange(P + n, device=o.device)
        rows = j[P + n - m:]
        for h in range(H):
            kv = h * Hk // H
            x, _ = _exact_scores(st["q"][z, :m, h].double(), k[:, kv], st, h, rows, j)
            o[z, :m, h] = _logistic(x).masked_fill_(j[None] > rows[:, None], 0.0) @ v[:, kv]
    return o
