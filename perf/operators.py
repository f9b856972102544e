"""Cases of the paged key-value cache operators: appending to the cache, the
decode step that reads it, the attention weights that its keys receive, and
the eviction that keeps the keys with the largest weights.

A paged cache is a pool of pages [P, Hkv, page, Dh] for K and one for V, a
table [B, pages] of page numbers and the lengths [B]: row t of sequence b
lies in page table[b, t // page], at row t % page.

Each case is run either in its plain form (elementary torch operations in 32
bits) or through the library's entry points; exact() states the same results
in 64 bits, one sequence and head at a time.
"""
import math

import torch

own = False

HEADS = ((32, 8), (32, 32), (32, 1), (16, 8), (8, 8), (8, 1), (4, 2))
PAGES = (8, 16, 24, 32, 64, 128, 256)
HEAD_SIZES = (64, 128, 256)


def listed():
    decode = dict(op="decode", window=0, weights=False)
    return [
        # one user's request, early in its answer: the latency of a step
        dict(decode, name="decode_one_short", B=1, Hq=32, Hkv=8, Dh=128, page=16, lmin=517, lmax=517),
        # a full server: 16 requests with long contexts, bound by memory bandwidth
        dict(decode, name="decode_batch_long", B=16, Hq=32, Hkv=8, Dh=128, page=64, lmin=16384,
             lmax=32768),
        # one K/V head for each query head, small heads, requests of every age
        dict(decode, name="decode_mha_ragged", B=8, Hq=32, Hkv=32, Dh=64, page=16, lmin=1, lmax=4096),
        # the Gemma-2B head layout under a sliding window
        dict(decode, name="decode_mqa_window", B=16, Hq=8, Hkv=1, Dh=256, page=32, lmin=16384,
             lmax=32768, window=4096),
        # a step that also records which keys it attended to, as eviction needs
        dict(decode, name="decode_weights", B=4, Hq=32, Hkv=8, Dh=128, page=16, lmin=16384,
             lmax=32768, weights=True),
        # every step of a server: one new token for each of 64 requests
        dict(op="append", name="append_tokens", B=64, Hkv=8, Dh=128, page=16, S=1, lmax=4096),
        # prompts of different lengths, padded to one length, written to the cache at once
        dict(op="append", name="append_prompts", B=4, Hkv=8, Dh=128, page=64, S=4096, lmax=4096),
        # the weights that the keys of a short prompt received, one K/V head for each query head
        dict(op="key_weights", name="key_weights_mha_short", B=2, Hq=32, Hkv=32, S=1024, Dh=128,
             queries=0, window=0, lmin=1024),
        # the same for one long prompt with grouped heads
        dict(op="key_weights", name="key_weights_gqa_long", B=1, Hq=32, Hkv=8, S=8192, Dh=128,
             queries=0, window=0, lmin=8192),
        # only a prompt's last 64 queries vote: padded long prompts
        dict(op="key_weights", name="key_weights_last64", B=4, Hq=32, Hkv=8, S=32768, Dh=64,
             queries=64, window=0, lmin=16384),
        # one request just over its budget
        dict(op="evict", name="evict_one_small", B=1, Hkv=8, Dh=64, page=16, lmin=1100, lmax=1100,
             budget=1024, recent=128),
        # a full server cut back to 4096 keys a request
        dict(op="evict", name="evict_batch_long", B=16, Hkv=8, Dh=128, page=64, lmin=16384,
             lmax=32768, budget=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op)
            for op in ("decode", "append", "key_weights", "evict")}
    op = rng.choice(("decode", "decode", "append", "key_weights", "evict"))
    while True:
        Hq, Hkv = rng.choice(HEADS)
        Dh = rng.choice(HEAD_SIZES)
        c = dict(op=op, Hkv=Hkv, Dh=Dh)
        if op == "decode":
            lmax = _log(rng, 1, 32768)
            c.update(B=_log(rng, 1, 64), Hq=Hq, page=rng.choice(PAGES), lmin=_log(rng, 1, lmax),
                     lmax=lmax, window=rng.choice((0, 0, _log(rng, 1, lmax))),
                     weights=rng.random() < 0.4)
        elif op == "append":
            S = _log(rng, 1, 4096)
            c.update(B=_log(rng, 1, 64), page=rng.choice(PAGES), S=S, lmax=_log(rng, S, 8192))
        elif op == "key_weights":
            S = _log(rng, 1, rng.choice((8192, 32768)))
            queries = 0 if S <= 8192 and rng.random() < 0.6 else _log(rng, 1, min(S, 512))
            c.update(B=_log(rng, 1, 8), Hq=Hq, S=S, queries=queries,
                     window=rng.choice((0, 0, _log(rng, 1, S))), lmin=_log(rng, 1, S))
        else:
            lmax = _log(rng, 2, 32768)
            budget = _log(rng, 1, lmax)
            c.update(B=_log(rng, 1, 16), page=rng.choice(PAGES), lmin=_log(rng, 1, lmax), lmax=lmax,
                     budget=budget, recent=rng.randint(0, budget))
        if _cost(c) <= most[op]:
            return c


def _cost(c):
    """The largest bytes (or the plain form's score matrix) that a case can come to."""
    if c["op"] == "decode":
        return c["B"] * c["Hkv"] * c["lmax"] * c["Dh"]
    if c["op"] == "append":
        return c["B"] * c["Hkv"] * c["S"] * c["Dh"]
    if c["op"] == "key_weights":
        return c["B"] * c["Hq"] * c["S"] * (c["queries"] or c["S"]) * c["Dh"]
    return c["B"] * c["Hkv"] * c["lmax"] * c["Dh"]


def work(case):
    c = case
    half = (c.get("lmin", 0) + c.get("lmax", c.get("S", 0))) / 2   # the mean length
    if c["op"] == "decode":
        seen = min(half, c["window"]) if c["window"] else half
        rows = c["B"] * c["Hkv"] * seen
        bytes_ = rows * c["Dh"] * 4 + 4 * c["B"] * c["Hq"] * c["Dh"]
        if c["weights"]:
            bytes_ += 4 * c["B"] * c["Hkv"] * half
        return {"bytes": bytes_, "flops": 4 * c["Dh"] * c["B"] * c["Hq"] * seen}
    if c["op"] == "append":
        rows = c["B"] * c["Hkv"] * (c["S"] if c["S"] == 1 else (c["S"] + 1) / 2)
        return {"bytes": rows * c["Dh"] * 8, "flops": 0}
    if c["op"] == "key_weights":
        n = int(half)
        nq = min(n, c["queries"] or n)
        pairs = nq * n - nq * (nq - 1) / 2
        if c["window"]:
            pairs = min(pairs, nq * c["window"])
        keys = min(n, nq + c["window"]) if c["window"] else n
        return {"bytes": c["B"] * (c["Hq"] * nq * (2 * c["Dh"] + 4) + c["Hkv"] * keys * 2 * c["Dh"]
                                   + 4 * c["Hkv"] * n),
                "flops": 2 * c["Dh"] * c["B"] * c["Hq"] * pairs}
    kept = min(half, c["budget"])
    return {"bytes": c["B"] * c["Hkv"] * (kept * (c["Dh"] * 8 + 4) + 8 * half), "flops": 0}


# ---------------------------------------------------------------------------
# inputs

def _lengths(gen, B, lo, hi):
    return torch.randint(lo, hi + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _paged(gen, c, cols, spare=0):
    """Pools and a table [B, cols] of pages in random order; `spare` further columns of pages."""
    B, page = c["B"], c["page"]
    pages = B * (cols + spare)
    pools = [_normal(gen, pages, c["Hkv"], page, c["Dh"]) for _ in range(2)]
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    return pools, order[:B * cols].view(B, cols), order[B * cols:].view(B, spare)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"c": c}
    B, Hkv, Dh = c["B"], c["Hkv"], c["Dh"]
    if c["op"] == "decode":
        cols = -(-c["lmax"] // c["page"])
        (s["kp"], s["vp"]), s["table"], _ = _paged(gen, c, cols)
        s["seqlens"] = _lengths(gen, B, c["lmin"], c["lmax"])
        s["q"] = _normal(gen, B, c["Hq"], 1, Dh)
        if c["weights"]:
            s["weights"] = torch.zeros(B, Hkv, cols * c["page"], device="cuda")
    elif c["op"] == "append":
        cols = -(-c["lmax"] // c["page"])
        (s["kp"], s["vp"]), s["table"], _ = _paged(gen, c, cols)
        s["k"], s["v"] = _normal(gen, B, Hkv, c["S"], Dh), _normal(gen, B, Hkv, c["S"], Dh)
        s["newlens"] = _lengths(gen, B, 1, c["S"])
        before = torch.rand(B, generator=gen, device="cuda") * (c["lmax"] + 1 - s["newlens"])
        s["seqlens"] = torch.minimum(s["newlens"] + before.to(torch.int32),
                                     torch.full_like(s["newlens"], c["lmax"]))
    elif c["op"] == "key_weights":
        S = c["S"]
        s["q"], s["k"] = _normal(gen, B, c["Hq"], S, Dh), _normal(gen, B, Hkv, S, Dh)
        s["seqlens"] = _lengths(gen, B, c["lmin"], S)
        s["weights"] = torch.zeros(B, Hkv, S, device="cuda")
        s["lse"] = torch.zeros(B, c["Hq"], S, device="cuda")
        # the log-sum-exps that the prompt's forward pass left behind
        pos = torch.arange(S, device="cuda")
        for b, n in enumerate(s["seqlens"].tolist()):
            nq = min(n, c["queries"] or n)
            for h in range(c["Hq"]):
                z = s["q"][b, h, n - nq:n].float() @ s["k"][b, h * Hkv // c["Hq"], :n].float().t()
                i = pos[n - nq:n, None]
                seen = pos[None, :n] <= i
                if c["window"]:
                    seen &= pos[None, :n] > i - c["window"]
                s["lse"][b, h, n - nq:n] = (z * Dh ** -0.5).masked_fill_(~seen, -math.inf).logsumexp(-1)
    else:
        cols, spare = -(-c["lmax"] // c["page"]), -(-c["budget"] // c["page"])
        (s["kp"], s["vp"]), s["table"], s["table_out"] = _paged(gen, c, cols, spare)
        s["seqlens"] = _lengths(gen, B, c["lmin"], c["lmax"])
        # accumulated weights: a few keys hold most of the mass
        s["weights"] = torch.empty(B, Hkv, cols * c["page"], device="cuda").exponential_(
            generator=gen).pow_(3)
        s["weights_out"] = torch.zeros_like(s["weights"])
    return s


# ---------------------------------------------------------------------------
# one pass

def run(state):
    if own:
        return _call(state)
    return {"decode": _plain_decode, "append": _plain_append, "key_weights": _plain_key_weights,
            "evict": _plain_evict}[state["c"]["op"]](state)


def _call(s):
    import causal_head_self_gb300 as chs
    c = s["c"]
    if c["op"] == "decode":
        if not c["weights"]:
            return chs.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["seqlens"],
                                         window=c["window"])
        o = chs.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["seqlens"],
                                  window=c["window"], weights=s["weights"], accumulate=False)
        return o, s["weights"]
    if c["op"] == "append":
        chs.attn_paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["seqlens"],
                              s["newlens"])
        return s["kp"], s["vp"]
    if c["op"] == "key_weights":
        return chs.attn_key_weights(s["q"], s["k"], s["lse"], s["weights"], s["seqlens"],
                                    queries=c["queries"], window=c["window"], accumulate=False)
    newlens, keep = chs.attn_cache_evict(s["kp"], s["vp"], s["weights"], s["table"], s["seqlens"],
                                         c["budget"], c["recent"], table_out=s["table_out"],
                                         weights_out=s["weights_out"])
    return s["kp"], s["vp"], s["weights_out"], newlens, keep


def _rows(pool, table):
    """The rows of a paged pool in order, [B, Hkv, rows, Dh]."""
    B, cols = table.shape
    return pool[table.long()].transpose(1, 2).reshape(B, pool.shape[1], cols * pool.shape[2],
                                                      pool.shape[3])


def _plain_decode(s):
    c = s["c"]
    B, Hq, Hkv, Dh = c["B"], c["Hq"], c["Hkv"], c["Dh"]
    k, v = _rows(s["kp"], s["table"]).float(), _rows(s["vp"], s["table"]).float()
    T = k.shape[2]
    t, n = torch.arange(T, device="cuda"), s["seqlens"][:, None]
    seen = t < n
    if c["window"]:
        seen &= t >= n - c["window"]
    z = (s["q"].float().view(B, Hkv, Hq // Hkv, Dh) * Dh ** -0.5) @ k.transpose(2, 3)
    z.masked_fill_(~seen[:, None, None], -math.inf)
    p = (z - z.amax(-1, keepdim=True)).exp_()
    p /= p.sum(-1, keepdim=True)
    o = (p @ v).view(B, Hq, 1, Dh).to(torch.bfloat16)
    if not c["weights"]:
        return o
    return o, torch.where((t < n)[:, None], p.sum(2), s["weights"])


def _plain_append(s):
    c = s["c"]
    i = torch.arange(c["S"], device="cuda")
    real = i < s["newlens"][:, None]
    t = (s["seqlens"] - s["newlens"])[:, None] + i
    b, j = real.nonzero(as_tuple=True)
    t = t[b, j]
    page, row = s["table"][b, t // c["page"]].long(), t % c["page"]
    s["kp"][page, :, row] = s["k"][b, :, j]
    s["vp"][page, :, row] = s["v"][b, :, j]
    return s["kp"], s["vp"]


def _plain_key_weights(s):
    c = s["c"]
    B, Hq, Hkv, S, Dh = c["B"], c["Hq"], c["Hkv"], c["S"], c["Dh"]
    nq = min(S, c["queries"] or S)
    n = s["seqlens"].long()[:, None]
    j = torch.arange(S, device="cuda")
    i = (n - nq).clamp(min=0) + torch.arange(nq, device="cuda")   # positions of the voting queries
    at = i.clamp(max=S - 1)[:, None, :].expand(B, Hq, nq)
    q = s["q"].gather(2, at[..., None].expand(B, Hq, nq, Dh)).float() * Dh ** -0.5
    z = q.view(B, Hkv, -1, Dh) @ s["k"].float().transpose(2, 3)
    z -= s["lse"].gather(2, at).view(B, Hkv, -1, 1)
    seen = (j <= i[..., None]) & (i < n)[..., None]
    if c["window"]:
        seen &= j > i[..., None] - c["window"]
    p = z.exp_().view(B, Hkv, Hq // Hkv, nq, S).masked_fill_(~seen[:, None, None], 0.0)
    return torch.where((j < n)[:, None], p.sum((2, 3)), s["weights"])


def _plain_evict(s):
    c = s["c"]
    B, Hkv, page, budget = c["B"], c["Hkv"], c["page"], c["budget"]
    w, n = s["weights"], s["seqlens"].long()[:, None, None]
    T = w.shape[2]
    t = torch.arange(T, device="cuda")
    newlens = s["seqlens"].clamp(max=budget)
    rank = torch.where(t >= n - c["recent"], math.inf, w).masked_fill(t >= n, -math.inf)
    first = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    i = torch.arange(budget, device="cuda")
    real = i < newlens[:, None, None]
    keep = first.masked_fill(~real, T).sort(dim=-1).values
    kept = keep.clamp(max=T - 1)
    out = w.gather(2, kept)
    back = s["weights_out"].masked_fill((t < n) & (t >= newlens[:, None, None]), 0.0)
    back[..., :budget] = torch.where(real, out, back[..., :budget])
    b, j = real[:, 0].nonzero(as_tuple=True)
    heads = torch.arange(Hkv, device="cuda")
    src = kept[b, :, j]                                           # [kept rows, Hkv]
    to, row = s["table_out"][b, j // page].long(), j % page
    for pool in (s["kp"], s["vp"]):
        pool[to[:, None], heads, row[:, None]] = \
            pool[s["table"][b[:, None], src // page].long(), heads, src % page]
    return (s["kp"], s["vp"], back, newlens, torch.where(real, keep, -1).to(torch.int32))


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions

def _sequence(pool, table, n, h):
    """Rows 0 .. n-1 of one sequence and head."""
    page = pool.shape[2]
    return torch.cat([pool[p, h] for p in table[:-(-n // page)].tolist()])[:n].double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    B, Hkv, Dh = c["B"], c["Hkv"], c["Dh"]
    if c["op"] in ("decode", "key_weights"):
        G = c["Hq"] // Hkv
        w = s["weights"].double() if "weights" in s else None
    if c["op"] == "decode":
        o = torch.empty(B, c["Hq"], 1, Dh, device="cuda", dtype=torch.float64)
        for b, n in enumerate(s["seqlens"].tolist()):
            lo = max(0, n - c["window"]) if c["window"] else 0
            for g in range(Hkv):
                k = _sequence(s["kp"], s["table"][b], n, g)[lo:]
                v = _sequence(s["vp"], s["table"][b], n, g)[lo:]
                p = torch.softmax(s["q"][b, g * G:(g + 1) * G, 0].double() @ k.t() / math.sqrt(Dh), -1)
                o[b, g * G:(g + 1) * G, 0] = p @ v
                if w is not None:
                    w[b, g, :lo] = 0
                    w[b, g, lo:n] = p.sum(0)
        return o if w is None else (o, w)
    if c["op"] == "key_weights":
        for b, n in enumerate(s["seqlens"].tolist()):
            first = max(0, n - c["queries"]) if c["queries"] else 0
            w[b, :, :n] = 0
            for h in range(c["Hq"]):
                z = s["q"][b, h, first:n].double() @ s["k"][b, h // G, :n].double().t() / math.sqrt(Dh)
                p = torch.exp(z - s["lse"][b, h, first:n, None].double()).tril(first)
                if c["window"]:
                    p = p.triu(first - c["window"] + 1)
                w[b, h // G, :n] += p.sum(0)
        return w
    if c["op"] == "append":
        k, v, kp, vp = (s[x].cpu() for x in ("k", "v", "kp", "vp"))
        table, page = s["table"].tolist(), c["page"]
        for b, (n, new) in enumerate(zip(s["seqlens"].tolist(), s["newlens"].tolist())):
            for i in range(new):
                at, row = divmod(n - new + i, page)
                kp[table[b][at], :, row], vp[table[b][at], :, row] = k[b, :, i], v[b, :, i]
        return kp, vp
    keep = torch.full((B, Hkv, c["budget"]), -1, dtype=torch.int32)
    back, page = s["weights_out"], c["page"]
    for b, n in enumerate(s["seqlens"].tolist()):
        m = min(n, c["budget"])
        back[b, :, m:n] = 0
        for g in range(Hkv):
            old = n - c["recent"] if n > c["budget"] else 0
            values = s["weights"][b, g, :n].tolist()
            kept = sorted(range(old), key=lambda t: (-values[t], t))[:m - (n - old)]
            kept = sorted(kept) + list(range(old, n))
            keep[b, g, :m] = torch.tensor(kept, dtype=torch.int32)
            kept = torch.tensor(kept, device="cuda")
            back[b, g, :m] = s["weights"][b, g][kept]
            to = torch.arange(m, device="cuda")
            for pool in (s["kp"], s["vp"]):
                pool[s["table_out"][b, to // page].long(), g, to % page] = \
                    pool[s["table"][b, kept // page].long(), g, kept % page]
    return s["kp"], s["vp"], back, s["seqlens"].clamp(max=c["budget"]), keep
