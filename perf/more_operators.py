"""Cases of the operators on packed tokens: attention over sequences of
different lengths that lie one behind another, forward and as a training step;
rotary positions, alone and together with the write to the paged cache; and
the plan of a serving step, which hands out pages and says where each new
token goes.

Packed tokens are rows [T, H, Dh]: sequence b holds rows cu[b] .. cu[b+1] - 1,
and rows behind the last sequence belong to none.

Each case is run either in its plain form (elementary torch operations in 32
bits) or through the library's entry points; exact() states the same results
in 64 bits, one sequence at a time.
"""
import math
import random

import torch

own = False

HEADS = ((32, 8), (32, 32), (32, 1), (16, 8), (8, 8), (8, 1), (4, 2))
PAGES = (8, 16, 24, 32, 64, 128, 256)
HEAD_SIZES = (64, 128, 256)


def listed():
    attn = dict(window=0, causal=True, pad=0, salt=0)
    rope = dict(interleaved=False, inverse=False, scaling="none", factor=1.0, base=10000.0, salt=0)
    return [
        # a few short requests that arrived together: the latency of a small prefill
        dict(attn, op="fwd", name="fwd_requests_short", B=16, Hq=32, Hkv=8, Dh=128, lmin=1, lmax=128),
        # a server's prefill step: prompts of every length, the buffer longer than their sum
        dict(attn, op="fwd", name="fwd_prompts_ragged", B=16, Hq=32, Hkv=8, Dh=128, lmin=64, lmax=4096,
             pad=37),
        # four long documents, bound by the tensor cores
        dict(attn, op="fwd", name="fwd_prompts_long", B=4, Hq=32, Hkv=8, Dh=128, lmin=4096, lmax=16384),
        # the large head size with a sliding window
        dict(attn, op="fwd", name="fwd_window_wide", B=6, Hq=16, Hkv=8, Dh=256, lmin=512, lmax=8192,
             window=2048),
        # a training step over a batch packed from documents of very different lengths
        dict(attn, op="train", name="train_documents", B=24, Hq=32, Hkv=8, Dh=128, lmin=16, lmax=2048),
        # the same with one K/V head for each query head and small heads
        dict(attn, op="train", name="train_mha_small", B=8, Hq=32, Hkv=32, Dh=64, lmin=128, lmax=4096,
             pad=61),
        # the queries and keys of a packed batch, in every layer's forward pass
        dict(rope, op="rope", name="rope_batch", T=16384, Hq=32, Hkv=8, Dh=128, rot=128, far=8192),
        # part of each head in neighbouring pairs, positions far beyond the trained ones; the
        # gradient's way back
        dict(rope, op="rope", name="rope_far_back", T=4001, Hq=16, Hkv=8, Dh=256, rot=64, far=1000000,
             interleaved=True, inverse=True, scaling="yarn", factor=32.0),
        # one new token for each of 64 requests: every layer of a decode step
        dict(rope, op="append", name="append_step", T=64, Hq=32, Hkv=8, Dh=128, rot=128, far=32768,
             page=16, pad=0),
        # the tokens of a prefill step
        dict(rope, op="append", name="append_prompts", T=16384, Hq=32, Hkv=8, Dh=128, rot=128, far=16384,
             page=64, pad=19, scaling="turns", factor=8.0, base=500000.0),
        # one new token for each of 64 requests: pages and slots of a decode step
        dict(op="plan", name="plan_step", B=64, page=16, lmax=8192, grow=1, T=64, mixed=False),
        # a large server's step: prompts admitted, requests finished, drafts taken back
        dict(op="plan", name="plan_mixed", B=2048, page=64, lmax=32768, grow=512, T=262144, mixed=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op)
            for op in ("fwd", "train", "rope", "append", "plan")}
    op = rng.choice(("fwd", "fwd", "train", "train", "rope", "append", "plan"))
    while True:
        Hq, Hkv = rng.choice(HEADS)
        Dh = rng.choice(HEAD_SIZES)
        c = dict(op=op, salt=rng.randrange(1 << 20))
        if op in ("fwd", "train"):
            lmax = _log(rng, 1, 16384)
            causal = rng.random() < 0.85
            # (the plain form goes by sequence and K/V head)
            c.update(B=_log(rng, 1, min(256, 1024 // Hkv)), Hq=Hq, Hkv=Hkv, Dh=Dh, lmin=_log(rng, 1, lmax), lmax=lmax,
                     causal=causal, window=rng.choice((0, 0, _log(rng, 1, lmax))) if causal else 0,
                     pad=rng.choice((0, _log(rng, 1, 300))))
        elif op in ("rope", "append"):
            scaling = rng.choice(("none", "none", "linear", "base", "turns", "yarn"))
            c.update(T=_log(rng, 1, 16384), Hq=Hq, Hkv=Hkv, Dh=Dh,
                     rot=rng.choice((Dh, Dh, Dh // 2, Dh // 4, 16)), far=_log(rng, 1, 1000000),
                     interleaved=rng.random() < 0.5, inverse=op == "rope" and rng.random() < 0.5,
                     scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 8.0, 40.0)),
                     base=rng.choice((10000.0, 500000.0)))
            if op == "append":
                c.update(page=rng.choice(PAGES), pad=rng.choice((0, _log(rng, 1, 100))))
        else:
            mixed = rng.random() < 0.6
            B, grow = _log(rng, 1, 4096), _log(rng, 1, 4096) if mixed else rng.choice((1, 1, 4))
            c.update(B=B, page=rng.choice(PAGES), lmax=_log(rng, 1, 32768), grow=grow,
                     T=B * grow, mixed=mixed)
        if _cost(c) <= most[op]:
            return c


def _cost(c):
    if c["op"] in ("fwd", "train"):
        return sum(l * l for l in _lengths(c)) * c["Hq"] * c["Dh"]
    if c["op"] in ("rope", "append"):
        return c["T"] * (c["Hq"] + c["Hkv"]) * c["Dh"]
    return c["T"] + c["B"] * (c["lmax"] // c["page"])


def _lengths(c):
    """The case's lengths, spread over the logarithm of their range (the seed orders them)."""
    rng = random.Random(c["salt"] * 7919 + c["B"])
    return [_log(rng, c["lmin"], c["lmax"]) for _ in range(c["B"])]


def _pairs(c):
    """The (query, key) pairs that the mask leaves, of one head."""
    total = 0
    for n in _lengths(c):
        if not c["causal"]:
            total += n * n
        else:
            w = min(n, c["window"] or n)
            total += w * (w + 1) // 2 + (n - w) * w
    return total


def work(case):
    c = case
    if c["op"] in ("fwd", "train"):
        rows = sum(_lengths(c)) * c["Dh"] * 2
        if c["op"] == "fwd":
            return {"bytes": rows * (2 * c["Hq"] + 2 * c["Hkv"]),
                    "flops": 4 * c["Dh"] * c["Hq"] * _pairs(c)}
        return {"bytes": rows * (4 * c["Hq"] + 4 * c["Hkv"]),
                "flops": 14 * c["Dh"] * c["Hq"] * _pairs(c)}
    if c["op"] == "rope":
        rows = c["T"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 4 * rows * c["Dh"] + 4 * c["T"], "flops": 3 * rows * c["rot"]}
    if c["op"] == "append":
        # q and k read and written, k and v written to the pages, v read
        rows = c["T"] * (2 * c["Hq"] + 5 * c["Hkv"])
        return {"bytes": 2 * rows * c["Dh"] + 8 * c["T"],
                "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    return {"bytes": 8 * c["T"] + 16 * c["B"] + 8 * (c["T"] // c["page"]), "flops": 0}


# ---------------------------------------------------------------------------
# inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    s = {"c": c}
    if c["op"] in ("fwd", "train"):
        lens = _lengths(c)
        rng.shuffle(lens)
        first = [0]
        for n in lens:
            first.append(first[-1] + n)
        T, Hq, Hkv, Dh = first[-1] + c["pad"], c["Hq"], c["Hkv"], c["Dh"]
        s["first"], s["cu"] = first, _int32(first)
        # one projection's output: queries, keys and values of a token side by side
        qkv = _normal(gen, T, Hq + 2 * Hkv, Dh)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["o"] = torch.zeros(T, Hq, Dh, device="cuda", dtype=torch.bfloat16)
        if c["op"] == "train":
            s["do"] = _normal(gen, T, Hq, Dh)
            s["lse"] = torch.zeros(Hq, T, device="cuda")
            s["dq"] = torch.zeros(T, Hq, Dh, device="cuda", dtype=torch.bfloat16)
            s["dk"], s["dv"] = (torch.zeros(T, Hkv, Dh, device="cuda", dtype=torch.bfloat16)
                                for _ in range(2))
    elif c["op"] in ("rope", "append"):
        T, Hq, Hkv, Dh = c["T"] + c.get("pad", 0), c["Hq"], c["Hkv"], c["Dh"]
        qkv = _normal(gen, T, Hq + 2 * Hkv, Dh)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["positions"] = torch.randint(0, c["far"], (T,), generator=gen, device="cuda",
                                       dtype=torch.int32)
        s["q_out"] = torch.zeros(T, Hq, Dh, device="cuda", dtype=torch.bfloat16)
        s["k_out"] = torch.zeros(T, Hkv, Dh, device="cuda", dtype=torch.bfloat16)
        if c["op"] == "append":
            page = c["page"]
            pages = -(-T // page) + 8
            s["kp"], s["vp"] = _normal(gen, pages, Hkv, page, Dh), _normal(gen, pages, Hkv, page, Dh)
            order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
            t = torch.arange(T, device="cuda", dtype=torch.int32)
            s["slots"] = order[(t // page).long()] * page + t % page
            s["positions"][c["T"]:] = -1   # rows behind the last token
            s["slots"][c["T"]:] = -1
        s["turns"], s["amplitude"] = _frequencies(c)
        if own:
            import causal_head_self_gb300 as chs
            s["rope"] = chs.attn_rope_frequencies(c["rot"], c["base"], scaling=c["scaling"],
                                                  factor=c["factor"], original_len=8192)
    else:
        B, page, lmax, grow, T = c["B"], c["page"], c["lmax"], c["grow"], c["T"]
        lens, delta = [], []
        for b in range(B):
            kind = rng.random() if c["mixed"] else 1.0
            if kind < 0.15:      # a prompt is admitted
                lens.append(0)
                delta.append(_log(rng, 1, grow))
            elif kind < 0.25:    # a request is finished
                lens.append(_log(rng, 1, lmax))
                delta.append(-lens[-1])
            elif kind < 0.35:    # drafted tokens are taken back
                lens.append(_log(rng, 1, lmax))
                delta.append(-min(lens[-1], rng.randint(0, 8)))
            elif kind < 0.40:    # an empty place
                lens.append(0)
                delta.append(0)
            else:
                lens.append(_log(rng, 1, lmax))
                delta.append(rng.randint(1, grow) if c["mixed"] else grow)
        cols = -(-(lmax + grow) // page)
        held = [-(-n // page) for n in lens]
        need = sum(-(-max(n + d, 0) // page) for n, d in zip(lens, delta))
        spare = max(need - sum(held), 0) + 16
        order = torch.randperm(B * cols + 16, generator=gen, device="cuda").to(torch.int32)
        column = torch.arange(cols, device="cuda")
        used = column < torch.tensor(held, device="cuda")[:, None]
        s["table"] = torch.full((B, cols), -1, device="cuda", dtype=torch.int32)
        s["table"][used] = order[:sum(held)]
        s["num_pages"] = B * cols + 16
        s["free"] = torch.full((s["num_pages"],), -1, device="cuda", dtype=torch.int32)
        s["free"][:spare] = order[sum(held):sum(held) + spare]
        s["num_free"] = _int32([spare])
        s["seqlens"], s["delta"] = _int32(lens), _int32(delta)
        s["seqlens_out"], s["num_free_out"] = torch.zeros_like(s["seqlens"]), _int32([0])
    return s


def _frequencies(c):
    """The turns per token of each pair, in 64 bits, and the factor on the rotated values."""
    rot, base, factor = c["rot"], c["base"], c["factor"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    if c["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    turns = base ** (-2 * i / rot) / (2 * math.pi)
    if c["scaling"] == "linear":
        turns = turns / factor
    if c["scaling"] in ("turns", "yarn"):
        low, high = (1.0, 4.0) if c["scaling"] == "turns" else (1.0, 32.0)
        keep = ((8192 * turns - low) / (high - low)).clamp(0, 1)
        turns = turns * (keep + (1 - keep) / factor)
    return turns, 0.1 * math.log(factor) + 1 if c["scaling"] == "yarn" else 1.0


# ---------------------------------------------------------------------------
# one pass

def run(state):
    if own:
        return _call(state)
    return {"fwd": _plain_fwd, "train": _plain_train, "rope": _plain_rope, "append": _plain_append,
            "plan": _plain_plan}[state["c"]["op"]](state)


def _call(s):
    import causal_head_self_gb300 as chs
    c = s["c"]
    if c["op"] == "fwd":
        return chs.attn_fwd_packed(s["q"], s["k"], s["v"], s["cu"], s["o"], causal=c["causal"],
                                   window=c["window"])
    if c["op"] == "train":
        mask = dict(causal=c["causal"], window=c["window"])
        chs.attn_fwd_packed(s["q"], s["k"], s["v"], s["cu"], s["o"], s["lse"], **mask)
        chs.attn_bwd_packed(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["cu"], s["dq"],
                            s["dk"], s["dv"], **mask)
        return s["o"], s["dq"], s["dk"], s["dv"]
    if c["op"] == "rope":
        return chs.attn_rope(s["q"], s["k"], s["positions"], s["rope"], s["q_out"], s["k_out"],
                             interleaved=c["interleaved"], inverse=c["inverse"])
    if c["op"] == "append":
        chs.attn_rope_append(s["q"], s["k"], s["v"], s["positions"], s["rope"], s["kp"], s["vp"],
                             s["slots"], s["q_out"], s["k_out"], interleaved=c["interleaved"])
        return s["q_out"], s["k_out"], s["kp"], s["vp"]
    cu, positions, slots = chs.attn_cache_plan(
        s["delta"], s["seqlens"], s["table"], s["free"], s["num_free"], rows=c["T"], page=c["page"],
        num_pages=s["num_pages"], seqlens_out=s["seqlens_out"], num_free_out=s["num_free_out"])
    return s["seqlens_out"], s["table"], s["free"], s["num_free_out"], cu, positions, slots


def _hidden(n, c):
    """The (query, key) pairs of a sequence of n that the mask hides."""
    i = torch.arange(n, device="cuda")
    hidden = torch.zeros(n, n, device="cuda", dtype=torch.bool)
    if c["causal"]:
        hidden = i[None] > i[:, None]
    if c["window"]:
        hidden = hidden | (i[None] <= i[:, None] - c["window"])
    return hidden


def _weights(s, a, z, g, hidden):
    """Queries, keys, values [.., n, Dh] of the sequence at rows a .. z - 1 and K/V head g, and the
    softmax weights of the group's query heads."""
    c = s["c"]
    G = c["Hq"] // c["Hkv"]
    q = s["q"][a:z, g * G:(g + 1) * G].float().transpose(0, 1)
    k, v = s["k"][a:z, g].float(), s["v"][a:z, g].float()
    p = (q * c["Dh"] ** -0.5) @ k.t()
    p.masked_fill_(hidden, -math.inf)
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    p /= p.sum(-1, keepdim=True)
    return q, k, v, p


def _plain_fwd(s):
    c, first, o = s["c"], s["first"], torch.zeros_like(s["o"])
    G = c["Hq"] // c["Hkv"]
    for a, z in zip(first, first[1:]):
        hidden = _hidden(z - a, c)
        for g in range(c["Hkv"]):
            _, _, v, p = _weights(s, a, z, g, hidden)
            o[a:z, g * G:(g + 1) * G] = (p @ v).transpose(0, 1)
    return o


def _plain_train(s):
    c, first, scale = s["c"], s["first"], s["c"]["Dh"] ** -0.5
    G = c["Hq"] // c["Hkv"]
    o, dq, dk, dv = (torch.zeros_like(s[x]) for x in ("o", "dq", "dk", "dv"))
    for a, z in zip(first, first[1:]):
        hidden = _hidden(z - a, c)
        for g in range(c["Hkv"]):
            heads = slice(g * G, (g + 1) * G)
            q, k, v, p = _weights(s, a, z, g, hidden)
            do, out = s["do"][a:z, heads].float().transpose(0, 1), p @ v
            ds = do @ v.t()
            ds -= (do * out).sum(-1, keepdim=True)
            ds *= p
            o[a:z, heads] = out.transpose(0, 1)
            dv[a:z, g] = (p.transpose(1, 2) @ do).sum(0)
            dq[a:z, heads] = (ds @ k).transpose(0, 1) * scale
            dk[a:z, g] = (ds.transpose(1, 2) @ q).sum(0) * scale
    return o, dq, dk, dv


def _rotated(x, out, s):
    """x [T, H, Dh] with its first `rot` values turned by their positions, in 32 bits."""
    c = s["c"]
    rot = c["rot"]
    angle = s["positions"].double()[:, None] * (2 * math.pi * s["turns"])
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    if c["inverse"]:
        sin = -sin
    x = x.float()
    y = x.clone()
    first = slice(0, rot, 2) if c["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if c["interleaved"] else slice(rot // 2, rot)
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return torch.where((s["positions"] >= 0)[:, None, None], y.to(torch.bfloat16), out)


def _plain_rope(s):
    return _rotated(s["q"], s["q_out"], s), _rotated(s["k"], s["k_out"], s)


def _plain_append(s):
    q, k = _rotated(s["q"], s["q_out"], s), _rotated(s["k"], s["k_out"], s)
    t = (s["slots"] >= 0).nonzero()[:, 0]
    slot, page = s["slots"][t].long(), s["c"]["page"]
    s["kp"][slot // page, :, slot % page] = k[t]
    s["vp"][slot // page, :, slot % page] = s["v"][t]
    return q, k, s["kp"], s["vp"]


def _plain_plan(s):
    c, table, free = s["c"], s["table"].clone(), s["free"].clone()
    page, T, B = c["page"], c["T"], c["B"]
    before, delta = s["seqlens"].long(), s["delta"].long()
    after = before + delta
    had, has = (before + page - 1) // page, (after + page - 1) // page
    column = torch.arange(table.shape[1], device="cuda")
    back = table[(column >= has[:, None]) & (column < had[:, None])]   # pages given back, in order
    F = s["num_free"].long()
    stack = torch.cat([free[:int(F)], back])
    wanted = (column >= had[:, None]) & (column < has[:, None])
    taken = int(wanted.sum())
    left = stack.numel() - taken
    table[wanted] = stack.flip(0)[:taken]
    kept = max(left - int(F), 0)
    free[int(F):int(F) + kept] = stack[int(F):int(F) + kept]
    new = delta.clamp(min=0)
    cu = torch.zeros(B + 1, device="cuda", dtype=torch.long)
    cu[1:] = new.cumsum(0)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    real = t < cu[-1]
    positions = torch.where(real, before[b] + t - cu[b], -1)
    at = positions.clamp(min=0)
    slots = table[b, (at // page).clamp(max=table.shape[1] - 1)].long() * page + at % page
    return (after.int(), table, free, F.new_tensor([left]).int(), cu.int(), positions.int(),
            torch.where(real, slots, -1).int())


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("fwd", "train"):
        return _exact_attention(c, s)
    if c["op"] == "plan":
        return _exact_plan(c, s)
    pairs = []
    inverse = -1.0 if c["inverse"] else 1.0
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.double()
        for i, turns in enumerate(s["turns"].tolist()):
            one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
            # the angle as a complex number on the unit circle, times the pair as another
            z = torch.polar(torch.full_like(s["positions"], s["amplitude"], dtype=torch.float64),
                            inverse * 2 * math.pi * (s["positions"].double() * turns))
            pair = torch.complex(y[..., one], y[..., two]) * z[:, None]
            y[..., one], y[..., two] = pair.real, pair.imag
        y[s["positions"] < 0] = out[s["positions"] < 0].double()
        pairs.append(y)
    if c["op"] == "rope":
        return tuple(pairs)
    kp, vp = s["kp"].double(), s["vp"]
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            kp[slot // c["page"], :, slot % c["page"]] = pairs[1][t]
            vp[slot // c["page"], :, slot % c["page"]] = s["v"][t]
    return pairs[0], pairs[1], kp, vp


def _exact_attention(c, s):
    train = c["op"] == "train"
    o = torch.zeros(s["o"].shape, device="cuda", dtype=torch.float64)
    grads = [torch.zeros(s[x].shape, device="cuda", dtype=torch.float64) for x in ("q", "k", "v")]
    for a, z in zip(s["first"], s["first"][1:]):
        n = z - a
        seen = torch.ones(n, n, device="cuda", dtype=torch.bool)
        if c["causal"]:
            seen = seen.tril()
        if c["window"]:
            seen = seen.triu(1 - c["window"])
        for h in range(c["Hq"]):
            g = h * c["Hkv"] // c["Hq"]
            x = [t[a:z, i].double().requires_grad_(train)
                 for t, i in ((s["q"], h), (s["k"], g), (s["v"], g))]
            scores = torch.where(seen, x[0] @ x[1].t() / math.sqrt(c["Dh"]), -math.inf)
            y = torch.softmax(scores, -1) @ x[2]
            o[a:z, h] = y.detach()
            if train:
                for grad, d, i in zip(grads, torch.autograd.grad(y, x, s["do"][a:z, h].double()),
                                      (h, g, g)):
                    grad[a:z, i] += d
    return (o, *grads) if train else o


def _exact_plan(c, s):
    page = c["page"]
    lens, delta, table = s["seqlens"].tolist(), s["delta"].tolist(), s["table"].tolist()
    free, num_free = s["free"].tolist(), s["num_free"].item()
    stack = free[:num_free]
    for b, (n, d) in enumerate(zip(lens, delta)):
        stack += [table[b][i] for i in range(-(-(n + d) // page), -(-n // page))]
    cu, positions, slots = [0], [], []
    for b, (n, d) in enumerate(zip(lens, delta)):
        for i in range(-(-n // page), -(-(n + d) // page)):
            table[b][i] = stack.pop()
        for t in range(n, n + d):
            positions.append(t)
            slots.append(table[b][t // page] * page + t % page)
        cu.append(len(positions))
    free[num_free:len(stack)] = stack[num_free:]
    rest = [-1] * (c["T"] - len(positions))
    return (_int32([n + d for n, d in zip(lens, delta)]), _int32(table), _int32(free),
            _int32([len(stack)]), _int32(cu), _int32(positions + rest), _int32(slots + rest))
