"""Paged-cache test helpers: caches with pages in random order whose unused
rows hold NaN and infinities and whose unused table entries hold nonsense, and
the operators in 64 bits from their definitions, one row at a time."""
import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2   # a rounding to bf16, relative to the value


def make_cache(lens, Hkv, Dh, page, cols, seed, spare=0, first_used=None):
    """(kpages, vpages, table, seqlens) on the CPU.  Rows that hold no key are
    NaN or +-inf; table entries past a sequence's pages (and before row
    first_used[b]) are not page numbers at all."""
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    P = B * cols + spare
    pools = []
    for _ in range(2):
        junk = torch.tensor([math.nan, math.inf, -math.inf])
        pool = junk[torch.randint(0, 3, (P, Hkv, page, 1), generator=gen)].expand(P, Hkv, page, Dh)
        pools.append(pool.to(torch.bfloat16).clone())
    order = torch.randperm(P, generator=gen).to(torch.int32)
    table = order[:B * cols].view(B, cols).clone()
    nonsense = torch.tensor([-1, -(2 ** 31), 2 ** 31 - 1, P, P + 5], dtype=torch.int32)
    for b, n in enumerate(lens):
        lo = 0 if first_used is None else max(0, first_used[b])
        for c in range(cols):
            if c * page >= n or (c + 1) * page <= lo:
                table[b, c] = nonsense[(b + c) % 5]
        for t in range(lo, n):
            for pool in pools:
                pool[table[b, t // page], :, t % page] = torch.randn(
                    (Hkv, Dh), generator=gen).to(torch.bfloat16)
    return (*pools, table, torch.tensor(lens, dtype=torch.int32))


def rows(pool, table_row, lo, hi, g):
    """Rows [lo, hi) of one sequence and head in 64 bits."""
    page = pool.shape[2]
    return torch.stack([pool[table_row[t // page], g, t % page] for t in range(lo, hi)]).double()


def decode(q, kp, vp, table, lens, window=0, scale=0.0):
    """(o, its tolerance, weights, their relative tolerance): weights are rows
    [0, lens[b]) of a [B, Hkv, cols * page] tensor, the others 0."""
    B, Hq, _, Dh = q.shape
    Hkv, page = kp.shape[1], kp.shape[2]
    G, T = Hq // Hkv, table.shape[1] * page
    scale = scale or 1 / math.sqrt(Dh)
    o, tol = torch.zeros(B, Hq, 1, Dh, dtype=torch.float64), torch.zeros(B, Hq, 1, Dh, dtype=torch.float64)
    w, worst = torch.zeros(B, Hkv, T, dtype=torch.float64), 0.0
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        lo = max(0, n - window) if window > 0 else 0
        for g in range(Hkv):
            k, v = rows(kp, table[b], lo, n, g), rows(vp, table[b], lo, n, g)
            qg = q[b, g * G:(g + 1) * G, 0].double()
            p = torch.softmax(scale * qg @ k.t(), -1)
            # Dh products are added in 32 bits, each addition off by at most
            # 2^-23 of the sum of their sizes (truncated); a score's error moves a
            # weight and the sum of weights by that much each
            delta = Dh * 2.0 ** -23 * float((scale * qg.abs() @ k.abs().t()).max())
            worst = max(worst, 2 * delta + 2.0 ** -18)   # 2^-18: exp2 and the 32-bit sums
            o[b, g * G:(g + 1) * G, 0] = p @ v
            # the weights and the output are each rounded to bf16 once
            tol[b, g * G:(g + 1) * G, 0] = HALF_BF16 * ((p @ v).abs() + p @ v.abs()) + worst * (p @ v.abs())
            w[b, g, lo:n] = p.sum(0)
    return o, tol, w, worst


def key_weights(q, k, lse, lens, queries=0, causal=True, window=0, scale=0.0):
    """(weights [B, Hkv, S], relative tolerance)."""
    B, Hq, S, Dh = q.shape
    Hkv = k.shape[1]
    scale = scale or 1 / math.sqrt(Dh)
    w, worst = torch.zeros(B, Hkv, S, dtype=torch.float64), 0.0
    for b, n in enumerate(lens):
        first = max(0, n - queries) if queries else 0
        if n == 0:
            continue
        for h in range(Hq):
            g = h * Hkv // Hq
            qh, kg = q[b, h, first:n].double(), k[b, g, :n].double()
            p = torch.exp(scale * qh @ kg.t() - lse[b, h, first:n, None].double())
            i, j = torch.arange(first, n)[:, None], torch.arange(n)[None]
            seen = torch.ones(n - first, n, dtype=torch.bool)
            if causal:
                seen &= j <= i
                if window > 0:
                    seen &= j > i - window
            w[b, g, :n] += torch.where(seen, p, 0.0).sum(0)
            x = float((scale * qh.abs() @ kg.abs().t()).max()) + float(lse[b, h, first:n].abs().max())
            # the score as above; the exponent (of size x / ln 2) and the 32-bit
            # normaliser are rounded once each
            worst = max(worst, (Dh * 2.0 ** -23 + 2.0 ** -23) * x + 2.0 ** -18)
    return w, worst


def evict(weights, lens, budget, recent):
    """(newlens, keep): the rows that stay, -1 behind them."""
    B, Hkv, _ = weights.shape
    keep = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens.tolist()):
        for g in range(Hkv):
            if n <= budget:
                kept = list(range(n))
            else:
                x = weights[b, g].tolist()
                x = [-math.inf if math.isnan(y) else y for y in x]
                is_nan = weights[b, g].isnan().tolist()
                old = sorted(range(n - recent), key=lambda t: (is_nan[t], -x[t], t))
                kept = sorted(old[:budget - recent]) + list(range(n - recent, n))
            keep[b, g, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
    return lens.clamp(max=budget), keep


def evict_apply(kp, vp, weights, table, lens, budget, recent, table_out=None, weights_out=None):
    """What attn_cache_evict leaves in (kpages, vpages, weights_out), and (newlens, keep)."""
    newlens, keep = evict(weights, lens, budget, recent)
    in_place = table_out is None
    table_out = table if in_place else table_out
    w_out = weights.clone() if weights_out is None else weights_out.clone()
    nk, nv = kp.clone(), vp.clone()
    page = kp.shape[2]
    for b, n in enumerate(lens.tolist()):
        m = int(newlens[b])
        for g in range(kp.shape[1]):
            kept = keep[b, g, :m].tolist()
            for i, t in enumerate(kept):
                for new, old in ((nk, kp), (nv, vp)):
                    new[table_out[b, i // page], g, i % page] = old[table[b, t // page], g, t % page]
            w_out[b, g, :m] = weights[b, g][kept]
            w_out[b, g, m:min(n, w_out.shape[2])] = 0
    return nk, nv, w_out, newlens, keep
