"""The paged key-value cache on the GPU: append, decode, key weights and
eviction against their definitions in 64 bits (tests/paged_ref.py).  Rows that
hold no key are NaN or infinite and unused table entries are not page numbers,
so any use of either shows."""
import math
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import causal_head_self_gb300 as chs
import paged_ref as ref
from causal_head_self_gb300 import build as _build
from causal_head_self_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def gpu(*xs):
    return [x.to("cuda") for x in xs]


def same_bits(a, b):
    """Equal as bit patterns (NaN rows included)."""
    a, b = a.cpu(), b.cpu()
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.view(kind), b.view(kind))


def status_ok():
    assert chs.attn_status() == chs.ATTN_OK


def queries(B, Hq, Dh, seed):
    gen = torch.Generator().manual_seed(seed + 101)
    return torch.randn((B, Hq, 1, Dh), generator=gen).to(torch.bfloat16)


# ---------------------------------------------------------------- append

# (Hkv, Dh, page, cols, S, lengths after, new rows or None for all)
APPEND = [
    (2, 64, 8, 5, 1, [1, 8, 9, 40], None),
    (1, 128, 16, 4, 1, [0, 17, 64], [0, 1, 1]),
    (3, 256, 24, 3, 7, [7, 30, 72, 0, 24], [7, 5, 0, 0, 1]),
    (8, 128, 64, 3, 130, [130, 192, 131], None),
    (2, 64, 128, 2, 200, [200, 250, 3], [200, 1, 3]),
    (4, 64, 16, 300, 4100, [4100, 4800], [4099, 4100]),   # more rows than a wave takes
]


@pytest.mark.parametrize("Hkv,Dh,page,cols,S,lens,new", APPEND)
def test_append_writes_its_rows_and_nothing_else(Hkv, Dh, page, cols, S, lens, new):
    B = len(lens)
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=S)
    gen = torch.Generator().manual_seed(S)
    k, v = (torch.randn((B, Hkv, S, Dh), generator=gen).to(torch.bfloat16) for _ in range(2))
    nl = None if new is None else torch.tensor(new, dtype=torch.int32)
    dk, dv, dkp, dvp, dt, dsl = gpu(k, v, kp, vp, table, sl)
    chs.attn_paged_append(dk, dv, dkp, dvp, dt, dsl, None if nl is None else nl.cuda())
    status_ok()
    for b, n in enumerate(lens):
        m = (S if new is None else new[b]) if n else 0
        for i in range(m):
            t = n - m + i
            kp[table[b, t // page], :, t % page] = k[b, :, i]
            vp[table[b, t // page], :, t % page] = v[b, :, i]
    assert same_bits(dkp, kp) and same_bits(dvp, vp)


def test_append_reports_impossible_lengths_and_pages():
    kp, vp, table, sl = gpu(*ref.make_cache([5, 5, 5, 5], 1, 64, 8, 2, seed=0))
    k = torch.zeros(4, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    before = kp.clone()
    bad = [([5, 5, 5, 17], None), ([5, 5, 5, -1], None), ([5, 5, 5, 2], None),
           ([5, 5, 5, 5], [0, 0, 0, 4]), ([5, 5, 5, 5], [0, 0, 0, -1])]
    for lens, new in bad:
        chs.attn_paged_append(k, k, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              torch.tensor(new or [0, 0, 0, 3], dtype=torch.int32, device="cuda"))
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
        assert same_bits(kp, before)
    for page in (-1, kp.shape[0]):
        t = table.clone()
        t[2, 0] = page
        chs.attn_paged_append(k, k, kp, vp, t, sl, torch.tensor([0, 0, 3, 0], dtype=torch.int32,
                                                                device="cuda"))
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
        assert same_bits(kp, before)


# ---------------------------------------------------------------- decode

# (Hq, Hkv, Dh, page, cols, lengths, window)
DECODE = [
    (4, 4, 64, 8, 4, [0, 1, 7, 8, 9, 32], 0),             # one query head per K/V head
    (8, 2, 128, 16, 40, [1, 127, 128, 129, 640], 0),      # tiles end at, before and after a length
    (8, 2, 128, 16, 40, [600, 0, 300, 0, 0, 13], 0),      # empty slots between
    (4, 1, 256, 32, 12, [1, 63, 64, 65, 384], 0),
    (4, 2, 64, 24, 30, [719, 100, 24, 25], 0),            # pages of no power of two
    (4, 2, 128, 40, 9, [360, 41], 0),
    (8, 1, 256, 72, 5, [300, 73], 0),
    (2, 1, 128, 128, 3, [384, 129], 0),
    (2, 1, 64, 256, 2, [257, 512, 3], 0),                 # several tiles per page
    (2, 2, 128, 1000, 1, [777, 1000], 0),                 # a linear cache
    (32, 1, 128, 16, 30, [480, 33], 0),                   # 32 heads: four copies fill the rows
    (33, 1, 128, 16, 20, [300, 1], 0),                    # past it: one copy
    (64, 1, 64, 16, 20, [320, 129], 0),
    (128, 1, 128, 16, 12, [190, 64], 0),
    (160, 1, 64, 8, 30, [240, 5], 0),                     # two row blocks
    (96, 2, 256, 16, 16, [256, 70], 0),
    (8, 2, 128, 16, 40, [640, 200, 128, 129, 130], 1),    # windows: one key,
    (8, 2, 128, 16, 40, [640, 200, 128, 129, 0], 128),    # a tile,
    (4, 1, 64, 8, 50, [400, 77, 390], 77),                # odd,
    (4, 1, 256, 24, 20, [480, 100, 65], 65),
    (4, 4, 128, 16, 12, [190, 5], 1000),                  # wider than the sequence
    (40, 1, 128, 16, 30, [480, 470], 200),
]


@pytest.mark.parametrize("Hq,Hkv,Dh,page,cols,lens,window", DECODE)
def test_decode_matches_the_definition(Hq, Hkv, Dh, page, cols, lens, window):
    first = [n - window if window else 0 for n in lens]   # pages before the window are gone too
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=Hq + page, first_used=first)
    q = queries(len(lens), Hq, Dh, seed=page)
    o, tol, w, rtol = ref.decode(q, kp, vp, table, sl, window=window)
    args = gpu(q, kp, vp, table, sl)
    got = chs.attn_decode_paged(*args, window=window)
    status_ok()
    assert ((got.cpu().double() - o).abs() <= tol).all()
    # the same with the step's weights: replaced, then added to
    T = cols * page
    weights = torch.full((len(lens), Hkv, T + 3), 7.0, device="cuda")
    again = chs.attn_decode_paged(*args, window=window, weights=weights, accumulate=False)
    status_ok()
    assert same_bits(again, got)
    for accumulate in (False, True):
        if accumulate:
            chs.attn_decode_paged(*args, window=window, weights=weights)
            status_ok()
        # one more 32-bit rounding of the sum for the addition
        want = (2 if accumulate else 1) * w
        x = weights.cpu().double()
        for b, n in enumerate(lens):
            assert ((x[b, :, :n] - want[b, :, :n]).abs() <= (rtol + 2.0 ** -24) * want[b, :, :n]).all()
            assert (x[b, :, n:] == 7.0).all()   # behind the sequence: left alone


def widen(table, page, rows=13000):
    """The table with unused columns behind it, for more keys than a short step holds."""
    more = -(-rows // page) - table.shape[1]
    return torch.cat([table, torch.full((table.shape[0], more), -1, dtype=torch.int32)], 1)


@pytest.mark.parametrize("Hq,Hkv,Dh,page,cols,lens,window", DECODE)
def test_decode_with_a_wide_table_matches_the_definition(Hq, Hkv, Dh, page, cols, lens, window):
    first = [n - window if window else 0 for n in lens]
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=Hq + page, first_used=first)
    q = queries(len(lens), Hq, Dh, seed=page)
    o, tol, w, rtol = ref.decode(q, kp, vp, table, sl, window=window)
    args = gpu(q, kp, vp, widen(table, page), sl)
    got = chs.attn_decode_paged(*args, window=window)
    weights = torch.full((len(lens), Hkv, args[3].shape[1] * page), 7.0, device="cuda")
    again = chs.attn_decode_paged(*args, window=window, weights=weights, accumulate=False)
    status_ok()
    assert same_bits(again, got)
    assert ((got.cpu().double() - o).abs() <= tol).all()
    x = weights.cpu().double()
    for b, n in enumerate(lens):
        assert ((x[b, :, :n] - w[b, :, :n]).abs() <= (rtol + 2.0 ** -24) * w[b, :, :n]).all()
        assert (x[b, :, n:] == 7.0).all()


def test_decode_with_a_scale_and_large_scores():
    # scores of about +-1000: only the largest weights survive, none overflows
    lens = [300, 129]
    kp, vp, table, sl = ref.make_cache(lens, 2, 128, 16, 20, seed=3)
    q = queries(2, 8, 128, seed=4) * 8
    o, _, w, _ = ref.decode(q, kp, vp, table, sl, scale=1.5)
    weights = torch.zeros(2, 2, 320, device="cuda")
    got = chs.attn_decode_paged(*gpu(q, kp, vp, table, sl), scale=1.5, weights=weights)
    status_ok()
    # a score of size c is off by up to Dh 2^-23 c, and a weight by e to that:
    # c <= 1.5 * 128 * 8 * 4.5^2 bounds |q| |k| far above, so take the sum's own size
    c = 1.5 * float((q.double().abs().amax() * 4.5 * 128))
    rel = math.expm1(2 * 128 * 2.0 ** -23 * c)
    assert ((weights.cpu().double() - w).abs() <= rel * w + 1e-30).all()
    top = o.abs().amax()
    assert ((got.cpu().double() - o).abs() <= (2 * ref.HALF_BF16 + rel) * 4 * top).all()


def test_decode_of_a_linear_cache_agrees_with_attn_decode():
    q, kc, vc, sl = gpu(*inputs.decode_inputs(3, 8, 2, 640, 128, 1, 640, seed=5))
    table = torch.arange(3, dtype=torch.int32, device="cuda").view(3, 1)
    a = chs.attn_decode(q, kc, vc, sl, window=200).double()
    b = chs.attn_decode_paged(q, kc, vc, table, sl, window=200).double()
    status_ok()
    # both within 2 roundings of |v| <= 6 of the exact result
    assert ((a - b).abs() <= 2 * 2 * ref.HALF_BF16 * 6).all()


def test_decode_of_one_sequence_over_every_multiprocessor():
    # a long sequence is cut into one share per CTA; a ragged batch beside it
    q, kc, vc, sl = inputs.decode_inputs(4, 8, 2, 16384, 64, 1, 16384, seed=6)
    sl[0], sl[2] = 16384, 1
    dq, dk, dv, dsl = gpu(q, kc, vc, sl)
    order = torch.randperm(4 * 1024, generator=torch.Generator().manual_seed(1))
    pk, pv = (torch.empty(4096, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for pool, c in ((pk, dk), (pv, dv)):
        pool[order.cuda()] = c.view(4, 2, 1024, 16, 64).transpose(1, 2).reshape(4096, 2, 16, 64)
    table = order.to(torch.int32).view(4, 1024).cuda()
    got = chs.attn_decode_paged(dq, pk, pv, table, dsl).cpu().double()
    status_ok()
    for b, n in enumerate(sl.tolist()):
        for h in range(8):
            p = torch.softmax(q[b, h, 0].double() @ kc[b, h // 4, :n].double().t() / 8, -1)
            v = vc[b, h // 4, :n].double()
            tol = ref.HALF_BF16 * ((p @ v).abs() + p @ v.abs()) + 2.0 ** -12 * (p @ v.abs())
            assert ((got[b, h, 0] - p @ v).abs() <= tol).all()


def test_decode_of_many_short_sequences():
    lens = [(7 * b) % 40 for b in range(150)]   # more units than CTAs, empty ones among them
    kp, vp, table, sl = ref.make_cache(lens, 2, 64, 8, 5, seed=8)
    q = queries(150, 4, 64, seed=9)
    o, tol, w, rtol = ref.decode(q, kp, vp, table, sl)
    weights = torch.zeros(150, 2, 40, device="cuda")
    got = chs.attn_decode_paged(*gpu(q, kp, vp, table, sl), weights=weights, accumulate=False)
    status_ok()
    assert ((got.cpu().double() - o).abs() <= tol).all()
    assert ((weights.cpu().double() - w).abs() <= rtol * w).all()


def test_decode_reports_impossible_lengths_and_pages():
    lens = [20, 30, 40]
    kp, vp, table, sl = ref.make_cache(lens, 2, 64, 8, 5, seed=10)
    q = queries(3, 4, 64, seed=11)
    o, tol, _, _ = ref.decode(q, kp, vp, table, sl)
    dq, dk, dv, dt, dsl = gpu(q, kp, vp, table, sl)
    for n in (-1, 41, 2 ** 31 - 1, -(2 ** 31)):
        bad = dsl.clone()
        bad[1] = n
        got = chs.attn_decode_paged(dq, dk, dv, dt, bad).cpu().double()
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
        assert (got[1] == 0).all()                                       # that sequence alone
        assert ((got - o).abs() <= tol)[[0, 2]].all()
    for page in (-1, kp.shape[0], 2 ** 31 - 1):
        bad = dt.clone()
        bad[2, 1] = page
        chs.attn_decode_paged(dq, dk, dv, bad, dsl)
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
    chs.attn_decode_paged(dq, dk, dv, dt, dsl)
    status_ok()


def test_pool_offsets_past_32_bits():
    # 2^31 elements and more in each pool: the last pages lie past a 32-bit offset
    P, Hkv, page, Dh = 2 ** 31 // (8 * 64 * 128) + 40, 8, 64, 128
    kp, vp = (torch.zeros(P, Hkv, page, Dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 31
    table = torch.arange(P - 6, P, dtype=torch.int32, device="cuda").view(2, 3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((2, Hkv, 150, Dh), generator=gen, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    sl = torch.tensor([150, 150], dtype=torch.int32, device="cuda")
    chs.attn_paged_append(k, v, kp, vp, table, sl)
    status_ok()
    q = queries(2, 8, Dh, seed=12).cuda()
    got = chs.attn_decode_paged(q, kp, vp, table, sl).double()
    status_ok()
    p = torch.softmax(torch.einsum("bhd,bhtd->bht", q[:, :, 0].double(), k.double()) * Dh ** -0.5, -1)
    o = torch.einsum("bht,bhtd->bhd", p, v.double())[:, :, None]
    a = torch.einsum("bht,bhtd->bhd", p, v.double().abs())[:, :, None]
    assert ((got - o).abs() <= ref.HALF_BF16 * (o.abs() + a) + 2.0 ** -12 * a).all()
    w = torch.rand(2, Hkv, 192, device="cuda", generator=gen)
    to = torch.arange(P - 8, P - 6, dtype=torch.int32, device="cuda").view(2, 1)
    newlens, keep = chs.attn_cache_evict(kp, vp, w, table, sl, 40, 10, table_out=to)
    status_ok()
    for b in range(2):
        for g in range(Hkv):
            assert torch.equal(kp[P - 8 + b, g, :40], k[b, g, keep[b, g].long()])
            assert torch.equal(vp[P - 8 + b, g, :40], v[b, g, keep[b, g].long()])


# ---------------------------------------------------------------- key weights

# (Hq, Hkv, S, Dh, lengths, queries, causal, window)
KEY_WEIGHTS = [
    (2, 2, 1, 64, [1], 0, True, 0),
    (4, 2, 129, 128, [129, 128, 1, 0], 0, True, 0),
    (4, 1, 300, 64, [300, 77], 0, True, 0),
    (2, 1, 260, 256, [260, 131], 0, True, 0),
    (8, 2, 400, 128, [400, 399, 20], 1, True, 0),         # only the last query votes
    (8, 2, 400, 128, [400, 399, 20], 32, True, 0),
    (4, 4, 333, 64, [333, 200], 150, True, 0),
    (4, 2, 400, 128, [400, 140], 0, True, 1),             # each query sees itself alone
    (4, 2, 400, 128, [400, 140], 0, True, 100),
    (4, 2, 400, 64, [400, 300], 64, True, 129),           # keys that no voting query sees
    (4, 2, 257, 128, [257, 100], 0, False, 0),
    (4, 2, 257, 256, [257, 100], 17, False, 0),
    (32, 1, 600, 64, [600, 513], 0, True, 0),             # one K/V head: a cluster per item
    (12, 1, 300, 128, [300, 130], 40, True, 0),           # several heads per tile, the last not full
    (5, 1, 300, 256, [300, 299], 64, True, 70),
    (3, 3, 500, 64, [500, 3], 5, True, 0),
    (8, 2, 400, 64, [400, 0, 64, 63, 129], 64, True, 0),  # one tile of 256 voting rows
    (8, 2, 400, 128, [400, 65, 1], 50, True, 0),          # ... with rows that pad each head
    (4, 2, 700, 64, [700, 128, 127], 128, True, 0),
    (6, 2, 300, 128, [300, 200], 16, False, 0),           # 96 rows: one and a half pieces
    (8, 1, 300, 256, [300, 131], 16, True, 0),            # 128 rows, the most at head size 256
    (9, 1, 300, 256, [300, 131], 16, True, 0),            # one head too many for that
    (2, 1, 300, 64, [300, 290], 129, True, 0),
]


@pytest.mark.parametrize("Hq,Hkv,S,Dh,lens,nq,causal,window", KEY_WEIGHTS)
def test_key_weights_match_the_definition(Hq, Hkv, S, Dh, lens, nq, causal, window):
    B = len(lens)
    q, k, _ = inputs.prefill_inputs(B, Hq, Hkv, S, Dh, seed=S + Dh)
    # the log-sum-exps of the real rows, in 64 bits and rounded once; the rows
    # behind the last are NaN in every input
    lse = torch.full((B, Hq, S), math.nan)
    for b, n in enumerate(lens):
        for h in range(Hq if n else 0):
            z = q[b, h, :n].double() @ k[b, h * Hkv // Hq, :n].double().t() / math.sqrt(Dh)
            i, j = torch.arange(n)[:, None], torch.arange(n)[None]
            hidden = (j > i) if causal else torch.zeros(n, n, dtype=torch.bool)
            if window:
                hidden |= j <= i - window
            lse[b, h, :n] = torch.logsumexp(z.masked_fill(hidden, -math.inf), -1).float()
        q[b, :, n:], k[b, :, n:] = math.nan, math.inf
    want, rtol = ref.key_weights(q, k, lse, lens, queries=nq, causal=causal, window=window)
    weights = torch.full((B, Hkv, S + 5), 3.0, device="cuda")
    dq, dk, dl, sl = gpu(q, k, lse, torch.tensor(lens, dtype=torch.int32))
    args = dict(queries=nq, causal=causal, window=window)
    chs.attn_key_weights(dq, dk, dl, weights, sl, accumulate=False, **args)
    status_ok()
    first = weights.clone()
    for b, n in enumerate(lens):
        x = first[b].cpu().double()
        assert ((x[:, :n] - want[b, :, :n]).abs() <= rtol * want[b, :, :n]).all()
        assert (x[:, n:] == 3.0).all()   # behind the sequence: left alone
    chs.attn_key_weights(dq, dk, dl, weights, sl, **args)   # added to
    status_ok()
    for b, n in enumerate(lens):
        assert torch.equal(weights[b, :, :n], first[b, :, :n] + first[b, :, :n])
        assert (weights[b, :, n:] == 3.0).all()


@pytest.mark.parametrize("B,Hq,Hkv,S,Dh,nq,window", [
    (3, 32, 8, 2500, 64, 0, 0),          # CTAs walk several items
    (2, 16, 8, 1900, 256, 0, 500),
    (8, 32, 32, 1030, 128, 33, 0),
    (1, 8, 8, 2000, 128, 0, 0),          # a cluster of two per item
    (1, 8, 1, 4000, 64, 0, 0),
    (6, 32, 8, 5000, 64, 64, 0),         # queries that stay: shares of several units
    (3, 16, 8, 3000, 256, 60, 0),
    (7, 8, 8, 1024, 128, 7, 0),
])
def test_key_weights_of_many_tiles(B, Hq, Hkv, S, Dh, nq, window):
    gen = torch.Generator(device="cuda").manual_seed(S)
    q = torch.randn((B, Hq, S, Dh), generator=gen, device="cuda").to(torch.bfloat16)
    k = torch.randn((B, Hkv, S, Dh), generator=gen, device="cuda").to(torch.bfloat16)
    lens = [S - 137 * b for b in range(B)]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # any normaliser will do: the true ones, in 32 bits
    _, lse = chs.attn_fwd_lse(q, k, k, window=window)
    w = torch.zeros(B, Hkv, S, device="cuda")
    chs.attn_key_weights(q, k, lse, w, sl, queries=nq, window=window)
    status_ok()
    again = torch.zeros_like(w)
    chs.attn_key_weights(q, k, lse, again, sl, queries=nq, window=window, accumulate=False)
    assert same_bits(w, again)
    j = torch.arange(S, device="cuda")
    for b, n in enumerate(lens):
        i = torch.arange(max(0, n - nq) if nq else 0, n, device="cuda")[:, None]
        seen = (j[:n] <= i) & ((j[:n] > i - window) if window else True)
        want = torch.zeros(Hkv, n, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            z = q[b, h, i[:, 0]].double() @ k[b, h * Hkv // Hq, :n].double().t() * Dh ** -0.5
            p = torch.exp(z - lse[b, h, i].double())
            want[h * Hkv // Hq] += torch.where(seen, p, 0.0).sum(0)
        # as in paged_ref.key_weights with |q| . |k| <= 6 Dh and |lse| <= 20
        rel = (Dh + 1) * 2.0 ** -23 * (6 * Dh ** 0.5 + 20) + 2.0 ** -18
        assert ((w[b, :, :n].double() - want).abs() <= rel * want).all()
        assert (w[b, :, n:] == 0).all()


def test_key_weights_of_a_whole_prompt_from_its_forward_pass():
    # every query's weights sum to 1, so a head group's sum to G S
    B, Hq, Hkv, S, Dh = 2, 8, 2, 700, 128
    q, k, v = gpu(*inputs.prefill_inputs(B, Hq, Hkv, S, Dh, seed=31))
    _, lse = chs.attn_fwd_lse(q, k, v)
    weights = torch.zeros(B, Hkv, S, device="cuda")
    chs.attn_key_weights(q, k, lse, weights)
    status_ok()
    total = weights.double().sum(-1)
    # the forward's log-sum-exp is in 32 bits, of scores in 32 bits (see above)
    assert ((total / (Hq // Hkv * S) - 1).abs() <= 2 * (128 + 1) * 2.0 ** -23 * 20 + 2.0 ** -17).all()


def test_key_weights_of_many_sequences():
    # more sequences than a CTA keeps lengths of; most of them short or empty
    B, Hq, Hkv, S, Dh = 300, 2, 1, 130, 64
    lens = [(37 * b) % 131 for b in range(B)]
    q, k, _ = inputs.prefill_inputs(B, Hq, Hkv, S, Dh, seed=9)
    lse = torch.full((B, Hq, S), 5.0)
    want, rtol = ref.key_weights(q, k, lse, lens)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, Hkv, S, device="cuda")
    chs.attn_key_weights(*gpu(q, k, lse), w, sl)
    status_ok()
    assert ((w.cpu().double() - want).abs() <= rtol * want).all()
    want, rtol = ref.key_weights(q, k, lse, lens, queries=9)
    w.zero_()
    chs.attn_key_weights(*gpu(q, k, lse), w, sl, queries=9)
    status_ok()
    assert ((w.cpu().double() - want).abs() <= rtol * want).all()


def test_key_weights_offsets_past_32_bits():
    # queries of 2^31 elements: the last head's lie past a 32-bit offset
    B, Hq, Hkv, S, Dh, nq = 2, 256, 2, 32768, 128, 16
    q = torch.empty(B, Hq, S, Dh, dtype=torch.bfloat16, device="cuda")
    assert q.numel() >= 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(4)
    q[:, :, S - nq:] = torch.randn((B, Hq, nq, Dh), generator=gen, device="cuda").to(torch.bfloat16)
    k = torch.randn((B, Hkv, S, Dh), generator=gen, device="cuda").to(torch.bfloat16)
    lse = torch.full((B, Hq, S), 10.0, device="cuda")
    w = torch.zeros(B, Hkv, S, device="cuda")
    chs.attn_key_weights(q, k, lse, w, queries=nq)
    status_ok()
    i = torch.arange(S - nq, S, device="cuda")[:, None]
    for g in range(Hkv):
        want = torch.zeros(S, dtype=torch.float64, device="cuda")
        for h in range(g * 128, g * 128 + 128):
            p = torch.exp(q[1, h, S - nq:].double() @ k[1, g].double().t() * Dh ** -0.5 - 10)
            want += torch.where(torch.arange(S, device="cuda") <= i, p, 0.0).sum(0)
        rel = (Dh + 1) * 2.0 ** -23 * (6 * Dh ** 0.5 + 10) + 2.0 ** -18   # (as above)
        assert ((w[1, g].double() - want).abs() <= rel * want).all()


def test_key_weights_report_impossible_lengths():
    q, k, _ = gpu(*inputs.prefill_inputs(2, 2, 2, 140, 64, seed=1))
    lse = torch.zeros(2, 2, 140, device="cuda")
    for n in (-1, 141):
        w = torch.full((2, 2, 140), 5.0, device="cuda")
        chs.attn_key_weights(q, k, lse, w, torch.tensor([n, 0], dtype=torch.int32, device="cuda"))
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
        assert (w == 5.0).all()


# ---------------------------------------------------------------- eviction

# (Hkv, Dh, page, cols, lengths, budget, recent)
EVICT = [
    (2, 64, 8, 5, [40, 17, 16, 15, 0], 16, 4),
    (1, 128, 16, 20, [320, 100, 300], 100, 0),        # no recent rows
    (2, 64, 16, 10, [160, 31, 30], 30, 30),           # only recent rows
    (3, 256, 24, 8, [190, 1], 1, 0),
    (2, 64, 8, 5, [40, 33], 1, 1),
    (2, 128, 32, 8, [256, 200], 255, 100),            # one row goes
    (1, 64, 64, 80, [5000, 4097, 4096], 1500, 64),    # more than a tile of rows
    (1, 64, 8, 4, [32, 20], 60, 8),                   # a budget past what the table holds
]


@pytest.mark.parametrize("Hkv,Dh,page,cols,lens,budget,recent", EVICT)
@pytest.mark.parametrize("values", ["spread", "ties", "special"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_keeps_the_largest_weights(Hkv, Dh, page, cols, lens, budget, recent, values, in_place):
    B = len(lens)
    cols_out = max(1, -(-min(budget, cols * page) // page))
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=budget, spare=B * cols_out)
    gen = torch.Generator().manual_seed(budget + recent)
    T = cols * page
    w = torch.rand((B, Hkv, T + 2), generator=gen) ** 8
    if values == "ties":
        w = (w * 3).round()                           # 0, 1, 2 and 3 only
    elif values == "special":
        odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, -1.0])
        pick = torch.randint(0, 14, w.shape, generator=gen)
        w = torch.where(pick < 7, odd[pick.clamp(max=6)], w)
    used = set(table.flatten().tolist())
    free = [x for x in range(kp.shape[0]) if x not in used]
    to = None if in_place else torch.tensor(free[:B * cols_out], dtype=torch.int32).view(B, cols_out)
    w_out = None if in_place else torch.full((B, Hkv, min(budget, T) + 1), 9.0)
    want = ref.evict_apply(kp, vp, w, table, sl, budget, recent, to, w_out)
    dkp, dvp, dw, dt, dsl = gpu(kp, vp, w, table, sl)
    dto, dwo = (None, None) if in_place else gpu(to, w_out)
    newlens, keep = chs.attn_cache_evict(dkp, dvp, dw, dt, dsl, budget, recent, table_out=dto,
                                         weights_out=dwo)
    status_ok()
    assert same_bits(newlens, want[3]) and same_bits(keep, want[4])
    assert same_bits(dkp, want[0]) and same_bits(dvp, want[1])
    got_w = dw if in_place else dwo
    # (a kept -0 keeps its sign)
    assert same_bits(got_w, want[2])
    if not in_place:
        assert same_bits(dw, w)


# rows that fit in a block's shared memory, and more; clustered values, so that
# every digit decides, and equal ones
@pytest.mark.parametrize("n,budget,recent,steps", [(70001, 20000, 1000, 4000), (45056, 9000, 0, 9),
                                                   (45041, 45040, 7, 1), (60000, 1, 0, 2 ** 20)])
def test_evict_of_long_sequences_matches_a_sort(n, budget, recent, steps):
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = -(-n // 16)
    w = 1.0 + torch.randint(0, steps, (1, 2, 16 * pages), generator=gen, device="cuda") * 2.0 ** -23
    kp, vp = (torch.randn(pages, 2, 16, 64, generator=gen, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    k0 = kp.clone()
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(1, pages)
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    w0 = w.clone()
    newlens, keep = chs.attn_cache_evict(kp, vp, w, table, sl, budget, recent)
    status_ok()
    assert newlens.tolist() == [budget]
    for g in range(2):
        top = w0[0, g, :n - recent].sort(descending=True, stable=True).indices[:budget - recent]
        want = torch.cat([top.sort().values, torch.arange(n - recent, n, device="cuda")])
        assert torch.equal(keep[0, g].long(), want)
        assert torch.equal(w[0, g, :budget], w0[0, g, want]) and (w[0, g, budget:n] == 0).all()
        assert torch.equal(w[0, g, n:], w0[0, g, n:])
        i = torch.arange(budget, device="cuda")
        assert torch.equal(kp[table[0, i // 16].long(), g, i % 16],
                           k0[table[0, want // 16].long(), g, want % 16])


def test_evict_reports_impossible_lengths_and_pages():
    kp, vp, table, sl = gpu(*ref.make_cache([40, 30], 1, 64, 8, 5, seed=10))
    w = torch.rand(2, 1, 40, device="cuda")
    before, w0 = kp.clone(), w.clone()
    for n in (-1, 41):
        bad = torch.tensor([n, 0], dtype=torch.int32, device="cuda")
        newlens, keep = chs.attn_cache_evict(kp, vp, w, table, bad, 16, 4)
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
        assert same_bits(kp, before) and torch.equal(w, w0) and (keep == -1).all()
    for page in (-1, kp.shape[0]):
        bad = table.clone()
        bad[1, 0] = page
        chs.attn_cache_evict(kp.clone(), vp.clone(), w.clone(), bad, sl, 16, 4)
        assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG


# ---------------------------------------------------------------- together

def test_prompt_decode_and_eviction_together():
    """A padded batch as a server runs it: the prompts' forward pass, their keys'
    weights, the cache filled and cut back, then decode steps that append, attend
    and add to the weights, and a second eviction in place."""
    B, Hq, Hkv, Dh, S, page, budget, recent = 3, 8, 2, 128, 300, 16, 128, 32
    prompt = [300, 211, 90]
    q, k, v = inputs.prefill_inputs(B, Hq, Hkv, S, Dh, seed=77)
    dq, dk, dv = gpu(q, k, v)
    sl = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    _, lse = chs.attn_fwd_lse(dq, dk, dv)
    cols = -(-S // page)
    kp, vp = (torch.full((2 * B * cols, Hkv, page, Dh), math.nan, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    order = torch.randperm(2 * B * cols, generator=torch.Generator().manual_seed(5)).to(torch.int32)
    table, small = (x.view(B, cols).cuda() for x in order.chunk(2))
    weights, w_out = (torch.zeros(B, Hkv, cols * page, device="cuda") for _ in range(2))
    chs.attn_key_weights(dq, dk, lse, weights, sl, queries=100)
    chs.attn_paged_append(dk, dv, kp, vp, table, sl, sl)
    new, keep = chs.attn_cache_evict(kp, vp, weights, table, sl, budget, recent, table_out=small,
                                     weights_out=w_out)
    status_ok()
    # the reference's own cache: per (sequence, head) lists of rows
    want_new, want_keep = ref.evict(weights.cpu(), sl.cpu(), budget, recent)
    assert same_bits(new, want_new) and same_bits(keep, want_keep)
    K = [[[k[b, g, t] for t in want_keep[b, g, :want_new[b]]] for g in range(Hkv)] for b in range(B)]
    V = [[[v[b, g, t] for t in want_keep[b, g, :want_new[b]]] for g in range(Hkv)] for b in range(B)]
    W = [[[float(weights[b, g, t]) for t in want_keep[b, g, :want_new[b]]] for g in range(Hkv)]
         for b in range(B)]
    lens = new
    gen = torch.Generator().manual_seed(6)
    for step in range(40):
        lens = lens + 1
        k1, v1 = (torch.randn((B, Hkv, 1, Dh), generator=gen).to(torch.bfloat16) for _ in range(2))
        q1 = torch.randn((B, Hq, 1, Dh), generator=gen).to(torch.bfloat16)
        chs.attn_paged_append(k1.cuda(), v1.cuda(), kp, vp, small, lens)
        o = chs.attn_decode_paged(q1.cuda(), kp, vp, small, lens, weights=w_out)
        for b in range(B):
            for g in range(Hkv):
                K[b][g].append(k1[b, g, 0])
                V[b][g].append(v1[b, g, 0])
                p = torch.softmax(q1[b, 4 * g:4 * g + 4, 0].double() @ torch.stack(K[b][g]).double().t()
                                  / math.sqrt(Dh), -1)
                vv = torch.stack(V[b][g]).double()
                got = o[b, 4 * g:4 * g + 4, 0].cpu().double()
                a = p @ vv.abs()
                assert ((got - p @ vv).abs() <= ref.HALF_BF16 * ((p @ vv).abs() + a) + 2.0 ** -12 * a).all()
                W[b][g] = [x + y for x, y in zip(W[b][g] + [0.0], p.sum(0).tolist())]
    status_ok()
    for b in range(B):
        for g in range(Hkv):
            n = int(lens[b])
            x = w_out[b, g, :n].cpu().double()
            # each step adds a weight that is right to 2^-12 and rounds once
            assert ((x - torch.tensor(W[b][g])).abs() <= (2.0 ** -12 + 40 * 2.0 ** -24) * x).all()
    before = w_out.clone()
    new, keep = chs.attn_cache_evict(kp, vp, w_out, small, lens, budget, recent)
    status_ok()
    want_new, want_keep = ref.evict(before.cpu(), lens.cpu(), budget, recent)
    assert same_bits(new, want_new) and same_bits(keep, want_keep)
    for b in range(B):
        for g in range(Hkv):
            for i, t in enumerate(want_keep[b, g, :want_new[b]].tolist()):
                at = small[b, i // page], g, i % page
                assert torch.equal(kp[at].cpu(), K[b][g][t]) and torch.equal(vp[at].cpu(), V[b][g][t])


def _step(s):
    chs.attn_paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["sl"])
    chs.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["sl"], s["o"], weights=s["w"],
                          accumulate=False)
    chs.attn_cache_evict(s["kp"], s["vp"], s["w"], s["table"], s["sl"], 48, 8, table_out=s["to"],
                         weights_out=s["wo"], newlens=s["new"], keep=s["keep"])


def _state(seed, lens, Hq=8, Hkv=2, Dh=128, page=16, cols=40):
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed, spare=8 * len(lens))
    used = set(table.flatten().tolist())
    free = [x for x in range(kp.shape[0]) if x not in used][:3 * len(lens)]
    B = len(lens)
    gen = torch.Generator().manual_seed(seed)
    s = dict(kp=kp, vp=vp, table=table, sl=sl, q=queries(B, Hq, Dh, seed),
             k=torch.randn((B, Hkv, 1, Dh), generator=gen).to(torch.bfloat16),
             v=torch.randn((B, Hkv, 1, Dh), generator=gen).to(torch.bfloat16),
             o=torch.zeros(B, Hq, 1, Dh, dtype=torch.bfloat16), w=torch.zeros(B, Hkv, cols * page),
             wo=torch.zeros(B, Hkv, cols * page), to=torch.tensor(free, dtype=torch.int32).view(B, 3),
             new=torch.zeros(B, dtype=torch.int32), keep=torch.zeros(B, Hkv, 48, dtype=torch.int32))
    return {k: v.cuda() for k, v in s.items()}


def _all_same(a, b):
    return all(same_bits(a[k], b[k]) for k in a)


def test_graphs_replay_bit_for_bit_and_share_nothing():
    lens = [[600, 64, 30], [100, 640, 5]]
    eager = [_state(i, x) for i, x in enumerate(lens)]
    states = [_state(i, x) for i, x in enumerate(lens)]
    for s in eager:
        _step(s)
    status_ok()
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(s)
        graphs.append(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):   # both at once, on two streams
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    status_ok()
    assert all(_all_same(a, b) for a, b in zip(states, eager))


def test_calls_on_two_streams_at_once():
    lens = [[640, 300, 77], [400, 1, 639]]
    eager = [_state(10 + i, x) for i, x in enumerate(lens)]
    states = [_state(10 + i, x) for i, x in enumerate(lens)]
    for s in eager:
        _step(s)
    streams = [torch.cuda.Stream() for _ in lens]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(states, streams):
            with torch.cuda.stream(stream):
                _step(s)
    # an explicit stream takes its allocations there too
    outs = [chs.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["sl"], stream=stream)
            for s, stream in zip(states, streams)]
    torch.cuda.synchronize()
    status_ok()
    assert all(_all_same(a, b) for a, b in zip(states, eager))
    assert all(same_bits(o, s["o"]) for o, s in zip(outs, eager))


@pytest.mark.parametrize("B,Hq,Hkv,S,Dh,queries,window", [
    (50, 40, 8, 663, 64, 6, 83), (60, 24, 8, 1283, 64, 7, 171), (120, 8, 8, 280, 256, 38, 25),
    (100, 8, 8, 512, 256, 126, 13), (33, 3, 3, 2493, 128, 12, 15), (188, 33, 3, 150, 128, 70, 8)])
def test_key_weights_where_most_keys_have_no_query(B, Hq, Hkv, S, Dh, queries, window):
    # long runs of key blocks without a tile, between blocks that have some
    gen = torch.Generator(device="cuda").manual_seed(S)
    q, k = (torch.randn((B, h, S, Dh), generator=gen, device="cuda").to(torch.bfloat16)
            for h in (Hq, Hkv))
    lse = torch.randn((B, Hq, S), generator=gen, device="cuda") + 6
    sl = torch.randint(0, S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.full((B, Hkv, S), 3.0, device="cuda")
    chs.attn_key_weights(q, k, lse, w, sl, queries=queries, window=window, accumulate=False)
    status_ok()
    worst = 0.0
    for b, n in enumerate(sl.tolist()):
        first = max(0, n - queries)
        lo = max(0, first - window + 1)   # the first key that any of them sees
        assert (w[b, :, n:] == 3.0).all() and (w[b, :, :min(lo, n)] == 0.0).all()
        i, j = (torch.arange(x, n, device="cuda") for x in (first, lo))
        seen = (j <= i[:, None]) & (j > i[:, None] - window)
        kg = k[b, :, lo:n].double().repeat_interleave(Hq // Hkv, 0)
        qh = q[b, :, first:n].double()
        p = torch.exp(qh @ kg.transpose(1, 2) * Dh ** -0.5 - lse[b, :, first:n, None].double())
        want = torch.where(seen, p, 0.0).sum(1).view(Hkv, Hq // Hkv, -1).sum(1)
        # (paged_ref.key_weights' bound, with |q| . |k| / sqrt(Dh) <= 6 sqrt(Dh) and |lse| <= 12)
        rel = (Dh + 1) * 2.0 ** -23 * (6 * Dh ** 0.5 + 12) + 2.0 ** -18
        assert ((w[b, :, lo:n].double() - want).abs() <= rel * want).all()


@pytest.mark.parametrize("queries,Hq", [(0, 8), (40, 8), (40, 40)])
def test_key_weights_replay_bit_for_bit_on_two_streams(queries, Hq):
    B, Hkv, S, Dh = 2, 2, 700, 64
    q, k, v = gpu(*inputs.prefill_inputs(B, Hq, Hkv, S, Dh, seed=31))
    sl = torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    _, lse = chs.attn_fwd_lse(q, k, v)
    weights = torch.zeros(3, B, Hkv, S, device="cuda")
    for _ in range(3):
        chs.attn_key_weights(q, k, lse, weights[0], sl, queries=queries)
    graphs = []
    for w in weights[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chs.attn_key_weights(q, k, lse, w, sl, queries=queries)
        graphs.append(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):   # both at once; each replay adds
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    status_ok()
    assert weights[0].any() and all(same_bits(w, weights[0]) for w in weights[1:])


@pytest.mark.parametrize("Hq", [4, 40])
def test_sequences_may_share_pages(Hq):
    # a common prefix, and one page again and again
    lens, Hkv, Dh, page, cols = [200, 150, 96], 1, 128, 16, 13
    kp, vp, table, sl = gpu(*ref.make_cache(lens, Hkv, Dh, page, cols, seed=3))
    table[1, :6] = table[0, :6]
    table[2, :6] = table[0, 0]
    q = queries(3, Hq, Dh, seed=4).cuda()
    w = torch.zeros(3, Hkv, cols * page, device="cuda")
    got = chs.attn_decode_paged(q, kp, vp, table, sl, weights=w)
    # the same rows in pages of their own
    own = torch.arange(3 * cols, dtype=torch.int32, device="cuda").view(3, cols)
    used = torch.arange(cols, device="cuda") * page < sl[:, None]
    at = torch.where(used, table, 0).long().flatten()
    w2 = torch.zeros_like(w)
    want = chs.attn_decode_paged(q, kp[at].contiguous(), vp[at].contiguous(), own, sl, weights=w2)
    status_ok()
    assert same_bits(got, want) and same_bits(w, w2)


def test_empty_batches():
    kp, vp, table, sl = gpu(*ref.make_cache([5], 2, 64, 8, 2, seed=0))
    none, no_lens = table[:0], sl[:0]
    q = torch.zeros(0, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    kv, w = torch.zeros(0, 2, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 2, 16).cuda()
    before = kp.clone()
    assert chs.attn_decode_paged(q, kp, vp, none, no_lens, weights=w).shape == q.shape
    chs.attn_paged_append(kv, kv, kp, vp, none, no_lens)
    chs.attn_paged_append(torch.zeros(1, 2, 0, 64, dtype=torch.bfloat16).cuda(),
                          torch.zeros(1, 2, 0, 64, dtype=torch.bfloat16).cuda(), kp, vp, table, sl)
    new, keep = chs.attn_cache_evict(kp, vp, w, none, no_lens, 4)
    assert new.shape == (0,) and keep.shape == (0, 2, 4)
    chs.attn_key_weights(q, kv, torch.zeros(0, 4, 1, device="cuda"), w, no_lens)
    status_ok()
    assert same_bits(kp, before)


def _wide_state(seed, lens):
    s = _state(seed, lens)
    s["table"] = widen(s["table"].cpu(), 16).cuda()
    for name in ("w", "wo"):
        s[name] = torch.zeros(*s[name].shape[:2], s["table"].shape[1] * 16, device="cuda")
    return s


@pytest.mark.parametrize("B,Hq,Hkv,Dh", [(2, 16, 16, 256), (4, 32, 8, 128), (12, 6, 3, 64), (1, 130, 1, 128)])
def test_asking_for_weights_does_not_change_the_output(B, Hq, Hkv, Dh):
    gen = torch.Generator(device="cuda").manual_seed(Dh)
    page, cols = 64, 220
    kp, vp = (torch.randn((B * cols, Hkv, page, Dh), generator=gen, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    table = torch.randperm(B * cols, generator=gen, device="cuda").to(torch.int32).view(B, cols)
    sl = torch.randint(1, cols * page + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    q = queries(B, Hq, Dh, seed=Dh).cuda()
    weights = torch.zeros(B, Hkv, cols * page, device="cuda")
    o = chs.attn_decode_paged(q, kp, vp, table, sl)
    assert same_bits(o, chs.attn_decode_paged(q, kp, vp, table, sl, weights=weights))
    status_ok()


def test_steps_with_wide_tables_share_nothing():
    lens = [[600, 64, 30], [100, 640, 5]]
    eager = [_wide_state(i, x) for i, x in enumerate(lens)]
    states = [_wide_state(i, x) for i, x in enumerate(lens)]
    for s in eager:
        _step(s)
    status_ok()
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(s)
        graphs.append(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    status_ok()
    assert all(_all_same(a, b) for a, b in zip(states, eager))


def test_wide_tables_withheld_tile_times_out_then_recovers():
    s, want = _wide_state(20, [300, 20, 129]), _wide_state(20, [300, 20, 129])
    _step(want)
    status_ok()
    chs.attn_debug_inject_fault(3)
    try:
        chs.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["sl"])
        assert chs.attn_status() == chs.ATTN_ERR_TIMEOUT
    finally:
        chs.attn_debug_inject_fault(0)
    _step(s)
    status_ok()
    assert _all_same(s, want)


FIRST_CALL_CAPTURED = """
import torch, causal_head_self_gb300 as chs
assert chs.attn_status() == chs.ATTN_OK      # (the library's own state is made here)
q = torch.ones(3, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
kv = torch.ones(3, 2, 20, 64, dtype=torch.bfloat16, device="cuda")
pages = torch.zeros(2, 9, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
sl = torch.full((3,), 20, dtype=torch.int32, device="cuda")
w, w_out = torch.zeros(2, 3, 2, 24, device="cuda")
lse = torch.zeros(3, 8, 20, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    chs.attn_paged_append(kv, kv, *pages, table, sl)
    o = chs.attn_decode_paged(q, *pages, table, sl, weights=w)
    chs.attn_key_weights(q.expand(3, 8, 20, 64).contiguous(), kv, lse, w_out[..., :20].contiguous(), sl)
    new, keep = chs.attn_cache_evict(*pages, w, table, sl, 10, 2, weights_out=w_out)
graph.replay()
torch.cuda.synchronize()
assert chs.attn_status() == chs.ATTN_OK
assert (o == 1).all() and new.tolist() == [10] * 3
assert keep[0, 0].tolist() == list(range(8)) + [18, 19]
print("captured")
"""


def test_every_call_may_be_captured_at_its_first_use():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], capture_output=True, text=True,
                       timeout=120, cwd=Path(__file__).resolve().parent.parent)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr


def test_workspace_of_a_decode_step():
    q, sl = queries(2, 8, 128, seed=1).cuda(), torch.tensor([70, 9], dtype=torch.int32, device="cuda")
    kp, vp, table, _ = ref.make_cache([70, 9], 2, 128, 16, 5, seed=2)
    kp, vp, table, wide = gpu(kp, vp, table, widen(table, 16))
    assert chs.attn_decode_paged_workspace(q, kp, table) == 0
    assert chs.attn_decode_paged_workspace(q, kp, table, weights=True) > 0
    want = chs.attn_decode_paged(q, kp, vp, table, sl)
    need = chs.attn_decode_paged_workspace(q, kp, wide)
    # a workspace of just that size, and nothing written behind it
    ws = torch.full((need + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    got = chs.attn_decode_paged(q, kp, vp, wide, sl, workspace=ws[:need])
    assert (ws[need:] == 0x5a).all()
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7, atol=1e-4)
    with pytest.raises(chs.AttnError) as e:
        chs.attn_decode_paged(q, kp, vp, wide, sl, workspace=ws[:need - 1])
    assert e.value.code == chs.ATTN_ERR_SCRATCH_LIMIT
    # a window makes the step short again
    chs.attn_decode_paged(q, kp, vp, wide, sl, window=64, workspace=ws[:0])
    status_ok()


def test_withheld_tile_times_out_then_recovers():
    s, want = _state(20, [300, 20, 129]), _state(20, [300, 20, 129])
    _step(want)
    status_ok()
    chs.attn_debug_inject_fault(3)
    try:
        chs.attn_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["sl"])
        assert chs.attn_status() == chs.ATTN_ERR_TIMEOUT
    finally:
        chs.attn_debug_inject_fault(0)
    _step(s)
    status_ok()
    assert _all_same(s, want)


@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_decode_of_more_tiles_than_the_ring_holds(Dh):
    # shares of about 30 tiles per CTA, several units each: the ring of tiles wraps
    # many times, also inside a unit
    B, Hkv, page, cols = 16, 8, 16, 256
    gen = torch.Generator(device="cuda").manual_seed(Dh)
    kp, vp = (torch.randn((B * cols, Hkv, page, Dh), generator=gen, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    table = torch.randperm(B * cols, generator=gen, device="cuda").to(torch.int32).view(B, cols)
    sl = torch.randint(1, cols * page + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    sl[0] = cols * page
    q = torch.randn((B, 16, 1, Dh), generator=gen, device="cuda").to(torch.bfloat16)
    weights = torch.zeros(B, Hkv, cols * page, device="cuda")
    got = chs.attn_decode_paged(q, kp, vp, table, sl, weights=weights)
    status_ok()
    for b, n in enumerate(sl.tolist()):
        k, v = (x[table[b].long()].transpose(0, 1).reshape(Hkv, cols * page, Dh)[:, :n].double()
                for x in (kp, vp))
        z = q[b, :, 0].view(Hkv, 2, Dh).double() @ k.transpose(1, 2) * Dh ** -0.5
        p = torch.softmax(z, -1)
        o, a = (p @ v).view(16, Dh), (p @ v.abs()).view(16, Dh)
        # (delta of paged_ref.decode with |q| . |k| <= 6 Dh: 2 * 6 Dh^1.5 2^-23)
        rel = 12 * Dh ** 1.5 * 2.0 ** -23 + 2.0 ** -18
        assert ((got[b, :, 0].double() - o).abs() <= ref.HALF_BF16 * (o.abs() + a) + rel * a).all()
        w = p.sum(1)
        assert ((weights[b, :, :n].double() - w).abs() <= rel * w).all()
