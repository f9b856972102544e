"""The paged cache's calls on the GPU at sizes, values and settings that the
other tests do not reach."""
import math

import pytest
import torch

import causal_head_self_gb300 as chs
import paged_ref as ref
from causal_head_self_gb300 import build as _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def same_bits(a, b):
    return a.shape == b.shape and torch.equal(a.view(torch.int32), b.view(torch.int32))


def status_ok():
    assert chs.attn_status() == chs.ATTN_OK


# The columns of all heads together, 128 a head where every query votes and 16 where one
# does, pass 32 bits.
@pytest.mark.parametrize("Hq,queries", [(2 ** 24 + 16, 0), (2 ** 27 + 16, 1)])
def test_key_weights_of_more_columns_than_32_bits_count(Hq, queries):
    q = torch.zeros(1, Hq, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, Hq, 1, device="cuda")
    w = torch.full((1, 1, 1), 7.0, device="cuda")
    chs.attn_key_weights(q, k, lse, w, queries=queries, accumulate=False)
    status_ok()
    # each head adds e^0: whole numbers that 24 bits hold in each part of the sum, and at its end
    assert w.item() == Hq


@pytest.mark.parametrize("Hq,Hkv,S,Dh,window", [
    (8, 2, 17, 128, 0), (4, 4, 32, 64, 0), (12, 1, 30, 64, 0), (8, 2, 40, 64, 9), (2, 2, 100, 128, 0),
    (8, 2, 128, 256, 0), (2, 1, 300, 64, 40)])
def test_every_row_votes_however_it_is_said(Hq, Hkv, S, Dh, window):
    gen = torch.Generator().manual_seed(S)
    q, k = (torch.randn((2, h, S, Dh), generator=gen).to(torch.bfloat16) for h in (Hq, Hkv))
    lse = 5 + torch.randn((2, Hq, S), generator=gen)
    lens = [S, S - 5]
    want, rtol = ref.key_weights(q, k, lse, lens, window=window)
    q, k, lse, sl = (x.cuda() for x in (q, k, lse, torch.tensor(lens, dtype=torch.int32)))
    got = []
    for queries in (0, S, S + 1, 64 * S, 2 ** 31 - 1, -1):
        w = torch.zeros(2, Hkv, S, device="cuda")
        chs.attn_key_weights(q, k, lse, w, sl, queries=queries, window=window)
        status_ok()
        got.append(w)
    assert ((got[0].cpu().double() - want).abs() <= rtol * want).all()
    assert all(same_bits(w, got[0]) for w in got)


# (Hq, Hkv, S, Dh, queries, causal, window): the general kernel, the same with several heads
# per tile, and the one for few voting queries, whose tiles are padded here
SPECIAL = [(2, 2, 300, 64, 0, True, 0), (4, 2, 260, 128, 0, True, 90), (2, 1, 200, 256, 0, False, 0),
           (12, 1, 300, 128, 40, True, 0), (5, 1, 300, 64, 20, True, 70),
           (8, 2, 300, 64, 20, True, 0), (3, 1, 150, 128, 7, True, 0), (5, 1, 200, 256, 9, True, 0),
           (6, 2, 300, 64, 33, False, 0), (4, 2, 300, 128, 128, True, 0)]


@pytest.mark.parametrize("kind", ["lse +inf", "lse -inf", "lse nan", "key -inf", "key +inf", "query nan"])
@pytest.mark.parametrize("Hq,Hkv,S,Dh,queries,causal,window", SPECIAL)
def test_key_weights_of_values_that_are_not_numbers(Hq, Hkv, S, Dh, queries, causal, window, kind):
    gen = torch.Generator().manual_seed(S + Hq)
    lens, G = [S, S - 30], Hq // Hkv
    q, k = (torch.randn((2, h, S, Dh), generator=gen).to(torch.bfloat16) for h in (Hq, Hkv))
    lse = 5 + torch.randn((2, Hq, S), generator=gen)
    for b, n in enumerate(lens):
        first = n - (queries or n)
        rows = torch.arange(first, n)[torch.rand(n - first, generator=gen) < 0.3]
        if kind.startswith("lse"):
            lse[b, 0, rows] = float(kind[4:])
            lse[b, Hq - 1, n - 1] = float(kind[4:])
        elif kind.startswith("key"):
            # its scores are infinite, not NaN: each query has the same sign there
            q[b, :, :, 0] = q[b, :, :, 0].abs().clamp(min=0.1)
            k[b, 0, ::7, 0] = float(kind[4:])
        else:
            q[b, 0, first + (n - first) // 2] = math.nan
        lse[b, :, n:], q[b, :, n:], k[b, :, n:] = math.nan, math.nan, math.nan
    want = torch.zeros(2, Hkv, S, dtype=torch.float64)
    for b, n in enumerate(lens):
        i = torch.arange(n - (queries or n), n)[:, None]
        j = torch.arange(n)[None]
        seen = (j <= i) if causal else torch.ones(len(i), n, dtype=torch.bool)
        if window:
            seen &= j > i - window
        for h in range(Hq):
            z = q[b, h, i[:, 0]].double() @ k[b, h // G, :n].double().t() * Dh ** -0.5
            p = torch.exp(z - lse[b, h, i].double())
            want[b, h // G, :n] += torch.where(seen, p, 0.0).sum(0)
    w = torch.zeros(2, Hkv, S, device="cuda")
    chs.attn_key_weights(q.cuda(), k.cuda(), lse.cuda(), w, torch.tensor(lens, dtype=torch.int32).cuda(),
                         queries=queries, causal=causal, window=window, accumulate=False)
    status_ok()
    got = w.cpu().double()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    finite = want.isfinite()
    # (paged_ref.key_weights' bound, with |q| . |k| / sqrt(Dh) <= 6 sqrt(Dh) and |lse| <= 12)
    rel = (Dh + 1) * 2.0 ** -23 * (6 * Dh ** 0.5 + 12) + 2.0 ** -18
    assert ((got - want).abs()[finite] <= rel * want[finite]).all()


# ---------------------------------------------------------------- decode

def widen(table, page, rows=13000):
    """The table with unused columns behind it: more rows than the one-launch form takes."""
    more = -(-rows // page) - table.shape[1]
    return torch.cat([table, torch.full((table.shape[0], more), -1, dtype=torch.int32)], 1)


def course(name, n, gen):
    """Scores over n keys: rising by far more than 2^8 a tile, by less than that, falling, any."""
    t = torch.arange(n) / max(n - 1, 1)
    return {"rising": 400 * t, "creeping": 3.0 / 128 * torch.arange(n), "falling": 400 - 400 * t,
            "any": 100 * torch.randn(n, generator=gen)}[name]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scores", ["rising", "creeping", "falling", "any"])
@pytest.mark.parametrize("Hq,Hkv,Dh,page,cols,lens", [
    (8, 2, 128, 16, 40, [640, 300, 2]), (4, 4, 64, 24, 30, [719, 130]), (4, 1, 256, 32, 12, [384, 65]),
    (40, 1, 128, 16, 30, [470, 129]), (160, 1, 64, 8, 40, [320, 7])])
def test_decode_of_scores_that_move_the_maximum(Hq, Hkv, Dh, page, cols, lens, scores, wide):
    gen = torch.Generator().manual_seed(Hq + Dh)
    B, G = len(lens), Hq // Hkv
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=Dh)
    u = torch.randint(0, 2, (Dh,), generator=gen) * 2.0 - 1
    # q . k = 8 f a about, with a head's factor f in [1/2, 1] and a key's score a
    f = 0.5 + 0.5 * torch.rand((B, Hq, 1, 1), generator=gen)
    q = (f * u + torch.randn((B, Hq, 1, Dh), generator=gen) / 50).to(torch.bfloat16)
    for b, n in enumerate(lens):
        a = course(scores, n, gen)
        for t in range(n):
            kp[table[b, t // page], :, t % page] = (
                a[t] / 8 * u + torch.randn((Hkv, Dh), generator=gen) / 50).to(torch.bfloat16)
    args = [x.cuda() for x in (q, kp, vp, widen(table, page) if wide else table, sl)]
    weights = torch.zeros(B, Hkv, args[3].shape[1] * page, device="cuda")
    got = chs.attn_decode_paged(*args, scale=8.0 / Dh, weights=weights, accumulate=False)
    status_ok()
    got, weights = got.cpu().double(), weights.cpu().double()
    for b, n in enumerate(lens):
        for g in range(Hkv):
            k, v = ref.rows(kp, table[b], 0, n, g), ref.rows(vp, table[b], 0, n, g)
            qg = q[b, g * G:(g + 1) * G, 0].double()
            p = torch.softmax(8.0 / Dh * qg @ k.t(), -1)
            # As in paged_ref.decode, with the sizes of this head's and these keys' products
            # (Dh additions in 32 bits, and 2^-22 for the scaling and the maximum's removal);
            # a weight is off by e to twice that, and 2^-18 for exp2 and the sums.  P is rounded
            # to bf16 and n products are added in 32 bits.
            size = 8.0 / Dh * qg.abs() @ k.abs().t()
            rel = torch.expm1(2 * size.max() * (Dh * 2.0 ** -23 + 2.0 ** -22)) + 2.0 ** -18
            assert rel < 1 / 16   # (so that no zero and no other row's result would do)
            o, a = p @ v, p @ v.abs()
            tol = ref.HALF_BF16 * (o.abs() + a) + (rel + n * 2.0 ** -23) * a
            assert ((got[b, g * G:(g + 1) * G, 0] - o).abs() <= tol).all()
            assert n < 2 or (tol < o.abs()).double().mean() > 0.5
            w = p.sum(0)
            # (a weight below 2^-126, the least normal number, may be 0)
            assert ((weights[b, g, :n] - w).abs() <= rel * w + G * 2.0 ** -126).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kind", ["key -inf", "every key -inf", "key +inf", "query nan"])
@pytest.mark.parametrize("Hq,Hkv,Dh,page,cols,lens", [
    (8, 2, 128, 16, 40, [640, 300, 2]), (4, 1, 256, 32, 12, [384, 65]), (40, 1, 64, 16, 30, [470, 129])])
def test_decode_of_visible_keys_that_are_not_numbers(Hq, Hkv, Dh, page, cols, lens, kind, wide):
    gen = torch.Generator().manual_seed(Hq)
    B, G = len(lens), Hq // Hkv
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=Hq)
    # (a score is infinite, not NaN: each query has the same sign there)
    q = torch.randn((B, Hq, 1, Dh), generator=gen).to(torch.bfloat16)
    q[..., 0] = q[..., 0].abs().clamp(min=0.1)
    if kind == "query nan":
        q[0, 1] = math.nan
    else:
        value = math.inf if kind == "key +inf" else -math.inf
        for t in range(0, lens[0], 1 if kind == "every key -inf" else 3):
            kp[table[0, t // page], 0, t % page, 0] = value
    args = [x.cuda() for x in (q, kp, vp, widen(table, page) if wide else table, sl)]
    weights = torch.zeros(B, Hkv, args[3].shape[1] * page, device="cuda")
    got = chs.attn_decode_paged(*args, weights=weights, accumulate=False)
    status_ok()
    got, weights = got.cpu().double(), weights.cpu().double()
    for b, n in enumerate(lens):
        for g in range(Hkv):
            k, v = ref.rows(kp, table[b], 0, n, g), ref.rows(vp, table[b], 0, n, g)
            p = torch.softmax(Dh ** -0.5 * q[b, g * G:(g + 1) * G, 0].double() @ k.t(), -1)
            o, a, w = p @ v, p @ v.abs(), p.sum(0)
            # (paged_ref.decode's bound, with |q| . |k| <= 6 Dh)
            rel = 12 * Dh ** 1.5 * 2.0 ** -23 + 2.0 ** -18
            for x, y, tol in ((got[b, g * G:(g + 1) * G, 0], o,
                               ref.HALF_BF16 * (o.abs() + a) + (rel + n * 2.0 ** -23) * a),
                              (weights[b, g, :n], w, rel * w)):
                assert torch.equal(x.isnan(), y.isnan())
                assert ((x - y).abs() <= tol)[~y.isnan()].all()
