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
