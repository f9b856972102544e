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
