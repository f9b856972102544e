"""What the paged cache's operators owe beyond the wide bounds: the decode step's
weights are held in two bf16 parts where they meet V (up to 16 query heads per
K/V head), so that its output is off by its own rounding and little more."""
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


def widen(table, page, rows=13000):
    """The table with unused columns behind it: more rows than the one-launch form takes."""
    more = -(-rows // page) - table.shape[1]
    return torch.cat([table, torch.full((table.shape[0], more), -1, dtype=torch.int32)], 1)


def narrow_decode(q, kp, vp, table, lens, window=0, scale=0.0):
    """(o in 64 bits, its tolerance, weights, their tolerance)."""
    B, Hq, _, Dh = q.shape
    Hkv, T = kp.shape[1], table.shape[1] * kp.shape[2]
    G = Hq // Hkv
    scale = scale or 1 / math.sqrt(Dh)
    o, tol = (torch.zeros(B, Hq, 1, Dh, dtype=torch.float64) for _ in range(2))
    w, wtol = (torch.zeros(B, Hkv, T, dtype=torch.float64) for _ in range(2))
    for b, n in enumerate(lens.tolist()):
        lo = max(0, n - window) if window > 0 else 0
        for g in range(Hkv if n else 0):
            k, v = ref.rows(kp, table[b], lo, n, g), ref.rows(vp, table[b], lo, n, g)
            qg = q[b, g * G:(g + 1) * G, 0].double()
            p = torch.softmax(scale * qg @ k.t(), -1)
            out, size = p @ v, p @ v.abs()
            # A score is a sum of Dh products in 32 bits, each addition off by at most 2^-23
            # of the sum of their sizes (truncated), and it is scaled and has the maximum
            # taken off in 32 bits (2^-22 of its size covers both roundings and the fused
            # one): the exponent's error.  It moves a weight, and the sum of weights, by e to
            # that; 2^-18: exp2 and the 32-bit sums.
            sizes = scale * qg.abs() @ k.abs().t()
            delta = float((sizes * (Dh * 2.0 ** -23 + 2.0 ** -22)).max())
            rel = math.expm1(2 * delta) + 2.0 ** -18
            # P is two bf16 parts, each cut off (not rounded) after 8 bits, 2^-7 of what it
            # stands for: 2^-14 of a weight is left; the products of both parts, 2 n, are added
            # in 32 bits (2^-23 each)
            rel_o = rel + 2.0 ** -14 + 2 * (n - lo) * 2.0 ** -23
            at = slice(g * G, (g + 1) * G)
            o[b, at, 0] = out
            # ... and the output is rounded once, from a value that is off by rel_o already
            tol[b, at, 0] = ref.HALF_BF16 * (out.abs() + rel_o * size) + rel_o * size
            w[b, g, lo:n], wtol[b, g, lo:n] = p.sum(0), (rel + 2.0 ** -24) * p.sum(0)
    return o, tol, w, wtol


# (Hq, Hkv, Dh, page, cols, lengths, window): up to 16 query heads per K/V head
CASES = [
    (4, 4, 64, 8, 16, [2, 7, 128, 60], 0),
    (8, 2, 128, 16, 40, [3, 127, 300, 640], 0),
    (16, 1, 128, 16, 30, [480, 33], 0),
    (30, 2, 64, 24, 20, [470, 0, 5], 0),
    (4, 1, 256, 32, 12, [5, 65, 384], 0),
    (2, 2, 256, 16, 16, [256, 70], 0),
    (4, 1, 64, 8, 50, [400, 77, 390], 77),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,Dh,page,cols,lens,window", CASES)
def test_decode_rounds_its_output_once(Hq, Hkv, Dh, page, cols, lens, window, wide):
    kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=Hq + Dh)
    q = torch.randn((len(lens), Hq, 1, Dh), generator=torch.Generator().manual_seed(Dh)).to(torch.bfloat16)
    o, tol, _, _ = narrow_decode(q, kp, vp, table, sl, window=window)
    table = widen(table, page) if wide else table
    got = chs.attn_decode_paged(*(x.cuda() for x in (q, kp, vp, table, sl)), window=window)
    assert chs.attn_status() == chs.ATTN_OK
    assert ((got.cpu().double() - o).abs() <= tol).all()
