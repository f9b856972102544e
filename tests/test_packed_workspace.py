"""The workspace that attn_fwd_packed asks for: what the query answers is
enough for the call, whatever the number of K/V heads, on both sides of every
limit of the rule by which CTAs list their own items (64 sequences, 1024 blocks
of 128 or 256 rows, 32 items a CTA).  workspace=None allocates the query's
answer, so a call that needs more than it raises."""
import itertools

import pytest
import torch

import causal_head_self_gb300 as chs

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -11   # as in packed_ref.py


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# 128 * 1024 and 256 * 1024 rows: the most blocks of one listing
ROWS = (4000, 131071, 131072, 140000, 200003, 262143, 262144)


@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("Hq", [1, 4, 6, 8, 16])
def test_query_and_call_agree(Dh, Hq):
    """Sequences without rows: the call is the listing alone."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # rows at which the items of 128- and of 256-row blocks reach 32 for each CTA
    edges = [block * (32 * sms * ctas // Hq) + d
             for block, ctas in ((128, 1), (128, 2), (256, 1)) for d in (-70 * block, -block, 0, block)]
    edges = [T for T in edges if 0 < T <= 300000]
    most = max(ROWS + tuple(edges))
    store = torch.zeros(most * 3 * Hq * Dh, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(most * Hq * Dh, dtype=torch.bfloat16, device="cuda")
    for T, B in itertools.product(ROWS + tuple(edges), (1, 2, 11, 12, 40, 63, 64, 65, 200)):
        cu = i32([0] * (B + 1))
        for Hkv in (h for h in range(1, Hq + 1) if Hq % h == 0):
            x = store[:T * (Hq + 2 * Hkv) * Dh].view(T, Hq + 2 * Hkv, Dh)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            o = out[:T * Hq * Dh].view(T, Hq, Dh)
            need = chs.attn_packed_workspace(q, cu)
            try:
                chs.attn_fwd_packed(q, k, v, cu, o)
            except chs.AttnError as e:
                raise AssertionError((T, B, Hq, Hkv, Dh, need)) from e
    assert chs.attn_status() == chs.ATTN_OK


def windowed(q, k, v, w):
    """Rows i of one sequence's head over keys i - w < j <= i, and the bound of packed_ref.py."""
    n, Dh = q.shape
    pad = torch.zeros(w - 1, Dh, dtype=torch.float64, device=q.device)
    K = torch.cat([pad, k.double()]).unfold(0, w, 1)    # [n, Dh, w]
    V = torch.cat([pad, v.double()]).unfold(0, w, 1)
    s = torch.einsum("nd,ndw->nw", q.double(), K) * Dh ** -0.5
    j = torch.arange(n, device=q.device)[:, None] - (w - 1) + torch.arange(w, device=q.device)
    p = torch.softmax(s.masked_fill(j < 0, -torch.inf), -1)
    y = torch.einsum("nw,ndw->nd", p, V)
    a = torch.einsum("nw,ndw->nd", p, V.abs())
    return y, (1 + U) * (U + F) * a + U * y.abs()


@pytest.mark.parametrize("T,B,Hq,Hkv,Dh", [
    (131071, 16, 8, 1, 64), (131072, 16, 8, 1, 64), (140000, 12, 8, 2, 64), (140000, 40, 8, 4, 64),
    (262143, 64, 4, 1, 64), (262144, 64, 4, 1, 64), (131071, 64, 8, 2, 128), (131072, 64, 8, 1, 128),
    (131072, 64, 8, 8, 128)])
def test_long_buffers_of_few_sequences(T, B, Hq, Hkv, Dh):
    gen = torch.Generator("cuda").manual_seed(T + B)
    x = torch.randn(T, Hq + 2 * Hkv, Dh, generator=gen, device="cuda", dtype=torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    lens = [T // B - 5 * (b % 3) for b in range(B)]
    first = [0]
    for n in lens:
        first.append(first[-1] + n)
    cu, w = i32(first), 16
    o = chs.attn_fwd_packed(q, k, v, cu, window=w)
    ws = torch.empty(max(chs.attn_packed_workspace(q, cu), 1), dtype=torch.uint8, device="cuda")
    assert torch.equal(chs.attn_fwd_packed(q, k, v, cu, window=w, workspace=ws)[:first[-1]], o[:first[-1]])
    assert chs.attn_status() == chs.ATTN_OK
    for b in (0, B // 2, B - 1):
        a, z = first[b], first[b + 1]
        for h in (0, Hq - 1):
            g = h * Hkv // Hq
            want, bound = windowed(q[a:z, h], k[a:z, g], v[a:z, g], w)
            assert bool(((o[a:z, h].double() - want).abs() <= bound).all()), (b, h)
