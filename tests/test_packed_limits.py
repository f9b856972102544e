"""Packed calls and rotations past 2^31 elements, where 32-bit offsets would
wrap, and the ends of the arguments' ranges."""
import pytest
import torch

import causal_head_self_gb300 as chs
import packed_ref as ref
from causal_head_self_gb300 import inputs

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_tensors_of_2_31_elements():
    T, Hq, Hkv, Dh, W = 1 << 18, 64, 8, 128, 100
    d = torch.device("cuda")
    q = inputs.device_normal_bf16((1, Hq, T, Dh), 1, d)[0].transpose(0, 1)      # heads first
    k = inputs.device_normal_bf16((1, 1, T, Hkv * Dh), 2, d)[0, 0].view(T, Hkv, Dh)
    v = inputs.device_normal_bf16((1, 1, T, Hkv * Dh), 3, d)[0, 0].view(T, Hkv, Dh)
    dout = inputs.device_normal_bf16((1, 1, T, Hq * Dh), 4, d)[0, 0].view(T, Hq, Dh)
    assert q.numel() == 1 << 31
    lens = [100000, 0, 1, 130000, 32142]
    cu = ref.offsets(lens)
    assert cu[-1] == T - 1
    o, lse = torch.zeros(T, Hq, Dh, dtype=torch.bfloat16, device=d), torch.zeros(Hq, T, device=d)
    chs.attn_fwd_packed(q, k, v, i32(cu), o, lse, window=W)
    grads = chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), window=W)
    assert chs.attn_status() == chs.ATTN_OK
    # a row's results need the rows a window to either side of it
    for at in (200, 99998, 100000, 100500, 229000, T - 3000, T - 2):
        lo = max(a for a in cu if a <= at)
        hi = min(z for z in cu if z > at)
        a, z = max(lo, at - W + 1), min(hi, at + W)
        rows = slice(a, z)
        want, L, bound, dwant, dbound = ref.attention(q[rows], k[rows], v[rows], [0, z - a], True, W,
                                                      dout=dout[rows])
        r = at - a
        ref.check(o[at], want[r], bound[r], at)
        assert float((lse[:, at].double() - L[:, r]).abs().max()) < ref.F
        for got, w, b in zip(grads, dwant, dbound):
            ref.check(got[at], w[r], b[r], at)
    del o, grads, dout
    # rotation in place, and back to where it was (two roundings)
    pos = torch.arange(T, dtype=torch.int32, device=d)
    handle = chs.attn_rope_frequencies(Dh)
    kept = q[T - 5:].clone()
    chs.attn_rope(q, k, pos, handle, q, k)
    assert not torch.equal(q[T - 5:], kept)
    chs.attn_rope(q, k, pos, handle, q, k, inverse=True)
    assert chs.attn_status() == chs.ATTN_OK
    near = (q[T - 5:].double() - kept.double()).abs()
    assert float(near.max()) <= 2 * 2.0 ** -8 * 1.5 * float(kept.double().abs().max())


def test_a_sequence_of_more_blocks_than_the_listing_has_bins():
    T, W = 300000, 64
    d = torch.device("cuda")
    q, k, v, dout = (inputs.device_normal_bf16((1, 1, T, 64), i, d)[0, 0].view(T, 1, 64) for i in range(4))
    cu, lse = [0, 299000, 299001, T], torch.zeros(1, T, device=d)
    for causal_window in (W, 0):   # (without a window as a check of the listing alone: one head)
        o = chs.attn_fwd_packed(q, k, v, i32(cu), None, lse, window=causal_window)
        grads = chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), window=causal_window)
        assert chs.attn_status() == chs.ATTN_OK
        assert not o.isnan().any() and not any(g.isnan().any() for g in grads)
        for at in (5, 127, 150000, 298990, 299000, T - 3):
            lo = max(a for a in cu if a <= at)
            hi = min(z for z in cu if z > at)
            if causal_window:
                a, z = max(lo, at - W + 1), min(hi, at + W)
                want, _, bound, dwant, dbound = ref.attention(q[a:z], k[a:z], v[a:z], [0, z - a], True, W,
                                                              dout=dout[a:z])
                for got, w, b in zip((o, *grads), (want, *dwant), (bound, *dbound)):
                    ref.check(got[at], w[at - a], b[at - a], at)
            else:
                rows = slice(lo, at + 1)
                p = torch.softmax(k[rows, 0].double() @ q[at, 0].double() / 8, 0)
                y, size = p @ v[rows, 0].double(), p @ v[rows, 0].double().abs()
                assert bool(((o[at, 0].double() - y).abs() <= (1 + ref.U) * (ref.U + ref.F) * size
                             + ref.U * y.abs()).all())


def test_pools_of_2_31_elements():
    P, Hkv, page, Dh, T = 32768, 8, 64, 128, 300
    kp = torch.zeros(P, Hkv, page, Dh, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    assert kp.numel() == 1 << 31
    gen = torch.Generator("cuda").manual_seed(0)
    q, k, v = ref.layouts(T, 8, Hkv, Dh, "fused", gen)
    slots = torch.arange(T, dtype=torch.int32, device="cuda") * 6991 % (P * page)
    slots[-1], slots[-2] = P * page - 1, (P // 2) * page
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    handle = chs.attn_rope_frequencies(Dh)
    ko = torch.zeros(T, Hkv, Dh, dtype=torch.bfloat16, device="cuda")
    chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots, None, ko)
    assert chs.attn_status() == chs.ATTN_OK
    at = slots.long()
    assert torch.equal(kp[at // page, :, at % page], ko) and torch.equal(vp[at // page, :, at % page], v)
    assert int((kp != 0).sum()) == int((ko != 0).sum())


@pytest.mark.parametrize("window", [2 ** 31 - 1, 700, 0])
def test_windows_longer_than_the_sequences(window):
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v = ref.layouts(700, 4, 2, 64, "fused", gen)
    cu = i32([0, 300, 700])
    o, lse = torch.zeros(700, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 700, device="cuda")
    chs.attn_fwd_packed(q, k, v, cu, o, lse, window=window)
    grads = chs.attn_bwd_packed(q, k, v, o, o, lse, cu, window=window)
    assert chs.attn_status() == chs.ATTN_OK
    want, _, bound, dwant, dbound = ref.attention(q, k, v, [0, 300, 700], dout=o)
    ref.check(o, want, bound)
    for got, w, b in zip(grads, dwant, dbound):
        ref.check(got, w, b)


@pytest.mark.parametrize("scale", [1e-4, 1.0])
def test_scales(scale):
    # nearly equal weights, and weights of a few keys alone
    gen = torch.Generator("cuda").manual_seed(2)
    q, k, v = ref.layouts(400, 4, 2, 64, "fused", gen)
    dout = ref.layouts(400, 4, 2, 64, "contiguous", gen)[0]
    cu, lse = [0, 130, 400], torch.zeros(4, 400, device="cuda")
    o = chs.attn_fwd_packed(q, k, v, i32(cu), None, lse, scale=scale)
    grads = chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), scale=scale)
    assert chs.attn_status() == chs.ATTN_OK
    want, _, bound, dwant, dbound = ref.attention(q, k, v, cu, scale=scale, dout=dout)
    # scores of up to about 40 at scale 1: an fp32 error of 64 * 2^-24 * 64 * 3 of a weight
    ref.check(o, want, bound)
    for got, w, b in zip(grads, dwant, dbound):
        ref.check(got, w, b)


@pytest.mark.parametrize("Dh,n", [(64, 700), (128, 700), (128, 5000), (256, 700)])
def test_a_wait_that_runs_out(Dh, n):
    # (the host's test hook: a copy is withheld, the waits give up after 2 s)
    gen = torch.Generator("cuda").manual_seed(3)
    q, k, v = ref.layouts(n, 2, 1, Dh, "fused", gen)
    cu, lse = i32([0, n]), torch.zeros(2, n, device="cuda")
    try:
        chs.attn_debug_inject_fault(1)
        chs.attn_fwd_packed(q, k, v, cu)
        assert chs.attn_status() == chs.ATTN_ERR_TIMEOUT
        chs.attn_debug_inject_fault(4)
        chs.attn_bwd_packed(q, k, v, q, q, lse, cu)
        assert chs.attn_status() == chs.ATTN_ERR_TIMEOUT
    finally:
        chs.attn_debug_inject_fault(0)
    assert chs.attn_status() == chs.ATTN_OK
    o = chs.attn_fwd_packed(q, k, v, cu, None, lse)
    grads = chs.attn_bwd_packed(q, k, v, o, o, lse, cu)
    assert chs.attn_status() == chs.ATTN_OK
    want, _, bound, dwant, dbound = ref.attention(q, k, v, [0, n], dout=o)
    ref.check(o, want, bound)
    for got, w, b in zip(grads, dwant, dbound):
        ref.check(got, w, b)
