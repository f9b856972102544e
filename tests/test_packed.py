"""Attention over packed sequences on the GPU, against the 64-bit reference."""
import pytest
import torch

import causal_head_self_gb300 as chs
import packed_ref as ref

pytestmark = pytest.mark.gpu

LENS = {
    "one": [1],
    "edges": [1, 2, 127, 128, 129, 0, 255, 256, 257, 1, 0],
    "ragged": [300, 7, 1023, 64, 65, 511],
    "long": [2100, 33, 1700],
}
HEADS = [(4, 2), (3, 3), (6, 1), (8, 2)]
AHEAD, BEHIND = 5, 9


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(lens, Hq, Hkv, Dh, kind="fused", seed=0):
    """Inputs whose rows of no sequence are NaN, outputs of another value."""
    gen = torch.Generator("cuda").manual_seed(seed)
    cu = ref.offsets(lens, AHEAD)
    T = cu[-1] + BEHIND
    q, k, v = ref.layouts(T, Hq, Hkv, Dh, kind, gen)
    dout = ref.layouts(T, Hq, Hkv, Dh, kind, gen)[0]
    for x in (q, k, v, dout):
        x[:AHEAD] = x[cu[-1]:] = float("nan")
    return q, k, v, dout, cu, T


def outside_is(x, value, cu, rows=0):
    x = x.transpose(0, rows)
    return bool((x[:cu[0]] == value).all()) and bool((x[cu[-1]:] == value).all())


def run(q, k, v, dout, cu, causal, window, scale=0.0, kind="fused"):
    T, Hq, Dh = q.shape
    Hkv = k.shape[1]
    o, lse = torch.full_like(q, 7), torch.full((Hq, T), 7.0, device="cuda")
    if kind == "fused":
        dx = torch.full((T, Hq + 2 * Hkv, Dh), 7, dtype=torch.bfloat16, device="cuda")
        grads = dx[:, :Hq], dx[:, Hq:Hq + Hkv], dx[:, Hq + Hkv:]
    else:
        grads = torch.full_like(q, 7), torch.full_like(k, 7), torch.full_like(v, 7)
    mask = dict(causal=causal, window=window, scale=scale)
    assert chs.attn_fwd_packed(q, k, v, i32(cu), o, lse, **mask) is o
    chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), *grads, **mask)
    assert chs.attn_status() == chs.ATTN_OK
    return o, lse, grads


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_forward_and_gradients(Dh, lens, causal, window):
    Hq, Hkv = HEADS[(len(lens) + Dh // 64) % len(HEADS)]
    kind = ["fused", "heads_first", "contiguous", "wide"][(len(LENS[lens]) + Dh // 64) % 4]
    q, k, v, dout, cu, T = case(LENS[lens], Hq, Hkv, Dh, kind)
    o, lse, grads = run(q, k, v, dout, cu, causal, window, kind=kind)
    real = slice(cu[0], cu[-1])
    want, L, bound, dwant, dbound = ref.attention(q, k, v, cu, causal, window, dout=dout)
    ref.check(o[real], want[real], bound[real], "o")
    # (a relative error of every weight's is an absolute one of the logarithm)
    assert float((lse[:, real] - L[:, real]).abs().max()) < ref.F
    for name, got, w, b in zip(("dq", "dk", "dv"), grads, dwant, dbound):
        ref.check(got[real], w[real], b[real], name)
    assert all(outside_is(x, 7, cu) for x in (o, *grads)) and outside_is(lse, 7, cu, 1)


@pytest.mark.parametrize("kind", ["fused", "heads_first", "contiguous", "wide"])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_strides(Dh, kind):
    q, k, v, dout, cu, T = case([130, 1, 258], 4, 2, Dh, kind, seed=3)
    o, lse, grads = run(q, k, v, dout, cu, True, 0, kind=kind)
    same = [x.contiguous() for x in (q, k, v, dout)]
    o2, lse2, grads2 = run(*same, cu, True, 0, kind="contiguous")
    assert torch.equal(o.contiguous(), o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a.contiguous(), b) for a, b in zip(grads, grads2))


@pytest.mark.parametrize("axis", [0, 1, 2, 3])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_parts_of_one_tensor(Dh, axis):
    # q, k, v and their gradients are parts of one tensor each: [3, T, H, Dh], [T, 3, H, Dh],
    # [T, H, 3, Dh], [H, 3, T, Dh]
    gen = torch.Generator("cuda").manual_seed(9)
    H, cu = 3, [0, 200, 201, 330]
    T = cu[-1]
    shape = [(3, T, H, Dh), (T, 3, H, Dh), (T, H, 3, Dh), (H, 3, T, Dh)][axis]
    x = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    dx = torch.zeros_like(x)

    def parts(y):
        return y.unbind(axis) if axis < 3 else [z.transpose(0, 1) for z in y.unbind(1)]
    q, k, v = parts(x)
    dout = torch.randn(T, H, Dh, generator=gen, device="cuda").to(torch.bfloat16)
    lse = torch.zeros(H, T, device="cuda")
    o = chs.attn_fwd_packed(q, k, v, i32(cu), None, lse)
    chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), *parts(dx))
    assert chs.attn_status() == chs.ATTN_OK
    same = [y.contiguous() for y in (q, k, v)]
    assert torch.equal(o, chs.attn_fwd_packed(*same, i32(cu)))
    for a, b in zip(parts(dx), chs.attn_bwd_packed(*same, o, dout, lse, i32(cu))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("stride", [4, 8, 9999])
def test_one_row_of_one_head(Dh, stride):
    # an axis of one entry has any stride: softmax over one key, whose gradient is 0 but dv's
    x = torch.randn(4, Dh, device="cuda").to(torch.bfloat16)
    q, k, v, dout = (y.as_strided((1, 1, Dh), (stride, stride + 3, 1)) for y in x)
    o, lse = torch.zeros(1, 1, Dh, device="cuda", dtype=torch.bfloat16), torch.zeros(1, 1, device="cuda")
    out = [torch.zeros_like(o) for _ in range(3)]
    places = [y.as_strided((1, 1, Dh), (stride, stride + 3, 1)) for y in (o, *out)]
    chs.attn_fwd_packed(q, k, v, i32([0, 1]), places[0], lse)
    chs.attn_bwd_packed(q, k, v, places[0], dout, lse, i32([0, 1]), *places[1:])
    assert chs.attn_status() == chs.ATTN_OK
    assert torch.equal(o[0, 0], v[0, 0]) and torch.equal(out[2][0, 0], dout[0, 0])
    want, L, bound, dwant, dbound = ref.attention(q, k, v, [0, 1], dout=dout)
    assert abs(float(lse) - float(L)) < ref.F
    for got, w, b in zip(out, dwant, dbound):
        ref.check(got, w, b)


@pytest.mark.parametrize("Dh,n", [(64, 2560), (128, 768), (128, 2560), (256, 768)])
def test_one_sequence_is_the_batch_form(Dh, n):
    gen = torch.Generator("cuda").manual_seed(5)
    q, k, v = ref.layouts(n, 8, 2, Dh, "heads_first", gen)
    dout = ref.layouts(n, 8, 2, Dh, "heads_first", gen)[0]
    lse = torch.zeros(8, n, device="cuda")
    o = chs.attn_fwd_packed(q, k, v, i32([0, n]), None, lse, window=333)
    grads = chs.attn_bwd_packed(q, k, v, o, dout, lse, i32([0, n]), window=333)
    batch = [x.transpose(0, 1)[None].contiguous() for x in (q, k, v, dout)]
    o2, lse2 = chs.attn_fwd_lse(*batch[:3], window=333)
    grads2 = chs.attn_bwd(*batch[:3], o2, batch[3], lse2, window=333)
    assert chs.attn_status() == chs.ATTN_OK
    # each within its bound of the same values (the two may choose tiles of other sizes)
    _, _, bound, _, bounds = ref.attention(q, k, v, [0, n], True, 333, dout=dout)
    assert bool(((o.double() - o2[0].transpose(0, 1).double()).abs() <= 2 * bound).all())
    assert float((lse - lse2[0]).abs().max()) < 2 * ref.F
    for a, b, bound in zip(grads, grads2, bounds):
        assert bool(((a.double() - b[0].transpose(0, 1).double()).abs() <= 2 * bound).all())


@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_sequence_keeps_to_itself(Dh, value):
    lens = [100, 30, 200, 1, 129, 127]
    q, k, v, dout, cu, T = case(lens, 4, 2, Dh)
    o, lse, grads = run(q, k, v, dout, cu, True, 0)
    for b in (1, 3, 4):
        for x in (q, k, v, dout):
            x[cu[b]:cu[b + 1]] = value
    o2, lse2, grads2 = run(q, k, v, dout, cu, True, 0)
    for b in (0, 2, 5):
        rows = slice(cu[b], cu[b + 1])
        assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])
        assert all(torch.equal(x[rows], y[rows]) for x, y in zip(grads, grads2))


@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_many_sequences(Dh):
    # more sequences than the listing has warps, more tiles than SMs
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (1500,), generator=gen).tolist()
    q, k, v, dout, cu, T = case(lens, 2, 1, Dh, "contiguous")
    o, lse, grads = run(q, k, v, dout, cu, True, 0, kind="contiguous")
    real = slice(cu[0], cu[-1])
    want, L, bound, dwant, dbound = ref.attention(q, k, v, cu, dout=dout)
    ref.check(o[real], want[real], bound[real], "o")
    for name, got, w, b in zip(("dq", "dk", "dv"), grads, dwant, dbound):
        ref.check(got[real], w[real], b[real], name)


@pytest.mark.parametrize("Dh,lens", [(64, [3000, 5, 2500]), (128, [3300, 2900, 900]),
                                     (128, [700, 900, 40, 1300]), (256, [2000, 1300])])
def test_several_items_a_cta(Dh, lens):
    # many heads: every SM takes several blocks, of its own list and of the launch's
    q, k, v, dout, cu, T = case(lens, 32, 4, Dh)
    real = slice(cu[0], cu[-1])
    want, _, bound = ref.attention(q, k, v, cu, True, 600)
    whole, _, wide = ref.attention(q, k, v, cu, False)
    o, p = torch.full_like(q, 7), torch.full_like(q, 7)
    chs.attn_fwd_packed(q, k, v, i32(cu), o, window=600)
    chs.attn_fwd_packed(q, k, v, i32(cu), p, causal=False)
    assert chs.attn_status() == chs.ATTN_OK
    ref.check(o[real], want[real], bound[real], "causal")
    ref.check(p[real], whole[real], wide[real], "not causal")
    assert outside_is(o, 7, cu) and outside_is(p, 7, cu)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 7), (False, 0)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 1), (4, 2), (16, 2), (3, 3)])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_short_sequences(Dh, Hq, Hkv, causal, window):
    # lengths about those where two and four heads share a tile, few sequences and many
    # (62 rows on average: folded in the backward pass too)
    few = [1, 2, 31, 32, 33, 63, 64, 65, 0, 100, 16, 129, 300, 5]
    for lens in (few, few * 6):
        q, k, v, dout, cu, T = case(lens, Hq, Hkv, Dh, "heads_first" if Dh == 128 else "fused", seed=Hq)
        o, lse = torch.full_like(dout, 7), torch.full((Hq, T), 7.0, device="cuda")
        chs.attn_fwd_packed(q, k, v, i32(cu), o, lse, causal=causal, window=window)
        assert chs.attn_status() == chs.ATTN_OK
        real = slice(cu[0], cu[-1])
        grads = [torch.full_like(x, 7) for x in (dout, k, v)]
        chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), *grads, causal=causal, window=window)
        assert chs.attn_status() == chs.ATTN_OK
        want, L, bound, dwant, dbound = ref.attention(q, k, v, cu, causal, window, dout=dout)
        ref.check(o[real], want[real], bound[real], len(lens))
        for name, got, w, b in zip(("dq", "dk", "dv"), grads, dwant, dbound):
            ref.check(got[real], w[real], b[real], name)
            assert outside_is(got, 7, cu)
        assert float((lse[:, real] - L[:, real]).abs().max()) < ref.F
        assert outside_is(o, 7, cu) and outside_is(lse, 7, cu, 1)


def test_workspaces():
    gen = torch.Generator("cuda").manual_seed(0)
    q, k, v = ref.layouts(2000, 4, 2, 128, "fused", gen)
    cu = i32([0, 700, 2000])
    assert chs.attn_packed_workspace(q, cu) == 0          # few sequences: none
    many = i32(list(range(0, 2001, 20)))
    need = chs.attn_packed_workspace(q, many)
    assert need > 0
    back = chs.attn_packed_workspace(q, cu, backward=True)
    want = chs.attn_fwd_packed(q, k, v, many)
    with pytest.raises(chs.AttnError):
        chs.attn_fwd_packed(q, k, v, many, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    ws = torch.full((max(need, back),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(chs.attn_fwd_packed(q, k, v, many, workspace=ws), want)
    lse = torch.zeros(4, 2000, device="cuda")
    o = chs.attn_fwd_packed(q, k, v, cu, None, lse, workspace=ws)
    grads = chs.attn_bwd_packed(q, k, v, o, o, lse, cu, workspace=ws)
    again = chs.attn_bwd_packed(q, k, v, o, o, lse, cu)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)) and chs.attn_status() == chs.ATTN_OK


def test_gradients_against_differences():
    # a step of the loss sum(o * dout) along a direction; 64-bit reference at both ends
    q, k, v, dout, cu, T = case([70, 130], 4, 2, 64, "contiguous", seed=9)
    for x in (q, k, v, dout):
        x[:AHEAD] = x[cu[-1]:] = 0
    o, lse, grads = run(q, k, v, dout, cu, True, 50, kind="contiguous")
    gen = torch.Generator("cuda").manual_seed(2)
    real = slice(cu[0], cu[-1])
    bounds = ref.attention(q, k, v, cu, True, 50, dout=dout)[4]
    for i, g in enumerate(grads):
        step = torch.randn(g.shape, generator=gen, device="cuda", dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            x = [t.double() for t in (q, k, v)]
            x[i] = x[i] + sign * 1e-5 * step
            y = ref.attention(*x, cu, True, 50)[0]
            ends.append(float((y * dout.double()).sum()))
        slope = (ends[0] - ends[1]) / 2e-5
        got = float((g.double() * step)[real].sum())
        # the gradient's own bound along the direction, and the difference's cubic term
        assert abs(got - slope) <= float((bounds[i] * step.abs()).sum()) + 1e-4 * abs(slope)


@pytest.mark.parametrize("lens,causal,window", [([2, 5, 9, 3, 30] * 8, True, 0), ([40, 90, 130] * 4, True, 0),
                                                ([900, 1400], True, 20), ([3, 17, 32] * 8, False, 0)])
@pytest.mark.parametrize("Dh", [64, 128, 256])
def test_few_keys_lose_no_precision(Dh, lens, causal, window):
    """Where queries see few keys nothing averages rounding errors out.  The gradients' relative error
    (2-norm) is that of one rounding: half a step is uniform in +-2^-8 of a value's binade, which is
    at most 2^-8 / sqrt(3) = 0.00226 of the values; the parts that P and dS are held to (2^-16) and
    D's (fp32) add a twentieth of it at most where a row's keys are more than 32."""
    q, k, v, dout, cu, T = case(lens, 4, 2, Dh, "contiguous", seed=1)
    o, lse, grads = run(q, k, v, dout, cu, causal, window, kind="contiguous")
    real = slice(cu[0], cu[-1])
    dwant = ref.attention(q, k, v, cu, causal, window, dout=dout)[3]
    for got, w in zip(grads, dwant):
        off = float((got[real].double() - w[real]).norm() / w[real].norm())
        assert off <= 1.05 * 2.0 ** -8 / 3 ** 0.5, off


def test_no_rows_and_no_sequences():
    x = torch.full((0, 4, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    assert chs.attn_fwd_packed(x, x, x, i32([0, 0])).shape == (0, 4, 64)
    y = torch.ones(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(y, 7)
    chs.attn_fwd_packed(y, y, y, i32([0]), o)
    assert bool((o == 7).all())
    for cu in (i32([3, 3, 3]), i32([6] * 100)):
        chs.attn_fwd_packed(y, y, y, cu, o)
        lse = torch.zeros(4, 6, device="cuda")
        chs.attn_bwd_packed(y, y, y, y, y, lse, cu, o, torch.empty_like(o), torch.empty_like(o))
    assert bool((o == 7).all()) and chs.attn_status() == chs.ATTN_OK


@pytest.mark.parametrize("cu", [[0, 9, 5, 12], [-1, 4, 8, 12], [0, 4, 8, 13], [3, 2, 8, 12]])
def test_unsound_offsets_write_nothing(cu):
    gen = torch.Generator("cuda").manual_seed(0)
    q, k, v = ref.layouts(12, 4, 2, 128, "fused", gen)
    dout = torch.ones(12, 4, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(dout, 7), torch.full((4, 12), 7.0, device="cuda")
    chs.attn_fwd_packed(q, k, v, i32(cu), o, lse)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
    grads = [torch.full_like(x, 7) for x in (q, k, v)]
    chs.attn_bwd_packed(q, k, v, dout, dout, lse, i32(cu), *grads)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
    assert all(bool((x == 7).all()) for x in (o, lse, *grads))


def test_captured_calls_follow_new_offsets():
    gen = torch.Generator("cuda").manual_seed(4)
    T, Hq, Hkv, Dh = 1500, 4, 2, 128
    q, k, v = ref.layouts(T, Hq, Hkv, Dh, "fused", gen)
    dout = ref.layouts(T, Hq, Hkv, Dh, "contiguous", gen)[0]
    cu = i32([0, 700, 700, 1500])
    o, lse = torch.zeros(T, Hq, Dh, dtype=torch.bfloat16, device="cuda"), torch.zeros(Hq, T, device="cuda")
    grads = [torch.zeros_like(x) for x in (dout, k, v)]
    grads = [x.contiguous() for x in grads]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def step():
        chs.attn_fwd_packed(q, k, v, cu, o, lse)
        chs.attn_bwd_packed(q, k, v, o, dout, lse, cu, *grads)
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for offsets in ([0, 1, 64, 1500], [10, 400, 1100, 1400]):
        cu.copy_(i32(offsets))
        for x in (o, *grads):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (o, *grads)]
        want, _, bound, dwant, dbound = ref.attention(q, k, v, offsets, dout=dout)
        for a, b, c in zip(got, (want, *dwant), (bound, *dbound)):
            ref.check(a, b, c)
    assert chs.attn_status() == chs.ATTN_OK


def test_two_streams_at_once():
    gen = torch.Generator("cuda").manual_seed(6)
    sets = []
    for lens in ([900, 5, 300], [64, 2000]):
        cu = ref.offsets(lens)
        q, k, v = ref.layouts(cu[-1], 8, 2, 128, "fused", gen)
        sets.append((q, k, v, ref.layouts(cu[-1], 8, 2, 128, "contiguous", gen)[0], i32(cu)))

    def both(s, stream=None):
        q, k, v, dout, cu = s
        lse = torch.zeros(8, q.shape[0], device="cuda")
        o = torch.zeros_like(dout)
        grads = [torch.zeros_like(x) for x in (q, k, v)]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            chs.attn_fwd_packed(q, k, v, cu, o, lse, stream=stream)
            chs.attn_bwd_packed(q, k, v, o, dout, lse, cu, *grads, stream=stream)
        return (o, lse, *grads)
    alone = [both(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    at_once = [both(s, x) for s, x in zip(sets, streams)]
    torch.cuda.synchronize()
    assert chs.attn_status() == chs.ATTN_OK
    for a, b in zip(alone, at_once):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
