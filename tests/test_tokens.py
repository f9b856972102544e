"""Rotary positions, their write to the paged cache and the plan of a serving
step on the GPU, against 64-bit formulas and host loops; then a whole step."""
import math
import random

import pytest
import torch

import causal_head_self_gb300 as chs
import packed_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8   # half a step of bf16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=None, n=8192):
    """Radians per token in 64 bits, and the amplitude."""
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "base":
        base *= factor ** (rot / (rot - 2))
        f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling in ("turns", "yarn"):
        high = high or (4.0 if scaling == "turns" else 32.0)
        for i, x in enumerate(f):
            keep = min(1, max(0, (n * x / (2 * math.pi) - low) / (high - low)))
            f[i] = keep * x + (1 - keep) * x / factor
    return f, 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def turned(x, positions, freqs, interleaved=False, inverse=False):
    """x [..., rows, Dh] turned in 64 bits, and the bound: products and sums in fp32 with cosines
    and sines to 2^-21 of 1, one rounding to bf16."""
    f, amplitude = freqs
    rot = 2 * len(f)
    a = positions.double()[..., None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    cos, sin = amplitude * a.cos(), amplitude * a.sin() * (-1 if inverse else 1)
    one = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    two = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    x = x.double()
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    size = (x[..., one].abs() + x[..., two].abs()) * amplitude * 2.0 ** -21
    for part in (one, two):
        bound[..., part] = U * y[..., part].abs() + (1 + U) * size
    return y, bound


def close(got, want):
    y, bound = want
    err = (got.double() - y).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


ROPES = [
    (64, 64, False, "none", 1.0), (64, 16, True, "linear", 4.0), (128, 128, False, "yarn", 32.0),
    (128, 64, True, "turns", 8.0), (256, 256, True, "none", 1.0), (256, 48, False, "base", 40.0),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T", [1, 3, 64, 1000, 6007])
@pytest.mark.parametrize("Dh,rot,interleaved,scaling,factor", ROPES)
def test_rope(Dh, rot, interleaved, scaling, factor, T, inverse):
    gen = torch.Generator("cuda").manual_seed(T)
    Hq, Hkv = (8, 2) if T < 6000 else (5, 3)
    q, k, _ = ref.layouts(T, Hq, Hkv, Dh, ["fused", "heads_first", "wide"][T % 3], gen)
    pos = torch.randint(0, 2 ** 31 - 1 if T % 2 else 5000, (T,), generator=gen, device="cuda",
                        dtype=torch.int32)
    pos[::7] = -3   # left out
    handle = chs.attn_rope_frequencies(rot, scaling=scaling, factor=factor)
    exact = frequencies(rot, scaling=scaling, factor=factor)
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    chs.attn_rope(q, k, pos, handle, qo, ko, interleaved=interleaved, inverse=inverse)
    assert chs.attn_status() == chs.ATTN_OK
    there = pos >= 0
    # the 64-bit formula's own angle is good to 2^-52 of it: 2^31 * 2^-52 at the largest position
    for x, y in ((q, qo), (k, ko)):
        close(y[there].transpose(0, 1), turned(x[there].transpose(0, 1), pos[there], exact,
                                               interleaved, inverse))
        assert bool((y[~there] == 7).all())
        assert torch.equal(y[there][..., rot:], x[there][..., rot:])
    # in place: the same bits
    want_q, want_k = torch.where(there[:, None, None], qo, q), torch.where(there[:, None, None], ko, k)
    chs.attn_rope(q, k, pos, handle, q, k, interleaved=interleaved, inverse=inverse)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)


@pytest.mark.parametrize("Dh,rot", [(64, 64), (128, 64), (256, 256)])
def test_rope_of_a_batch(Dh, rot):
    gen = torch.Generator("cuda").manual_seed(1)
    B, Hq, Hkv, S = 3, 4, 1, 37
    q = torch.randn(B, Hq, S, Dh, generator=gen, device="cuda").to(torch.bfloat16)
    k = torch.randn(B, S, Hkv, Dh, generator=gen, device="cuda").to(torch.bfloat16).transpose(1, 2)
    pos = torch.randint(0, 9999, (B, S), generator=gen, device="cuda", dtype=torch.int32)
    handle = chs.attn_rope_frequencies(rot)
    qo, ko = chs.attn_rope(q, k, pos, handle)
    assert chs.attn_status() == chs.ATTN_OK
    for x, y in ((q, qo), (k, ko)):
        close(y, turned(x, pos[:, None], frequencies(rot)))


@pytest.mark.parametrize("axis", [1, 2])
def test_rope_inside_one_tensor(axis):
    # queries and keys as parts of a projection's output [T, 3, H, Dh] or [T, H, 3, Dh], in place
    gen = torch.Generator("cuda").manual_seed(2)
    T, H, Dh = 70, 3, 128
    x = torch.randn((T, 3, H, Dh) if axis == 1 else (T, H, 3, Dh), generator=gen,
                    device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    handle = chs.attn_rope_frequencies(Dh)
    q, k, v = x.unbind(axis)
    want = chs.attn_rope(q.contiguous(), k.contiguous(), pos, handle)
    kept = v.clone()
    chs.attn_rope(q, k, pos, handle, q, k)
    assert chs.attn_status() == chs.ATTN_OK
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


def test_rope_gradient_and_infinities():
    # <turn(x), y> = <x, turn back(y)>: the inverse carries gradients; values that are not
    # turned are copied whatever they are
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(50, 4, 128, generator=gen, device="cuda").to(torch.bfloat16)
    y = torch.randn(50, 4, 128, generator=gen, device="cuda").to(torch.bfloat16)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    handle = chs.attn_rope_frequencies(64, scaling="yarn", factor=8.0)
    tx, _ = chs.attn_rope(x, x, pos, handle)
    ty, _ = chs.attn_rope(y, y, pos, handle, inverse=True)
    one, two = (tx.double() * y.double()), (x.double() * ty.double())
    # each side's rounding: u of each product (and the cosines' 2^-21)
    assert abs(float(one.sum() - two.sum())) <= (U + 2.0 ** -19) * float(one.abs().sum() + two.abs().sum())
    x[:, :, 64:] = float("nan")
    x[:, :, 65] = float("inf")
    again, _ = chs.attn_rope(x, x, pos, handle)
    assert torch.equal(again[..., :64], tx[..., :64])
    assert bool(again[..., 64].isnan().all()) and bool((again[..., 65] == float("inf")).all())


def pools(P, Hkv, page, Dh):
    return (torch.full((P, Hkv, page, Dh), 7, dtype=torch.bfloat16, device="cuda") for _ in range(2))


@pytest.mark.parametrize("k_out", [True, False])
@pytest.mark.parametrize("T", [1, 64, 3001])
@pytest.mark.parametrize("Dh,rot,interleaved,scaling,factor", ROPES + [(128, 0, False, "none", 1.0)])
def test_rope_append(Dh, rot, interleaved, scaling, factor, T, k_out):
    gen = torch.Generator("cuda").manual_seed(T + rot)
    Hq, Hkv, page = 6, 2, 24
    P = T // page + 5
    q, k, v = ref.layouts(T, Hq, Hkv, Dh, "fused", gen)
    pos = torch.randint(0, 100000, (T,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(P * page, generator=gen, device="cuda")[:T].to(torch.int32)
    pos[5::11] = -1       # left out altogether
    slots[3::13] = -1     # turned, not cached
    if rot:
        handle = chs.attn_rope_frequencies(rot, scaling=scaling, factor=factor)
    else:
        handle = chs.RopeFrequencies(torch.empty(0, dtype=torch.int64, device="cuda"), 1.0)
    kp, vp = pools(P, Hkv, page, Dh)
    want_q, want_k = chs.attn_rope(q, k, pos, handle, q.clone(), k.clone(), interleaved=interleaved)
    before = q.clone(), k.clone()
    qo, ko = torch.full_like(q, 3), torch.full_like(k, 3)
    chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots, qo, ko if k_out else None,
                         interleaved=interleaved)
    assert chs.attn_status() == chs.ATTN_OK
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    there = pos >= 0
    assert torch.equal(qo[there], want_q[there]) and bool((qo[~there] == 3).all())
    if k_out:
        assert torch.equal(ko[there], want_k[there]) and bool((ko[~there] == 3).all())
    t = (there & (slots >= 0)).nonzero()[:, 0]
    expect_k, expect_v = pools(P, Hkv, page, Dh)
    at = slots[t].long()
    expect_k[at // page, :, at % page] = want_k[t]
    expect_v[at // page, :, at % page] = v[t]
    assert torch.equal(kp, expect_k) and torch.equal(vp, expect_v)
    # queries and keys in place
    chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots, None, k, interleaved=interleaved)
    assert torch.equal(q[there], want_q[there]) and torch.equal(k[there], want_k[there])
    assert torch.equal(kp, expect_k) and torch.equal(vp, expect_v)


def test_rope_append_of_a_decode_step():
    # [B, H, 1, Dh], as attn_decode_paged takes the queries
    gen = torch.Generator("cuda").manual_seed(4)
    B, Hq, Hkv, Dh, page = 5, 4, 2, 128, 8
    q, k, v = (torch.randn(B, h, 1, Dh, generator=gen, device="cuda").to(torch.bfloat16)
               for h in (Hq, Hkv, Hkv))
    pos, slots = i32([[7], [100000], [0], [-1], [12]]), i32([[5], [31], [0], [-1], [-1]])
    kp, vp = pools(4, Hkv, page, Dh)
    handle = chs.attn_rope_frequencies(Dh)
    want_q, want_k = chs.attn_rope(q, k, pos, handle, q.clone(), k.clone())
    qo, _ = chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots)
    assert chs.attn_status() == chs.ATTN_OK and qo is q and torch.equal(q, want_q)
    for b, s in enumerate([5, 31, 0]):
        assert torch.equal(kp[s // page, :, s % page], want_k[b, :, 0])
        assert torch.equal(vp[s // page, :, s % page], v[b, :, 0])
    assert int((vp != 7).sum()) == 3 * Hkv * Dh


def test_slots_outside_the_pools():
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    kp, vp = pools(3, 2, 8, 64)
    handle = chs.attn_rope_frequencies(64)
    chs.attn_rope_append(q, q.clone(), q.clone(), i32([0, 1, 2, 3]), handle, kp, vp,
                         i32([24, 5, 2 ** 31 - 1, -5]), torch.zeros_like(q))
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
    assert int((vp != 7).sum()) == 2 * 64 and bool((vp[0, :, 5] == 1).all())


# ---------------------------------------------------------------- the plan

def plan_case(rng, B, page, lmax, grow, spare=8):
    lens, delta = [], []
    for _ in range(B):
        n = rng.choice((0, rng.randint(0, lmax)))
        lens.append(n)
        delta.append(rng.choice((0, -n, -rng.randint(0, n), rng.randint(0, grow), rng.randint(0, grow))))
    cols = -(-(lmax + grow) // page) + 1
    held = [-(-n // page) for n in lens]
    need = sum(max(0, -(-(n + d) // page)) for n, d in zip(lens, delta))
    free = max(0, need - sum(held)) + spare
    P = sum(held) + free + 3
    pages = list(range(P))
    rng.shuffle(pages)
    table = [[-9] * cols for _ in range(B)]
    for b in range(B):
        for i in range(held[b]):
            table[b][i] = pages.pop()
    stack = [pages.pop() for _ in range(free)]
    return lens, delta, table, stack, P


def plan_by_hand(lens, delta, table, stack, page):
    table, stack = [list(r) for r in table], list(stack)
    for b, (n, d) in enumerate(zip(lens, delta)):
        for i in range(-(-(n + d) // page), -(-n // page)):
            stack.append(table[b][i])
    cu, positions, slots = [0], [], []
    for b, (n, d) in enumerate(zip(lens, delta)):
        for i in range(-(-n // page), -(-(n + d) // page)):
            table[b][i] = stack.pop()
        for t in range(n, n + d):
            positions.append(t)
            slots.append(table[b][t // page] * page + t % page)
        cu.append(len(positions))
    return table, stack, cu, positions, slots


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,page,lmax,grow", [
    (1, 8, 0, 1), (1, 16, 100, 5), (5, 24, 300, 40), (64, 16, 1000, 1), (33, 64, 200, 700),
    (1025, 16, 60, 3), (3000, 8, 90, 20), (8192, 8, 20, 2), (2, 256, 5000, 9000), (300, 16, 700, 400)])
def test_plan(B, page, lmax, grow, in_place):
    rng = random.Random(B + page)
    lens, delta, table, stack, P = plan_case(rng, B, page, lmax, grow)
    want_table, want_stack, cu, positions, slots = plan_by_hand(lens, delta, table, stack, page)
    T = len(positions) + rng.choice((0, 1, 50))
    capacity = P
    free = i32(stack + [-7] * (capacity - len(stack)))
    seqlens, num_free, tab = i32(lens), i32([len(stack)]), i32(table)
    outs = {} if in_place else dict(seqlens_out=torch.zeros_like(seqlens), num_free_out=i32([0]))
    for again in range(1 if in_place else 2):   # (apart from the inputs: the same once more)
        got = chs.attn_cache_plan(i32(delta), seqlens, tab, free, num_free, rows=T, page=page,
                                  num_pages=P, **outs)
        assert chs.attn_status() == chs.ATTN_OK
        if not in_place:
            assert seqlens.tolist() == lens and num_free.tolist() == [len(stack)]
        after = outs.get("seqlens_out", seqlens)
        height = outs.get("num_free_out", num_free)
        assert after.tolist() == [n + d for n, d in zip(lens, delta)]
        assert height.tolist() == [len(want_stack)] and free[:len(want_stack)].tolist() == want_stack
        assert tab.tolist() == want_table
        rest = [-1] * (T - len(positions))
        assert [x.tolist() for x in got] == [cu, positions + rest, slots + rest]


def plan(lens, delta, table, stack, T, page=8, num_pages=100, capacity=None):
    capacity = capacity or len(stack) + 20
    state = dict(seqlens=i32(lens), table=i32(table), free_pages=i32(stack + [-7] * (capacity - len(stack))),
                 num_free=i32([len(stack)]))
    before = {k: v.clone() for k, v in state.items()}
    got = chs.attn_cache_plan(i32(delta), **state, rows=T, page=page, num_pages=num_pages)
    same = {k: torch.equal(v, before[k]) for k, v in state.items()}
    return [x.tolist() for x in got], state, same


def test_plan_is_all_or_nothing():
    table = [[3, -1, -1], [4, 5, -1]]
    # (a change past the table's 24 rows is not the step's failure but its sequence's)
    got, state, _ = plan([5, 9], [20, 1], table, [6], 30)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
    assert state["seqlens"].tolist() == [5, 10] and got[0] == [0, 0, 1]
    got, _, same = plan([5, 9], [19, 1], table, [6], 30)
    assert chs.attn_status() == chs.ATTN_ERR_NO_MEMORY and all(same.values())
    assert got == [[0, 0, 0], [-1] * 30, [-1] * 30]
    # a buffer for fewer rows than there are tokens takes the first ones'
    got, state, _ = plan([5, 9], [3, 3], table, [6, 7], 5)
    assert chs.attn_status() == chs.ATTN_OK and state["seqlens"].tolist() == [8, 12]
    assert got == [[0, 3, 6], [5, 6, 7, 9, 10], [29, 30, 31, 41, 42]]
    # the stack may not pass its capacity
    got, _, same = plan([5, 9], [-5, 0], table, [6], 4, capacity=1)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG and all(same.values())
    # pages that one sequence gives back serve another
    got, state, _ = plan([5, 9], [4, -9], table, [], 4)
    assert chs.attn_status() == chs.ATTN_OK
    assert state["table"].tolist()[0] == [3, 5, -1] and state["num_free"].tolist() == [1]
    assert state["free_pages"].tolist()[0] == 4
    assert got[2] == [29, 30, 31, 40]


@pytest.mark.parametrize("T", [0, 1, 5000, 20000])
def test_a_plan_of_no_sequences(T):
    none, table = i32([]), torch.empty((0, 4), dtype=torch.int32, device="cuda")
    num_free, height = i32([2]), i32([-9])
    out = [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (1, T, T)]
    cu, positions, slots = chs.attn_cache_plan(none, none, table, i32([5, 6, 7]), num_free, rows=T, page=8,
                                               num_pages=9, num_free_out=height, cu_seqlens=out[0],
                                               positions=out[1], slots=out[2])
    assert chs.attn_status() == chs.ATTN_OK and height.tolist() == [2]
    assert cu.tolist() == [0] and bool((positions == -1).all()) and bool((slots == -1).all())


@pytest.mark.parametrize("n,d", [(-1, 3), (25, 0), (20, 5), (5, -6), (2 ** 31 - 1, 1), (0, -(2 ** 31))])
def test_a_length_out_of_range_leaves_its_sequence(n, d):
    got, state, _ = plan([5, n, 9], [1, d, 8], [[3, -1, -1], [8, 9, 9], [4, 5, -1]], [6, 7], 10)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG
    assert state["seqlens"].tolist() == [6, n, 17] and got[0] == [0, 1, 1, 9]
    assert state["table"].tolist() == [[3, -1, -1], [8, 9, 9], [4, 5, 7]]
    assert got[2][:9] == [29] + [41, 42, 43, 44, 45, 46, 47, 56]


def test_page_numbers_outside_the_pool():
    got, _, _ = plan([5], [4], [[200, -1, -1]], [3], 4)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG and got[2] == [-1, -1, -1, 24]
    got, _, _ = plan([5], [4], [[2, -1, -1]], [-3], 4)
    assert chs.attn_status() == chs.ATTN_ERR_INVALID_ARG and got[2] == [21, 22, 23, -1]


# ---------------------------------------------------------------- a server's steps

def test_prompts_then_tokens():
    """Prompts are planned, turned and cached, and attended to; then each request takes tokens of
    its own, one is finished and another admitted; all captured in one graph per kind of step."""
    gen = torch.Generator("cuda").manual_seed(8)
    Hq, Hkv, Dh, page, P, cols, B = 8, 2, 128, 16, 64, 12, 4
    kp, vp = pools(P, Hkv, page, Dh)
    handle, exact = chs.attn_rope_frequencies(Dh), frequencies(Dh)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    num_free, seqlens = i32([P]), i32([0] * B)
    keys = [torch.zeros(0, Hkv, Dh, device="cuda", dtype=torch.bfloat16) for _ in range(B)]
    values = [x.clone() for x in keys]

    def tokens(n):
        return ref.layouts(n, Hq, Hkv, Dh, "fused", gen)

    def note(delta, cu, pos, k, v):
        """What the cache holds: the library's own turned keys, checked against the formula."""
        for b, d in enumerate(delta):
            a, z = cu[b], cu[b + 1]
            if d < 0:
                keys[b], values[b] = keys[b][:len(keys[b]) + d], values[b][:len(values[b]) + d]
            n = len(keys[b])
            assert pos[a:z].tolist() == list(range(n, n + z - a))
            keys[b], values[b] = torch.cat([keys[b], k[a:z]]), torch.cat([values[b], v[a:z]])

    # a prefill step: three prompts in a buffer that is longer than their sum
    delta = [70, 1, 0, 129]
    T = sum(delta) + 11
    q, k, v = tokens(T)
    k0 = k.clone()
    cu, pos, slots = chs.attn_cache_plan(i32(delta), seqlens, table, free, num_free, rows=T, page=page,
                                         num_pages=P)
    chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots, None, k)
    o = torch.zeros(T, Hq, Dh, dtype=torch.bfloat16, device="cuda")
    chs.attn_fwd_packed(q, k, v, cu, o)
    assert chs.attn_status() == chs.ATTN_OK
    n = sum(delta)
    close(k[:n].transpose(0, 1), turned(k0[:n].transpose(0, 1), pos[:n], exact))
    want, _, bound = ref.attention(q, k, v, cu.tolist())
    ref.check(o, want, bound)
    note(delta, cu.tolist(), pos, k, v)

    # decode steps: one token each; request 1 is finished, place 2 starts with a token
    for delta in ([1, 1, 0, 1], [1, -2, 1, 1], [1, 0, 1, -3], [1, 0, 1, 1]):
        T = B
        q, k, v = tokens(T)
        cu, pos, slots = chs.attn_cache_plan(i32(delta), seqlens, table, free, num_free, rows=T,
                                             page=page, num_pages=P)
        chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots, None, k)
        first = cu.tolist()
        note(delta, first, pos, k, v)
        assert seqlens.tolist() == [len(x) for x in keys]
        held = sum(-(-len(x) // page) for x in keys)
        assert num_free.tolist() == [P - held]
        used = [table[b, :-(-len(keys[b]) // page)].tolist() for b in range(B)]
        pages = sum(used, []) + free[:P - held].tolist()
        assert sorted(pages) == list(range(P))   # every page once
        query = torch.zeros(B, Hq, 1, Dh, dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            if delta[b] == 1:
                query[b, :, 0] = q[first[b]]
        got = chs.attn_decode_paged(query, kp, vp, table, seqlens)
        assert chs.attn_status() == chs.ATTN_OK
        for b in range(B):
            if not len(keys[b]):
                assert bool((got[b] == 0).all())
                continue
            K = keys[b].double().repeat_interleave(Hq // Hkv, 1).transpose(0, 1)
            V = values[b].double().repeat_interleave(Hq // Hkv, 1).transpose(0, 1)
            p = torch.softmax(query[b].double() @ K.transpose(1, 2) * Dh ** -0.5, -1)
            want = p @ V
            err = (got[b].double() - want).abs()
            assert bool((err <= (1 + U) * (U + ref.F) * (p @ V.abs()) + U * want.abs()).all())


def test_captured_plan_and_rotation():
    # one graph, replayed while lengths grow in place
    gen = torch.Generator("cuda").manual_seed(3)
    Hq, Hkv, Dh, page, P, B = 4, 2, 64, 8, 40, 3
    kp, vp = pools(P, Hkv, page, Dh)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free, num_free = torch.arange(P, dtype=torch.int32, device="cuda"), i32([P])
    seqlens, delta = i32([0, 0, 0]), i32([1, 1, 1])
    q, k, v = ref.layouts(B, Hq, Hkv, Dh, "fused", gen)
    qo = torch.zeros(B, Hq, Dh, dtype=torch.bfloat16, device="cuda")
    cu, pos, slots = i32([0] * 4), i32([0] * 3), i32([0] * 3)
    handle = chs.attn_rope_frequencies(Dh)
    stream = torch.cuda.Stream()

    def step():
        chs.attn_cache_plan(delta, seqlens, table, free, num_free, rows=B, page=page, num_pages=P,
                            cu_seqlens=cu, positions=pos, slots=slots)
        chs.attn_rope_append(q, k, v, pos, handle, kp, vp, slots, qo)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for n in range(2, 20):
        graph.replay()
        torch.cuda.synchronize()
        assert seqlens.tolist() == [n] * 3 and pos.tolist() == [n - 1] * 3
        assert num_free.tolist() == [P - 3 * -(-n // page)]
        at = slots.long()
        close(kp[at // page, :, at % page].transpose(0, 1),
              turned(k.transpose(0, 1), pos, frequencies(Dh)))
    assert chs.attn_status() == chs.ATTN_OK
