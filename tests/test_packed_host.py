"""Argument checks of the packed calls, the rotations and the plan.  They come
before any CUDA call, so made-up (aligned, disjoint) addresses are safe: nothing
is dereferenced or launched."""
import ctypes
import math

import pytest
import torch

import causal_head_self_gb300 as chs
from causal_head_self_gb300 import _binding
from causal_head_self_gb300 import build as _build

INVALID, UNSUPPORTED, OK = chs.ATTN_ERR_INVALID_ARG, chs.ATTN_ERR_UNSUPPORTED, chs.ATTN_OK
SCRATCH = chs.ATTN_ERR_SCRATCH_LIMIT


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _binding.load()


def ptr(i):
    return (i + 1) << 40


def rows(i, H=4, Dh=128, **change):
    """Tensor number i: rows of H heads, packed densely."""
    x = dict(data=ptr(i), batch=1 << 20, row=H * Dh, head=Dh)
    x.update(change)
    return _binding.Rows(x["data"], x["batch"], x["row"], x["head"])


SHAPE = dict(B=2, Hq=4, Hkv=2, T=40, Dh=128, causal=1, window=0, scale=0.0)
HEADS = dict(q=4, k=2, v=2, o=4, dout=4, dq=4, dk=2, dv=2)


def fwd(lib, lse=ptr(20), cu=ptr(21), ws=ptr(22), ws_bytes=1 << 20, tensors=None, **shape):
    t = {n: rows(i, HEADS[n]) for i, n in enumerate("qkvo")}
    t.update(tensors or {})
    s = dict(SHAPE, **shape)
    return lib.attn_fwd_packed(*t.values(), lse, cu, ws, ws_bytes, s["B"], s["Hq"], s["Hkv"], s["T"],
                               s["Dh"], s["causal"], s["window"], s["scale"], None)


def bwd(lib, lse=ptr(20), cu=ptr(21), ws=ptr(22), ws_bytes=1 << 20, tensors=None, **shape):
    t = {n: rows(i, HEADS[n]) for i, n in enumerate(("q", "k", "v", "o", "dout", "dq", "dk", "dv"))}
    t.update(tensors or {})
    s = dict(SHAPE, **shape)
    t = list(t.values())
    return lib.attn_bwd_packed(*t[:5], lse, *t[5:], cu, ws, ws_bytes, s["B"], s["Hq"], s["Hkv"], s["T"],
                               s["Dh"], s["causal"], s["window"], s["scale"], None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("change,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Dh=96), UNSUPPORTED), (dict(causal=2), INVALID),
    (dict(causal=0, window=3), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(T=2 ** 31 - 1), INVALID), (dict(B=1 << 25), INVALID),        # padded rows
    (dict(T=1 << 30, Hq=1 << 9, Hkv=1 << 9), INVALID),                 # tiles times heads
    (dict(B=0), OK), (dict(T=0), OK)])
def test_packed_shapes(lib, call, change, code):
    assert call(lib, **change) == code


@pytest.mark.parametrize("call,names", [(fwd, ["q", "k", "v", "o"]),
                                        (bwd, ["q", "k", "v", "o", "dout", "dq", "dk", "dv"])])
def test_packed_tensors(lib, call, names):
    outputs = ["o"] if call is fwd else ["dq", "dk", "dv"]
    for i, n in enumerate(names):
        H = HEADS[n]
        for bad in (dict(data=None), dict(data=ptr(i) + 8), dict(row=H * 128 + 4), dict(head=132),
                    dict(row=120), dict(head=0), dict(row=-512), dict(head=1 << 39),
                    dict(row=1 << 38, head=1 << 38)):
            if bad == dict(row=1 << 38, head=1 << 38) and n not in outputs:
                continue   # (rows over heads: only an output's elements have to be distinct)
            assert call(lib, tensors={n: rows(i, H, **bad)}) == INVALID, (n, bad)
        if n in outputs:
            assert call(lib, tensors={n: rows(i, H, row=(H - 1) * 128)}) == INVALID
            for j, m in enumerate(names):
                if m != n:
                    assert call(lib, tensors={n: rows(j, H, data=ptr(j) + 256)}) == INVALID, (n, m)
            assert call(lib, lse=ptr(i)) == INVALID and call(lib, ws=ptr(i)) == INVALID
            assert call(lib, cu=ptr(i)) == INVALID
    for bad in (dict(cu=None), dict(cu=ptr(21) + 2), dict(lse=ptr(20) + 2), dict(ws=None),
                dict(ws=ptr(22) + 128), dict(ws=ptr(21)), dict(ws=ptr(20)), dict(ws=ptr(0))):
        assert call(lib, **bad) == INVALID, bad
    if call is bwd:
        assert call(lib, ws_bytes=255) == SCRATCH
        assert call(lib, lse=None) == INVALID


def test_slices_of_one_tensor_are_apart(lib):
    # q, k, v (and their gradients) along the heads of one projection pass the checks of
    # overlap: what stops the call is the workspace's size, the last check
    def slices(base, names, skip=0):
        out, at = {}, 0
        for n in names:
            out[n] = rows(0, data=base + at * 256, row=8 * 128)
            at += HEADS[n] - skip
        return out
    few = dict(ws_bytes=256)
    both = dict(slices(ptr(0), "qkv"), **slices(ptr(1), ("dq", "dk", "dv")),
                o=rows(2), dout=rows(3))
    order = ["q", "k", "v", "o", "dout", "dq", "dk", "dv"]
    assert bwd(lib, tensors={n: both[n] for n in order}, **few) == SCRATCH
    both.update(slices(ptr(1), ("dq", "dk", "dv"), skip=1))   # a head too close
    assert bwd(lib, tensors={n: both[n] for n in order}, **few) == INVALID
    # an output between the inputs' heads of the same tensor
    t = slices(ptr(0), "qkv")
    t["o"] = rows(0, data=ptr(0) + 4 * 256, row=8 * 128)
    assert fwd(lib, tensors=t, **few) == INVALID


@pytest.mark.parametrize("order", ["rows, part, head", "rows, head, part", "part, rows, head",
                                   "part, head, rows", "head, part, rows"])
def test_parts_of_one_tensor_are_apart(lib, order):
    # as many K/V heads as query heads: q, k, v (and their gradients) are the three parts of a
    # tensor with an axis of them, wherever that lies
    T, H, Dh, size = 40, 4, 128, dict(rows=40, part=3, head=4)
    step, at = {}, Dh
    for axis in reversed(order.split(", ")):
        step[axis], at = at, at * size[axis]

    def part(i, n, by=0):
        return rows(i, data=ptr(i) + 2 * (n * step["part"] + by), row=step["rows"], head=step["head"])
    t = dict(q=part(0, 0), k=part(0, 1), v=part(0, 2), o=rows(2), dout=rows(3), dq=part(1, 0),
             dk=part(1, 1), dv=part(1, 2))
    few = dict(ws_bytes=256, Hkv=H)   # the workspace's size is the last check
    assert bwd(lib, tensors=t, **few) == SCRATCH
    for off in (-8, 8):
        assert bwd(lib, tensors=dict(t, dk=part(1, 1, off)), **few) == INVALID
    assert bwd(lib, tensors=dict(t, dv=part(1, 1)), **few) == INVALID
    assert bwd(lib, tensors=dict(t, dv=part(0, 2)), **few) == INVALID
    # a rotation in place (one that is sound would be launched: only what is refused here)
    inside = dict(B=1, S=T, Hq=H, Hkv=H, q=part(0, 0), qo=part(0, 0), k=part(0, 1), ko=part(0, 1))
    assert rope(lib, **dict(inside, ko=part(0, 1, 8))) == INVALID
    assert rope(lib, **dict(inside, k=part(0, 0, 64), ko=part(0, 0, 64))) == INVALID


def test_packed_workspace_queries(lib):
    # (the forward's answer depends on the GPU: only its refusals here)
    n = ctypes.c_size_t()
    assert lib.attn_bwd_packed_workspace(3, 8, 1000, ctypes.byref(n)) == OK
    assert n.value >= 2 * 16 * (1000 // 128 + 3) + 2 * 4 * 8 * 1000
    assert lib.attn_bwd_packed_workspace(3, 8, 1000, None) == INVALID
    for bad in ((-1, 8, 1000), (3, 0, 1000), (3, 8, -1), (3, 8, 2 ** 31 - 1), (1 << 25, 8, 1000)):
        assert lib.attn_bwd_packed_workspace(*bad, ctypes.byref(n)) == INVALID, bad
        assert lib.attn_fwd_packed_workspace(*bad, 128, 1, ctypes.byref(n)) == INVALID, bad
    assert lib.attn_fwd_packed_workspace(3, 8, 1000, 96, 1, ctypes.byref(n)) == UNSUPPORTED
    assert lib.attn_fwd_packed_workspace(3, 8, 1000, 128, 2, ctypes.byref(n)) == INVALID
    assert lib.attn_fwd_packed_workspace(3, 8, 1000, 128, 1, None) == INVALID


def rope(lib, append=False, q=None, qo=None, k=None, ko="given", v=None, positions=ptr(20),
         turns=ptr(21), slots=ptr(22), kp=ptr(23), vp=ptr(24), Hq=4, Hkv=2, P=9, page=16, B=2, S=20,
         Dh=128, rot=128, interleaved=0, inverse=0, amplitude=1.0):
    q, qo, k, v = q or rows(0), qo or rows(1), k or rows(2, 2), v or rows(4, 2)
    ko = rows(3, 2) if ko == "given" else ko
    if append:
        return lib.attn_rope_append(q, qo, Hq, k, ko, v, Hkv, positions, turns, amplitude, kp, vp, slots,
                                    P, page, B, S, Dh, rot, interleaved, None)
    return lib.attn_rope(q, qo, Hq, k, ko, Hkv, positions, turns, amplitude, B, S, Dh, rot, interleaved,
                         inverse, None)


@pytest.mark.parametrize("append", [False, True])
def test_rope_refusals(lib, append):
    def call(**change):
        return rope(lib, append, **change)
    for bad in (dict(B=-1), dict(S=-1), dict(Hq=-1), dict(Hkv=-1), dict(Hq=0, Hkv=0), dict(rot=8),
                dict(rot=144), dict(rot=-16), dict(interleaved=2), dict(amplitude=math.inf),
                dict(amplitude=math.nan), dict(B=1 << 16, S=1 << 15), dict(positions=None),
                dict(positions=ptr(20) + 2), dict(turns=None), dict(turns=ptr(21) + 4),
                dict(q=rows(0, data=ptr(0) + 2)), dict(q=rows(0, row=500)), dict(q=rows(0, head=-128)),
                dict(qo=rows(1, row=0)), dict(qo=rows(1, head=64)), dict(qo=rows(1, row=256)),
                dict(ko=rows(3, 2, batch=2560)),           # batches over one another
                dict(qo=rows(0, data=ptr(0) + 256)),       # neither the input nor apart from it
                dict(qo=rows(2)), dict(ko=rows(0, 2)), dict(ko=rows(1, 2)),
                dict(positions=ptr(1)), dict(turns=ptr(3))):
        assert call(**bad) == INVALID, bad
    assert call(Dh=96) == UNSUPPORTED
    assert call(B=0) == OK and call(S=0) == OK
    if not append:
        assert call(inverse=2) == INVALID and call(ko=None) == INVALID
        return
    for bad in (dict(Hkv=0), dict(P=0), dict(page=0), dict(P=1 << 27, page=16), dict(slots=None),
                dict(slots=ptr(22) + 2), dict(kp=None), dict(vp=ptr(24) + 8), dict(vp=ptr(23) + 256),
                dict(kp=ptr(0)), dict(vp=ptr(1)), dict(kp=ptr(4)), dict(vp=ptr(20)), dict(kp=ptr(21)),
                dict(vp=ptr(22)), dict(v=rows(4, 2, data=None)), dict(qo=rows(4)), dict(slots=ptr(1)),
                dict(ko=rows(4, 2))):
        assert call(**bad) == INVALID, bad
    assert call(page=12) == UNSUPPORTED


def test_rope_frequencies(lib):
    handle = chs.attn_rope_frequencies(64, 500000.0, device="cpu")
    assert handle.amplitude == 1.0 and handle.turns.shape == (32,)
    for i, t in enumerate(handle.turns.tolist()):
        want = 500000.0 ** (-2 * i / 64) / (2 * math.pi)
        # 64-bit arithmetic on both sides, and the unit of the table: 2^-64
        assert abs(t / 2.0 ** 64 - want) <= 2.0 ** -50 * want + 2.0 ** -64
    yarn = chs.attn_rope_frequencies(64, scaling="yarn", factor=4.0, original_len=4096, device="cpu")
    plain = chs.attn_rope_frequencies(64, device="cpu")
    assert yarn.amplitude == pytest.approx(0.1 * math.log(4.0) + 1, rel=1e-6)
    assert yarn.turns[0] == plain.turns[0]                        # many turns: kept
    assert abs(int(yarn.turns[-1]) * 4 / int(plain.turns[-1]) - 1) < 1e-12   # under one: divided
    for bad in (dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=272), dict(base=0.5),
                dict(base=math.nan), dict(scaling="linear", factor=0.5),
                dict(scaling="base", factor=math.inf), dict(scaling="turns", factor=2.0, low=4.0),
                dict(scaling="yarn", factor=2.0, original_len=0)):
        with pytest.raises(chs.AttnError):
            chs.attn_rope_frequencies(**dict(dict(rotary_dim=64, device="cpu"), **bad))
    with pytest.raises(ValueError):
        chs.attn_rope_frequencies(64, scaling="other", device="cpu")
    out, amp = (ctypes.c_ulonglong * 128)(), ctypes.c_float()
    f = lib.attn_rope_frequencies
    assert f(None, ctypes.addressof(amp), 64, 1e4, 0, 1.0, 1.0, 4.0, 8192.0) == INVALID
    assert f(ctypes.addressof(out), None, 64, 1e4, 0, 1.0, 1.0, 4.0, 8192.0) == INVALID
    assert f(ctypes.addressof(out), ctypes.addressof(amp), 64, 1e4, 5, 1.0, 1.0, 4.0, 8192.0) == INVALID


def plan(lib, ptrs=None, B=3, cols=4, page=16, P=9, capacity=9, T=20):
    names = ["delta", "seqlens", "seqlens_out", "table", "free", "num_free", "num_free_out", "cu",
             "positions", "slots"]
    p = {n: ptr(i) for i, n in enumerate(names)}
    p.update(ptrs or {})
    return lib.attn_cache_plan(*p.values(), B, cols, page, P, capacity, T, None)


def test_plan_refusals(lib):
    for bad in (dict(B=-1), dict(cols=0), dict(page=0), dict(P=0), dict(T=-1), dict(capacity=0),
                dict(cols=1 << 20, page=1 << 11), dict(P=1 << 27), dict(T=2 ** 31 - 1)):
        assert plan(lib, **bad) == INVALID, bad
    assert plan(lib, page=12) == UNSUPPORTED and plan(lib, B=8193) == UNSUPPORTED
    assert plan(lib, {"free": None}, B=0) == INVALID and plan(lib, {"cu": None}, B=0) == INVALID
    names = ["delta", "seqlens", "seqlens_out", "table", "free", "num_free", "num_free_out", "cu",
             "positions", "slots"]
    outputs = ["seqlens_out", "table", "free", "num_free_out", "cu", "positions", "slots"]
    for i, n in enumerate(names):
        assert plan(lib, {n: None}) == INVALID and plan(lib, {n: ptr(i) + 2}) == INVALID
        for o in outputs:
            pair = {n, o}
            if n == o or pair in ({"seqlens", "seqlens_out"}, {"num_free", "num_free_out"}):
                continue
            assert plan(lib, {o: ptr(i)}) == INVALID, (n, o)
    assert plan(lib, {"seqlens_out": ptr(1) + 4}) == INVALID   # neither in place nor apart


def test_python_checks_before_the_library():
    x = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        chs.attn_fwd_packed(x, x, x, cu)              # not on a GPU
    with pytest.raises(ValueError):
        chs.attn_fwd_packed(x[0], x, x, cu)
    with pytest.raises(TypeError):
        chs.attn_fwd_packed([1], x, x, cu)
    with pytest.raises(ValueError):
        chs.attn_fwd_packed(x, x, x, cu, window=2 ** 31)
    handle = chs.attn_rope_frequencies(64, device="cpu")
    with pytest.raises(TypeError):
        chs.attn_rope(x, x, cu, handle)
    with pytest.raises(ValueError):
        chs.attn_rope(x[0], x, cu, handle)
    with pytest.raises(ValueError):
        chs.attn_cache_plan(cu, cu, cu, cu, cu, rows=1, page=8, num_pages=4)
