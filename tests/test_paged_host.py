"""Argument checks of the paged cache's entry points.  They come before any
CUDA call, so made-up (aligned, disjoint) addresses are safe: nothing is
dereferenced or launched."""
import ctypes

import pytest
import torch

import causal_head_self_gb300 as chs
import paged_ref as ref
from causal_head_self_gb300 import _binding
from causal_head_self_gb300 import build as _build

INVALID, UNSUPPORTED, OK = chs.ATTN_ERR_INVALID_ARG, chs.ATTN_ERR_UNSUPPORTED, chs.ATTN_OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _binding.load()


def ptr(i):
    return (i + 1) << 34


def append(lib, ptrs=None, B=2, Hkv=2, S=4, P=10, page=16, cols=4, Dh=128):
    ptrs = ptrs or [ptr(i) for i in range(7)]
    return lib.attn_paged_append(*ptrs, B, Hkv, S, P, page, cols, Dh, None)


SHAPES = [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(P=0), INVALID), (dict(cols=0), INVALID),
    (dict(page=0), INVALID), (dict(page=-8), INVALID), (dict(Dh=96), UNSUPPORTED),
    (dict(page=12), UNSUPPORTED), (dict(page=1), UNSUPPORTED),
    (dict(page=1 << 20, cols=1 << 11), INVALID),    # 2^31 rows
    (dict(P=1 << 30, Hkv=2), INVALID),              # 2^31 (page, head) pairs
    (dict(B=0), OK),
]


@pytest.mark.parametrize("change,code", SHAPES)
def test_every_call_checks_the_caches_shape(lib, change, code):
    assert append(lib, **change) == code
    assert decode(lib, **change) == code
    assert evict(lib, **change) == code


def bad_pointers(call, n, optional=(), align=16, skip=()):
    for i in range(n):
        if i in skip:
            continue
        ptrs = [ptr(j) for j in range(n)]
        if i not in optional:
            ptrs[i] = None
            assert call(ptrs) == INVALID, f"null {i}"
        ptrs[i] = ptr(i) + 2
        assert call(ptrs) == INVALID, f"misaligned {i}"


def test_append_refusals(lib):
    assert append(lib, S=-1) == INVALID
    assert append(lib, S=0) == OK
    assert append(lib, B=1 << 15, Hkv=1 << 6, S=1 << 10, P=1) == INVALID   # 2^31 rows
    bad_pointers(lambda p: append(lib, p), 7, optional=(6,))
    for out in (2, 3):
        for other in range(7):
            if other != out:
                p = [ptr(i) for i in range(7)]
                p[other] = p[out] + 64   # inside the pool
                assert append(lib, p) == INVALID


def decode(lib, ptrs=None, weights=ptr(6), stride=64, acc=1, ws=ptr(7), ws_bytes=1 << 20, B=2, Hq=8,
           Hkv=2, P=10, page=16, cols=4, Dh=128, window=0, scale=0.0):
    ptrs = ptrs or [ptr(i) for i in range(6)]
    if stride == 64:
        stride = max(64, min(cols * page, 2 ** 31 - 1)) if cols > 0 and page > 0 else 64
    return lib.attn_decode_paged(*ptrs, weights, stride, acc, ws, ws_bytes, B, Hq, Hkv, P, page, cols,
                                 Dh, window, scale, None)


def test_decode_refusals(lib):
    assert decode(lib, Hq=7) == INVALID
    assert decode(lib, Hq=0) == INVALID
    assert decode(lib, stride=63) == INVALID
    assert decode(lib, acc=2) == INVALID
    assert decode(lib, scale=-1.0) == INVALID
    assert decode(lib, scale=float("nan")) == INVALID
    assert decode(lib, scale=float("inf")) == INVALID
    assert decode(lib, B=1 << 20, Hkv=1 << 5, Hq=1 << 5, P=1) == INVALID       # units
    assert decode(lib, B=1 << 16, Hkv=8, page=1024, cols=1024, P=1) == INVALID   # tiles
    bad_pointers(lambda p: decode(lib, p), 6)
    assert decode(lib, weights=ptr(6) + 2) == INVALID
    assert decode(lib, ws=None) == INVALID
    assert decode(lib, ws=ptr(7) + 128) == INVALID
    base = [ptr(i) for i in range(6)]
    for i in (0, 1, 2, 3, 4):                      # the output over an input
        assert decode(lib, base[:5] + [base[i]]) == INVALID
        assert decode(lib, weights=base[i]) == INVALID
        assert decode(lib, ws=base[i]) == INVALID
    assert decode(lib, weights=base[5]) == INVALID
    assert decode(lib, ws=base[5]) == INVALID
    assert decode(lib, ws=ptr(6)) == INVALID       # the workspace over the weights


def test_decode_workspace_query_checks_its_arguments(lib):
    n = ctypes.c_size_t()
    f = lib.attn_decode_paged_workspace
    assert f(2, 7, 2, 16, 4, 128, 0, ctypes.byref(n)) == INVALID
    assert f(2, 8, 2, 12, 4, 128, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(2, 8, 2, 16, 4, 80, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(2, 8, 2, 16, 4, 128, 0, None) == INVALID


def key_weights(lib, ptrs=None, stride=40, B=2, Hq=4, Hkv=2, S=40, Dh=128, queries=0, causal=1,
                window=0, acc=1, scale=0.0):
    ptrs = ptrs or [ptr(i) for i in range(5)]
    return lib.attn_key_weights(*ptrs, stride, B, Hq, Hkv, S, Dh, queries, causal, window, acc, scale,
                                None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), INVALID), (dict(S=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(Dh=96), UNSUPPORTED), (dict(causal=2), INVALID), (dict(causal=0, window=3), INVALID),
    (dict(stride=39), INVALID), (dict(acc=-1), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=1e-19), INVALID),   # lse / scale would not stay finite
    (dict(B=0), OK), (dict(S=0), OK),
])
def test_key_weights_argument_checks(lib, change, code):
    assert key_weights(lib, **change) == code


def test_key_weights_pointer_checks(lib):
    bad_pointers(lambda p: key_weights(lib, p), 5, optional=(3,))
    for other in range(4):
        p = [ptr(i) for i in range(5)]
        p[4] = p[other]
        assert key_weights(lib, p) == INVALID


def evict(lib, ptrs=None, stride=None, budget=32, recent=8, table_out=ptr(5), cols_out=2,
          w_out=ptr(6), stride_out=64, B=2, Hkv=2, P=10, page=16, cols=4, Dh=128):
    kp, vp, w, table, sl, new, keep = ptrs or [ptr(i) for i in (0, 1, 2, 3, 4, 7, 8)]
    if stride is None:
        stride = max(64, min(cols * page, 2 ** 31 - 1)) if cols > 0 and page > 0 else 64
    return lib.attn_cache_evict(kp, vp, w, stride, table, sl, budget, recent, table_out, cols_out,
                                w_out, stride_out, new, keep, B, Hkv, P, page, cols, Dh, None)


def test_evict_refusals(lib):
    assert evict(lib, budget=0) == INVALID
    assert evict(lib, recent=-1) == INVALID
    assert evict(lib, recent=33) == INVALID
    assert evict(lib, stride=63) == INVALID
    assert evict(lib, stride_out=31) == INVALID
    assert evict(lib, cols_out=1) == INVALID       # 16 rows for 32
    assert evict(lib, cols_out=0) == INVALID
    # in place: one table, one weights tensor
    assert evict(lib, table_out=ptr(3), cols_out=2) == INVALID
    assert evict(lib, w_out=ptr(2), stride_out=65) == INVALID
    names = (0, 1, 2, 3, 4, 7, 8)

    def call(p):
        return evict(lib, p)
    for i in range(7):
        p = [ptr(j) for j in names]
        p[i] = None
        assert call(p) == INVALID
        p[i] = ptr(names[i]) + 2
        assert call(p) == INVALID
    for i in (0, 1, 5, 6):                         # what is written over anything else
        for j in range(7):
            if i != j:
                p = [ptr(x) for x in names]
                p[i] = p[j]
                assert call(p) == INVALID, (i, j)
    for j in (0, 1, 3, 4, 7, 8):                   # the new weights over anything else
        assert evict(lib, w_out=ptr(j)) == INVALID
    assert evict(lib, w_out=ptr(2) + 256) == INVALID


def test_the_binding_refuses_cpu_tensors_and_wrong_types(lib):
    kp, vp, table, sl = ref.make_cache([5, 9], 2, 64, 8, 2, seed=0)
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 2, 16)
    for call in (lambda: chs.attn_decode_paged(q, kp, vp, table, sl),
                 lambda: chs.attn_paged_append(q, q, kp, vp, table, sl),
                 lambda: chs.attn_cache_evict(kp, vp, w, table, sl, 4),
                 lambda: chs.attn_key_weights(q, q, w, w),
                 lambda: chs.attn_decode_paged(q, kp.float(), vp, table, sl)):
        with pytest.raises(TypeError):
            call()


def test_the_binding_refuses_what_32_bits_cannot_hold():
    # (2^32 + 5 would reach the library as 5)
    kp, vp, table, sl = ref.make_cache([5, 9], 2, 64, 8, 2, seed=0)
    q, w, big = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16), 2**32 + 5
    wide = torch.zeros(1, dtype=torch.int32).expand(2, big)
    for call in (lambda: chs.attn_decode_paged(q, kp, vp, table, sl, window=big),
                 lambda: chs.attn_decode_paged(q, kp, vp, wide, sl),
                 lambda: chs.attn_cache_evict(kp, vp, w, table, sl, big),
                 lambda: chs.attn_cache_evict(kp, vp, w, table, sl, 4, -big),
                 lambda: chs.attn_key_weights(q, q, w, w, queries=big),
                 lambda: chs.attn_key_weights(q, q, w, w, window=big),
                 lambda: _binding._rows_of("weights", torch.zeros(1).expand(2, 2, big), 2, 2, 0)):
        with pytest.raises(ValueError):
            call()


def test_reference_eviction_by_hand():
    w = torch.tensor([[[5.0, 1.0, 5.0, 2.0, 9.0, 0.0, 0.0]]])
    newlens, keep = ref.evict(w, torch.tensor([6], dtype=torch.int32), 4, 1)
    assert newlens.tolist() == [4] and keep.tolist() == [[[0, 2, 4, 5]]]
    newlens, keep = ref.evict(w, torch.tensor([6], dtype=torch.int32), 2, 0)
    assert keep.tolist() == [[[0, 4]]]             # of two equal weights the lower row
