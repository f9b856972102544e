"""Paged-cache cases run against the range-checked build of the library
(started by tests/test_checked_paged.py in a process of its own with
CHS_ATTN_CHECK=1): append, decode with weights, key weights and eviction, with
ragged lengths, windows and pages of several sizes.  Exits non-zero on the first
failure."""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_head_self_gb300 as chs  # noqa: E402
import paged_ref as ref  # noqa: E402
from causal_head_self_gb300 import inputs  # noqa: E402


def status_ok(what):
    rc = chs.attn_status()
    assert rc == chs.ATTN_OK, f"{what}: {chs.error_string(rc)}"


def decode_cases():
    for Hq, Hkv, Dh, page, cols, lens, window in [
            (8, 2, 128, 16, 40, [1, 600, 0, 640, 129], 0), (4, 4, 64, 8, 30, [240, 77], 100),
            (8, 1, 256, 24, 20, [480, 65], 0), (160, 1, 64, 16, 20, [320, 5], 0),
            (40, 1, 128, 72, 6, [430, 73], 65)]:
        kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=page,
                                           first_used=[n - window if window else 0 for n in lens])
        gen = torch.Generator().manual_seed(page)
        q = torch.randn((len(lens), Hq, 1, Dh), generator=gen).to(torch.bfloat16)
        o, tol, w, rtol = ref.decode(q, kp, vp, table, sl, window=window)
        weights = torch.zeros(len(lens), Hkv, cols * page, device="cuda")
        got = chs.attn_decode_paged(*(x.cuda() for x in (q, kp, vp, table, sl)), window=window,
                                    weights=weights)
        status_ok("decode")
        assert ((got.cpu().double() - o).abs() <= tol).all()
        assert ((weights.cpu().double() - w).abs() <= rtol * w).all()


def key_weight_cases():
    for Hq, Hkv, S, Dh, nq, window in [(4, 2, 300, 128, 0, 0), (12, 1, 257, 64, 20, 0),
                                       (2, 2, 260, 256, 0, 100), (32, 1, 600, 64, 0, 0)]:
        q, k, v = inputs.prefill_inputs(2, Hq, Hkv, S, Dh, seed=S)
        _, lse = chs.attn_fwd_lse(q.cuda(), k.cuda(), v.cuda(), window=window)
        lens = [S, S - 131]
        want, rtol = ref.key_weights(q, k, lse.cpu(), lens, queries=nq, window=window)
        w = torch.zeros(2, Hkv, S, device="cuda")
        chs.attn_key_weights(q.cuda(), k.cuda(), lse, w,
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), queries=nq,
                             window=window)
        status_ok("key weights")
        assert ((w.cpu().double() - want).abs() <= rtol * want).all()


def cache_cases():
    lens = [300, 17, 120]
    kp, vp, table, sl = ref.make_cache(lens, 2, 128, 16, 20, seed=1, spare=9)
    w = torch.rand((3, 2, 320), generator=torch.Generator().manual_seed(1))
    used = set(table.flatten().tolist())
    free = [x for x in range(kp.shape[0]) if x not in used][:9]
    to = torch.tensor(free, dtype=torch.int32).view(3, 3)
    for target in (to, None):
        want = ref.evict_apply(kp, vp, w, table, sl, 40, 8, target)
        d = [x.cuda() for x in (kp, vp, w, table, sl)]
        new, keep = chs.attn_cache_evict(*d, 40, 8, table_out=None if target is None else target.cuda())
        status_ok("evict")
        assert torch.equal(keep.cpu(), want[4]) and torch.equal(new.cpu(), want[3])
        for got, ref_ in ((d[0], want[0]), (d[1], want[1])):
            assert torch.equal(got.cpu().view(torch.int16), ref_.view(torch.int16))
    k = torch.randn((3, 2, 7, 128)).to(torch.bfloat16)
    d = [x.cuda() for x in (k, k, kp, vp, table, sl)]
    chs.attn_paged_append(*d, torch.tensor([7, 3, 0], dtype=torch.int32, device="cuda"))
    status_ok("append")
    assert torch.equal(d[2][table[0, 18], :, 5 + 6].cpu(), k[0, :, 6]) and math.isfinite(float(k.sum()))


if __name__ == "__main__":
    assert chs._binding.LIB_PATH.endswith("_check.so"), chs._binding.LIB_PATH
    for case in (decode_cases, key_weight_cases, cache_cases):
        case()
        print(case.__name__, "ok", flush=True)
