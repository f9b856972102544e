"""Packed sequences against the range-checked build (started by
tests/test_checked_packed.py with CHS_ATTN_CHECK=1): every kernel that walks
them, its own list and the launch's, folded tiles, both kinds of D, rotations
and plans.  Exits non-zero on the first failure."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_head_self_gb300 as chs  # noqa: E402
import packed_ref as ref  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status_ok(what):
    rc = chs.attn_status()
    assert rc == chs.ATTN_OK, f"{what}: {chs.error_string(rc)}"


def attention_cases():
    short = [1, 33, 64, 2, 0, 17, 65, 32, 128, 129]
    for Dh in (64, 128, 256):
        for lens, Hq, Hkv, causal, window in [(short, 8, 2, True, 0), (short * 9, 4, 1, True, 0),
                                              ([300, 1, 700], 4, 4, True, 50), ([5000], 2, 1, True, 0),
                                              (short, 4, 2, False, 0), ([400, 90], 4, 2, True, 20)]:
            gen = torch.Generator("cuda").manual_seed(Dh)
            cu = ref.offsets(lens, 3)
            T = cu[-1] + 2
            q, k, v = ref.layouts(T, Hq, Hkv, Dh, "fused", gen)
            dout = ref.layouts(T, Hq, Hkv, Dh, "heads_first", gen)[0]
            lse = torch.zeros(Hq, T, device="cuda")
            o = torch.zeros(T, Hq, Dh, dtype=torch.bfloat16, device="cuda")
            grads = [torch.zeros(T, h, Dh, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
            chs.attn_fwd_packed(q, k, v, i32(cu), o, lse, causal=causal, window=window)
            status_ok("forward")
            chs.attn_bwd_packed(q, k, v, o, dout, lse, i32(cu), *grads, causal=causal, window=window)
            status_ok("backward")
            want, _, bound, dwant, dbound = ref.attention(q, k, v, cu, causal, window, dout=dout)
            ref.check(o, want, bound)
            for got, w, b in zip(grads, dwant, dbound):
                ref.check(got, w, b)


def token_cases():
    gen = torch.Generator("cuda").manual_seed(0)
    T, Hkv, page, P, Dh = 50, 2, 8, 20, 64
    q, k, v = ref.layouts(T, 4, Hkv, Dh, "fused", gen)
    kp, vp = (torch.zeros(P, Hkv, page, Dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((3, 7), -1, dtype=torch.int32, device="cuda")
    seqlens, num_free = i32([0, 0, 0]), i32([P])
    cu, pos, slots = chs.attn_cache_plan(i32([20, 1, 25]), seqlens, table,
                                         torch.arange(P, dtype=torch.int32, device="cuda"), num_free, rows=T,
                                         page=page, num_pages=P)
    ko = torch.zeros(T, Hkv, Dh, dtype=torch.bfloat16, device="cuda")
    chs.attn_rope_append(q, k, v, pos, chs.attn_rope_frequencies(Dh), kp, vp, slots, None, ko)
    status_ok("tokens")
    at = slots[:46].long()
    assert torch.equal(kp[at // page, :, at % page], ko[:46])
    assert torch.equal(vp[at // page, :, at % page], v[:46])


if __name__ == "__main__":
    attention_cases()
    token_cases()
    print("packed_cases ok")
