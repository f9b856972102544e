"""The forms of the paged cache's kernels that checked_paged_cases.py does not
reach, against the range-checked build (started by
tests/test_checked_paged_forms.py with CHS_ATTN_CHECK=1): decode steps over wide
tables (the line of tiles, with four copies of the heads and with one), key
weights of few voting queries, an append of more rows than a wave takes, and an
eviction whose rows do not fit in a block.  Exits non-zero on the first failure."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_head_self_gb300 as chs  # noqa: E402
import paged_ref as ref  # noqa: E402


def status_ok(what):
    rc = chs.attn_status()
    assert rc == chs.ATTN_OK, f"{what}: {chs.error_string(rc)}"


def wide_decode_cases():
    for Hq, Hkv, Dh, page, cols, lens, window in [
            (8, 2, 128, 16, 40, [1, 600, 0, 640, 129], 0), (4, 4, 64, 8, 30, [240, 77], 100),
            (8, 1, 256, 24, 20, [480, 65], 0), (32, 1, 128, 40, 12, [480, 3], 0),
            (160, 1, 64, 16, 20, [320, 5], 0), (33, 1, 256, 16, 20, [300, 65], 70)]:
        kp, vp, table, sl = ref.make_cache(lens, Hkv, Dh, page, cols, seed=page,
                                           first_used=[n - window if window else 0 for n in lens])
        q = torch.randn((len(lens), Hq, 1, Dh),
                        generator=torch.Generator().manual_seed(page)).to(torch.bfloat16)
        o, tol, w, rtol = ref.decode(q, kp, vp, table, sl, window=window)
        # room for more rows than a step in one launch takes, window or not
        more = torch.full((len(lens), -(-13000 // page) - cols), -1, dtype=torch.int32)
        table = torch.cat([table, more], 1)
        weights = torch.zeros(len(lens), Hkv, table.shape[1] * page, device="cuda")
        got = chs.attn_decode_paged(*(x.cuda() for x in (q, kp, vp, table, sl)), window=window,
                                    weights=weights)
        status_ok("decode")
        assert ((got.cpu().double() - o).abs() <= tol).all()
        assert ((weights[..., :w.shape[2]].cpu().double() - w).abs() <= rtol * w).all()


def few_voting_queries_cases():
    for Hq, Hkv, S, Dh, nq in [(8, 2, 500, 64, 64), (4, 1, 300, 128, 20), (5, 1, 300, 64, 33),
                               (4, 2, 260, 256, 17), (3, 3, 30, 128, 0)]:
        gen = torch.Generator().manual_seed(S)
        q, k = (torch.randn((2, h, S, Dh), generator=gen).to(torch.bfloat16) for h in (Hq, Hkv))
        lse = 5 + torch.randn((2, Hq, S), generator=gen)
        lens = [S, S - 11]
        want, rtol = ref.key_weights(q, k, lse, lens, queries=nq)
        w = torch.zeros(2, Hkv, S, device="cuda")
        chs.attn_key_weights(q.cuda(), k.cuda(), lse.cuda(), w,
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), queries=nq)
        status_ok("key weights")
        assert ((w.cpu().double() - want).abs() <= rtol * want).all()


def long_cases():
    B, Hkv, S, Dh, page = 2, 8, 1300, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    cols = -(-S // page)
    table = torch.randperm(B * cols, generator=gen, device="cuda").to(torch.int32).view(B, cols)
    k = torch.randn((B, Hkv, S, Dh), generator=gen, device="cuda").to(torch.bfloat16)
    kp, vp = (torch.zeros(B * cols, Hkv, page, Dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    chs.attn_paged_append(k, -k, kp, vp, table, torch.full((B,), S, dtype=torch.int32, device="cuda"))
    status_ok("append")
    rows = kp[table.long()].transpose(1, 2).reshape(B, Hkv, cols * page, Dh)
    assert torch.equal(rows[:, :, :S], k)
    rows = vp[table.long()].transpose(1, 2).reshape(B, Hkv, cols * page, Dh)
    assert torch.equal(rows[:, :, :S], -k)
    n, budget, recent = 50001, 7000, 500
    cols = -(-n // page)
    for to in (None, cols + torch.arange(-(-budget // page), dtype=torch.int32, device="cuda")[None]):
        kp = torch.randn((cols + 440, 1, page, 64), generator=gen, device="cuda").to(torch.bfloat16)
        vp, k0 = kp.clone(), kp[:cols].reshape(-1, 64).clone()
        w = torch.rand((1, 1, cols * page), generator=gen, device="cuda")
        top = w[0, 0, :n - recent].sort(descending=True, stable=True).indices[:budget - recent]
        want = torch.cat([top.sort().values, torch.arange(n - recent, n, device="cuda")])
        table = torch.arange(cols, dtype=torch.int32, device="cuda")[None]
        new, keep = chs.attn_cache_evict(kp, vp, w, table,
                                         torch.tensor([n], dtype=torch.int32, device="cuda"), budget,
                                         recent, table_out=to)
        status_ok("evict")
        assert new.tolist() == [budget] and torch.equal(keep[0, 0].long(), want)
        first = 0 if to is None else cols * page
        for pool in (kp, vp):
            assert torch.equal(pool.reshape(-1, 64)[first:first + budget], k0[want])


if __name__ == "__main__":
    assert chs._binding.LIB_PATH.endswith("_check.so"), chs._binding.LIB_PATH
    for case in (wide_decode_cases, few_voting_queries_cases, long_cases):
        case()
        print(case.__name__, "ok", flush=True)
