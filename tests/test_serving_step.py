"""A server's steps captured in two graphs that live side by side and share the
cache: prompts (plan, rotation with the write to the pages, packed attention)
and tokens (plan, rotation with the write, paged decode).  They are replayed
with changing lengths, which the graphs read on the GPU alone; after each replay
the cache is compared with what was put into it, and the attention with 64 bits.
(test_tokens.py makes such steps by eager calls.)"""
import random

import pytest
import torch

import causal_head_self_gb300 as chs
import packed_ref as ref
from test_tokens import U, close, frequencies, i32, pools, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,Dh,page", [(8, 2, 128, 16), (4, 4, 64, 8), (8, 1, 256, 64)])
def test_two_captured_steps_share_a_cache(Hq, Hkv, Dh, page):
    gen = torch.Generator("cuda").manual_seed(Dh)
    rng = random.Random(Dh)
    B, P, room, T = 5, 96, 400, 320   # T: rows of the prompts' buffer
    cols = -(-room // page)
    kp, vp = pools(P, Hkv, page, Dh)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    num_free, seqlens, delta = i32([P]), i32([0] * B), i32([0] * B)
    handle, exact = chs.attn_rope_frequencies(Dh), frequencies(Dh)
    stream = torch.cuda.Stream()

    def buffers(rows):
        q, k, v = ref.layouts(rows, Hq, Hkv, Dh, "fused", gen)
        return dict(q=q, k=k, v=v, turned=torch.zeros(rows, Hkv, Dh, dtype=torch.bfloat16, device="cuda"),
                    qo=torch.zeros(rows, Hq, Dh, dtype=torch.bfloat16, device="cuda"),
                    cu=i32([0] * (B + 1)), pos=i32([0] * rows), slots=i32([0] * rows))

    def tokens_of(x, rows):
        chs.attn_cache_plan(delta, seqlens, table, free, num_free, rows=rows, page=page, num_pages=P,
                            cu_seqlens=x["cu"], positions=x["pos"], slots=x["slots"])
        chs.attn_rope_append(x["q"], x["k"], x["v"], x["pos"], handle, kp, vp, x["slots"], x["qo"],
                             x["turned"])

    prompts, tokens = buffers(T), buffers(B)
    prompts["o"] = torch.zeros(T, Hq, Dh, dtype=torch.bfloat16, device="cuda")
    tokens["o"] = torch.zeros(B, Hq, 1, Dh, dtype=torch.bfloat16, device="cuda")

    def prompt_step():
        tokens_of(prompts, T)
        chs.attn_fwd_packed(prompts["qo"], prompts["turned"], prompts["v"], prompts["cu"], prompts["o"])

    def token_step():
        tokens_of(tokens, B)
        first = tokens["cu"][:-1].long().clamp(max=B - 1)   # a place's token, where it has one
        tokens["query"] = tokens["qo"][first].unsqueeze(2)
        chs.attn_decode_paged(tokens["query"], kp, vp, table, seqlens, tokens["o"])

    graphs = []
    stream.wait_stream(torch.cuda.current_stream())
    for step in (prompt_step, token_step):   # (no lengths change: nothing is written)
        with torch.cuda.stream(stream):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        graphs.append(graph)
    torch.cuda.synchronize()
    assert chs.attn_status() == chs.ATTN_OK and seqlens.tolist() == [0] * B

    held = [[torch.zeros(0, Hkv, Dh, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for _ in range(B)]

    def replay(graph, x, change):
        for t in (x["q"], x["k"], x["v"]):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        before = seqlens.tolist()
        delta.copy_(i32(change))
        graph.replay()
        assert chs.attn_status() == chs.ATTN_OK
        lens = [n + d for n, d in zip(before, change)]
        assert seqlens.tolist() == lens
        cu = x["cu"].tolist()
        assert cu == ref.offsets([max(d, 0) for d in change])
        n = cu[-1]
        want = sum((list(range(a, a + d)) for a, d in zip(before, change)), [])
        assert x["pos"].tolist() == want + [-1] * (len(x["pos"]) - n)
        for src, dst in (("k", "turned"), ("q", "qo")):
            close(x[dst][:n].transpose(0, 1), turned(x[src][:n].transpose(0, 1), x["pos"][:n], exact))
        pages = []
        for b in range(B):
            own = table[b, :-(-lens[b] // page)].tolist()
            pages += own
            kept = before[b] + min(change[b], 0)
            for i, (pool, new) in enumerate(((kp, x["turned"]), (vp, x["v"]))):
                held[b][i] = torch.cat([held[b][i][:kept], new[cu[b]:cu[b + 1]]])
                rows = pool[own].transpose(1, 2).reshape(-1, Hkv, Dh)[:lens[b]]
                assert torch.equal(rows, held[b][i])
        assert sorted(pages + free[:num_free.item()].tolist()) == list(range(P))   # each once
        return cu, lens

    for turn in range(4):
        # all places start again: prompts of every length, some places empty
        first = [0] * B if turn == 0 else [-n for n in seqlens.tolist()]
        if turn:
            replay(graphs[1], tokens, first)
        cu, _ = replay(graphs[0], prompts, [rng.choice((0, 1, 17, rng.randint(2, 64))) for _ in range(B)])
        want, _, bound = ref.attention(prompts["qo"], prompts["turned"], prompts["v"], cu)
        n = cu[-1]
        ref.check(prompts["o"][:n], want[:n], bound[:n])
        for _ in range(6):
            lens = seqlens.tolist()
            change = [1 if rng.random() < 0.7 else -rng.randint(0, min(a, 5)) for a in lens]
            _, lens = replay(graphs[1], tokens, change)
            for b in range(B):
                if lens[b] == 0:
                    assert bool((tokens["o"][b] == 0).all())
                    continue
                K, V = (t.double().repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for t in held[b])
                p = torch.softmax(tokens["query"][b].double() @ K.transpose(1, 2) * Dh ** -0.5, -1)
                y = p @ V
                err = (tokens["o"][b].double() - y).abs()
                assert bool((err <= (1 + U) * (U + ref.F) * (p @ V.abs()) + U * y.abs()).all())
