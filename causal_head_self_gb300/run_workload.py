"""Run one named workload through the C ABI a few times (for profilers).

    python -m causal_head_self_gb300.run_workload <workload> [--iters N]

Workload names are the keys of causal_head_self_gb300.inputs.WORKLOADS.
Inputs are generated on the host, copied to cuda:0 once, and the kernel
launches run back to back on the current stream; the device status is
checked at the end.
"""
from __future__ import annotations

import argparse
import sys

import torch

import causal_head_self_gb300 as chs
from causal_head_self_gb300 import inputs


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("workload", choices=sorted(inputs.WORKLOADS))
    ap.add_argument("--iters", type=int, default=3)
    args = ap.parse_args(argv)
    w = inputs.WORKLOADS[args.workload]
    dev = torch.device("cuda", 0)
    if w["kind"] == "prefill":
        q, k, v = (x.to(dev) for x in inputs.workload_inputs(args.workload))
        o = torch.empty_like(q)
        for _ in range(args.iters):
            chs.attn_fwd(q, k, v, o, causal=bool(w["causal"]), window=w["window"])
    elif w["kind"] == "backward":
        q, k, v, do = (x.to(dev) for x in inputs.workload_inputs(args.workload))
        o, lse = chs.attn_fwd_lse(q, k, v, causal=bool(w["causal"]), window=w["window"])
        for _ in range(args.iters):
            chs.attn_bwd(q, k, v, o, do, lse, causal=bool(w["causal"]), window=w["window"])
    elif w["kind"] == "chunk":
        q, kc, vc = (x.to(dev) for x in inputs.workload_inputs(args.workload))
        for _ in range(args.iters):
            chs.attn_fwd_chunk(q, kc, vc, w["start"], causal=bool(w["causal"]), window=w["window"])
    elif w["kind"] == "ring":
        q, kc, vc, sl = (x.to(dev) for x in inputs.decode_inputs(
            w["B"], w["Hq"], w["Hkv"], w["Tmax"], w["Dh"], w["lmin"], w["lmax"], w["seed"]))
        for _ in range(args.iters):
            chs.attn_decode_ring(q, kc, vc, sl, window=w["window"])
    elif w["kind"] == "paged":
        kp, vp, table, _, sl = inputs.paged_inputs(w["B"], w["Hkv"], w["Tmax"], w["Dh"], w["page"],
                                                   w["lmin"], w["lmax"], w["seed"], dev)
        q = inputs.device_normal_bf16((w["B"], w["Hq"], 1, w["Dh"]), w["seed"] + 2, dev)
        weights = torch.zeros((w["B"], w["Hkv"], w["Tmax"]), device=dev) if w["weights"] else None
        for _ in range(args.iters):
            chs.attn_decode_paged(q, kp, vp, table, sl, window=w["window"], weights=weights)
    elif w["kind"] == "key_weights":
        q, k, v = (inputs.device_normal_bf16((w["B"], h, w["S"], w["Dh"]), w["seed"] + i, dev)
                   for i, h in enumerate((w["Hq"], w["Hkv"], w["Hkv"])))
        _, lse = chs.attn_fwd_lse(q, k, v)
        weights = torch.zeros((w["B"], w["Hkv"], w["S"]), device=dev)
        for _ in range(args.iters):
            chs.attn_key_weights(q, k, lse, weights, queries=w["queries"])
    elif w["kind"] == "evict":
        spare = (w["budget"] + w["page"] - 1) // w["page"]
        kp, vp, table, to, sl = inputs.paged_inputs(w["B"], w["Hkv"], w["Tmax"], w["Dh"], w["page"],
                                                    w["lmin"], w["lmax"], w["seed"], dev, spare)
        weights = torch.rand((w["B"], w["Hkv"], w["Tmax"]), device=dev)
        kept = torch.zeros_like(weights)
        for _ in range(args.iters):
            chs.attn_cache_evict(kp, vp, weights, table, sl, w["budget"], w["recent"],
                                 table_out=to, weights_out=kept)
    elif w["kind"] == "packed":
        first = [0]
        for n in w["lens"]:
            first.append(first[-1] + n)
        T, Hq, Hkv = first[-1], w["Hq"], w["Hkv"]
        cu = torch.tensor(first, dtype=torch.int32, device=dev)
        x = inputs.device_normal_bf16((1, 1, T, (2 * Hq + 2 * Hkv) * w["Dh"]), w["seed"], dev)
        q, k, v, dout = x.view(T, -1, w["Dh"]).split((Hq, Hkv, Hkv, Hq), 1)
        lse = torch.empty((Hq, T), device=dev)
        for _ in range(args.iters):
            o = chs.attn_fwd_packed(q, k, v, cu, None, lse)
            chs.attn_bwd_packed(q, k, v, o, dout, lse, cu)
    elif w["kind"] == "rope":
        T, Hq, Hkv = w["T"], w["Hq"], w["Hkv"]
        x = inputs.device_normal_bf16((1, 1, T, (Hq + Hkv) * w["Dh"]), w["seed"], dev)
        q, k = x.view(T, -1, w["Dh"]).split((Hq, Hkv), 1)
        positions = torch.arange(T, dtype=torch.int32, device=dev)
        frequencies = chs.attn_rope_frequencies(w["Dh"], device=dev)
        for _ in range(args.iters):
            chs.attn_rope(q, k, positions, frequencies)
    else:
        q, kc, vc, sl = (x.to(dev) for x in inputs.workload_inputs(args.workload))
        o = torch.empty_like(q)
        for _ in range(args.iters):
            chs.attn_decode(q, kc, vc, sl, o, window=w["window"])
    torch.cuda.synchronize(dev)
    rc = chs.attn_status()
    print(f"{args.workload}: {args.iters} launches, status {chs.error_string(rc)}")
    return 0 if rc == chs.ATTN_OK else 1


if __name__ == "__main__":
    sys.exit(main())
