#!/usr/bin/env python
"""Decodes a batch of sequences through a stack of decoder layers: paged cache append with position
rotation, single-token attention, the norms around it and the quantized MoE block, on random weights.

    python examples/decode_layer.py [--layers 2] [--seqs 8] [--past 1000] [--steps 20] [--kv bf16|f16|e4m3]

Prints the time of a step (all layers, one token of every sequence)."""
import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import quantized_expert_decode_gb300 as q  # noqa: E402
import synth  # noqa: E402
from quantized_expert_decode_gb300.device import DeviceBlock  # noqa: E402
from quantized_expert_decode_gb300.layer import DecodeLayer, PagedCache  # noqa: E402


def build(layers, seqs, past, steps, fmt, q_heads=16, kv_heads=2, dim=128, page=64):
    cfg = dict(synth.config(1), T=seqs)
    h = cfg["H"]
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    inv_freq = (1e4 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).float().cuda()
    stack = []
    for i in range(layers):
        pages = seqs * (-(-(past + steps) // page))
        scale = torch.full((kv_heads,), 0.05, device="cuda") if fmt == q.COLI_KV_E4M3 else None
        cache = PagedCache(seqs, pages, page, kv_heads, dim, fmt, past + steps, scale, scale)
        w_qkv = rand((q_heads + 2 * kv_heads) * dim, h) / h ** 0.5
        w_o = rand(h, q_heads * dim) / (q_heads * dim) ** 0.5
        ones = torch.ones(h, device="cuda")
        stack.append(DecodeLayer(DeviceBlock(synth.make_block(cfg, seed=i)), cache, w_qkv, w_o, ones, ones, inv_freq, q_heads))
    # the sequences' past, appended in one call per layer
    if past:
        n = seqs * past
        seq = torch.arange(seqs, dtype=torch.int32, device="cuda").repeat_interleave(past)
        pos = torch.arange(past, dtype=torch.int32, device="cuda").repeat(seqs)
        d = q.make_append_desc(n, 0, seqs, stack[0].cache.width, q.COLI_ACT_F32, dim)
        for layer in stack:
            for s in range(seqs):
                layer.cache.grow(s, past)
            q.coli_kv_append(d, layer.cache.desc, None, rand(n, kv_heads, dim), rand(n, kv_heads, dim), inv_freq, seq, pos,
                             layer.cache.table, None, layer.err)
    return stack, rand(seqs, h)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--past", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--kv", default="bf16", choices=["bf16", "f16", "e4m3"])
    a = ap.parse_args()
    fmt = {"bf16": q.COLI_KV_BF16, "f16": q.COLI_KV_F16, "e4m3": q.COLI_KV_E4M3}[a.kv]
    stack, resid = build(a.layers, a.seqs, a.past, a.steps, fmt)
    h = resid.shape[1]
    stream = torch.cuda.current_stream()
    xn = torch.empty_like(resid)
    q.coli_moe_rmsnorm(resid, torch.ones(h, device="cuda"), 1e-5, xn, a.seqs, h, stream)
    times = []
    for _ in range(a.steps):
        at = [layer.cache.grow(s) for layer in stack for s in range(a.seqs)][: a.seqs]
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        lens = pos + 1
        torch.cuda.synchronize()
        t = time.perf_counter()
        for layer in stack:
            xn = layer.step(xn, resid, pos, lens, stream)
        torch.cuda.synchronize()
        times.append(time.perf_counter() - t)
    for layer in stack:
        layer.check(stream)
    times.sort()
    print(f"{a.layers} layers, {a.seqs} sequences of {a.past}..{a.past + a.steps} tokens, {a.kv} cache: "
          f"{times[len(times) // 2] * 1e6:.0f} us a step, residual rms {float(resid.square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
