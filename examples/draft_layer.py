#!/usr/bin/env python
"""Decodes a batch of sequences with drafted tokens through a stack of decoder layers on random weights: each step
drafts a tree of tokens behind every sequence's last one, all nodes go through the layers in one pass, the target's
probabilities accept a path of them, and its cached rows move up behind the committed tokens.

    python examples/draft_layer.py [--layers 2] [--seqs 8] [--past 500] [--steps 10] [--wide 2] [--deep 3] [--near 0.5]

The draft is the target's own distribution with noise (`--near`: how much), as no drafting model is at hand; its
tokens are drawn before the pass from the previous step's probabilities. Prints the time of a step's pass and
the tokens that a step gained."""
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
from quantized_expert_decode_gb300.layer import DecodeLayer, Nodes, PagedCache  # noqa: E402


def tree_of(wide, deep):
    """The root, and below it `wide` nodes, each followed by a chain to depth `deep`, in the order of their depth."""
    parents, above = [-1], [0] * wide
    for _ in range(deep):
        here = range(len(parents), len(parents) + wide)
        parents += above
        above = list(here)
    return parents


def build(layers, seqs, pages, page, vocab, q_heads=16, kv_heads=2, dim=128):
    cfg = dict(synth.config(1), T=seqs)
    h = cfg["H"]
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    inv_freq = (1e4 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).float().cuda()
    cache = PagedCache(seqs, pages, page, kv_heads, dim, layers=layers)
    ones, head_ones = torch.ones(h, device="cuda"), torch.ones(dim, device="cuda")
    stack = [DecodeLayer(DeviceBlock(synth.make_block(cfg, seed=i)), cache, rand((q_heads + 2 * kv_heads) * dim, h) / h ** 0.5,
                         rand(h, q_heads * dim) / (q_heads * dim) ** 0.5, ones, ones, inv_freq, q_heads, q_norm=head_ones,
                         k_norm=head_ones, layer=i) for i in range(layers)]
    return stack, cache, rand(vocab, h), rand(vocab, h) / h ** 0.5 * 3


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--past", type=int, default=500)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--wide", type=int, default=2)
    ap.add_argument("--deep", type=int, default=3)
    ap.add_argument("--near", type=float, default=0.5)
    ap.add_argument("--vocab", type=int, default=1000)
    a = ap.parse_args()
    page, tree = 16, tree_of(a.wide, a.deep)
    n, rows = len(tree), a.seqs * len(tree)
    pages = a.seqs * (-(-(a.past + (a.steps + 1) * n) // page) + 1)
    stack, cache, embed, head = build(a.layers, a.seqs, pages, page, a.vocab)
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = dict(dtype=torch.int32, device="cuda")
    # the sequences' past: random rows
    total = a.seqs * a.past
    if total:
        seq = torch.arange(a.seqs, **ints).repeat_interleave(a.past)
        pos = torch.arange(a.past, **ints).repeat(a.seqs)
        d = q.make_norm_append_desc(total, 0, a.seqs, cache.width, q.COLI_ACT_F32, cache.dim, eps=1e-5)
        for s in range(a.seqs):
            cache.grow(s, a.past)
        for layer in stack:
            k, v = (torch.randn(total, cache.heads, cache.dim, generator=g, device="cuda") for _ in range(2))
            q.coli_norm_append(d, layer.desc, None, k, v, None, layer.k_norm, layer.inv_freq, seq, pos, None, cache.table, None,
                               layer.err, torch.cuda.current_stream())
    drafts = [layer.drafts(rows, n) for layer in stack]
    verify = q.make_verify_desc(a.seqs, rows, n, a.vocab)
    path, count, token = torch.empty(a.seqs, n, **ints), torch.empty(a.seqs, **ints), torch.zeros(a.seqs, **ints)
    parent = torch.tensor(tree, device="cuda")
    err = torch.zeros(1, **ints)
    target = torch.full((rows, a.vocab), 1.0 / a.vocab, device="cuda")
    gained, times = [], []
    for _ in range(a.steps):
        # each node's token is drawn from its parent's row of the draft, here what the target said last time, with noise
        noisy = target.clamp(min=1e-9).log() + a.near * torch.randn(rows, a.vocab, generator=g, device="cuda")
        draft = torch.softmax(noisy, 1)
        up = (torch.arange(a.seqs, device="cuda")[:, None] * n + parent.clamp(min=0)[None, :]).flatten()
        tokens = torch.multinomial(draft[up], 1, generator=g)[:, 0].int().view(a.seqs, n)
        tokens[:, 0] = token
        past = list(cache.tokens)
        for s in range(a.seqs):
            cache.grow(s, n)
        nodes = Nodes(past, [tree] * a.seqs)
        torch.cuda.synchronize()
        t = time.perf_counter()
        resid = embed[tokens.flatten()]
        x = resid * torch.rsqrt(resid.square().mean(1, keepdim=True) + 1e-5)
        for layer, d in zip(stack, drafts):
            x = layer.draft_step(d, x, resid, nodes)
        target = torch.softmax(x @ head.T, 1)
        uniform = torch.rand(rows, generator=g, device="cuda")
        stream = torch.cuda.current_stream()
        q.coli_draft_verify(verify, target, draft, tokens, nodes.parent, uniform, nodes.first, path, count, token, err, stream)
        cache.compact(nodes.past, path, count, err, stream)
        taken = count.tolist()  # (waits for the pass)
        times.append(time.perf_counter() - t)
        for s in range(a.seqs):
            cache.cut(s, past[s] + taken[s])
        gained += taken
    q.coli_moe_check(err)
    for layer, d in zip(stack, drafts):
        layer.check(drafts=d)
    times.sort()
    print(f"{a.layers} layers, {a.seqs} sequences, trees of {n} nodes: {times[len(times) // 2] * 1e6:.0f} us a step, "
          f"{sum(gained) / len(gained):.2f} tokens of a sequence a step")


if __name__ == "__main__":
    main()
