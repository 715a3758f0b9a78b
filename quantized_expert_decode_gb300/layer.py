"""A decoder layer's decode step around the MoE block: the paged cache, its page tables, and the
calls in the order a layer makes them. Allocation, bookkeeping of pages and the two plain
projections (library products); everything else runs in the library's kernels."""
from __future__ import annotations

import torch

from . import (COLI_ACT_F32, COLI_GATE_NONE, COLI_KV_BF16, COLI_KV_E4M3, COLI_KV_F16, coli_attn_decode,
               coli_attn_workspace_bytes, coli_block_norms, coli_kv_append, coli_moe_check, coli_moe_forward,
               make_append_desc, make_attn_desc, make_kv_cache, make_norms_desc)

_TORCH = {COLI_KV_BF16: torch.bfloat16, COLI_KV_F16: torch.float16, COLI_KV_E4M3: torch.float8_e4m3fn}


class PagedCache:
    """Pools of `pages` pages for keys and values, and a page table for `seqs` sequences. Pages are handed
    out as sequences grow and come back when a sequence ends; nothing is copied or cleared. The table is
    written on torch's current stream."""

    def __init__(self, seqs, pages, page_size, heads, dim, fmt=COLI_KV_BF16, max_tokens=None, k_scale=None,
                 v_scale=None, device="cuda"):
        self.seqs, self.page_size, self.heads, self.dim, self.fmt = seqs, page_size, heads, dim, fmt
        self.device = torch.device(device)
        self.width = -(-(max_tokens or pages * page_size) // page_size)
        pool = (pages, heads, page_size, dim)
        self.k = torch.empty(pool, dtype=_TORCH[fmt], device=self.device)
        self.v = torch.empty(pool, dtype=_TORCH[fmt], device=self.device)
        self.k_scale, self.v_scale = k_scale, v_scale
        self.table = torch.full((seqs, self.width), -1, dtype=torch.int32, device=self.device)
        self.free = list(range(pages - 1, -1, -1))
        self.held = [[] for _ in range(seqs)]
        self.tokens = [0] * seqs
        self.desc = make_kv_cache(self.k, self.v, fmt, pages, page_size, heads, dim, k_scale=k_scale, v_scale=v_scale)

    def grow(self, seq, n=1):
        """Makes room for n more tokens of a sequence; returns the position of the first."""
        at = self.tokens[seq]
        want = -(-(at + n) // self.page_size)
        if want > self.width or want - len(self.held[seq]) > len(self.free):
            raise MemoryError("the cache has no page left")
        new = [self.free.pop() for _ in range(want - len(self.held[seq]))]
        if new:
            first = len(self.held[seq])
            self.table[seq, first:want] = torch.tensor(new, dtype=torch.int32, device=self.device)
            self.held[seq] += new
        self.tokens[seq] = at + n
        return at

    def end(self, seq):
        self.free += reversed(self.held[seq])
        self.held[seq], self.tokens[seq] = [], 0
        self.table[seq].fill_(-1)


class DecodeLayer:
    """One decoder layer's step for one new token of every sequence (slot), fp32 activations:
    attention over the cache, the norms around it, the MoE block (`block`, a DeviceBlock), and the norm
    that the next layer reads.

      w_qkv [(q_heads + 2 kv_heads) * dim, H], w_o [H, q_heads * dim]; mid_w, next_w [H]: the norms in
      front of the block and of the next layer; attn_post_w, block_post_w [H] or None: norms of what
      attention and block give back, before the residual takes it."""

    def __init__(self, block, cache: PagedCache, w_qkv, w_o, mid_w, next_w, inv_freq, q_heads, eps=1e-5, window=0,
                 interleaved=False, attn_post_w=None, block_post_w=None):
        self.block, self.cache, self.q_heads, self.eps = block, cache, q_heads, eps
        self.w_qkv, self.w_o, self.inv_freq = w_qkv, w_o, inv_freq
        self.mid_w, self.next_w, self.attn_post_w, self.block_post_w = mid_w, next_w, attn_post_w, block_post_w
        n, h, d, kh = cache.seqs, w_o.shape[0], cache.dim, cache.heads
        dev = cache.device
        row = (q_heads + 2 * kh) * d
        block.set_tokens(n)
        # q, k and v are slices of one projection's rows; q is rotated where it lies
        self.append = make_append_desc(n, q_heads, n, cache.width, COLI_ACT_F32, 2 * inv_freq.numel(), interleaved,
                                       q_stride=row, k_stride=row, v_stride=row, q_out_stride=row)
        self.attn = make_attn_desc(n, q_heads, cache.width, COLI_ACT_F32, d ** -0.5, window=window, q_stride=row)
        self.norms = make_norms_desc(n, h, COLI_ACT_F32, COLI_GATE_NONE, eps, eps)
        ws_bytes = coli_attn_workspace_bytes(self.attn, cache.desc)
        if ws_bytes == 0:
            raise ValueError("the attention does not take this cache with these heads and sequences")
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.heads_out = torch.empty(n, q_heads * d, device=dev)
        self.block_out = torch.empty(n, h, device=dev)

    def step(self, xn, resid, pos, lens, stream=None, seq=None):
        """xn [n, H]: the normalised input, resid [n, H] the residual (updated in place), pos and lens [n]
        int32: each sequence's new position and its tokens with the new one. Returns the next layer's xn.

        seq [n] int32, needed where a slot is idle (its sequence has ended and none has taken its place): -1 for
        such a slot, its own number for any other. Nothing is cached for an idle slot and its attention is 0, as
        its lens must be; its rows of xn and resid go through the block and mean nothing.

        Everything runs on one stream: torch's current one, or `stream` (a torch stream or a handle). What is
        given must be ready on the current stream, and the result is: another `stream` waits for the current one
        before the step, and the current one for it after. Can be captured into a graph (after one step outside
        it, which sets up the library products)."""
        now, on = self._streams(stream)
        if on is None:
            return self._run(xn, resid, pos, lens, seq, now)
        on.wait_stream(now)
        try:
            with torch.cuda.stream(on):
                out = self._run(xn, resid, pos, lens, seq, on)
        finally:  # what is under way still reads the arguments
            now.wait_stream(on)
        out.record_stream(now)  # it is on's memory
        return out

    def _streams(self, stream):
        """torch's current stream, and the one given if that is another."""
        dev = self.cache.device
        now = torch.cuda.current_stream(dev)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        return now, None if stream is None or stream.cuda_stream == now.cuda_stream else stream

    def _run(self, xn, resid, pos, lens, seq, stream):
        c, d, qd = self.cache, self.cache.dim, self.q_heads * self.cache.dim
        kd = c.heads * d
        qkv = xn @ self.w_qkv.T
        q, k, v = qkv[:, :qd], qkv[:, qd:qd + kd], qkv[:, qd + kd:]
        coli_kv_append(self.append, c.desc, q, k, v, self.inv_freq, seq, pos, c.table, q, self.err, stream)
        coli_attn_decode(self.attn, c.desc, q, c.table, lens, self.heads_out, None, self.err, self.ws, self.ws.numel(),
                         stream)
        y = self.heads_out @ self.w_o.T
        mid = torch.empty_like(y)
        coli_block_norms(self.norms, y, resid, self.attn_post_w, None, self.mid_w, resid, mid, stream)
        b = self.block
        coli_moe_forward(b.desc, mid, b.Wr, b.bias, b.table, b.shared, self.block_out, None, None, b.ws, b.ws_bytes,
                         stream)
        out = torch.empty_like(y)
        coli_block_norms(self.norms, self.block_out, resid, self.block_post_w, None, self.next_w, resid, out, stream)
        return out

    def check(self, stream=None):
        """Raises if a kernel flagged an error since the last check (synchronises `stream`, or the current one)."""
        now, on = self._streams(stream)
        coli_moe_check(self.err, on or now)
        coli_moe_check(self.block.ws, on or now)
