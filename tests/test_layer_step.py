"""A decoder layer's steps (quantized_expert_decode_gb300/layer.py) against the same layer written down in
64 bits, the MoE block by the oracle: several steps, sequences of different lengths, an idle page freed
and used again. And the page bookkeeping alone, without a GPU.

Tolerance: the projections are fp32 library products (some 1e-6 relative), the cache rounds keys and
values to the same bits on both sides but for values next to a rounding border (one bf16 step, 2^-8, of
one element among hundreds summed), the block is within 1e-4 rms of the oracle: 1e-3 rms."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__._builder().build()
    import quantized_expert_decode_gb300 as q
    return q


def test_pages_are_handed_out_and_come_back(q):
    from quantized_expert_decode_gb300.layer import PagedCache
    c = PagedCache(2, 5, 4, 1, 16, max_tokens=16, device="cpu")
    assert [c.grow(0, 3), c.grow(0), c.grow(0)] == [0, 3, 4]
    assert c.grow(1, 9) == 0
    held = c.table[0, :2].tolist() + c.table[1, :3].tolist()
    assert sorted(held) == [0, 1, 2, 3, 4] and int((c.table >= 0).sum()) == 5
    with pytest.raises(MemoryError):
        c.grow(1, 4)
    assert c.tokens == [5, 9]
    c.end(0)
    assert c.grow(1, 4) == 9 and c.table[1, 3].item() in held[:2] and int((c.table[0] >= 0).sum()) == 0
    with pytest.raises(MemoryError):
        c.grow(1, 4)  # beyond the table


@pytest.mark.gpu
@pytest.mark.parametrize("window,interleaved,sandwich", [(0, False, False), (5, True, True)])
def test_steps_match_the_definition(q, window, interleaved, sandwich):
    import oracle
    import synth
    from quantized_expert_decode_gb300.device import DeviceBlock
    from quantized_expert_decode_gb300.layer import DecodeLayer, PagedCache
    oracle.build()
    rng = np.random.default_rng(7)
    blk = synth.make_block(0)
    n, h, qh, kh, d, eps = 4, blk["cfg"]["H"], 6, 2, 32, 1e-5
    f32 = lambda a: np.asarray(a, np.float32)  # noqa: E731
    w_qkv, w_o = f32(rng.standard_normal(((qh + 2 * kh) * d, h)) / h ** 0.5), f32(rng.standard_normal((h, qh * d)) / (qh * d) ** 0.5)
    w = [f32(rng.uniform(0.5, 1.5, h)) for _ in range(4)]
    inv = f32(1e4 ** (-np.arange(0, d, 2) / d))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    cache = PagedCache(n, 40, 4, kh, d, max_tokens=40)
    layer = DecodeLayer(DeviceBlock(blk), cache, dev(w_qkv), dev(w_o), dev(w[0]), dev(w[1]), dev(inv), qh, eps, window, interleaved,
                        dev(w[2]) if sandwich else None, dev(w[3]) if sandwich else None)
    resid = f32(rng.standard_normal((n, h)))
    norm = lambda x, g: x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * g.astype(np.float64)  # noqa: E731
    x64, r64 = norm(resid.astype(np.float64), w[1]), resid.astype(np.float64)
    tx, tr = dev(f32(x64)), dev(resid)
    past = [[] for _ in range(n)]
    bf16 = lambda a: torch.from_numpy(a).to(torch.bfloat16).double().numpy()  # noqa: E731
    for step in range(9):
        if step == 4:  # a sequence ends, another takes its place
            cache.end(2)
            past[2] = []
        at = [cache.grow(s) for s in range(n)]
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        tx = layer.step(tx, tr, pos, pos + 1)
        # the definition
        qkv = x64 @ w_qkv.T.astype(np.float64)
        xq, xk, xv = qkv[:, :qh * d].reshape(n, qh, d), qkv[:, qh * d:(qh + kh) * d].reshape(n, kh, d), qkv[:, (qh + kh) * d:].reshape(n, kh, d)
        ia = np.arange(0, d, 2) if interleaved else np.arange(d // 2)
        ib = ia + (1 if interleaved else d // 2)
        heads = np.zeros((n, qh, d))
        for s in range(n):
            t = at[s] * inv.astype(np.float64)
            turn = []
            for m in (xq[s], xk[s]):
                z = m.copy()
                z[:, ia] = m[:, ia] * np.cos(t) - m[:, ib] * np.sin(t)
                z[:, ib] = m[:, ib] * np.cos(t) + m[:, ia] * np.sin(t)
                turn.append(z)
            past[s].append((bf16(turn[1]), bf16(xv[s])))
            seen = past[s][-window:] if window else past[s]
            for j in range(qh):
                k, v = np.array([e[0][j // (qh // kh)] for e in seen]), np.array([e[1][j // (qh // kh)] for e in seen])
                p = k @ turn[0][j] * d ** -0.5
                p = np.exp(p - p.max())
                heads[s, j] = p @ v / p.sum()
        y = heads.reshape(n, -1) @ w_o.T.astype(np.float64)
        r64 = r64 + (norm(y, w[2]) if sandwich else y)
        mid = norm(r64, w[0])
        y = oracle.moe_forward(blk, x=f32(mid))[0].astype(np.float64)
        r64 = r64 + (norm(y, w[3]) if sandwich else y)
        x64 = norm(r64, w[1])
        for got, want in ((tr, r64), (tx, x64)):
            err = np.abs(got.cpu().numpy() - want).max()
            assert err <= 1e-3 * np.sqrt((want ** 2).mean()), (step, err)
    layer.check()
