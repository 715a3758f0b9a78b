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


class FakeStream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


@pytest.fixture
def fake(q, monkeypatch):
    """A layer on the CPU whose library calls only note the stream they are given, torch's current stream
    beside it and some arguments, on streams that are numbers."""
    import contextlib
    import types

    from quantized_expert_decode_gb300 import layer as mod
    log = []
    now = [FakeStream(7, log)]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    def note(name, at, **kept):
        def call(*a):
            log.append((name, a[at] if a[at] is None or isinstance(a[at], int) else a[at].cuda_stream, now[-1].cuda_stream,
                        *(a[i] for i in kept.values())))
        monkeypatch.setattr(mod, name, call)

    note("coli_kv_append", 11, seq=6)
    note("coli_attn_decode", 10)
    note("coli_block_norms", 8)
    note("coli_moe_forward", 11)
    note("coli_moe_check", 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0, log))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle, log))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s.cuda_stream)))
    block = types.SimpleNamespace(set_tokens=lambda n: None, desc=None, Wr=None, bias=None, table=None, shared=None, ws=None,
                                  ws_bytes=0)
    cache = mod.PagedCache(2, 8, 4, 1, 16, device="cpu")
    layer = mod.DecodeLayer(block, cache, torch.zeros(64, 32), torch.zeros(32, 32), None, None, torch.ones(8), 2)
    x = torch.zeros(2, 32)
    at = torch.zeros(2, dtype=torch.int32)
    return types.SimpleNamespace(layer=layer, cache=cache, log=log, now=now, args=(x, x.clone(), at, at + 1))


def test_a_step_runs_on_one_stream(fake):
    # the projections run on torch's current stream: every library call's stream is the one that is current then
    calls = lambda: [e for e in fake.log if e[0].startswith("coli")]  # noqa: E731
    fake.layer.step(*fake.args)
    fake.layer.check()
    assert [e[0] for e in fake.log] == ["coli_kv_append", "coli_attn_decode", "coli_block_norms", "coli_moe_forward",
                                        "coli_block_norms", "coli_moe_check", "coli_moe_check"]
    assert all(e[1:3] == (7, 7) for e in calls())
    for given, handle in ((FakeStream(9, fake.log), 9), (9, 9), (0, 0)):
        # another stream: it waits for the current one, which then waits for it, and the result is used on both
        fake.log.clear()
        fake.layer.step(*fake.args, given)
        assert all(e[1:3] == (handle, handle) for e in calls()) and len(calls()) == 5
        assert fake.log[0] == ("wait", handle, 7) and fake.log[-2:] == [("wait", 7, handle), ("record", 7)]
    fake.log.clear()
    fake.layer.step(*fake.args, FakeStream(7, fake.log))
    fake.layer.check(9)
    assert [e[1:3] for e in calls()] == [(7, 7)] * 5 + [(9, 7)] * 2 and len(fake.log) == 7


def test_a_step_hands_the_slots_on(fake):
    # which slots append, -1 for an idle one
    seq = torch.tensor([-1, 1], dtype=torch.int32)
    for given in (None, seq):
        fake.log.clear()
        fake.layer.step(*fake.args, seq=given)
        assert fake.log[0][0] == "coli_kv_append" and fake.log[0][3] is given


@pytest.mark.parametrize("seqs,q_heads", [(2049, 2), (2, 3), (2, 2048)])
def test_a_layer_that_the_attention_refuses_is_not_built(q, seqs, q_heads):
    import types

    from quantized_expert_decode_gb300.layer import DecodeLayer, PagedCache
    block = types.SimpleNamespace(set_tokens=lambda n: None)
    cache = PagedCache(seqs, 2, 4, 2, 16, max_tokens=4, device="cpu")
    with pytest.raises(ValueError):
        DecodeLayer(block, cache, torch.zeros((q_heads + 4) * 16, 8), torch.zeros(8, q_heads * 16), None, None, torch.ones(8), q_heads)


def run_steps(mode, fmt, n, steps=6):
    """The outputs of some steps of a layer, the same layer and inputs for every mode: on the default stream, on a
    side stream that is torch's current one, on a stream that is not (by its handle, the default one beside a side stream),
    or replayed from a graph."""
    import synth
    from quantized_expert_decode_gb300.device import DeviceBlock
    from quantized_expert_decode_gb300.layer import DecodeLayer, PagedCache
    blk = synth.make_block(0)
    h, qh, kh, d = blk["cfg"]["H"], 6, 2, 32
    g = torch.Generator("cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    scale = torch.full((kh,), 0.05, device="cuda") if fmt == 3 else None
    cache = PagedCache(n, 10 * n, 4, kh, d, fmt, k_scale=scale, v_scale=scale)
    ones = torch.ones(h, device="cuda")
    layer = DecodeLayer(DeviceBlock(blk), cache, rand((qh + 2 * kh) * d, h) / h ** 0.5, rand(h, qh * d) / (qh * d) ** 0.5, ones, ones,
                        torch.rand(d // 2, device="cuda", generator=g), qh)
    x, r = rand(n, h), rand(n, h)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(pos)
    torch.cuda.synchronize()
    side, out, graph, y = torch.cuda.Stream(), [], None, None
    with torch.cuda.stream(side if mode in ("current", "graph", "zero") else torch.cuda.default_stream()):
        for i in range(steps):
            at = [cache.grow(s) for s in range(n)]
            torch.cuda._sleep(2_000_000)  # what does not wait for the current stream runs ahead of it
            pos.copy_(torch.tensor(at, dtype=torch.int32))
            lens.copy_(pos + 1)
            if mode == "graph" and i == 1:
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph, stream=side):
                    y = layer.step(x, r, pos, lens)
            if graph is not None:
                graph.replay()
            else:
                given = {"other": (side,), "handle": (side.cuda_stream,), "zero": (0,)}.get(mode, ())
                y = layer.step(x, r, pos, lens, *given)
            x.copy_(y)
            out.append((x.clone(), r.clone()))
        layer.check()
    torch.cuda.synchronize()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [(1, 4), (2, 3), (3, 4), (1, 1)])
def test_steps_on_streams_and_in_graphs(q, fmt, n):
    # the same kernels on the same values; only the library products may take another order of sums (some 1e-6, which
    # may move a cached value over a rounding border: an e4m3 step is 2^-3 of one element among 32). What is read too
    # early is off by the size of the values.
    want = run_steps("default", fmt, n)
    for mode in ("current", "other", "handle", "zero", "graph"):
        for i, (got, ref) in enumerate(zip(run_steps(mode, fmt, n), want)):
            for a, b in zip(got, ref):
                assert float((a - b).abs().max()) <= 0.05 * float(b.square().mean().sqrt()), (mode, i)


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


@pytest.mark.gpu
@pytest.mark.parametrize("idle", [{2: (3, 6)}, {0: (2, 8), 3: (4, 5)}])
def test_idle_slots(q, idle):
    # Slots {slot: (first idle step, step of its next sequence)}: the other slots' rows are those of a batch without
    # idle slots, a slot's next sequence is its first one over again, nothing is flagged and nothing cached for an
    # idle slot. Rows are computed apart from each other but for the block's order of sums (1e-4 rms of its oracle).
    import synth
    from quantized_expert_decode_gb300.device import DeviceBlock
    from quantized_expert_decode_gb300.layer import DecodeLayer, PagedCache
    blk = synth.make_block(0)
    n, steps, h, qh, kh, d = 4, 9, blk["cfg"]["H"], 6, 2, 32
    g = torch.Generator("cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w_qkv, w_o, inv = rand((qh + 2 * kh) * d, h) / h ** 0.5, rand(h, qh * d) / (qh * d) ** 0.5, torch.rand(d // 2, device="cuda")
    ones, x0, r0 = torch.ones(h, device="cuda"), rand(n, h), rand(n, h)

    def run(idle):
        cache = PagedCache(n, 20, 4, kh, d)
        for pool in (cache.k, cache.v):
            pool.zero_()
        layer = DecodeLayer(DeviceBlock(blk), cache, w_qkv, w_o, ones, ones, inv, qh)
        x, r, out = x0.clone(), r0.clone(), []
        for step in range(steps):
            for s, (first, again) in idle.items():
                if step == first:
                    cache.end(s)
                if step == again:
                    x[s], r[s] = x0[s], r0[s]
            on = [not (s in idle and idle[s][0] <= step < idle[s][1]) for s in range(n)]
            at = [cache.grow(s) if on[s] else 0 for s in range(n)]
            pos, live = torch.tensor(at, dtype=torch.int32, device="cuda"), torch.tensor(on, device="cuda")
            seq = torch.arange(n, dtype=torch.int32, device="cuda").masked_fill(~live, -1) if idle else None
            pools = [cache.k.clone(), cache.v.clone()]
            x = layer.step(x, r, pos, (pos + 1) * live, seq=seq)
            layer.check()
            rows = {(int(cache.table[s, at[s] // 4]), at[s] % 4) for s in range(n) if on[s]}
            for pool, was in zip((cache.k, cache.v), pools):
                changed = (pool.view(torch.int16) != was.view(torch.int16)).any(3).any(1)
                assert {tuple(e) for e in changed.nonzero().tolist()} <= rows
            out.append((x.clone(), r.clone(), on))
        return out

    full, some = run({}), run(idle)
    for step in range(steps):
        for s in range(n):
            if not some[step][2][s]:
                continue
            like = step - idle[s][1] if s in idle and step >= idle[s][1] else step
            for a, b in zip(some[step][:2], full[like][:2]):
                assert float((a[s] - b[s]).abs().max()) <= 1e-3 * float(b[s].square().mean().sqrt()), (step, s)
