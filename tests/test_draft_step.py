"""A decoder layer's steps on drafted nodes (quantized_expert_decode_gb300/layer.py): the bookkeeping of shared pages and
of nodes, without a GPU; and, on one, nodes through a stack of layers against single-token steps along each
node's path, with the accepted path compacted, sequences forked and the decoding going on from there.

Tolerance of the steps: as in the tests of the single-token step, both sides are within 1e-3 rms of the layer in 64
bits (the cache rounds keys and values to the same bits on both sides but for values next to a rounding
border, the block is within 1e-4 rms of its oracle): 2e-3 rms of each other, for each layer that they went through."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__._builder().build()
    import quantized_expert_decode_gb300 as q
    return q


@pytest.fixture
def cache(q, monkeypatch):
    """A cache on the CPU whose page copies are noted."""
    from quantized_expert_decode_gb300.layer import PagedCache
    copies = []
    monkeypatch.setattr(PagedCache, "_copy", lambda self, src, dst: copies.append((src, dst)))
    c = PagedCache(4, 8, 4, 1, 16, max_tokens=24, device="cpu", layers=2)
    c.copies = copies
    return c


def held(c):
    """Every page is free or held, as often as it says, and the table names the held ones."""
    count = [0] * 8
    for s in range(4):
        assert c.table[s].tolist() == c.held[s] + [-1] * (c.width - len(c.held[s]))
        assert len(c.held[s]) == -(-c.tokens[s] // 4)
        for p in c.held[s]:
            count[p] += 1
    assert count == c.uses and sorted(c.free) == [p for p in range(8) if count[p] == 0]


def test_layers_share_a_table(cache):
    assert len(cache.k_pools) == len(cache.v_pools) == len(cache.descs) == len(cache.caches) == 2
    assert cache.k is cache.k_pools[0] and cache.desc is cache.descs[0]
    assert [d.k for d in cache.descs] == [k.data_ptr() for k in cache.k_pools]


def test_forked_sequences_share_full_pages(cache):
    c = cache
    c.grow(0, 10)
    c.fork(0, 1)
    held(c)
    assert c.held[1][:2] == c.held[0][:2] and c.held[1][2] != c.held[0][2] and c.tokens[1] == 10
    assert c.copies == [(c.held[0][2], c.held[1][2])]
    assert c.grow(1, 3) == 10 and c.grow(0) == 10
    held(c)
    c.end(0)
    held(c)
    assert c.uses[c.held[1][0]] == 1
    c.end(1)
    held(c)
    assert len(c.free) == 8


def test_a_fork_of_full_pages_copies_nothing(cache):
    c = cache
    c.grow(0, 8)
    c.fork(0, 1)
    c.fork(1, 2)
    held(c)
    assert c.copies == [] and c.uses[c.held[0][0]] == 3
    # what is appended goes to a page of its own
    c.grow(1, 2)
    held(c)
    assert c.held[1][2] not in c.held[0] + c.held[2]
    with pytest.raises(ValueError):
        c.fork(0, 1)
    with pytest.raises(ValueError):
        c.fork(0, 0)


def test_a_shared_page_is_copied_before_it_is_written(cache):
    c = cache
    c.grow(0, 8)
    c.fork(0, 1)
    c.cut(1, 6)  # into a page that sequence 0 holds too
    held(c)
    assert c.held[1] == c.held[0] and c.copies == []
    assert c.grow(1) == 6
    held(c)
    assert c.copies == [(c.held[0][1], c.held[1][1])] and c.held[1][1] != c.held[0][1]
    c.cut(0, 5)
    assert c.grow(0, 2) == 5  # alone on its page by now
    held(c)
    assert len(c.copies) == 1


def test_cut(cache):
    c = cache
    c.grow(0, 20)
    pages = list(c.held[0])
    for keep in (20, 17, 16, 9, 0):
        c.cut(0, keep)
        held(c)
        assert c.held[0] == pages[: -(-keep // 4)] and c.tokens[0] == keep
    for bad in (1, -1):
        with pytest.raises(ValueError):
            c.cut(0, bad)


def test_no_page_left(cache):
    c = cache
    c.grow(0, 22)
    c.grow(1, 8)
    held(c)
    with pytest.raises(MemoryError):
        c.fork(0, 2)  # its last page would be copied
    c.cut(0, 20)
    c.fork(0, 2)
    c.grow(3, 4)
    held(c)
    with pytest.raises(MemoryError):
        c.grow(2)
    c.cut(2, 18)
    with pytest.raises(MemoryError):
        c.grow(2)  # its page is shared: a copy is needed
    held(c)
    c.end(3)
    assert c.grow(2) == 18
    held(c)


def test_nodes(q):
    from quantized_expert_decode_gb300.layer import Nodes
    n = Nodes([10, 5, 7], [[-1, 0, 0, 1], [], [-1, -1, 1]], rows=9, device="cpu")
    assert (n.rows, n.nodes) == (9, 4)
    assert n.first.tolist() == [0, 4, 4, 7] and n.past.tolist() == [10, 5, 7]
    assert n.seq.tolist() == [0, 0, 0, 0, 2, 2, 2, -1, -1]
    assert n.pos.tolist() == [10, 11, 11, 12, 7, 7, 8, 0, 0] and n.place.tolist() == [10, 11, 12, 13, 7, 8, 9, 0, 0]
    assert n.parent.tolist() == [-1, 0, 0, 1, -1, -1, 1, -1, -1]
    for parents in ([[0]], [[-1, 1]], [[-2]]):
        with pytest.raises(ValueError):
            Nodes([0], parents, device="cpu")
    with pytest.raises(ValueError):
        Nodes([0], [[-1, 0]], rows=1, device="cpu")
    with pytest.raises(ValueError):
        Nodes([0], [[-1, 0]], nodes=1, device="cpu")


def test_a_step_takes_its_own_rows_only(q):
    from quantized_expert_decode_gb300.layer import DecodeLayer, Nodes, PagedCache
    block = types.SimpleNamespace(set_tokens=lambda n: None, desc=q.make_desc(1, 256, 128, 8, 2))
    cache = PagedCache(2, 8, 4, 1, 16, device="cpu")
    layer = DecodeLayer(block, cache, torch.zeros(64, 32), torch.zeros(32, 32), None, None, torch.ones(8), 2)
    d = layer.drafts(4, 3)
    x = torch.zeros(4, 32)
    for rows, nodes in ((5, [[-1, 0], [-1]]), (4, [[-1, 0, 1, 2], []])):
        with pytest.raises(ValueError):
            layer.draft_step(d, x, x, Nodes([0, 0], nodes, rows=rows, device="cpu"))
    with pytest.raises(ValueError):
        layer.draft_step(d, x[:3], x[:3], Nodes([0, 0], [[-1, 0], [-1]], rows=4, device="cpu"))
    for rows, nodes in ((0, 1), (4, 0), (4, 257)):
        with pytest.raises(ValueError):
            layer.drafts(rows, nodes)


# ------------------------------------------------------------------------------------ on a GPU
H, QH, KH, D, LAYERS, VOCAB = 256, 6, 2, 32, 2, 50


class Model:
    """A stack of layers with an embedding, the same weights for every instance."""

    def __init__(self, fmt=1, window=0, norms=True, seqs=3, page=4):
        import synth
        from quantized_expert_decode_gb300.device import DeviceBlock
        from quantized_expert_decode_gb300.layer import DecodeLayer, PagedCache
        g = torch.Generator("cuda").manual_seed(11)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        scale = torch.full((KH,), 0.05, device="cuda") if fmt == 3 else None
        self.cache = PagedCache(seqs, 60, page, KH, D, fmt, k_scale=scale, v_scale=scale, layers=LAYERS)
        for pool in self.cache.k_pools + self.cache.v_pools:
            pool.view(torch.uint8).fill_(0x7f if fmt == 3 else 0xff)  # NaN until it is written
        self.layers = []
        for i in range(LAYERS):
            blk = synth.make_block(0, seed=i)
            assert blk["cfg"]["H"] == H
            w = [torch.rand(H, device="cuda", generator=g) + 0.5 for _ in range(2)]
            qk = [torch.rand(D, device="cuda", generator=g) + 0.5 for _ in range(2)] if norms else [None, None]
            inv = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
            self.layers.append(DecodeLayer(DeviceBlock(blk), self.cache, rand((QH + 2 * KH) * D, H) / H ** 0.5,
                                           rand(H, QH * D) / (QH * D) ** 0.5, w[0], w[1], inv, QH, window=window, q_norm=qk[0],
                                           k_norm=qk[1], layer=i))
        self.embed = rand(VOCAB, H)
        self.drafts = {}

    def start(self, tokens):
        r = self.embed[torch.as_tensor(tokens, device="cuda")].clone()
        return r * torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-5), r

    def step(self, tokens, live=None):
        """One token of every sequence (None: idle); the last layer's output."""
        on = [t is not None for t in tokens]
        at = [self.cache.grow(s) if on[s] else 0 for s in range(len(on))]
        x, r = self.start([t or 0 for t in tokens])
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        mask = torch.tensor(on, device="cuda")
        seq = torch.arange(len(on), dtype=torch.int32, device="cuda").masked_fill(~mask, -1)
        for layer in self.layers:
            x = layer.step(x, r, pos, (pos + 1) * mask, seq=seq)
            layer.check()
        return x

    def step_nodes(self, parents, tokens, rows=None, stream=None):
        """Nodes of every sequence in one pass; room is made for them. The last layer's output."""
        from quantized_expert_decode_gb300.layer import Nodes
        past = list(self.cache.tokens)
        for s, p in enumerate(parents):
            self.cache.grow(s, len(p))
        nodes = Nodes(past, parents, rows=rows, nodes=16)
        x, r = self.start([t for row in tokens for t in row] + [0] * (nodes.rows - sum(map(len, tokens))))
        for layer in self.layers:
            key = (layer, nodes.rows)
            d = self.drafts.setdefault(key, layer.drafts(nodes.rows, 16)) if key not in self.drafts else self.drafts[key]
            x = layer.draft_step(d, x, r, nodes, stream)
            layer.check(drafts=d)
        return x, past


def along(past, tokens, **a):
    """The outputs at `tokens` stepped one at a time behind `past`, by a model of their own."""
    m = Model(seqs=1, **a)
    for t in past:
        m.step([t])
    return [m.step([t])[0] for t in tokens]


def near(got, want):
    assert float((got - want).abs().max()) <= 2e-3 * LAYERS * float(want.square().mean().sqrt())


TREES = [[-1, 0, 0, 1, 1, 2, 3], [-1], [-1, 0, 1, 2, 0]]
TOKENS = [[5, 7, 8, 9, 1, 2, 3], [4], [20, 21, 22, 23, 24]]
PASTS = [[1, 2, 3, 4, 5, 6, 7, 8, 9], [10, 11], [30, 31, 32, 33, 34, 35]]


def path_of(tree, i):
    line = []
    while i >= 0:
        line.insert(0, i)
        i = tree[i]
    return line


def filled(**a):
    m = Model(**a)
    for i in range(max(map(len, PASTS))):
        m.step([p[i] if i < len(p) else None for p in PASTS])
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,window,norms,rows", [(1, 0, True, None), (2, 5, True, 20), (1, 3, False, 16), (1, 0, True, 80)])
def test_nodes_are_as_steps_along_their_paths(q, fmt, window, norms, rows):
    kind = dict(fmt=fmt, window=window, norms=norms)
    m = filled(**kind)
    x, _ = m.step_nodes(TREES, TOKENS, rows)
    at = 0
    for past, tree, tokens in zip(PASTS, TREES, TOKENS):
        for leaf in [i for i in range(len(tree)) if i not in tree]:
            line = path_of(tree, leaf)
            for node, want in zip(line, along(past, [tokens[i] for i in line], **kind)):
                if rows != 80:
                    near(x[at + node], want)
                else:
                    # the block of more than 64 rows runs on 16-bit operands, 2e-2 rms of its oracle
                    assert float((x[at + node] - want).abs().max()) <= 0.1 * LAYERS * float(want.square().mean().sqrt())
        at += len(tree)


@pytest.mark.gpu
def test_an_8_bit_cache_takes_nodes(q):
    # an e4m3 step is 2^-3 of one element among 32: values next to a rounding border may differ by that
    m = filled(fmt=3)
    x, _ = m.step_nodes(TREES, TOKENS)
    at = 0
    for past, tree, tokens in zip(PASTS, TREES, TOKENS):
        line = path_of(tree, len(tree) - 1)
        for node, want in zip(line, along(past, [tokens[i] for i in line], fmt=3)):
            assert float((x[at + node] - want).abs().max()) <= 0.1 * float(want.square().mean().sqrt())
        at += len(tree)


@pytest.mark.gpu
def test_accepted_paths_go_on(q):
    # verify by the target's largest entries, compact, cut, and go on: as the same tokens stepped one at a time
    m = filled()
    head = torch.randn(VOCAB, H, device="cuda", generator=torch.Generator("cuda").manual_seed(12))
    text = [list(p) for p in PASTS]
    last = [40, 41, 42]  # each sequence's last token, not cached yet
    lengths = []
    for turn in range(4):
        # what the target wants next, by steps of its own, so that some drafted nodes are right
        wanted = []
        for s in range(3):
            toks, here = [last[s]], []
            for _ in range(3):
                y = along(text[s], toks)[-1]
                toks.append(int((head @ y).argmax()))
            wanted.append(toks[1:])
        trees, tokens = [], []
        for s in range(3):
            a, b, c = wanted[s]
            trees.append([-1, 0, 0, 2, 2, 4][: 6 - s])
            tokens.append([last[s], (a + 1) % VOCAB, a, (b + 1) % VOCAB, b if turn != 2 else (b + 2) % VOCAB, c][: 6 - s])
        x, past = m.step_nodes(trees, tokens)
        logits = x @ head.T
        flat = [t for row in trees for t in row]
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        path, count, token = ints([[0] * 6] * 3), ints([0] * 3), ints([0] * 3)
        first = ints([0, 6, 11, 15])
        q.coli_draft_verify(q.make_verify_desc(3, 15, 6, VOCAB, mode=q.COLI_VERIFY_GREEDY), logits, None,
                            ints([t for row in tokens for t in row]), ints(flat), None, first, path, count, token,
                            stream=torch.cuda.current_stream())
        m.cache.compact(ints(past), path, count)
        for s, (n, line) in enumerate(zip(count.tolist(), path.tolist())):
            assert 1 <= n
            lengths.append(n)
            m.cache.cut(s, past[s] + n)
            text[s] += [tokens[s][i] for i in line[:n]]
            last[s] = int(token[s])
    assert max(lengths) >= 3 and min(lengths) >= 2
    # what is cached now is what single steps cache
    x = m.step(last)
    for s in range(3):
        near(x[s], along(text[s], [last[s]])[0])


@pytest.mark.gpu
def test_forks_go_their_own_ways(q):
    m = Model(seqs=3)
    text = [3, 1, 4, 1, 5, 9, 2]
    for t in text:
        m.step([t, None, None])
    m.cache.fork(0, 1)
    m.cache.fork(1, 2)
    a = m.step([10, 20, 30])
    m.cache.cut(2, 4)  # into a shared page
    b = m.step([11, 21, 31])
    for s, (first, second) in enumerate(((10, 11), (20, 21))):
        want = along(text, [first, second])
        near(a[s], want[0])
        near(b[s], want[1])
    near(b[2], along(text[:4], [31])[0])


@pytest.mark.gpu
def test_steps_on_nodes_in_a_graph_and_on_a_stream(q):
    from quantized_expert_decode_gb300.layer import Nodes
    want, past = filled().step_nodes(TREES, TOKENS)
    side = torch.cuda.Stream()
    got, _ = filled().step_nodes(TREES, TOKENS, stream=side)
    near(got, want)
    m = filled()
    for s, p in enumerate(TREES):
        m.cache.grow(s, len(p))
    nodes = Nodes(past, TREES, nodes=16)
    drafts = [layer.drafts(nodes.rows, 16) for layer in m.layers]
    x0, r0 = m.start([t for row in TOKENS for t in row])
    x, r = x0.clone(), r0.clone()

    def run():
        y = x
        for layer, d in zip(m.layers, drafts):
            y = layer.draft_step(d, y, r, nodes)
        return y

    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = run()
        for _ in range(2):
            x.copy_(x0)
            r.copy_(r0)
            graph.replay()
    side.synchronize()
    near(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("args", [["--steps", "3"], ["--layers", "1", "--seqs", "3", "--past", "0", "--wide", "1", "--deep", "5", "--steps", "4"]])
def test_the_example_runs(q, args):
    import os
    import subprocess
    import sys
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_layer.py")
    r = subprocess.run([sys.executable, at, *args], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens of a sequence a step" in r.stdout
