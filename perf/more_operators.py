"""Workloads of a decoder's step on drafted tokens: each sequence brings a chain or a tree of drafted tokens (nodes),
the model sees them all in one pass, and what the target's probabilities accept stays in the cache.

Each case names one operator and its sizes. `run` computes a case in its plain form (elementary torch operations) or,
with `own` true, through the library's entry points:

  append   queries and keys are normalised per head, rotated by the nodes' positions, and keys and values are written
           to the nodes' places in the paged cache (a node's place is not its position: branches share positions)
  tree     every node attends to its sequence's cached tokens, to its ancestors among the nodes and to itself
  verify   the nodes are accepted or rejected by the target's probabilities, the draft's and given random numbers, and
           one more token is drawn
  compact  the cached rows of the accepted nodes move to the places behind the sequence's committed tokens
  copy     pages are copied for a sequence that is forked
"""
import math

import torch

own = False

DEVICE = "cuda"
ACT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KV = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
EPS = 1e-6
ROPE_BASE = 1e6


# ------------------------------------------------------------------------------------ the cases
def _append(name, seqs, nodes, past, heads, dim, rotary, interleaved, normed, act, kv, page, layout):
    return dict(name=name, op="append", seqs=seqs, nodes=nodes, past=past, q_heads=heads[0], kv_heads=heads[1], dim=dim,
                rotary=rotary, interleaved=interleaved, normed=normed, act=act, kv=kv, page=page, layout=layout)


def _tree(name, seqs, nodes, longest, ragged, chain, window, heads, dim, act, kv, page, layout):
    return dict(name=name, op="tree", seqs=seqs, nodes=nodes, longest=longest, ragged=ragged, chain=chain, window=window,
                q_heads=heads[0], kv_heads=heads[1], dim=dim, act=act, kv=kv, page=page, layout=layout)


def _verify(name, seqs, nodes, chain, vocab, draft, greedy, act):
    return dict(name=name, op="verify", seqs=seqs, nodes=nodes, chain=chain, vocab=vocab, draft=draft, greedy=greedy,
                act=act)


def _compact(name, layers, seqs, nodes, accepted, past, kv_heads, dim, kv, page, layout):
    return dict(name=name, op="compact", layers=layers, seqs=seqs, nodes=nodes, accepted=accepted, past=past,
                kv_heads=kv_heads, dim=dim, kv=kv, page=page, layout=layout)


def _copy(name, layers, pages, kv_heads, dim, kv, page, layout):
    return dict(name=name, op="copy", layers=layers, pages=pages, kv_heads=kv_heads, dim=dim, kv=kv, page=page,
                layout=layout)


def listed():
    return [
        # one chat's step: the last token and seven drafted ones, fp32 activations as the MoE block takes them: latency
        _append("append-one-draft", 1, 8, 4096, (16, 2), 128, 128, False, True, "f32", "bf16", 16, "hnd"),
        # a full server's step: 32 sequences with trees of up to 64 nodes, far positions, an 8-bit cache
        _append("append-batch-32", 32, 64, 200000, (48, 8), 128, 64, True, True, "bf16", "e4m3", 64, "hnd"),
        # one short chat, a small tree: latency
        _tree("tree-one-short", 1, 8, 500, False, False, 0, (16, 2), 128, "f32", "bf16", 16, "hnd"),
        # one long document and a large tree: the only parallelism is along the length
        _tree("tree-one-long", 1, 64, 131007, False, False, 0, (48, 8), 128, "bf16", "bf16", 64, "hnd"),
        # a batch of 32 sequences of all lengths, fp32 activations, one slot idle
        _tree("tree-batch-32", 32, 21, 8192, True, False, 0, (48, 8), 128, "f32", "bf16", 16, "hnd"),
        # a full server: many long sequences on an 8-bit cache, pages of whole tokens
        _tree("tree-batch-48-e4m3", 48, 16, 16384, False, False, 0, (64, 8), 128, "bf16", "e4m3", 64, "nhd"),
        # one chat's chain of five drafted tokens: latency
        _verify("verify-one-chain", 1, 6, True, 32000, True, False, "f32"),
        # a batch with trees and a large vocabulary
        _verify("verify-batch-32", 32, 32, False, 131072, True, False, "f32"),
        # what one chat's step accepted, over all layers: latency
        _compact("compact-one", 32, 1, 16, 4, 4000, 8, 128, "bf16", 16, "hnd"),
        # the same for a batch with long accepted paths
        _compact("compact-batch-64", 32, 64, 64, 9, 1000, 8, 128, "bf16", 64, "nhd"),
        # a fork of one sequence: its last, partly filled page, over all layers: latency
        _copy("copy-one-page", 32, 1, 8, 128, "bf16", 16, "hnd"),
        # prompts duplicated for many samples each: bandwidth
        _copy("copy-256-pages", 8, 256, 8, 128, "f16", 64, "hnd"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"], w["flops"]


def draw(rng):
    most = {}
    for c in listed():
        b, f = _cost(c)
        most[c["op"]] = (max(most.get(c["op"], (0, 0))[0], b), max(most.get(c["op"], (0, 0))[1], f))
    op = rng.choice(["append", "tree", "tree", "tree", "verify", "verify", "compact", "copy"])
    while True:
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
        group = rng.choice([1, 2, 4, 5, 6, 8, 12, 16])
        heads = (kv_heads * group, kv_heads)
        act, kv = rng.choice(sorted(ACT)), rng.choice(sorted(KV))
        page, layout = rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(["hnd", "nhd"])
        if op == "append":
            rotary = rng.choice([dim, dim, dim // 2, 0])
            c = _append("", _log_int(rng, 1, 64), _log_int(rng, 1, 100), _log_int(rng, 100, 300000), heads, dim, rotary,
                        rng.random() < 0.4, rng.random() < 0.8, act, kv, page, layout)
        elif op == "tree":
            window = _log_int(rng, 64, 4096) if rng.random() < 0.25 else 0
            c = _tree("", _log_int(rng, 1, 64), _log_int(rng, 1, 100), _log_int(rng, 16, 131072), rng.random() < 0.6,
                      rng.random() < 0.3, window, heads, dim, act, kv, page, layout)
        elif op == "verify":
            greedy = rng.random() < 0.25
            c = _verify("", _log_int(rng, 1, 64), _log_int(rng, 1, 64), rng.random() < 0.4, _log_int(rng, 1000, 150000),
                        not greedy and rng.random() < 0.7, greedy, rng.choice(["f32", "f32", "bf16", "f16"]))
        elif op == "compact":
            nodes = _log_int(rng, 3, 100)
            c = _compact("", rng.choice([1, 2, 28, 32, 61]), _log_int(rng, 1, 64), nodes, rng.randint(1, min(16, nodes // 2 + 1)),
                         _log_int(rng, 10, 4000), kv_heads, dim, kv, page, layout)
        else:
            c = _copy("", rng.choice([1, 2, 16, 28, 32, 61]), _log_int(rng, 1, 2000), kv_heads, dim, kv, page, layout)
        b, f = _cost(c)
        if b > most[op][0] or f > most[op][1] or heads[0] > 128:
            continue
        # the plain forms make every sequence as long as the longest, in 32 bits, and hold every row's scores
        if op == "tree" and (c["seqs"] * c["longest"] * kv_heads * dim > 48 * 16384 * 8 * 128 or
                             c["seqs"] * c["nodes"] * c["longest"] * heads[0] > 48 * 16 * 16384 * 64):
            continue
        if op == "verify" and c["seqs"] * c["nodes"] * c["vocab"] > 32 * 32 * 131072:
            continue
        # what a pass gives back: whole pools
        if op == "compact" and c["layers"] * _compact_pages(c) * page * kv_heads * dim > 1 << 30:
            continue
        del c["name"]
        return c


def _frac(i):
    return math.modf(0.61803398875 * (i + 1))[0]


def _past(case):
    """Committed tokens of each sequence (the same for every seed)."""
    n, top = case["seqs"], case["longest"]
    if not case["ragged"]:
        return [top - i % 3 if top > 3 else top for i in range(n)]
    lens = [int(top * _frac(i)) for i in range(n)]
    lens[n // 2] = top
    return lens


def _counts(case):
    """Nodes of each sequence: between half of the most and the most, in large batches one idle slot."""
    n, top = case["seqs"], case["nodes"]
    count = [top - int((top // 2) * _frac(3 * i)) for i in range(n)]
    count[n // 2] = top
    if n >= 8:
        count[3] = 0
    return count


def _accepted(case):
    """Nodes of each sequence's accepted path, the root among them: at most half of all."""
    n = case["nodes"]
    return [min((n + 1) // 2, 1 + int(case["accepted"] * (0.5 + 0.5 * _frac(i)))) for i in range(case["seqs"])]


def _compact_pages(case):
    return case["seqs"] * ((case["nodes"] + case["page"] - 1) // case["page"] + 1) + 4


def _size(name):
    return {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}[name]


def work(case):
    op = case["op"]
    if op == "append":
        n, qh, kh, d = sum(_counts(case)), case["q_heads"], case["kv_heads"], case["dim"]
        a, c = _size(case["act"]), _size(case["kv"])
        return {"bytes": n * d * (2 * qh * a + 2 * kh * (a + c)) + 16 * n + 2 * case["rotary"] + 8 * d,
                "flops": n * (qh + kh) * (3 * case["rotary"] + (4 * d if case["normed"] else 0))}
    if op == "tree":
        qh, kh, d, w = case["q_heads"], case["kv_heads"], case["dim"], case["window"]
        tokens = pairs = 0
        for past, n in zip(_past(case), _counts(case)):
            if n:
                seen = min(past, w - 1) if w else past
                tokens += seen + n
                pairs += n * (seen + 1)
        rows = sum(_counts(case))
        return {"bytes": tokens * kh * d * 2 * _size(case["kv"]) + rows * (qh * (2 * d * _size(case["act"]) + 4) + 4),
                "flops": 4 * pairs * qh * d}
    if op == "verify":
        rows = sum(1 for n in _counts(case) if n) * (2 if case["draft"] else 1)
        return {"bytes": rows * case["vocab"] * _size(case["act"]) + 16 * sum(_counts(case)), "flops": 2 * rows * case["vocab"]}
    row = case["kv_heads"] * case["dim"] * _size(case["kv"]) * 2 * case["layers"]
    if op == "compact":
        return {"bytes": 2 * row * sum(n - 1 for n in _accepted(case)) + 8 * case["seqs"], "flops": 0}
    return {"bytes": 2 * row * case["page"] * case["pages"] + 8 * case["pages"], "flops": 0}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _pool(case, pages, g):
    """One cache pool: [page][head][slot][dim] or [page][slot][head][dim] in memory."""
    order = (case["kv_heads"], case["page"]) if case["layout"] == "hnd" else (case["page"], case["kv_heads"])
    x = _randn(g, pages, *order, case["dim"])
    if case["kv"] == "e4m3":
        x = x.mul_(16.0)
    return x.to(KV[case["kv"]])


def _paged(case, pool):
    """The pool as [page][head][slot][dim], whatever its order in memory."""
    return pool if case["layout"] == "hnd" else pool.permute(0, 2, 1, 3)


def _scales(case, g):
    if case["kv"] != "e4m3":
        return None, None
    u = torch.rand(2, case["kv_heads"], generator=g, device=DEVICE) * 0.03 + 0.02
    return u[0].contiguous(), u[1].contiguous()


def _trees(case, seed):
    """The sequences' nodes one after another: where each sequence's begin, each node's sequence and index, its parent's
    index (-1: the root) and its depth. Nodes are in the order of their depth, as a drafter makes them."""
    count = _counts(case)
    cpu = torch.Generator().manual_seed(seed + 1)
    first, parents, depths = [0], [], []
    for n in count:
        u = torch.rand(max(n, 1), generator=cpu).tolist()
        if case.get("chain"):
            p = list(range(-1, n - 1))
        else:
            p = [-1] + sorted(int(u[i] * min(i, 1 + i * 0.7)) for i in range(1, n))
        d = []
        for i in range(n):
            d.append(0 if p[i] < 0 else d[p[i]] + 1)
        parents += p[:n]
        depths += d
        first.append(first[-1] + n)
    seq = [b for b, n in enumerate(count) for _ in range(n)]
    index = [i for n in count for i in range(n)]
    return [torch.tensor(x, dtype=torch.int32) for x in (first, seq, index, parents, depths)]


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed), seed)
    s["case"] = case
    if own:
        s["call"] = _PLAN[case["op"]](case, s)
    return s


def _prepare_append(case, g, seed):
    first, seq, index, _, depth = _trees(case, seed)
    n, b, ps = len(seq), case["seqs"], case["page"]
    cpu = torch.Generator().manual_seed(seed)
    past = (torch.rand(b, generator=cpu) * case["past"]).int()
    pos, place = past[seq.long()] + depth, past[seq.long()] + index
    width = int((case["past"] + case["nodes"]) // ps + 1)
    # pages that are written belong to one sequence alone; the earlier entries name pages shared by all
    key = torch.unique(seq.long() * width + place.long() // ps)
    pages = n // ps + 2 * b + 16
    page_of = torch.randperm(pages, generator=cpu)
    table = page_of[len(key) + torch.randint(0, 16, (b * width,), generator=cpu)]
    table[key] = page_of[: len(key)]
    act, rot, d = ACT[case["act"]], case["rotary"], case["dim"]
    ks, vs = _scales(case, g)
    weights = torch.rand(2, d, generator=g, device=DEVICE) + 0.5 if case["normed"] else [None, None]
    return dict(
        q=(_randn(g, n, case["q_heads"], d) * 2.0).to(act), k=(_randn(g, n, case["kv_heads"], d) * 2.0).to(act),
        v=_randn(g, n, case["kv_heads"], d).to(act), q_norm=weights[0], k_norm=weights[1], k_pool=_pool(case, pages, g),
        v_pool=_pool(case, pages, g), k_scale=ks, v_scale=vs, seq=seq.to(DEVICE), pos=pos.to(DEVICE), place=place.to(DEVICE),
        table=table.view(b, width).int().to(DEVICE),
        inv_freq=(ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEVICE))


def _prepare_tree(case, g, seed):
    first, _, _, parent, _ = _trees(case, seed)
    past, ps = torch.tensor(_past(case)), case["page"]
    used = (past + torch.tensor(_counts(case)) + ps - 1) // ps
    width, pages = max(1, int(used.max())), int(used.sum()) + 3
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.zeros(case["seqs"], width, dtype=torch.long)
    inside = torch.arange(width)[None, :] < used[:, None]
    table[inside] = perm[: int(used.sum())]
    ks, vs = _scales(case, g)
    rows = len(parent)
    return dict(
        q=(_randn(g, rows, case["q_heads"], case["dim"]) * 1.5).to(ACT[case["act"]]), k_pool=_pool(case, pages, g),
        v_pool=_pool(case, pages, g), k_scale=ks, v_scale=vs, first=first.to(DEVICE), past=past.int().to(DEVICE),
        parent=None if case["chain"] else parent.to(DEVICE), table=table.int().to(DEVICE), scale=1.0 / math.sqrt(case["dim"]))


def _prepare_verify(case, g, seed):
    first, seq, index, parent, _ = _trees(case, seed)
    rows, v = len(seq), case["vocab"]
    act = ACT[case["act"]]
    logits = _randn(g, rows, v).mul_(3.0)
    up = (first[seq.long()] + parent).clamp_(min=0).long().to(DEVICE)  # the row of a node's parent
    if case["greedy"]:
        # the draft's favourites, most of them the target's too; rounded logits have ties
        target = logits.to(act)
        likely = target.float().argmax(1)[up]
        other = torch.randint(0, v, (rows,), generator=g, device=DEVICE)
        keep = torch.rand(rows, generator=g, device=DEVICE) < 0.7
        return dict(target=target, draft=None, tokens=torch.where(keep, likely, other).int(), first=first.to(DEVICE),
                    parent=None if case["chain"] else parent.to(DEVICE), uniform=None)
    target = torch.softmax(logits, 1).to(act)
    logits += _randn(g, rows, v).mul_(0.7)
    draft = torch.softmax(logits, 1).to(act)
    del logits
    # each node's token is drawn from its parent's row of the draft
    running = draft.double().cumsum(1)
    at = torch.rand(rows, 1, generator=g, device=DEVICE, dtype=torch.float64) * running[up, -1:]
    tokens = torch.cat([torch.searchsorted(running[r:r + 1], a) for r, a in zip(up.tolist(), at.split(1))]).view(-1)
    return dict(target=target, draft=draft if case["draft"] else None, tokens=tokens.clamp_(max=v - 1).int(),
                first=first.to(DEVICE), parent=None if case["chain"] else parent.to(DEVICE),
                uniform=torch.rand(rows, generator=g, device=DEVICE))


def _prepare_compact(case, g, seed):
    b, ps, n = case["seqs"], case["page"], case["nodes"]
    cpu = torch.Generator().manual_seed(seed)
    count = _accepted(case)
    # an accepted node beside the root lies behind the places that the path goes to, so that a pass can be repeated
    path = torch.full((b, n), -1, dtype=torch.int32)
    for i, m in enumerate(count):
        path[i, :m] = torch.cat([torch.zeros(1), m + torch.randperm(n - m, generator=cpu)[: m - 1].sort().values]).int()
    past = (torch.rand(b, generator=cpu) * case["past"]).int()
    width = (case["past"] + n) // ps + 1
    pages = _compact_pages(case)
    perm = torch.randperm(pages, generator=cpu)
    table = torch.zeros(b, width, dtype=torch.long)
    per = (n + ps - 1) // ps + 1
    for i in range(b):
        at = int(past[i]) // ps
        mine = table[i, at:at + per]
        mine.copy_(perm[i * per:i * per + len(mine)])
    return dict(k_pools=[_pool(case, pages, g) for _ in range(case["layers"])],
                v_pools=[_pool(case, pages, g) for _ in range(case["layers"])], past=past.to(DEVICE), path=path.to(DEVICE),
                count=torch.tensor(count, dtype=torch.int32).to(DEVICE), table=table.int().to(DEVICE))


def _prepare_copy(case, g, seed):
    pages = 2 * case["pages"] + 2
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int().to(DEVICE)
    n = case["pages"]
    return dict(k_pools=[_pool(case, pages, g) for _ in range(case["layers"])],
                v_pools=[_pool(case, pages, g) for _ in range(case["layers"])], src=perm[:n].contiguous(),
                dst=perm[n:2 * n].contiguous())


_PREPARE = {"append": _prepare_append, "tree": _prepare_tree, "verify": _prepare_verify, "compact": _prepare_compact,
            "copy": _prepare_copy}


# ------------------------------------------------------------------------------------ the library's calls
def _cache(lib, case, k_pool, v_pool, k_scale=None, v_scale=None):
    ps, kh, d = case["page"], case["kv_heads"], case["dim"]
    token, head = (d, ps * d) if case["layout"] == "hnd" else (kh * d, d)
    fmt = {"bf16": lib.COLI_KV_BF16, "f16": lib.COLI_KV_F16, "e4m3": lib.COLI_KV_E4M3}[case["kv"]]
    return lib.make_kv_cache(k_pool, v_pool, fmt, k_pool.shape[0], ps, kh, d, page_stride=ps * kh * d, token_stride=token,
                             head_stride=head, k_scale=k_scale, v_scale=v_scale)


def _act(lib, case):
    return {"f32": lib.COLI_ACT_F32, "bf16": lib.COLI_ACT_BF16, "f16": lib.COLI_ACT_F16}[case["act"]]


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEVICE)


def _plan_append(case, s):
    import quantized_expert_decode_gb300 as lib
    desc = lib.make_norm_append_desc(len(s["seq"]), case["q_heads"], case["seqs"], s["table"].shape[1], _act(lib, case),
                                     case["rotary"], case["interleaved"], EPS)
    return dict(lib=lib, desc=desc, cache=_cache(lib, case, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]),
                q_out=torch.empty_like(s["q"]), err=_err())


def _plan_tree(case, s):
    import quantized_expert_decode_gb300 as lib
    desc = lib.make_tree_desc(case["seqs"], len(s["q"]), case["nodes"], case["q_heads"], s["table"].shape[1],
                              _act(lib, case), s["scale"], window=case["window"])
    cache = _cache(lib, case, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    n = lib.coli_tree_workspace_bytes(desc, cache)
    return dict(lib=lib, desc=desc, cache=cache, out=torch.empty_like(s["q"]),
                lse=torch.empty(s["q"].shape[:2], device=DEVICE), ws=torch.empty(n, dtype=torch.uint8, device=DEVICE),
                ws_bytes=n, err=_err())


def _plan_verify(case, s):
    import quantized_expert_decode_gb300 as lib
    desc = lib.make_verify_desc(case["seqs"], len(s["tokens"]), case["nodes"], case["vocab"], _act(lib, case),
                                lib.COLI_VERIFY_GREEDY if case["greedy"] else lib.COLI_VERIFY_SAMPLE)
    ints = dict(dtype=torch.int32, device=DEVICE)
    return dict(lib=lib, desc=desc, path=torch.empty(case["seqs"], case["nodes"], **ints),
                count=torch.empty(case["seqs"], **ints), token=torch.empty(case["seqs"], **ints), err=_err())


def _plan_pools(case, s):
    import quantized_expert_decode_gb300 as lib
    caches = lib.make_kv_caches([_cache(lib, case, k, v) for k, v in zip(s["k_pools"], s["v_pools"])])
    if case["op"] == "copy":
        return dict(lib=lib, caches=caches, err=_err())
    return dict(lib=lib, caches=caches, err=_err(),
                desc=lib.make_compact_desc(case["seqs"], case["nodes"], s["table"].shape[1], case["layers"]))


_PLAN = {"append": _plan_append, "tree": _plan_tree, "verify": _plan_verify, "compact": _plan_pools, "copy": _plan_pools}


def _own_append(s):
    c = s["call"]
    c["lib"].coli_norm_append(c["desc"], c["cache"], s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], s["inv_freq"],
                              s["seq"], s["pos"], s["place"], s["table"], c["q_out"], c["err"], torch.cuda.current_stream())
    return dict(q=c["q_out"], k=s["k_pool"], v=s["v_pool"])


def _own_tree(s):
    c = s["call"]
    c["lib"].coli_attn_tree(c["desc"], c["cache"], s["q"], s["first"], s["past"], s["parent"], s["table"], c["out"], c["lse"],
                            c["err"], c["ws"], c["ws_bytes"], torch.cuda.current_stream())
    return dict(out=c["out"], lse=c["lse"])


def _own_verify(s):
    c = s["call"]
    c["lib"].coli_draft_verify(c["desc"], s["target"], s["draft"], s["tokens"], s["parent"], s["uniform"], s["first"],
                               c["path"], c["count"], c["token"], c["err"], torch.cuda.current_stream())
    return dict(path=c["path"], count=c["count"], token=c["token"])


def _own_compact(s):
    c = s["call"]
    c["lib"].coli_kv_compact(c["desc"], c["caches"], s["past"], s["path"], s["count"], s["table"], c["err"],
                             torch.cuda.current_stream())
    return dict(k=s["k_pools"], v=s["v_pools"])


def _own_copy(s):
    c = s["call"]
    c["lib"].coli_kv_copy_pages(c["caches"], s["case"]["layers"], s["case"]["pages"], s["src"], s["dst"], c["err"],
                                torch.cuda.current_stream())
    return dict(k=s["k_pools"], v=s["v_pools"])


# ------------------------------------------------------------------------------------ the plain forms
def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _rotated(case, x, cos, sin):
    """x [token][head][dim] in 32 bits, its first `rotary` entries rotated."""
    rot = case["rotary"]
    if rot == 0:
        return x
    turn, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = turn[..., : rot // 2], turn[..., rot // 2:]
        turn = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turn, rest), dim=-1)


def _store(case, pool, page, slot, x, scale):
    """Writes x [token][head][dim] to the pool's pages, rounded to the cache's type."""
    view = _paged(case, pool)
    if case["kv"] == "e4m3":
        x = (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(KV["e4m3"]).view(torch.uint8)
        view = view.view(torch.uint8)
    else:
        x = x.to(view.dtype)
    view[page, :, slot] = x


def _plain_append(s):
    case = s["case"]
    # far positions lose their angle in 32 bits
    angle = (s["pos"].double()[:, None] * s["inv_freq"].double()[None, :])[:, None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    place = s["place"].long()
    page = s["table"][s["seq"].long(), place // case["page"]].long()
    slot = place % case["page"]
    _store(case, s["k_pool"], page, slot, _rotated(case, _normed(s["k"], s["k_norm"]), cos, sin), s["k_scale"])
    _store(case, s["v_pool"], page, slot, s["v"].float(), s["v_scale"])
    return dict(q=_rotated(case, _normed(s["q"], s["q_norm"]), cos, sin).to(s["q"].dtype), k=s["k_pool"], v=s["v_pool"])


def _dense(case, pool, table, scale):
    """The sequences' pages as [sequence][head][token][dim] in 32 bits."""
    view = _paged(case, pool)
    if case["kv"] == "e4m3":
        x = view.view(torch.uint8)[table].view(KV["e4m3"]).float()
    else:
        x = view[table].float()
    x = x.transpose(1, 2).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _related(case, s, index, seq):
    """[row][node] whether the node is the row's own or an ancestor's, and the rows' depths."""
    rows, n = len(index), case["nodes"]
    node = torch.arange(n, device=DEVICE)[None, :]
    if s["parent"] is None:
        return node <= index[:, None], index
    # the square of "is or is the parent of" until paths of all lengths are in it
    up = torch.zeros(case["seqs"], n, n, device=DEVICE)
    up[seq, index, index] = 1.0
    has = s["parent"] >= 0
    # (a root's own entry is written twice)
    up[seq, index, torch.where(has, s["parent"].long(), index)] = 1.0
    for _ in range(max(1, (n - 1).bit_length())):
        up = (up @ up).clamp(max=1.0)
    mine = up[seq, index]
    return mine > 0, mine.sum(1).long() - 1


def _plain_tree(s):
    case = s["case"]
    b, kh, d, n = case["seqs"], case["kv_heads"], case["dim"], case["nodes"]
    rows = len(s["q"])
    first, past = s["first"].long(), s["past"].long()
    seq = torch.searchsorted(first[1:], torch.arange(rows, device=DEVICE), right=True)
    index = torch.arange(rows, device=DEVICE) - first[seq]
    table = s["table"].long()
    k, v = _dense(case, s["k_pool"], table, s["k_scale"]), _dense(case, s["v_pool"], table, s["v_scale"])
    related, depth = _related(case, s, index, seq)
    # every sequence's rows beside each other, behind the last ones zeros
    q = torch.zeros(b, n, kh, case["q_heads"] // kh, d, device=DEVICE)
    q[seq, index] = s["q"].float().view(rows, kh, -1, d)
    t = torch.arange(k.shape[2], device=DEVICE)[None, :]
    own_past = past[seq][:, None]
    node = t - own_past
    inside = (node >= 0) & (node < n)
    seen = torch.where(inside, related.gather(1, node.clamp(0, n - 1)), t < own_past)
    if case["window"]:
        # a node's position is its depth behind the committed tokens
        node_depth = torch.zeros(b, n, dtype=torch.long, device=DEVICE)
        node_depth[seq, index] = depth
        position = torch.where(inside, own_past + node_depth[seq].gather(1, node.clamp(0, n - 1)), t)
        seen &= position > own_past + depth[:, None] - case["window"]
    mask = torch.zeros(b, n, k.shape[2], dtype=torch.bool, device=DEVICE)
    mask[seq, index] = seen
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [sequence][kv head][head of the group, node][dim]
    score = q @ k.transpose(2, 3) * s["scale"]
    score = score.view(b, kh, -1, n, k.shape[2]).masked_fill_(~mask[:, None, None], float("-inf")).flatten(2, 3)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = total.log() + top
    pick = lambda x: x.unflatten(2, (-1, n)).permute(0, 3, 1, 2, 4)[seq, index]  # noqa: E731
    return dict(out=pick(out).reshape(rows, -1, d).to(s["q"].dtype), lse=pick(lse).reshape(rows, -1))


def _plain_verify(s):
    case = s["case"]
    b, n, v = case["seqs"], case["nodes"], case["vocab"]
    ints = dict(dtype=torch.int32, device=DEVICE)
    first = s["first"].long()
    here, rows = first[:-1], first[1:] - first[:-1]
    live = rows > 0
    last = len(s["tokens"]) - 1
    at = torch.zeros(b, dtype=torch.long, device=DEVICE)  # the deepest accepted node
    path = torch.full((b, n), -1, **ints)
    path[:, 0] = torch.where(live, 0, -1)
    count = live.int()
    row = lambda i: (here + i).clamp(0, last)  # noqa: E731
    if case["greedy"]:
        best = s["target"].float().argmax(1)
    else:
        # the residual is max(target - away * draft, 0), of `mass` in all, or the target without rejected tokens;
        # sums and what is next to a border in 64 bits
        away, mass = torch.zeros(b, 1, device=DEVICE).double(), torch.ones(b, 1, device=DEVICE).double()
        gone = None if case["draft"] else torch.zeros(b, v, dtype=torch.bool, device=DEVICE)

    def residual():
        p = s["target"][row(at)].double()
        return p.masked_fill(gone, 0.0) if gone is not None else (p - away * s["draft"][row(at)].double()).clamp_(min=0.0)

    # nodes come behind their parents, so that one look at each in turn walks down the tree
    for i in range(1, n):
        r = row(i)
        parent = i - 1 if s["parent"] is None else s["parent"][r].long()
        child = live & (i < rows) & (parent == at)
        token = s["tokens"][r].long()
        if case["greedy"]:
            taken = child & (best[row(at)] == token)
        else:
            u = s["uniform"][r].double()[:, None]
            p = s["target"][row(at)].gather(1, token[:, None]).double()
            if case["draft"]:
                taken = child & ((away + u * mass) * s["draft"][row(at)].gather(1, token[:, None]).double() < p)[:, 0]
            else:
                taken = child & (u * mass < p.masked_fill(gone.gather(1, token[:, None]), 0.0))[:, 0]
            lost = child & ~taken
            if case["draft"]:
                away = torch.where(lost[:, None], away + mass, away)
            else:
                gone.scatter_(1, token[:, None], gone.gather(1, token[:, None]) | lost[:, None])
            mass = torch.where(lost[:, None], residual().sum(1, keepdim=True), mass)
            away, mass = away.masked_fill(taken[:, None], 0.0), mass.masked_fill(taken[:, None], 1.0)
            if gone is not None:
                gone &= ~taken[:, None]
        at = torch.where(taken, i, at)
        end = count.clamp(max=n - 1).long()[:, None]
        path.scatter_(1, end, torch.where(taken[:, None], i, path.gather(1, end)).int())
        count = count + taken.int()
    if case["greedy"]:
        token = best[row(at)]
    else:
        left = residual()
        left = torch.where(left.sum(1, keepdim=True) > 0, left, s["target"][row(at)].double())
        running = left.cumsum(1)
        over = running > s["uniform"][row(0)].double()[:, None] * running[:, -1:]
        token = over.int().argmax(1)
    return dict(path=path, count=count.int(), token=torch.where(live, token, -1).int())


def _plain_compact(s):
    case = s["case"]
    count, path = s["count"].long(), s["path"].long()
    i = torch.arange(path.shape[1], device=DEVICE)[None, :]
    # behind the end of its path a sequence's root is copied onto itself
    i = torch.where(i < count[:, None], i, 0).flatten()
    seq = torch.arange(len(count), device=DEVICE).repeat_interleave(path.shape[1])
    from_, to = s["past"].long()[seq] + path[seq, i], s["past"].long()[seq] + i
    table, ps = s["table"].long(), case["page"]
    fp, fs, tp, ts = table[seq, from_ // ps], from_ % ps, table[seq, to // ps], to % ps
    for pool in s["k_pools"] + s["v_pools"]:
        view = _paged(case, pool)
        if case["kv"] == "e4m3":
            view = view.view(torch.uint8)
        view[tp, :, ts] = view[fp, :, fs]
    return dict(k=s["k_pools"], v=s["v_pools"])


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for pool in s["k_pools"] + s["v_pools"]:
        view = pool.view(torch.uint8)
        view[dst] = view[src]
    return dict(k=s["k_pools"], v=s["v_pools"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "tree": _own_tree, "verify": _own_verify, "compact": _own_compact, "copy": _own_copy}[op](state)
    return {"append": _plain_append, "tree": _plain_tree, "verify": _plain_verify, "compact": _plain_compact,
            "copy": _plain_copy}[op](state)


# ------------------------------------------------------------------------------------ the definitions in 64 bits
def _exact_append(case, s):
    n, rot, ps = len(s["seq"]), case["rotary"], case["page"]
    place, seq = s["place"].long(), s["seq"].long()
    phase = torch.exp(1j * (s["pos"].double()[:, None, None] * s["inv_freq"].double()))

    def turn(x, w):
        x = x.double().clone()
        if w is not None:
            x = x * w.double() / (torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 / case["dim"] + EPS) ** 0.5
        if rot:
            if case["interleaved"]:
                pairs = x[..., :rot].unflatten(-1, (rot // 2, 2))
            else:
                pairs = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
            x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return x

    def put(pool, x, scale):
        p = pool.double()
        flat = p.view(-1, case["dim"])  # rows of one head and one token
        if scale is not None:
            x = torch.clamp(x / scale.double()[:, None], -E4M3_MAX, E4M3_MAX)
        h = torch.arange(case["kv_heads"], device=DEVICE)
        page, slot = s["table"].long().flatten()[seq * s["table"].shape[1] + place // ps], place % ps
        if case["layout"] == "hnd":
            row = (page[:, None] * case["kv_heads"] + h) * ps + slot[:, None]
        else:
            row = (page * ps + slot)[:, None] * case["kv_heads"] + h
        flat.index_copy_(0, row.flatten(), x.reshape(n * case["kv_heads"], case["dim"]))
        return p

    return dict(q=turn(s["q"], s["q_norm"]), k=put(s["k_pool"], turn(s["k"], s["k_norm"]), s["k_scale"]),
                v=put(s["v_pool"], s["v"].double(), s["v_scale"]))


def _lines(parent, n):
    """Each node's line of ancestors, itself last."""
    lines = []
    for i in range(n):
        up = i - 1 if parent is None else parent[i]
        lines.append((lines[up] if up >= 0 else []) + [i])
    return lines


def _exact_tree(case, s):
    qh, kh, d = case["q_heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(len(s["q"]), qh, d, dtype=torch.float64, device=DEVICE)
    lse = torch.full((len(s["q"]), qh), float("-inf"), dtype=torch.float64, device=DEVICE)
    first, parents = s["first"].tolist(), None if s["parent"] is None else s["parent"].tolist()
    for i, past in enumerate(s["past"].tolist()):
        r0, r1 = first[i], first[i + 1]
        if r0 == r1:
            continue
        lines = _lines(None if parents is None else parents[r0:r1], r1 - r0)
        start = max(0, past + 1 - case["window"]) if case["window"] else 0
        hide = torch.zeros(r1 - r0, past + r1 - r0 - start, dtype=torch.bool)
        hide[:, past - start:] = True
        for j, line in enumerate(lines):
            if case["window"]:
                hide[j, : max(0, past + len(line) - case["window"] - start)] = True
                line = line[-case["window"]:]
            hide[j, past - start + torch.tensor(line)] = False
        hide = hide.to(DEVICE)
        t = torch.arange(start, past + r1 - r0, device=DEVICE)
        page, slot = s["table"][i].long()[t // case["page"]], t % case["page"]
        for h in range(kh):
            def rows(pool, scale):
                raw = pool.view(torch.uint8) if case["kv"] == "e4m3" else pool
                x = raw[page, h, slot] if case["layout"] == "hnd" else raw[page, slot, h]
                x = x.view(pool.dtype).double()
                return x if scale is None else x * scale[h].double()
            mine = slice(h * (qh // kh), (h + 1) * (qh // kh))
            logit = torch.einsum("ngd,td->ngt", s["q"][r0:r1, mine].double(), rows(s["k_pool"], s["k_scale"])) * s["scale"]
            logit.masked_fill_(hide[:, None], float("-inf"))
            lse[r0:r1, mine] = torch.logsumexp(logit, 2)
            out[r0:r1, mine] = torch.einsum("ngt,td->ngd", torch.softmax(logit, 2), rows(s["v_pool"], s["v_scale"]))
    return dict(out=out, lse=lse)


def _exact_verify(case, s):
    first, tokens = s["first"].tolist(), s["tokens"].tolist()
    parents = None if s["parent"] is None else s["parent"].tolist()
    paths = torch.full((case["seqs"], case["nodes"]), -1, dtype=torch.int32)
    counts, drawn = [], []
    for b in range(case["seqs"]):
        r0, n = first[b], first[b + 1] - first[b]
        if n == 0:
            counts.append(0)
            drawn.append(-1)
            continue
        up = [-1] + [i - 1 if parents is None else parents[r0 + i] for i in range(1, n)]
        path, token = [0], None
        while token is None:
            here = path[-1]
            p = s["target"][r0 + here].double()
            children = [i for i in range(1, n) if up[i] == here]
            if case["greedy"]:
                best = int((p == p.max()).nonzero()[0])
                hits = [i for i in children if tokens[r0 + i] == best]
                if hits:
                    path.append(hits[0])
                else:
                    token = best
                continue
            # the residual as a distribution of its own, made smaller child by child
            rest, next_ = p.clone(), None
            norm = 1.0
            for i in children:
                x, u = tokens[r0 + i], float(s["uniform"][r0 + i])
                if case["draft"]:
                    q = s["draft"][r0 + here].double() * norm
                    if u * float(q[x]) < float(rest[x]):
                        next_ = i
                        break
                    rest = torch.relu(rest - q)
                else:
                    if u * norm < float(rest[x]):
                        next_ = i
                        break
                    rest[x] = 0.0
                norm = float(rest.sum())
            if next_ is not None:
                path.append(next_)
                continue
            if float(rest.sum()) == 0.0:
                rest = p
            line = torch.cumsum(rest, 0)
            token = int(torch.searchsorted(line, line[-1] * float(s["uniform"][r0]), right=True).clamp(max=case["vocab"] - 1))
        paths[b, : len(path)] = torch.tensor(path, dtype=torch.int32)
        counts.append(len(path))
        drawn.append(token)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEVICE)  # noqa: E731
    return dict(path=paths.to(DEVICE), count=ints(counts), token=ints(drawn))


def _exact_compact(case, s):
    table, past, path, count = (s[x].tolist() for x in ("table", "past", "path", "count"))
    ps = case["page"]

    def moved(pool):
        old, new = _paged(case, pool).double(), pool.double()
        view = _paged(case, new)
        for b in range(case["seqs"]):
            for i in range(1, count[b]):
                f, t = past[b] + path[b][i], past[b] + i
                view[table[b][t // ps], :, t % ps] = old[table[b][f // ps], :, f % ps]
        return new

    return dict(k=[moved(x) for x in s["k_pools"]], v=[moved(x) for x in s["v_pools"]])


def _exact_copy(case, s):
    def copied(pool):
        x = pool.double()
        return x.index_copy_(0, s["dst"].long(), pool.double().index_select(0, s["src"].long()))

    return dict(k=[copied(x) for x in s["k_pools"]], v=[copied(x) for x in s["v_pools"]])


def exact(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed), seed)
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify, "compact": _exact_compact,
            "copy": _exact_copy}[case["op"]](case, s)
