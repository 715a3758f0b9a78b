"""Workloads of the attention half of a decoder layer: the paged cache append, the single-token
attention over that cache and the norms around a block.

Each case names one operator and its sizes. `run` computes a case in its plain form (elementary
torch operations) or, with `own` true, through the library's entry points:

  append  keys and values of new tokens are rotated by position, converted to the cache's type and
          written to the sequences' pages; the queries are rotated by the same positions
  attend  one new token per sequence attends to its sequence's cached keys and values
  norms   r' = a * r + gate * norm(y), and the norm of r' that the next block reads
"""
import math

import torch

own = False

DEVICE = "cuda"
ACT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KV = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
POST_EPS, PRE_EPS = 1e-5, 1e-6
ROPE_BASE = 1e6


# ------------------------------------------------------------------------------------ the cases
def _append(name, seqs, tokens, past, heads, dim, rotary, interleaved, act, kv, page, layout):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, past=past, q_heads=heads[0], kv_heads=heads[1],
                dim=dim, rotary=rotary, interleaved=interleaved, act=act, kv=kv, page=page, layout=layout)


def _attend(name, seqs, longest, ragged, window, heads, dim, act, kv, page, layout):
    return dict(name=name, op="attend", seqs=seqs, longest=longest, ragged=ragged, window=window, q_heads=heads[0],
                kv_heads=heads[1], dim=dim, act=act, kv=kv, page=page, layout=layout)


def _norms(name, rows, width, act, post, pre, gate, scale):
    return dict(name=name, op="norms", rows=rows, width=width, act=act, post=post, pre=pre, gate=gate, resid_scale=scale)


def listed():
    return [
        # one sequence's next token at hidden size 2048, fp32 activations as the MoE block takes them: latency
        _append("append-one-token", 1, 1, 4096, (16, 2), 128, 128, False, "f32", "bf16", 16, "hnd"),
        # a continuous batch's decode step at hidden size 6144, far positions, an 8-bit cache, half of each head rotated
        _append("append-step-64", 64, 64, 200000, (48, 8), 128, 64, True, "bf16", "e4m3", 64, "hnd"),
        # a prefill batch of 2048 tokens from a few sequences, fp32 activations, pages of whole tokens
        _append("append-prompt-2048", 3, 2048, 5000, (48, 8), 128, 128, False, "f32", "f16", 16, "nhd"),
        # long prompts in one call, ragged
        _append("append-prompt-16411", 5, 16411, 9000, (64, 8), 128, 128, False, "bf16", "bf16", 64, "hnd"),
        # a chat's first answers: one short sequence, latency
        _attend("attend-one-short", 1, 333, False, 0, (16, 2), 128, "f32", "bf16", 16, "hnd"),
        # one long document: the only parallelism is along its length
        _attend("attend-one-long", 1, 131071, False, 0, (48, 8), 128, "bf16", "bf16", 64, "hnd"),
        # the batch of 32 independent sequences that the MoE block decodes, lengths all over the range, one slot idle
        _attend("attend-batch-32", 32, 8192, True, 0, (48, 8), 128, "f32", "bf16", 16, "hnd"),
        # a full server: many long sequences on an 8-bit cache
        _attend("attend-batch-64-e4m3", 64, 24576, False, 0, (64, 8), 128, "bf16", "e4m3", 64, "hnd"),
        # a layer with a sliding window and a key head for every query head, odd page size, pages of whole tokens
        _attend("attend-window", 16, 5000, True, 1024, (32, 32), 64, "f16", "f16", 24, "nhd"),
        # the norms between two blocks for one token: latency
        _norms("norms-one-token", 1, 6144, "f32", True, True, "none", 1.0),
        # the same for a batch of 32, its block gated element by element
        _norms("norms-batch-32", 32, 6144, "bf16", True, True, "element", 1.0),
        # a long prefill: bandwidth
        _norms("norms-prompt-4099", 4099, 6144, "f32", True, True, "channel", 0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    op = rng.choice(["append", "attend", "attend", "norms"])
    while True:
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
        group = rng.choice([1, 2, 4, 5, 6, 8, 12, 16])
        heads = (kv_heads * group, kv_heads)
        act, kv = rng.choice(sorted(ACT)), rng.choice(sorted(KV))
        page, layout = rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(["hnd", "nhd"])
        if op == "append":
            tokens = _log_int(rng, 1, 17000)
            seqs = tokens if tokens <= 64 and rng.random() < 0.6 else rng.randint(1, min(8, tokens))
            rotary = rng.choice([dim, dim, dim // 2, 0])
            c = _append("", seqs, tokens, _log_int(rng, 100, 300000), heads, dim, rotary, rng.random() < 0.4, act, kv,
                        page, layout)
        elif op == "attend":
            window = _log_int(rng, 64, 4096) if rng.random() < 0.25 else 0
            c = _attend("", _log_int(rng, 1, 64), _log_int(rng, 16, 131072), rng.random() < 0.6, window, heads, dim, act,
                        kv, page, layout)
        else:
            c = _norms("", _log_int(rng, 1, 8192), rng.choice([256, 1000, 2048, 4096, 5120, 6144, 8192, 12288]), act,
                       rng.random() < 0.7, rng.random() < 0.8, rng.choice(["none", "channel", "row", "element"]),
                       rng.choice([1.0, 0.5]))
        # the plain form of attend makes every sequence as long as the longest, in 32 bits
        dense = c["seqs"] * c["longest"] * kv_heads * dim if op == "attend" else 0
        if work(c)["bytes"] <= most[op] and heads[0] <= 128 and dense <= 64 * 24576 * 8 * 128:
            del c["name"]
            return c


def _lengths(case):
    """Cached tokens of each sequence, the new one included (the same for every seed)."""
    n, top = case["seqs"], case["longest"]
    if not case["ragged"]:
        return [top - i % 3 if top > 3 else top for i in range(n)]
    lens = [1 + int((top - 1) * math.modf(0.61803398875 * (i + 1))[0]) for i in range(n)]
    lens[n // 2] = top
    if n >= 8:
        lens[3] = 0  # an idle slot of the batch
    return lens


def _seen(case):
    w = case["window"]
    return [min(n, w) if w else n for n in _lengths(case)]


def _bytes(name):
    return {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}[name]


def work(case):
    if case["op"] == "append":
        n, qh, kh, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        a, c = _bytes(case["act"]), _bytes(case["kv"])
        return {"bytes": n * d * (2 * qh * a + 2 * kh * (a + c)) + 12 * n + 2 * case["rotary"],
                "flops": 3 * n * (qh + kh) * case["rotary"]}
    if case["op"] == "attend":
        t, qh, kh, d = sum(_seen(case)), case["q_heads"], case["kv_heads"], case["dim"]
        return {"bytes": t * kh * d * 2 * _bytes(case["kv"]) + case["seqs"] * qh * (2 * d * _bytes(case["act"]) + 4),
                "flops": 4 * t * qh * d}
    n, a = case["rows"] * case["width"], _bytes(case["act"])
    streams = 3 + (1 if case["pre"] else 0) + (1 if case["gate"] == "element" else 0)
    return {"bytes": n * a * streams + 8 * case["width"], "flops": 12 * n}


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


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed), seed)
    s["case"] = case
    if own:
        s["call"] = _PLAN[case["op"]](case, s)
    return s


def _prepare_append(case, g, seed):
    n, b, ps = case["tokens"], case["seqs"], case["page"]
    cpu = torch.Generator().manual_seed(seed)
    # new tokens per sequence (ragged), each sequence's past length, and so each token's position
    share = torch.rand(b, generator=cpu) + 0.25
    count = torch.ones(b, dtype=torch.long) + ((n - b) * share / share.sum()).floor().long()
    count[0] += n - int(count.sum())
    past = (torch.rand(b, generator=cpu) * case["past"]).long()
    seq = torch.repeat_interleave(torch.arange(b), count)
    first = torch.cumsum(count, 0) - count
    pos = past[seq] + torch.arange(n) - first[seq]
    width = int((case["past"] + n) // ps + 1)
    # pages that are written belong to one sequence alone; the earlier entries name pages shared by all
    key = torch.unique(seq * width + pos // ps)
    pages = n // ps + 2 * b + 16
    page_of = torch.randperm(pages, generator=cpu)
    table = page_of[len(key) + torch.randint(0, 16, (b * width,), generator=cpu)]
    table[key] = page_of[: len(key)]
    act = ACT[case["act"]]
    rot = case["rotary"]
    ks, vs = _scales(case, g)
    return dict(
        q=_randn(g, n, case["q_heads"], case["dim"]).to(act), k=_randn(g, n, case["kv_heads"], case["dim"]).to(act),
        v=_randn(g, n, case["kv_heads"], case["dim"]).to(act), k_pool=_pool(case, pages, g), v_pool=_pool(case, pages, g),
        k_scale=ks, v_scale=vs, seq=seq.int().to(DEVICE), pos=pos.int().to(DEVICE),
        table=table.view(b, width).int().to(DEVICE),
        inv_freq=(ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEVICE))


def _prepare_attend(case, g, seed):
    lens = torch.tensor(_lengths(case))
    ps = case["page"]
    used = (lens + ps - 1) // ps
    width = max(1, int(used.max()))
    pages = int(used.sum()) + 3
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.zeros(case["seqs"], width, dtype=torch.long)
    inside = torch.arange(width)[None, :] < used[:, None]
    table[inside] = perm[: int(used.sum())]
    ks, vs = _scales(case, g)
    return dict(
        q=(_randn(g, case["seqs"], case["q_heads"], case["dim"]) * 1.5).to(ACT[case["act"]]), k_pool=_pool(case, pages, g),
        v_pool=_pool(case, pages, g), k_scale=ks, v_scale=vs, lens=lens.int().to(DEVICE), table=table.int().to(DEVICE),
        scale=1.0 / math.sqrt(case["dim"]))


def _prepare_norms(case, g, seed):
    act = ACT[case["act"]]
    t, h = case["rows"], case["width"]
    gate = {"none": None, "channel": (h,), "row": (t,), "element": (t, h)}[case["gate"]]
    return dict(
        y=(_randn(g, t, h) * 0.3).to(act), resid=(_randn(g, t, h) * 3.0).to(act),
        post_w=torch.rand(h, generator=g, device=DEVICE) + 0.5 if case["post"] else None,
        pre_w=torch.rand(h, generator=g, device=DEVICE) + 0.5 if case["pre"] else None,
        gate=None if gate is None else torch.sigmoid(_randn(g, *gate)).to(act))


_PREPARE = {"append": _prepare_append, "attend": _prepare_attend, "norms": _prepare_norms}


# ------------------------------------------------------------------------------------ the library's calls
def _cache(lib, case, s):
    ps, kh, d = case["page"], case["kv_heads"], case["dim"]
    token, head = (d, ps * d) if case["layout"] == "hnd" else (kh * d, d)
    fmt = {"bf16": lib.COLI_KV_BF16, "f16": lib.COLI_KV_F16, "e4m3": lib.COLI_KV_E4M3}[case["kv"]]
    return lib.make_kv_cache(s["k_pool"], s["v_pool"], fmt, s["k_pool"].shape[0], ps, kh, d, page_stride=ps * kh * d,
                             token_stride=token, head_stride=head, k_scale=s["k_scale"], v_scale=s["v_scale"])


def _act(lib, case):
    return {"f32": lib.COLI_ACT_F32, "bf16": lib.COLI_ACT_BF16, "f16": lib.COLI_ACT_F16}[case["act"]]


def _plan_append(case, s):
    import quantized_expert_decode_gb300 as lib
    desc = lib.make_append_desc(case["tokens"], case["q_heads"], case["seqs"], s["table"].shape[1], _act(lib, case),
                                case["rotary"], case["interleaved"])
    return dict(lib=lib, desc=desc, cache=_cache(lib, case, s), q_out=torch.empty_like(s["q"]),
                err=torch.zeros(1, dtype=torch.int32, device=DEVICE))


def _plan_attend(case, s):
    import quantized_expert_decode_gb300 as lib
    desc = lib.make_attn_desc(case["seqs"], case["q_heads"], s["table"].shape[1], _act(lib, case), s["scale"],
                              window=case["window"])
    cache = _cache(lib, case, s)
    n = lib.coli_attn_workspace_bytes(desc, cache)
    return dict(lib=lib, desc=desc, cache=cache, out=torch.empty_like(s["q"]),
                lse=torch.empty(s["q"].shape[:2], device=DEVICE), ws=torch.empty(n, dtype=torch.uint8, device=DEVICE),
                ws_bytes=n, err=torch.zeros(1, dtype=torch.int32, device=DEVICE))


def _plan_norms(case, s):
    import quantized_expert_decode_gb300 as lib
    gate = {"none": lib.COLI_GATE_NONE, "channel": lib.COLI_GATE_CHANNEL, "row": lib.COLI_GATE_ROW,
            "element": lib.COLI_GATE_ELEMENT}[case["gate"]]
    desc = lib.make_norms_desc(case["rows"], case["width"], _act(lib, case), gate, POST_EPS, PRE_EPS, case["resid_scale"])
    return dict(lib=lib, desc=desc, resid=torch.empty_like(s["y"]), xn=torch.empty_like(s["y"]) if case["pre"] else None)


_PLAN = {"append": _plan_append, "attend": _plan_attend, "norms": _plan_norms}


def _own_append(s):
    c = s["call"]
    c["lib"].coli_kv_append(c["desc"], c["cache"], s["q"], s["k"], s["v"], s["inv_freq"], s["seq"], s["pos"], s["table"],
                            c["q_out"], c["err"], torch.cuda.current_stream())
    return dict(q=c["q_out"], k=s["k_pool"], v=s["v_pool"])


def _own_attend(s):
    c = s["call"]
    c["lib"].coli_attn_decode(c["desc"], c["cache"], s["q"], s["table"], s["lens"], c["out"], c["lse"], c["err"], c["ws"],
                              c["ws_bytes"], torch.cuda.current_stream())
    return dict(out=c["out"], lse=c["lse"])


def _own_norms(s):
    c = s["call"]
    c["lib"].coli_block_norms(c["desc"], s["y"], s["resid"], s["post_w"], s["gate"], s["pre_w"], c["resid"], c["xn"],
                              torch.cuda.current_stream())
    return dict(resid=c["resid"], xn=c["xn"])


# ------------------------------------------------------------------------------------ the plain forms
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
    pos = s["pos"].long()
    page = s["table"][s["seq"].long(), pos // case["page"]].long()
    slot = pos % case["page"]
    _store(case, s["k_pool"], page, slot, _rotated(case, s["k"].float(), cos, sin), s["k_scale"])
    _store(case, s["v_pool"], page, slot, s["v"].float(), s["v_scale"])
    return dict(q=_rotated(case, s["q"].float(), cos, sin).to(s["q"].dtype), k=s["k_pool"], v=s["v_pool"])


def _dense(case, pool, table, scale):
    """The sequences' pages as [sequence][head][token][dim] in 32 bits."""
    view = _paged(case, pool)
    if case["kv"] == "e4m3":
        x = view.view(torch.uint8)[table].view(KV["e4m3"]).float()
    else:
        x = view[table].float()
    x = x.transpose(1, 2).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attend(s):
    case = s["case"]
    b, kh, d = case["seqs"], case["kv_heads"], case["dim"]
    table = s["table"].long()
    k, v = _dense(case, s["k_pool"], table, s["k_scale"]), _dense(case, s["v_pool"], table, s["v_scale"])
    q = s["q"].float().view(b, kh, -1, d)
    t = torch.arange(k.shape[2], device=DEVICE)[None, :]
    lens = s["lens"].long()[:, None]
    seen = (t < lens) & (t >= lens - case["window"]) if case["window"] else t < lens
    score = (q @ k.transpose(2, 3) * s["scale"]).masked_fill(~seen[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = (total.log() + top).view(b, -1)
    return dict(out=out.view(b, -1, d).to(s["q"].dtype), lse=lse)


def _rms(x, w, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def _plain_norms(s):
    case = s["case"]
    z, r, gate = s["y"].float(), s["resid"].float(), s["gate"]
    if case["post"]:
        z = _rms(z, s["post_w"], POST_EPS)
    if gate is not None:
        z = z * (gate.float()[:, None] if case["gate"] == "row" else gate.float())
    r = case["resid_scale"] * r + z
    xn = _rms(r, s["pre_w"], PRE_EPS).to(s["y"].dtype) if case["pre"] else None
    return dict(resid=r.to(s["y"].dtype), xn=xn)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "norms": _own_norms}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "norms": _plain_norms}[op](state)


# ------------------------------------------------------------------------------------ the definitions in 64 bits
def _exact_append(case, s):
    n, rot, ps = case["tokens"], case["rotary"], case["page"]
    pos, seq = s["pos"].long(), s["seq"].long()
    phase = torch.exp(1j * (pos.double()[:, None, None] * s["inv_freq"].double()))

    def rotate(x):
        x = x.double().clone()
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
        page, slot = s["table"].long().flatten()[seq * s["table"].shape[1] + pos // ps], pos % ps
        if case["layout"] == "hnd":
            row = (page[:, None] * case["kv_heads"] + h) * ps + slot[:, None]
        else:
            row = (page * ps + slot)[:, None] * case["kv_heads"] + h
        flat.index_copy_(0, row.flatten(), x.reshape(n * case["kv_heads"], case["dim"]))
        return p

    return dict(q=rotate(s["q"]), k=put(s["k_pool"], rotate(s["k"]), s["k_scale"]),
                v=put(s["v_pool"], s["v"].double(), s["v_scale"]))


def _exact_attend(case, s):
    b, qh, kh, d = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(b, qh, d, dtype=torch.float64, device=DEVICE)
    lse = torch.full((b, qh), float("-inf"), dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(s["lens"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        t = torch.arange(first, n, device=DEVICE)
        if n == 0:
            continue
        page, slot = s["table"][i].long()[t // case["page"]], t % case["page"]
        for h in range(kh):
            def rows(pool, scale):
                raw = pool.view(torch.uint8) if case["kv"] == "e4m3" else pool
                x = raw[page, h, slot] if case["layout"] == "hnd" else raw[page, slot, h]
                x = x.view(pool.dtype).double()
                return x if scale is None else x * scale[h].double()
            mine = slice(h * (qh // kh), (h + 1) * (qh // kh))
            logit = torch.einsum("gd,td->gt", s["q"][i, mine].double(), rows(s["k_pool"], s["k_scale"])) * s["scale"]
            lse[i, mine] = torch.logsumexp(logit, 1)
            out[i, mine] = torch.einsum("gt,td->gd", torch.softmax(logit, 1), rows(s["v_pool"], s["v_scale"]))
    return dict(out=out, lse=lse)


def _exact_norms(case, s):
    y, r = s["y"].double(), s["resid"].double()
    if case["post"]:
        y = s["post_w"].double() * y / (torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / case["width"] + POST_EPS) ** 0.5
    if case["gate"] == "row":
        y = (y.T * s["gate"].double()).T
    elif case["gate"] != "none":
        y = y * s["gate"].double()
    r = y + r * case["resid_scale"]
    if not case["pre"]:
        return dict(resid=r, xn=None)
    return dict(resid=r, xn=s["pre_w"].double() * r
                / (torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / case["width"] + PRE_EPS) ** 0.5)


def exact(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed), seed)
    return {"append": _exact_append, "attend": _exact_attend, "norms": _exact_norms}[case["op"]](case, s)
