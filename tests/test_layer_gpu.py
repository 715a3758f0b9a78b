"""The layer operators (include/colilayer.h) against their definitions in 64 bits, on a GPU.

Tolerances. u = 2^-24 is the relative error of one fp32 rounding; an output rounded to type t adds
finfo(t).eps / 2 of its value (and, below its normal range, half its smallest step).

  append   the turn is a fraction in (-1/2, 1/2] rounded to a float (at most 2^-26), its cosine and
           sine are off by a few 2^-25 more: 2 pi 2^-24 of |a| + |b| covers both. A rotation is two
           products and a sum: 3 u of |a| + |b|. Values are copied: equal bits.
  attend   a score is q . k in fp32 partial sums of 16 products: at most dim / 16 + 4 roundings of
           A = scale * sum |q_i k_i|, the 22 bits kept of q another 2^-22 A, and the step to base 2
           4 u |s|. p is off by that relatively, numerator and denominator both; the sums over the
           tokens go through at most 32 + tokens / 64 roundings; p in parts keeps 16 bits (16-bit
           activations on a bf16 cache) or 22 bits (all others).
  norms    a row's sum of squares goes through at most 64 + 32 roundings of positive terms, half of
           which reach the factor; each element a few more: 64 u of the terms' magnitudes.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACT = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16), "f16": (2, torch.float16)}
KV = {"bf16": (1, torch.bfloat16), "f16": (2, torch.float16), "e4m3": (3, torch.float8_e4m3fn)}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10}


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import quantized_expert_decode_gb300 as q
    return q


def half_ulp(x, dtype):
    return x.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def close(got, want, bound):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    err = (got - want).abs().nan_to_num(0.0)
    bad = err > bound
    assert not bool(bad.any()), f"{int(bad.sum())} values off, worst {float((err / bound).max()):.3g} times the bound"


class Cache:
    """Paged pools of random contents; every value outside what a test writes or names is NaN."""

    def __init__(self, q, rng, fmt, pages, page_size, heads, dim, layout="hnd", scales=True):
        self.fmt, self.dtype = KV[fmt]
        self.ps, self.heads, self.dim, self.pages = page_size, heads, dim, pages
        shape = {"hnd": (pages, heads, page_size), "nhd": (pages, page_size, heads), "hpn": (heads, pages, page_size)}[layout]
        order = {"hnd": (0, 1, 2, 3), "nhd": (0, 2, 1, 3), "hpn": (1, 0, 2, 3)}[layout]
        nan = 0x7f if fmt == "e4m3" else 0x7fff
        raw = torch.uint8 if fmt == "e4m3" else torch.int16
        self.raw = [torch.full((*shape, dim), nan, dtype=raw, device="cuda") for _ in range(2)]
        self.k, self.v = (r.permute(*order) for r in self.raw)  # [page][head][slot][dim], as raw bits
        st = self.k.stride()
        self.scale = None
        if fmt == "e4m3" and scales:
            self.scale = torch.from_numpy(rng.uniform(0.02, 0.05, (2, heads)).astype(np.float32)).cuda()
        self.desc = q.make_kv_cache(self.raw[0], self.raw[1], self.fmt, pages, page_size, heads, dim, st[0], st[2], st[1],
                                    None if self.scale is None else self.scale[0],
                                    None if self.scale is None else self.scale[1])

    def factor(self, i):
        return torch.ones(self.heads, dtype=torch.float64, device="cuda") if self.scale is None else self.scale[i].double()

    def bits(self, x):
        """x rounded to the cache's type, as raw bits."""
        if self.dtype == torch.float8_e4m3fn:
            return x.clamp(-448, 448).to(self.dtype).view(torch.uint8)
        return x.to(self.dtype).view(torch.int16)

    def put(self, which, page, slot, x):
        (self.k, self.v)[which][page, :, slot] = self.bits(x)

    def rows(self, which, page, slot):
        """[token][head][dim] in 64 bits, unscaled."""
        x = (self.k, self.v)[which][page, :, slot].contiguous().view(self.dtype)
        return x.float().double()


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------ append
def rotate64(x, pos, inv_freq, rot, interleaved):
    """x [token][head][dim] rotated in 64 bits, and |a| + |b| of each element's pair."""
    x = x.double()
    out, mag = x.clone(), torch.zeros_like(x)
    if rot:
        t = (pos.double()[:, None] * inv_freq.double()[None, :])[:, None, :]
        ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        a, b = x[..., ia], x[..., ib]
        out[..., ia], out[..., ib] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return out, mag


def check_append(q, rng, act="f32", kv="bf16", heads=(8, 2), dim=64, rot=64, interleaved=False, page=16, layout="hnd",
                 seq=(0, 0, 1, 2), pos=(5, 6, 31, 0), pad=0, offset=0, base=1e4, scales=True):
    code, dtype = ACT[act]
    n, (qh, kh) = len(seq), heads
    seqs, width = max(max(seq) + 1, 1), max(pos) // page + 1
    c = Cache(q, rng, kv, seqs * min(width, 4) + 3, page, kh, dim, layout, scales)
    table = torch.from_numpy(rng.integers(0, c.pages, (seqs, width)).astype(np.int32))
    free = list(rng.permutation(c.pages))
    page_of = {}
    for b, p in zip(seq, pos):
        if b >= 0 and (b, p // page) not in page_of:
            page_of[b, p // page] = int(free.pop())
            table[b, p // page] = page_of[b, p // page]
    table = table.cuda()
    # one fused buffer [token][q heads, k heads, v heads], its rows padded and shifted
    row = (qh + 2 * kh) * dim + pad
    buf = (randn(rng, n * row + offset) * 3).to(dtype)
    x = buf[offset:].view(n, row)
    parts = [x[:, :qh * dim], x[:, qh * dim:(qh + kh) * dim], x[:, (qh + kh) * dim:(qh + 2 * kh) * dim]]
    xq, xk, xv = (p.unflatten(1, (-1, dim)) if p.shape[1] else p.reshape(n, 0, dim) for p in parts)
    inv = torch.from_numpy((base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)).cuda()
    tpos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    tseq = torch.tensor(seq, dtype=torch.int32, device="cuda")
    qo = torch.full((n, qh, dim), float("nan"), dtype=dtype, device="cuda")
    err = err_word()
    before = [c.k.clone(), c.v.clone()]
    d = q.make_append_desc(n, qh, seqs, width, code, rot, interleaved, row, row, row)
    q.coli_kv_append(d, c.desc, parts[0] if qh else None, parts[1], parts[2], inv if rot else None, tseq, tpos, table,
                     qo if qh else None, err)
    assert q.coli_moe_check(err) == q.COLI_MOE_OK
    angle = 2 * math.pi * 2.0 ** -24
    if qh:
        want, mag = rotate64(xq, tpos, inv, rot, interleaved)
        close(qo, want, half_ulp(want, dtype) + (angle + 3 * U) * mag)
    keep = [i for i in range(n) if seq[i] >= 0]
    pg = torch.tensor([page_of[seq[i], pos[i] // page] for i in keep], dtype=torch.long, device="cuda")
    sl = torch.tensor([pos[i] % page for i in keep], dtype=torch.long, device="cuda")
    want, mag = rotate64(xk, tpos, inv, rot, interleaved)
    f = c.factor(0)[None, :, None]
    want, mag = want[keep] / f, mag[keep] / f
    got = c.rows(0, pg, sl)
    lim = 448.0 if kv == "e4m3" else math.inf
    close(got, want.clamp(-lim, lim), half_ulp(want, c.dtype) + (angle + 4 * U) * mag * (1 + torch.finfo(c.dtype).eps))
    # values are only converted: the same bits as one rounding
    fv = c.factor(1).float()[None, :, None]
    assert torch.equal(c.v[pg, :, sl], c.bits(xv.float()[keep] / fv))
    # and nothing else has changed
    for now, was in zip((c.k, c.v), before):
        was[pg, :, sl] = now[pg, :, sl]
        assert torch.equal(now, was)


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("kv", sorted(KV))
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_types(q, act, kv, interleaved):
    check_append(q, np.random.default_rng(1), act, kv, interleaved=interleaved)


@pytest.mark.parametrize("dim,rot", [(16, 16), (80, 80), (80, 40), (96, 48), (128, 64), (256, 256), (128, 0), (128, 2), (128, 126),
                                     (64, 34)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_append_head_sizes(q, dim, rot, interleaved, act):
    check_append(q, np.random.default_rng(2), act, "bf16", (6, 3), dim, rot, interleaved)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "hpn"])
@pytest.mark.parametrize("page", [1, 3, 16, 24])
def test_append_pages(q, layout, page):
    check_append(q, np.random.default_rng(3), "bf16", "e4m3", (4, 4), 64, 32, page=page, layout=layout,
                 seq=(0, 0, 0, 1, 1, 2), pos=(7, 8, 9, 0, 1, 23))


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (4, 4), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("act", ["f32", "f16"])
def test_append_strides_and_alignment(q, pad, offset, act):
    check_append(q, np.random.default_rng(4), act, "f16", pad=pad, offset=offset)


def test_append_far_positions(q):
    # fp32 angles would be off by whole turns here
    far = (2 ** 31 // 1024 - 1) * 512
    check_append(q, np.random.default_rng(5), pos=(far, 999999, 65535, 65536), seq=(0, 1, 2, 3), page=1024)


def test_append_without_queries_and_scales(q):
    check_append(q, np.random.default_rng(6), "bf16", "e4m3", (0, 3), scales=False)


def test_append_many_tokens(q):
    for n in (63, 700, 5003):
        rng = np.random.default_rng(n)
        seq = np.sort(rng.integers(0, 3, n))
        pos = [int(i - np.searchsorted(seq, b)) for i, b in enumerate(seq)]
        check_append(q, rng, "bf16", "bf16", (5, 1), 64, 64, page=2048, seq=tuple(int(b) for b in seq), pos=tuple(pos))


def test_append_padding_tokens(q):
    check_append(q, np.random.default_rng(7), seq=(0, -1, 1, -1, -1), pos=(3, 0, 4, 0, 9))


def test_append_saturates_and_keeps_nan(q):
    rng = np.random.default_rng(8)
    c = Cache(q, rng, "e4m3", 2, 4, 1, 16, scales=False)
    x = torch.tensor([500.0, -1e9, float("inf"), -float("inf"), float("nan"), 448.0, 464.0, 0.0, -0.0, 2.0 ** -9, 2.0 ** -10,
                      2.0 ** -11, 17.0, 1.0625, 1.1875, -3.3], device="cuda").view(1, 1, 16)
    err = err_word()
    q.coli_kv_append(q.make_append_desc(1, 0, 1, 1, 0, 0), c.desc, None, x, x, None, None,
                     torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, dtype=torch.int32, device="cuda"), None, err)
    q.coli_moe_check(err)
    want = x.flatten().clamp(-448, 448).to(torch.float8_e4m3fn).float()
    for pool in (c.k, c.v):
        got = pool[1, 0, 0].contiguous().view(torch.float8_e4m3fn).float()
        assert torch.equal(got.nan_to_num(777.0), want.nan_to_num(777.0))


@pytest.mark.parametrize("scale", [1.0, 3.0, 0.75, 0.1, 7.0, 1.1, 2.0 ** -100, 2.0 ** -127, 3.0 * 2.0 ** -130, 2.0 ** -149, 2.0 ** 127, 3e38])
@pytest.mark.parametrize("rot", [0, 2])
def test_append_divides_by_the_scale(q, scale, rot):
    # values on and next to the borders between e4m3 values: the quotient's own side, as an IEEE division has it
    steps = torch.arange(0x7e, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    border = (steps[1:] + steps[:-1]) / 2
    s32 = torch.tensor(scale, dtype=torch.float32)
    x = torch.cat([steps, border]) * s32.double()
    x = torch.cat([x, x * (1 + 2.0 ** -23), x * (1 - 2.0 ** -23), -x, torch.tensor([math.inf, -math.inf, math.nan, 500 * scale])])
    x = x.float()
    n = -(-len(x) // 64)
    x = torch.cat([x, x.new_zeros(n * 64 - len(x))]).view(n, 1, 64)
    x[..., :2] = x[..., :2].nan_to_num(0.0, 0.0, 0.0)  # (turned by 0, an infinity would be NaN)
    x = x.cuda()
    c = Cache(q, np.random.default_rng(50), "e4m3", n, 1, 1, 64)
    c.scale.fill_(float(s32))
    err = err_word()
    # the odd rotary size takes the elements one by one; at position 0 it turns nothing
    q.coli_kv_append(q.make_append_desc(n, 0, n, 1, 0, rot), c.desc, None, x, x, torch.ones(1, device="cuda") if rot else None, None,
                     torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1),
                     None, err)
    assert q.coli_moe_check(err) == q.COLI_MOE_OK
    want = torch.from_numpy((x.cpu().numpy() / s32.numpy()).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
    want = want.float().nan_to_num(777.0)
    for pool in (c.k, c.v):
        got = pool[:, :, 0].contiguous().view(torch.float8_e4m3fn).float().cpu()
        assert torch.equal(got.nan_to_num(777.0), want)


def test_append_in_place_and_default_sequences(q):
    rng = np.random.default_rng(9)
    c = Cache(q, rng, "bf16", 4, 4, 2, 64)
    x, k = randn(rng, 3, 4, 64), randn(rng, 3, 2, 64)
    pos = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    inv = torch.rand(32, device="cuda")
    table = torch.tensor([[0], [2], [3]], dtype=torch.int32, device="cuda")
    want, mag = rotate64(x, pos, inv, 64, False)
    q.coli_kv_append(q.make_append_desc(3, 4, 3, 1, 0, 64), c.desc, x, k, k, inv, None, pos, table, x)
    close(x, want, half_ulp(want, torch.float32) + (2 * math.pi + 3) * U * mag)
    got = c.rows(1, table[:, 0].long(), pos.long())
    assert torch.equal(got, k.bfloat16().double())


def test_append_bad_places_are_skipped_and_flagged(q):
    rng = np.random.default_rng(10)
    for seq, pos, page in (((0, 9), (0, 1), 1), ((0, -2), (0, 1), 1), ((0, 1), (0, 8), 1), ((0, 1), (0, -1), 1),
                           ((0, 1), (0, 1), 4), ((0, 1), (0, 1), -1)):
        c = Cache(q, rng, "f16", 4, 4, 1, 64)
        x = randn(rng, 2, 1, 64)
        table = torch.tensor([[2, 3], [page, page]], dtype=torch.int32, device="cuda")
        err = err_word()
        qo = torch.zeros_like(x)
        q.coli_kv_append(q.make_append_desc(2, 1, 2, 2), c.desc, x, x, x, None,
                         torch.tensor(seq, dtype=torch.int32, device="cuda"),
                         torch.tensor(pos, dtype=torch.int32, device="cuda"), table, qo, err)
        assert q.coli_moe_check(err, raise_on_error=False) == q.COLI_MOE_EKERNEL
        assert q.coli_moe_check(err) == q.COLI_MOE_OK  # cleared
        assert torch.equal(qo, x)
        assert torch.equal(c.rows(0, 2, 0), x[0].half().double())
        assert int((c.k != 0x7fff).sum()) <= 64 and int((c.v != 0x7fff).sum()) <= 64


# ------------------------------------------------------------------------------------ attention
def fill(rng, c, lens, width=None):
    """A page table for the sequences and random contents for the tokens they hold."""
    used = [(n + c.ps - 1) // c.ps for n in lens]
    width = width or max(1, max(used))
    perm = rng.permutation(c.pages)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)  # entries behind the end are not read
    at = 0
    for b, (n, u) in enumerate(zip(lens, used)):
        table[b, :u] = torch.from_numpy(perm[at:at + u].astype(np.int32))
        at += u
        t = torch.arange(n)
        page, slot = table[b, t // c.ps].long().cuda(), (t % c.ps).cuda()
        for which in (0, 1):
            x = randn(rng, n, c.heads, c.dim)
            c.put(which, page, slot, x * (16 if c.dtype == torch.float8_e4m3fn else 1))
    return table.cuda()


def attend64(c, xq, table, lens, scale, window=0, skip=()):
    """out, lse, sum p |v| and A = max scale * sum |q k| of each row, in 64 bits."""
    b, qh, d = xq.shape
    g = qh // c.heads
    out = torch.zeros(b, qh, d, dtype=torch.float64, device="cuda")
    mass, lse = torch.zeros_like(out), torch.full((b, qh), -math.inf, dtype=torch.float64, device="cuda")
    amp = torch.zeros(b, qh, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        ts = [t for t in range(max(0, n - window) if window else 0, n) if (i, t // c.ps) not in skip]
        if not ts:
            continue
        t = torch.tensor(ts, device="cuda")
        page, slot = table[i].long()[t // c.ps], t % c.ps
        k = c.rows(0, page, slot) * c.factor(0)[None, :, None]
        v = c.rows(1, page, slot) * c.factor(1)[None, :, None]
        x = xq[i].double().view(c.heads, g, d)
        s = torch.einsum("hgd,thd->hgt", x, k) * scale
        p = torch.softmax(s, -1)
        out[i] = torch.einsum("hgt,thd->hgd", p, v).reshape(qh, d)
        mass[i] = torch.einsum("hgt,thd->hgd", p, v.abs()).reshape(qh, d)
        lse[i] = torch.logsumexp(s, -1).flatten()
        amp[i] = (torch.einsum("hgd,thd->hgt", x.abs(), k.abs()) * abs(scale)).amax(-1).flatten()
    return out, lse, mass, amp


def run_attend(q, c, xq, table, lens, scale, window=0, act="f32", err=None, stream=None, q_stride=0, out=None, out_stride=0):
    d = q.make_attn_desc(len(lens), xq.shape[1], table.shape[1], ACT[act][0], scale, window, q_stride, out_stride)
    n = q.coli_attn_workspace_bytes(d, c.desc)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    out = torch.full(xq.shape, float("nan"), dtype=ACT[act][1], device="cuda") if out is None else out
    lse = torch.full(xq.shape[:2], float("nan"), device="cuda")
    tl = lens if torch.is_tensor(lens) else torch.tensor(lens, dtype=torch.int32, device="cuda")
    q.coli_attn_decode(d, c.desc, xq, table, tl, out, lse, err, ws, n, stream)
    return out, lse


def check_attend(q, seed, lens, heads=(8, 2), dim=64, act="f32", kv="bf16", page=16, layout="hnd", window=0, boost=1.5,
                 scales=True):
    rng = np.random.default_rng(seed)
    qh, kh = heads
    c = Cache(q, rng, kv, sum((n + page - 1) // page for n in lens) + 2, page, kh, dim, layout, scales)
    table = fill(rng, c, lens)
    xq = (randn(rng, len(lens), qh, dim) * boost).to(ACT[act][1])
    scale = dim ** -0.5 * (1.0 if scales or kv != "e4m3" else 0.05)
    err = err_word()
    out, lse = run_attend(q, c, xq, table, lens, scale, window, act, err)
    assert q.coli_moe_check(err) == q.COLI_MOE_OK
    compare_attend(c, out, lse, attend64(c, xq, table, lens, scale, window), lens, act, kv)
    return c, xq, table, scale, out, lse


def compare_attend(c, out, lse, ref, lens, act, kv):
    want, wlse, mass, amp = ref
    n = max(max(lens), 1)
    ds = amp * ((c.dim / 16 + 4) * 2 * U + 2.0 ** -22 + 8 * U)
    sums = (32 + n / 64) * U
    parts = 2.0 ** -16 if (act != "f32" and kv == "bf16") else 2.0 ** -22
    empty = torch.isinf(wlse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    close(lse.masked_fill(empty, 0.0), wlse.masked_fill(empty, 0.0),
          ds + sums + 4 * U * (1 + wlse.masked_fill(empty, 0.0).abs()))
    close(out, want, half_ulp(want, ACT[act][1]) + (2 * ds + 2 * sums + parts)[..., None] * mass * 1.01
          if torch.is_tensor(ds) else 0)


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("kv", sorted(KV))
def test_attention_types(q, act, kv):
    check_attend(q, 11, [1, 77, 300, 0, 16, 17], act=act, kv=kv)


@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (8, 8), (16, 1), (12, 4), (24, 1), (10, 2), (40, 1), (17, 1), (64, 2), (128, 1)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_heads(q, heads, kv):
    check_attend(q, 12, [130, 5], heads, kv=kv, act="bf16")


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("kv", sorted(KV))
def test_attention_head_sizes(q, dim, kv):
    check_attend(q, 13, [150, 33, 2], (6, 2), dim, kv=kv)


@pytest.mark.parametrize("dim", [8, 24, 72, 120, 248])
def test_attention_odd_head_sizes(q, dim):
    check_attend(q, 14, [150, 33], (6, 2), dim, act="f16", kv="f16")
    check_attend(q, 14, [150, 33], (20, 1), dim, act="f32", kv="bf16")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1000, 4097])
def test_attention_lengths(q, n):
    check_attend(q, 15, [n], (4, 1), 128, page=16)
    check_attend(q, 15, [n, 0, n], (4, 2), 64, act="bf16", kv="e4m3", page=24)


@pytest.mark.parametrize("page", [1, 2, 3, 5, 8, 24, 48, 100, 128, 333])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "hpn"])
def test_attention_pages(q, page, layout):
    check_attend(q, 16, [334, 1, 97], (6, 3), 64, kv="f16", page=page, layout=layout)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 64, 100, 129, 500, 10 ** 6])
def test_attention_windows(q, window):
    check_attend(q, 17, [0, 1, 99, 100, 101, 500, 1300], (8, 2), 64, window=window, page=24)


def test_attention_windows_beyond_the_table(q):
    lens = [(i * 37) % 513 for i in range(63)] + [512]
    for window in (513, 2 ** 30, 2 ** 31 - 1):
        check_attend(q, 49, lens, (16, 8), 64, window=window)


def test_attention_long(q):
    check_attend(q, 18, [40000], (8, 1), 128, act="f32", kv="bf16", page=64)
    check_attend(q, 18, [70001], (5, 1), 64, act="bf16", kv="e4m3", page=32)
    check_attend(q, 18, [20011, 3, 0, 9000], (16, 2), 128, act="f16", kv="f16", page=16)


def test_attention_many_sequences(q):
    rng = np.random.default_rng(19)
    check_attend(q, 19, [int(x) for x in rng.integers(0, 60, 700)], (4, 2), 32, page=8)
    check_attend(q, 19, [int(x) for x in rng.integers(0, 400, 90)], (8, 8), 64, page=16, act="bf16")
    check_attend(q, 19, [0] * 40, (8, 8), 64)
    check_attend(q, 19, [0] * 30 + [3000] + [0] * 5, (8, 8), 64)


@pytest.mark.parametrize("seqs,ragged,kv", [(64, False, "bf16"), (64, True, "bf16"), (40, False, "f16"), (40, True, "e4m3"), (30, False, "bf16"),
                                            (160, True, "f16"), (320, True, "bf16")])
def test_attention_long_items_beyond_one_wave(q, seqs, ragged, kv):
    # 8 kv heads: more items than the GPU holds CTAs at once, or about as many, long ones: whole, cut evenly or
    # in runs that go on from item to item, as their lengths say
    rng = np.random.default_rng(seqs)
    top = 9000 if seqs <= 64 else 2500
    lens = [int(x) for x in rng.integers(0, top, seqs)] if ragged else [top - 300 + i % 5 for i in range(seqs)]
    check_attend(q, seqs, lens, (8, 8), 16, kv=kv, page=64)


@pytest.mark.parametrize("heads", [(16, 1), (9, 1), (24, 2), (50, 2)])
@pytest.mark.parametrize("act,kv", [("bf16", "bf16"), ("f32", "f16"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_attention_of_wide_groups_around_their_units(q, heads, act, kv):
    # 9 to 16 query heads of 81 to 128 elements: units of 128, 192, 256 or 384 tokens
    lens = [1, 191, 192, 193, 255, 257, 383, 384, 385, 0, 576, 769, 2305]
    check_attend(q, 41, lens, heads, 128, act=act, kv=kv, page=16)
    check_attend(q, 42, lens, heads, 96, act=act, kv=kv, page=7)
    check_attend(q, 43, lens + [12001], heads, 80, act=act, kv=kv, page=48, window=385)
    check_attend(q, 44, [i * 97 % 411 for i in range(500)], heads, 128, act=act, kv=kv, page=16)


def test_attention_short_sequences_in_wide_tables(q):
    # the table could name far longer sequences: what is decided by its width must not be wrong for short ones
    for seqs, width in ((3, 4000), (64, 200), (50, 1000)):
        rng = np.random.default_rng(seqs)
        c = Cache(q, rng, "bf16", seqs * 4 + 2, 16, 8, 64)
        lens = [int(x) for x in rng.integers(0, 60, seqs)]
        table = fill(rng, c, lens, width)
        xq = randn(rng, seqs, 16, 64)
        err = err_word()
        out, lse = run_attend(q, c, xq, table, lens, 0.125, err=err)
        assert q.coli_moe_check(err) == q.COLI_MOE_OK
        compare_attend(c, out, lse, attend64(c, xq, table, lens, 0.125), lens, "f32", "bf16")


def test_attention_most_sequences(q):
    check_attend(q, 20, [i % 3 for i in range(2048)], (2, 1), 16, page=2)


def test_attention_peaked_and_flat_scores(q):
    # one token takes all, scores of hundreds; and scores that are all but equal
    check_attend(q, 21, [300, 1000], (8, 2), 64, boost=60.0)
    check_attend(q, 21, [300, 1000], (8, 2), 64, boost=60.0, act="bf16", kv="f16")
    check_attend(q, 22, [300, 1000], (8, 2), 64, boost=1e-4)
    check_attend(q, 22, [300, 1000], (8, 2), 64, boost=0.0)


@pytest.mark.parametrize("act,kv,low,high,key", [("f32", "f16", 16, 30, 0), ("f32", "e4m3", 16, 30, 0), ("bf16", "f16", 16, 40, 0),
                                                 ("bf16", "e4m3", 16, 30, 0), ("f16", "f16", 10, 15, 9), ("f16", "e4m3", 12, 15, 7),
                                                 ("f32", "bf16", 20, 60, 0), ("bf16", "bf16", 20, 60, 0), ("f16", "bf16", 10, 15, 20)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_huge_scores(q, act, kv, low, high, key, sign):
    # One token's score is twice the others', all of them so large that they are many steps of 1 apart in fp32: its
    # value is the output, whatever the score's own rounding (p of the token is the whole sum: the parts' 22 or 16 bits).
    rng = np.random.default_rng(51)
    c = Cache(q, rng, kv, 20, 16, 2, 64, scales=False)
    lens = [200, 33, 64]
    table = fill(rng, c, lens)
    u = torch.from_numpy(rng.choice([-1.0, 1.0], (2, 64))).cuda() * 2.0 ** key
    best = [int(rng.integers(0, n)) for n in lens]
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        k = u.float()[None] * torch.where(t == best[b], 2.0, 1.0)[:, None, None]
        c.put(0, table[b].long()[t // 16], t % 16, k)
    size = torch.from_numpy(2.0 ** rng.uniform(low, high, (3, 16, 1)) * rng.uniform(0.9, 1.1, (3, 16, 64))).cuda()
    xq = (size * u.sign().repeat_interleave(8, 0)[None] * sign).to(ACT[act][1])
    out, lse = run_attend(q, c, xq, table, lens, 0.125 * sign, act=act)
    _, wlse, _, amp = attend64(c, xq, table, lens, 0.125 * sign)
    close(lse, wlse, amp * ((64 / 16 + 4) * 2 * U + 2.0 ** -22 + 8 * U) + 36 * U * wlse.abs())
    for b in range(3):
        v = c.rows(1, table[b].long()[best[b] // 16].view(1), torch.tensor([best[b] % 16], device="cuda"))[0]
        want = v.repeat_interleave(8, 0)
        parts = 2.0 ** -16 if act != "f32" and kv == "bf16" else 2.0 ** -22
        close(out[b], want, half_ulp(want, ACT[act][1]) + (parts + 8 * U) * want.abs())


def test_attention_large_and_small_values(q):
    # values far from 1 in the cache's own range, queries that make up for the keys
    for kv, f in (("bf16", 2.0 ** 60), ("bf16", 2.0 ** -60), ("f16", 2.0 ** 10), ("f16", 2.0 ** -12)):
        rng = np.random.default_rng(23)
        c = Cache(q, rng, kv, 20, 16, 2, 64)
        lens = [200, 31]
        table = fill(rng, c, lens)
        t = torch.arange(200, device="cuda")
        for which in (0, 1):
            for b, n in enumerate(lens):
                page, slot = table[b].long()[t[:n] // 16], t[:n] % 16
                c.put(which, page, slot, c.rows(which, page, slot) * f)
        xq = randn(rng, 2, 8, 64) / f
        out, lse = run_attend(q, c, xq, table, lens, 0.125)
        want, wlse, mass, amp = attend64(c, xq, table, lens, 0.125)
        compare_attend(c, out / f, lse, (want / f, wlse, mass / f, amp), lens, "f32", kv)


def test_attention_ignores_what_is_not_its_own(q):
    # NaN and infinities before the window, behind the end and on other pages: the same bits as without
    rng = np.random.default_rng(24)
    for kv, inf in (("bf16", 0x7f80), ("f16", 0x7c00), ("e4m3", 0x7f)):
        lens, window = [37, 250, 0, 64], 50
        got = []
        for poison in (False, True):
            rng = np.random.default_rng(24)
            c = Cache(q, rng, kv, 30, 16, 2, 64)
            table = fill(rng, c, lens)
            xq = randn(rng, 4, 8, 64)
            for b, n in enumerate(lens):
                t = torch.arange(0, max(0, n - window), device="cuda")
                tail = torch.arange(n, (n + 15) // 16 * 16, device="cuda")
                for u in (t, tail):
                    page, slot = table[b].long()[u // 16], u % 16
                    c.k[page, :, slot] = inf if poison else 0
                    c.v[page, :, slot] = inf if poison else 0
            got.append(run_attend(q, c, xq, table, lens, 0.125, window))
        for a, b in zip(*got):
            assert torch.equal(a, b)
        assert bool(torch.isfinite(got[0][0]).all())


def test_attention_nan_in_a_seen_place_reaches_its_heads_only(q):
    rng = np.random.default_rng(26)
    for which in (0, 1):
        c = Cache(q, rng, "f16", 8, 16, 2, 64)
        table = fill(rng, c, [50, 20])
        xq = randn(rng, 2, 8, 64)
        (c.k, c.v)[which][table[0, 1].long(), 1, 3, 7] = 0x7e00
        out, _ = run_attend(q, c, xq, table, [50, 20], 0.125)
        bad = torch.isnan(out)
        assert bool(bad[0, 4:, 7].all()) and not bool(bad[1].any()) and not bool(bad[0, :4].any())


def test_attention_bad_pages_are_left_out_and_flagged(q):
    rng = np.random.default_rng(27)
    for bad in (-1, 30, 2 ** 31 - 1, -2 ** 31):
        c = Cache(q, rng, "bf16", 30, 16, 2, 64)
        lens = [100, 10, 300]
        table = fill(rng, c, lens)
        table[0, 2], table[1, 0], table[2, 18] = bad, bad, bad
        xq = randn(rng, 3, 8, 64)
        err = err_word()
        out, lse = run_attend(q, c, xq, table, lens, 0.125, err=err)
        assert int(err.item()) == q.COLI_LAYER_BAD_PAGE
        assert q.coli_moe_check(err, raise_on_error=False) == q.COLI_MOE_EKERNEL
        ref = attend64(c, xq, table, lens, 0.125, skip={(0, 2), (1, 0), (2, 18)})
        compare_attend(c, out, lse, ref, lens, "f32", "bf16")
        assert bool((out[1] == 0).all())


def test_attention_bad_lengths_are_clamped_and_flagged(q):
    rng = np.random.default_rng(28)
    c = Cache(q, rng, "bf16", 10, 16, 1, 64)
    table = fill(rng, c, [48, 48, 20])
    xq = randn(rng, 3, 4, 64)
    for given in ([49, 48, 20], [2 ** 31 - 1, 48, 20], [48, -1, 20], [48, -2 ** 31, 20]):
        err = err_word()
        tl = torch.tensor(given, dtype=torch.int32, device="cuda")
        out, lse = run_attend(q, c, xq, table[:, :3], tl, 0.125, err=err)
        assert int(err.item()) == q.COLI_LAYER_BAD_POSITION
        seen = [min(max(n, 0), 48) for n in given]
        compare_attend(c, out, lse, attend64(c, xq, table, seen, 0.125), seen, "f32", "bf16")


def test_attention_at_the_longest_lengths(q):
    # tables that name all but 2^31 tokens on few pages; the window's end lies within a unit of 2^31
    rng = np.random.default_rng(48)
    for ps in (64, 1023):
        width = (2 ** 31 - 1) // ps
        top = width * ps
        c = Cache(q, rng, "f16", 3, ps, 2, 64)
        first_page = (top - 100) // ps
        table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
        table[:, first_page:] = torch.arange(width - first_page, dtype=torch.int32, device="cuda") % 2 + 1
        for t in range(top - 30, top):
            page = int(table[0, t // ps])
            for which in (0, 1):
                c.put(which, torch.tensor([page]), torch.tensor([t % ps]), randn(rng, 1, 2, 64))
        xq = randn(rng, 3, 4, 64)
        seen = [top, top, top - 1]
        for given, flag in (([top, 2 ** 31 - 1, top - 1], 0 if top == 2 ** 31 - 1 else q.COLI_LAYER_BAD_POSITION), (seen, 0)):
            err = err_word()
            out, lse = run_attend(q, c, xq, table, given, 0.125, 20, err=err)
            assert int(err.item()) == flag
            ref = attend64(c, xq, table, seen, 0.125, 20)
            compare_attend(c, out, lse, ref, [20], "f32", "f16")


def test_attention_strided_rows_and_no_lse(q):
    rng = np.random.default_rng(29)
    c = Cache(q, rng, "f16", 12, 16, 2, 80)
    lens = [33, 64, 7]
    table = fill(rng, c, lens)
    for act in sorted(ACT):
        buf = randn(rng, 3 * 1001 + 1).to(ACT[act][1])
        xq = buf[1:].view(3, 1001)[:, :640].unflatten(1, (8, 80))
        obuf = torch.full((3, 999), 7.0, dtype=ACT[act][1], device="cuda")
        out, lse = run_attend(q, c, xq, table, lens, 0.1, act=act, q_stride=1001, out=obuf, out_stride=999)
        compare_attend(c, obuf[:, :640].unflatten(1, (8, 80)), lse, attend64(c, xq, table, lens, 0.1), lens, act, "f16")
        assert bool((obuf[:, 640:] == 7.0).all())
        d = q.make_attn_desc(3, 8, table.shape[1], ACT[act][0], 0.1, 0, 1001, 999)
        ws = torch.empty(q.coli_attn_workspace_bytes(d, c.desc), dtype=torch.uint8, device="cuda")
        again = torch.zeros_like(obuf)
        q.coli_attn_decode(d, c.desc, xq, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), again, None, None, ws,
                           ws.numel())
        assert torch.equal(again[:, :640], obuf[:, :640])


def test_attention_behind_two_to_the_31_elements(q):
    # a pool of 2^32 + elements: pages at both ends
    rng = np.random.default_rng(30)
    pages, ps, kh, d = 2 ** 32 // (64 * 8 * 128) + 5, 64, 8, 128
    pool = [torch.empty(pages, kh, ps, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c = Cache(q, rng, "bf16", 1, ps, kh, d)
    c.pages, c.k, c.v = pages, pool[0].view(torch.int16), pool[1].view(torch.int16)
    c.desc = q.make_kv_cache(pool[0], pool[1], 1, pages, ps, kh, d)
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device="cuda")
    t = torch.arange(150, device="cuda")
    for which in (0, 1):
        c.put(which, table[0].long()[t // ps], t % ps, randn(rng, 150, kh, d))
    xq = randn(rng, 1, 16, d)
    new = randn(rng, 1, kh, d)
    pos = torch.tensor([149], dtype=torch.int32, device="cuda")
    q.coli_kv_append(q.make_append_desc(1, 0, 1, 3), c.desc, None, new, new, None, None, pos, table, None)
    assert torch.equal(c.rows(0, table[0, 2].long(), 149 % ps), new[0].bfloat16().double())
    out, lse = run_attend(q, c, xq, table, [150], 0.1)
    compare_attend(c, out, lse, attend64(c, xq, table, [150], 0.1), [150], "f32", "bf16")


def test_attention_repeats_on_streams_and_in_graphs(q):
    rng = np.random.default_rng(31)
    c = Cache(q, rng, "bf16", 400, 16, 2, 128)
    lens = [3000, 17, 0, 1500]
    table = fill(rng, c, lens)
    xq = randn(rng, 4, 16, 128)
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = run_attend(q, c, xq, table, tl, 0.1)
    d = q.make_attn_desc(4, 16, table.shape[1], 0, 0.1)
    ws = torch.empty(q.coli_attn_workspace_bytes(d, c.desc), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):  # back to back in one workspace
        q.coli_attn_decode(d, c.desc, xq, table, tl, out, lse, None, ws, ws.numel(), s)
    s.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    out.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q.coli_attn_decode(d, c.desc, xq, table, tl, out, lse, None, ws, ws.numel(), s)
        q.coli_attn_decode(d, c.desc, xq, table, tl, out, lse, None, ws, ws.numel(), s)
    for new in (lens, [1, 2500, 900, 0], lens):  # lengths are read at replay
        tl.copy_(torch.tensor(new, dtype=torch.int32))
        if new is not lens:
            old = table.clone()
            table[1] = table[0]
            table[2] = table[3]
        g.replay()
        torch.cuda.synchronize()
        if new is lens:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        else:
            compare_attend(c, out, lse, attend64(c, xq, table, new, 0.1), new, "f32", "bf16")
            table.copy_(old)


# ------------------------------------------------------------------------------------ norms
def check_norms(q, seed, rows, width, act="f32", gate="none", post=True, pre=True, scale=1.0, pad=0, offset=0, alias="",
                mag=1.0):
    rng = np.random.default_rng(seed)
    code, dtype = ACT[act]

    def make(scale_by):
        buf = (randn(rng, rows * (width + pad) + offset) * scale_by).to(dtype)
        return buf, buf[offset:].view(rows, width + pad)[:, :width]

    (yb, y), (rb, r) = make(0.3 * mag), make(3.0 * mag)
    eb, e = make(1.0)
    gv = {"none": None, "channel": e[0].contiguous(), "row": e[:, 0].contiguous(), "element": e}[gate]
    pw = randn(rng, width).abs() + 0.5 if post else None
    nw = randn(rng, width).abs() + 0.5 if pre else None
    z, y64, r64 = y.double(), y.double(), r.double()
    if post:
        z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-5) * pw.double()
    if gv is not None:
        z = z * (gv.double()[:, None] if gate == "row" else gv.double())
    want = scale * r64 + z
    size = (scale * r64).abs() + z.abs()
    rs = torch.rsqrt(want.square().mean(1, keepdim=True) + 1e-6)
    ob, o = make(0.0)
    xb, x = make(0.0)
    if alias == "resid":
        ob, o = rb, r
    if alias == "both":
        ob, o, xb, x = rb, r, yb, y
    if alias == "gate":
        xb, x = eb, e
    g = {"none": 0, "channel": 1, "row": 2, "element": 3}[gate]
    st = width + pad
    d = q.make_norms_desc(rows, width, code, g, 1e-5, 1e-6, scale, st, st, st if gate == "element" else 0, st, st)
    q.coli_block_norms(d, y, r, pw, gv, nw, o, x if pre else None)
    torch.cuda.synchronize()
    close(o, want, half_ulp(want, dtype) + 64 * U * size)
    if pre:
        xn = want * rs * nw.double()
        close(x, xn, half_ulp(xn, dtype) + 64 * U * (size * rs * nw.double() + xn.abs()))
    elif alias == "":
        assert bool((xb == 0).all())


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("gate", ["none", "channel", "row", "element"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_norms_parts(q, act, gate, post, pre):
    check_norms(q, 41, 5, 512, act, gate, post, pre, 0.5)


@pytest.mark.parametrize("width", [1, 2, 3, 7, 8, 31, 32, 33, 100, 255, 1000, 1001, 1024, 2048, 4096, 5120, 6144, 8191, 8192, 12288,
                                   16384, 16385, 20000, 32768, 50001, 65528, 65535, 65536])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_norms_widths(q, width, act):
    check_norms(q, 42, 3, width, act, "element")


@pytest.mark.parametrize("rows", [1, 2, 37, 152, 700, 5000])
def test_norms_rows(q, rows):
    check_norms(q, 43, rows, 1536, "bf16", "row")


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("act", ["f32", "f16"])
@pytest.mark.parametrize("gate", ["channel", "element"])
def test_norms_strides_and_alignment(q, pad, offset, act, gate):
    check_norms(q, 44, 9, 256, act, gate, pad=pad, offset=offset)


@pytest.mark.parametrize("alias,gate", [("resid", "channel"), ("both", "element"), ("gate", "element")])
@pytest.mark.parametrize("width", [640, 1001, 20000])
def test_norms_in_place(q, alias, gate, width):
    check_norms(q, 45, 6, width, "bf16", gate, alias=alias)


def test_norms_of_small_and_zero_rows(q):
    check_norms(q, 46, 4, 512, mag=1e-12)
    check_norms(q, 46, 4, 512, mag=0.0)
    check_norms(q, 46, 4, 512, mag=1e8, scale=0.0)


def test_norms_on_a_stream_and_in_a_graph(q):
    rng = np.random.default_rng(47)
    y, r, w = randn(rng, 8, 20000), randn(rng, 8, 20000), randn(rng, 20000)
    o, x, o2, x2 = (torch.empty_like(y) for _ in range(4))
    d = q.make_norms_desc(8, 20000, 0, 0, 1e-5, 1e-5)
    q.coli_block_norms(d, y, r, w, None, w, o, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q.coli_block_norms(d, y, r, w, None, w, o2, x2, s)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(x, x2)
