"""Host-side checks of include/colilayer.h: the binding declares what the header does, bad arguments
are refused with the documented codes before the GPU is touched, and the page arithmetic the kernels
share (csrc/kv_index.h) is right at its borders, on bad pages and behind 2^31 elements."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40  # a 256-byte aligned address never dereferenced: validation fails first


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__._builder().build()
    import quantized_expert_decode_gb300 as q
    return q


def test_header_and_binding_agree(q):
    with open(os.path.join(ROOT, "include", "colilayer.h")) as f:
        text = f.read()
    names = sorted(re.findall(r"^(?:int|size_t)\s+(coli_[a-z_]+)\s*\(", text, re.M))
    assert names == sorted(q.LAYER_EXPORTS)
    lib = ctypes.CDLL(q.LIB_PATH)
    for n in names:
        getattr(lib, n)
    for name, value in re.findall(r"^#define (COLI_(?:ACT|KV|GATE|LAYER)_\w+) (\d+)", text, re.M):
        assert getattr(q, name) == int(value), name


def test_struct_layouts_match_the_header(q, tmp_path):
    # sizes and the last field's offset as a C compiler sees them
    src = tmp_path / "l.c"
    names = {"coli_kv_cache": "head_stride", "coli_append_desc": "q_out_stride", "coli_attn_desc": "out_stride",
             "coli_norms_desc": "xn_stride"}
    body = "".join(f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {f}));' for n, f in names.items())
    src.write_text('#include <stdio.h>\n#include "colilayer.h"\nint main(void){' + body + "return 0;}")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, l.split())) for l in subprocess.run([str(exe)], capture_output=True, text=True,
                                                              check=True).stdout.splitlines()]
    want = [(ctypes.sizeof(getattr(q, n)), getattr(getattr(q, n), f).offset) for n, f in names.items()]
    assert got == want


def cache(q, **over):
    d = dict(k=FAKE, v=FAKE, fmt=1, pages=10, page_size=16, heads=4, dim=128)
    d.update(over)
    return q.make_kv_cache(**d)


BAD_CACHES = [(dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(fmt=0), "EINVAL"), (dict(fmt=4), "EINVAL"),
              (dict(pages=0), "EINVAL"), (dict(page_size=0), "EINVAL"), (dict(heads=0), "EINVAL"),
              (dict(heads=2000), "EINVAL"), (dict(dim=0), "EINVAL"), (dict(dim=100), "ENOTSUP"),
              (dict(dim=264), "ENOTSUP"), (dict(fmt=3, dim=72), "ENOTSUP"), (dict(k=FAKE + 8), "EALIGN"),
              (dict(v=FAKE + 2), "EALIGN"), (dict(token_stride=64), "EINVAL"), (dict(head_stride=-128), "EINVAL"),
              (dict(page_stride=0), "EINVAL"), (dict(token_stride=132), "EALIGN"), (dict(k_scale=FAKE + 1), "EALIGN")]


def append(lib, c=None, **over):
    d = dict(tokens=3, q_heads=8, seqs=3, table_width=5, act=0, rotary=64)
    a = dict(q=FAKE, k=FAKE, v=FAKE, inv_freq=FAKE, seq=FAKE, pos=FAKE, table=FAKE, q_out=FAKE, err=None)
    for k, v in over.items():
        (d if k not in a else a)[k] = v
    return lib.coli_kv_append(lib.make_append_desc(**d), c or cache(lib), raise_on_error=False, **a)


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(q, over, code):
    want = getattr(q, "COLI_MOE_" + code)
    c = cache(q, **over)
    assert append(q, c) == want
    d = q.make_attn_desc(2, 8, 5, 0, 0.1)
    assert q.coli_attn_workspace_bytes(d, c) == 0
    assert q.coli_attn_decode(d, c, FAKE, FAKE, FAKE, FAKE, ws=FAKE, ws_bytes=1 << 40, raise_on_error=False) == want


@pytest.mark.parametrize("over,code", [
    (dict(tokens=0), "EINVAL"), (dict(q_heads=-1), "EINVAL"), (dict(q_heads=2000), "EINVAL"), (dict(seqs=0), "EINVAL"),
    (dict(table_width=0), "EINVAL"), (dict(table_width=1 << 28), "EINVAL"), (dict(act=3), "EINVAL"),
    (dict(rotary=-2), "EINVAL"), (dict(rotary=63), "EINVAL"), (dict(rotary=130), "EINVAL"), (dict(interleaved=2), "EINVAL"),
    (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(pos=None), "EINVAL"), (dict(table=None), "EINVAL"),
    (dict(inv_freq=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(q_out=None), "EINVAL"), (dict(q_heads=0), "EINVAL"),
    (dict(seq=None, tokens=4), "EINVAL"), (dict(q_stride=1000), "EINVAL"), (dict(k_stride=511), "EINVAL"),
    (dict(v_stride=-1), "EINVAL"), (dict(q_stride=1100), "EINVAL"), (dict(q=FAKE + 2), "EALIGN"),
    (dict(k=FAKE + 1), "EALIGN"), (dict(err=FAKE + 2), "EALIGN"), (dict(pos=FAKE + 1), "EALIGN")])
def test_append_refusals(q, over, code):
    # q and q_out are the same rows here, so unequal strides are refused too
    assert append(q, **over) == getattr(q, "COLI_MOE_" + code)


@pytest.mark.parametrize("desc,args,code", [
    (dict(seqs=0), {}, "EINVAL"), (dict(seqs=2049), {}, "EINVAL"), (dict(q_heads=0), {}, "EINVAL"),
    (dict(q_heads=6), {}, "EINVAL"), (dict(q_heads=2048), {}, "EINVAL"), (dict(table_width=0), {}, "EINVAL"),
    (dict(table_width=1 << 27), {}, "EINVAL"), (dict(act=-1), {}, "EINVAL"), (dict(window=-1), {}, "EINVAL"),
    (dict(scale=float("nan")), {}, "EINVAL"), (dict(scale=float("inf")), {}, "EINVAL"), (dict(q_stride=8), {}, "EINVAL"),
    (dict(out_stride=-8), {}, "EINVAL"), ({}, dict(q=None), "EINVAL"), ({}, dict(out=None), "EINVAL"),
    ({}, dict(table=None), "EINVAL"), ({}, dict(lens=None), "EINVAL"), ({}, dict(q=FAKE + 1), "EALIGN"),
    ({}, dict(lens=FAKE + 2), "EALIGN"), ({}, dict(lse=FAKE + 2), "EALIGN"), ({}, dict(ws=None), "EWORKSPACE"),
    ({}, dict(ws=FAKE + 16), "EWORKSPACE"), ({}, dict(ws_bytes=0), "EWORKSPACE")])
def test_attention_refusals(q, desc, args, code):
    d = dict(seqs=2, q_heads=8, table_width=5, act=0, scale=0.1)
    d.update(desc)
    a = dict(q=FAKE, table=FAKE, lens=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(args)
    assert q.coli_attn_decode(q.make_attn_desc(**d), cache(q), raise_on_error=False, **a) == getattr(q, "COLI_MOE_" + code)
    if desc:
        assert q.coli_attn_workspace_bytes(q.make_attn_desc(**d), cache(q)) == 0


def test_attention_workspace(q):
    d = q.make_attn_desc(2, 8, 5, 0, 0.1)
    n = q.coli_attn_workspace_bytes(d, cache(q))
    assert n > 0 and n % 256 == 0
    assert q.coli_attn_decode(d, cache(q), FAKE, FAKE, FAKE, FAKE, ws=FAKE, ws_bytes=n - 1,
                              raise_on_error=False) == q.COLI_MOE_EWORKSPACE


@pytest.mark.parametrize("seqs,q_heads,width,window", [(64, 64, 32, 2 ** 31 - 1), (64, 64, 64, 2 ** 30), (2048, 8, 4, 2 ** 31 - 1),
                                                       (1, 8, 500, 8001), (5, 16, 31, 4096)])
def test_a_window_beyond_the_table_is_no_window(q, seqs, q_heads, width, window):
    # as many units, so the same workspace, as without a window
    c = cache(q, heads=8 if q_heads % 8 == 0 else 4)
    none, wide = (q.make_attn_desc(seqs, q_heads, width, 0, 0.1, window=w) for w in (0, window))
    assert q.coli_attn_workspace_bytes(wide, c) == q.coli_attn_workspace_bytes(none, c) > 0


@pytest.mark.parametrize("desc,args,code", [
    (dict(rows=0), {}, "EINVAL"), (dict(width=0), {}, "EINVAL"), (dict(width=65537), {}, "EINVAL"),
    (dict(act=5), {}, "EINVAL"), (dict(gate=4), {}, "EINVAL"), (dict(gate=1), {}, "EINVAL"),
    (dict(post_eps=-1.0), {}, "EINVAL"), (dict(pre_eps=float("nan")), {}, "EINVAL"),
    (dict(resid_scale=float("inf")), {}, "EINVAL"), (dict(y_stride=63), {}, "EINVAL"), (dict(xn_stride=-1), {}, "EINVAL"),
    ({}, dict(y=None), "EINVAL"), ({}, dict(resid=None), "EINVAL"), ({}, dict(resid_out=None), "EINVAL"),
    ({}, dict(gate=FAKE), "EINVAL"), ({}, dict(xn=None), "EINVAL"), ({}, dict(xn=2 * FAKE), "EINVAL"),
    (dict(resid_stride=80), dict(resid_out=3 * FAKE), "EINVAL"), ({}, dict(y=FAKE + 2), "EALIGN"),
    ({}, dict(post_w=FAKE + 2), "EALIGN")])
def test_norms_refusals(q, desc, args, code):
    d = dict(rows=2, width=64)
    d.update(desc)
    a = dict(y=FAKE, resid=3 * FAKE, post_w=FAKE, gate=None, pre_w=FAKE, resid_out=2 * FAKE, xn=4 * FAKE)
    a.update(args)
    assert q.coli_block_norms(q.make_norms_desc(**d), raise_on_error=False, **a) == getattr(q, "COLI_MOE_" + code)


# ---------------------------------------------------------------------- page arithmetic
@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv")
    src = d / "kv.cc"
    src.write_text('''
#include "kv_index.h"
using namespace colimoe;
extern "C" long long row(long long ps_, long long ts, long long hs, int pages, int page_size, const int *t, int width,
                         int tok, int h, int *why) {
    KvShape c{ps_, ts, hs, pages, page_size};
    return kv_row(c, t, width, tok, h, *why);
}
extern "C" void span(int n, int width, int page_size, int window, int *out) {
    kv_span(n, width, page_size, window, out[0], out[1], out[2]);
}
extern "C" int units(int tokens, int unit) { return kv_units(tokens, unit); }
extern "C" int unit_token(int first, int end, int unit, int u, int at) {
    int t;
    return kv_unit_token(first, end, unit, u, at, t) ? t : -1;
}
extern "C" int quotient(int size, int t) { return kv_quotient(kv_divide_by(size), t); }
''')
    so = d / "libkv.so"
    inc = os.path.join(ROOT, "quantized_expert_decode_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.row.restype = ctypes.c_longlong
    lib.row.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int] * 2 + [ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_void_p]
    return lib


def row(lib, table, tok, head=0, pages=1 << 20, ps=16, strides=(8192, 128, 2048)):
    arr = (ctypes.c_int * len(table))(*table)
    why = ctypes.c_int(-1)
    return lib.row(*strides, pages, ps, arr, len(table), tok, head, ctypes.byref(why)), why.value


def test_rows_follow_the_table(index):
    table = [7, 2, 900000]
    for tok in (0, 1, 15, 16, 31, 32, 47):
        for head in (0, 3):
            want = table[tok // 16] * 8192 + tok % 16 * 128 + head * 2048
            assert row(index, table, tok, head) == (want, 0)
    assert row(index, table, 32)[0] > 1 << 31  # 64-bit products


@pytest.mark.parametrize("ps", [1, 3, 24])
def test_rows_of_odd_pages(index, ps):
    table = list(range(50, 40, -1))
    for tok in range(10 * ps):
        assert row(index, table, tok, 1, ps=ps, strides=(1000, 16, 400))[0] == table[tok // ps] * 1000 + tok % ps * 16 + 400


def test_bad_pages_and_positions_have_no_row(index):
    assert row(index, [-1, 2], 3) == (-1, 1)
    assert row(index, [5, 2], 3, pages=5) == (-1, 1)
    assert row(index, [4, 2], 3, pages=5) == (4 * 8192 + 3 * 128, 0)
    assert row(index, [2 ** 31 - 1, 2], 3) == (-1, 1)
    assert row(index, [-2 ** 31, 2], 3) == (-1, 1)
    assert row(index, [1, 2], 32) == (-1, 2)
    assert row(index, [1, 2], -1) == (-1, 2)
    assert row(index, [1, 2], 2 ** 31 - 1) == (-1, 2)


@pytest.mark.parametrize("n,width,ps,window,want", [
    (0, 4, 16, 0, (0, 0, 0)), (1, 4, 16, 0, (0, 1, 0)), (64, 4, 16, 0, (0, 64, 0)), (65, 4, 16, 0, (0, 64, 2)),
    (-1, 4, 16, 0, (0, 0, 2)), (-2 ** 31, 4, 16, 5, (0, 0, 2)), (60, 4, 16, 10, (50, 60, 0)), (10, 4, 16, 10, (0, 10, 0)),
    (11, 4, 16, 10, (1, 11, 0)), (2 ** 31 - 1, 4, 16, 1, (63, 64, 2)), (5, 4, 16, 2 ** 31 - 1, (0, 5, 0))])
def test_spans(index, n, width, ps, window, want):
    out = (ctypes.c_int * 3)()
    index.span(n, width, ps, window, out)
    assert tuple(out) == want


@pytest.mark.parametrize("size", [1, 2, 3, 5, 7, 8, 16, 24, 48, 100, 333, 1000, 65535, 65536, 65537, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1])
def test_page_quotients(index, size):
    for m in [0, 1, 2, 3, 1000, (2 ** 31 - 1) // size - 1, (2 ** 31 - 1) // size]:
        for t in (m * size - 1, m * size, m * size + 1, m * size + size - 1):
            if 0 <= t < 2 ** 31:
                assert index.quotient(size, t) == t // size, (size, t)


@pytest.mark.parametrize("unit", [64, 128, 192, 256, 384])
@pytest.mark.parametrize("end", [1, 100, 5000, 2 ** 31 - 400, 2 ** 31 - 64, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("window", [0, 1, 20, 129, 385])
def test_units_up_to_the_longest_sequence(index, unit, end, window):
    # the places of the last unit pass 2^31, the tokens do not
    first = end - window if 0 < window < end else 0
    n = index.units(end - first, unit)
    assert n == -(-(end - first) // unit)
    for u in {0, n - 1}:
        for at in (0, 1, 15, 31, unit // 2, unit - 17, unit - 1):
            t = first + u * unit + at
            assert index.unit_token(first, end, unit, u, at) == (t if t < end else -1)


# ---------------------------------------------------------------------- how a call is laid out
@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    """attn_decode.cu's layout of a call, built for the host with the launches left out."""
    d = tmp_path_factory.mktemp("layout")
    src = d / "layout.cu"
    src.write_text('''
#include "attn_decode.cu"
namespace colimoe {
int num_sms() { return 152; }
cudaError_t launch_attn_bf16(const AttnParams &, const AttnWork &, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_attn_f16(const AttnParams &, const AttnWork &, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_attn_e4m3(const AttnParams &, const AttnWork &, int, cudaStream_t) { return cudaSuccess; }
}
extern "C" void layout(int fmt, int act, int dim, int heads, int kv_heads, int seqs, int width, int page_size, int window, double *out) {
    using namespace colimoe;
    AttnParams P{};
    P.fmt = fmt, P.act = act, P.dim = dim, P.q_heads = heads, P.kv_heads = kv_heads, P.seqs = seqs, P.table_width = width;
    P.window = window;
    P.cache = KvShape{(int64_t)kv_heads * page_size * dim, dim, (int64_t)page_size * dim, 1000, page_size};
    const Layout L = layout_of(P);
    out[0] = L.w.unit, out[1] = L.w.times.bytes, out[2] = L.w.whole, out[3] = L.grid, out[4] = (double)L.units;
}
''')
    from quantized_expert_decode_gb300 import build
    so = d / "liblayout.so"
    subprocess.run([os.path.join(build.cuda_home(), "bin", "nvcc"), *build.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I",
                    build.CSRC, "-I", build.INCLUDE, "--expt-relaxed-constexpr", str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def call(**a):
        d = dict(fmt=1, act=1, dim=128, heads=32, kv_heads=8, seqs=32, width=100, page_size=16, window=0)
        d.update(a)
        out = (ctypes.c_double * 5)()
        lib.layout(*d.values(), out)
        return dict(zip(("unit", "unit_us", "whole", "grid", "units"), out))
    return call


@pytest.mark.parametrize("fmt,size", [(1, 2), (2, 2), (3, 1)])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 256])
def test_a_units_time_is_of_the_bytes_it_has(layout, fmt, size, dim):
    # K and V of the head's own elements, not of the size that shared memory rounds it up to
    for heads in (8, 128):
        got = layout(fmt=fmt, dim=dim, heads=heads)
        assert got["unit_us"] == pytest.approx(got["unit"] * dim * 2 * size / 7.2e6, rel=1e-6)


@pytest.mark.parametrize("fmt,act,unit", [(1, 1, 192), (2, 0, 192), (3, 1, 384), (3, 0, 256)])
def test_long_items_of_wide_groups_are_cut(layout, fmt, act, unit):
    # 9 to 16 heads a kv head, 65 to 128 elements: whole items of few CTAs take longer than cut ones and their join
    # from 3 units on, from 5 where a quarter of the places is taken, from 9 where most are
    for dim, heads in ((128, 128), (96, 72)):
        for seqs, units, whole in ((1, 2, 1), (1, 3, 0), (4, 3, 0), (5, 3, 1), (5, 4, 1), (5, 5, 0), (8, 4, 1), (8, 5, 0), (8, 8, 0),
                                   (12, 5, 1), (12, 8, 1),
                                   (20, 6, 0)):
            got = layout(fmt=fmt, act=act, dim=dim, heads=heads, seqs=seqs, page_size=unit, width=units)
            assert got["unit"] == unit and (got["whole"] == 1) == bool(whole), (dim, seqs, units)
    # others as they were
    for dim, heads in ((128, 64), (64, 128), (256, 128)):
        unit = int(layout(fmt=fmt, act=act, dim=dim, heads=heads)["unit"])
        assert layout(fmt=fmt, act=act, dim=dim, heads=heads, seqs=1, page_size=unit, width=3)["whole"] == 1
        assert layout(fmt=fmt, act=act, dim=dim, heads=heads, seqs=10, page_size=unit, width=8)["whole"] == 1
