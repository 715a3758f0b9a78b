// attn_decode.cu — coli_attn_decode: how a call is laid out, and the join of the items that a run's
// border cut (attn_kernel.cuh has the streaming kernel).
#include "attn.h"
#include "host.h"
#include "pdl.cuh"

namespace colimoe {

namespace {

constexpr int kJoinThreads = 256;

// One block per (border between runs, head of the group): the block of an item's first cut adds up the
// partial sums of all runs that hold units of the item, in the order of the runs within each warp and
// the warps in order. Everything is scaled to the largest m, by exact powers of two.
template <int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams P, const AttnWork W, int shift) {
    constexpr int kWarps = kJoinThreads / 32, kPer = DP / 32;
    __shared__ float red[kWarps][DP];
    __shared__ float2 red_ml[kWarps];
    let_next_start();
    wait_for_previous();
    const int c = blockIdx.x + 1, runs = W.cuts[0].runs;
    const AttnCut cut = W.cuts[c];  // written if c < runs
    if (c >= runs || cut.b < 0) return;
    const int heads = 8 * W.nt, h = blockIdx.y;
    const int kh = cut.hv / W.chunks, group = P.q_heads / P.kv_heads, gh = (cut.hv - kh * W.chunks) * heads + h;
    if (gh >= group) return;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, c0 = c - 1;
    float o[kPer], l = 0.f, m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; j++) o[j] = 0.f;
#pragma unroll 4
    for (int r = c0 + w; r <= cut.last; r += kWarps) {
        const int64_t s = (int64_t)(2 * r + (r == c0 ? 1 : 0)) * heads + h;
        const float2 e = W.part_ml[s];
        Run<float, kPer> v;
        v.load(W.part_o + s * DP + lane * kPer);
        const float n = fmaxf(m, e.x), ref = n == -INFINITY ? 0.f : n;
        const float f0 = exp2f(m - ref), f1 = exp2f(e.x - ref);
        m = n;
        l = fmaf(l, f0, e.y * f1);
#pragma unroll
        for (int j = 0; j < kPer; j++) o[j] = fmaf(o[j], f0, v.e[j] * f1);
    }
#pragma unroll
    for (int j = 0; j < kPer; j++) red[w][lane * kPer + j] = o[j];
    if (lane == 0) red_ml[w] = make_float2(m, l);
    __syncthreads();
    float top = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
    for (int k = 0; k < kWarps; k++) top = fmaxf(top, red_ml[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int k = 0; k < kWarps; k++) {
        f[k] = exp2f(red_ml[k].x - ref);
        sum = fmaf(red_ml[k].y, f[k], sum);
    }
    const float vs = P.v_scale ? P.v_scale[kh] : 1.f;
    const int qh = kh * group + gh;
    for (int d = threadIdx.x; d < P.dim; d += kJoinThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; k++) v = fmaf(red[k][d], f[k], v);
        store_act(P.out, cut.b * P.out_stride + (int64_t)qh * P.dim + d, sum == 0.f ? 0.f : v / sum * vs, P.act);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[(int64_t)cut.b * P.q_heads + qh] = attn_lse(ref, sum, shift);
}

struct Layout {
    AttnWork w;
    int64_t units;  // at most
    int grid;
    size_t ml, o, total;
};

Layout layout_of(const AttnParams &P) {
    Layout L{};
    const int group = P.q_heads / P.kv_heads;
    L.w.dim = P.dim <= 64 ? 64 : P.dim <= 128 ? 128 : 256;
    L.w.use = P.dim > 64 && P.dim <= 96 ? 96 : L.w.dim;
    L.w.nt = group <= 8 ? 1 : 2;
    // q in one part where the cache's type (f16 for e4m3, scaled) holds it
    L.w.wide = P.act == COLI_ACT_F32 || (P.act == COLI_ACT_F16 && P.fmt == COLI_KV_BF16);
    L.w.chunks = (group + 8 * L.w.nt - 1) / (8 * L.w.nt);
    L.w.groups = P.kv_heads * L.w.chunks;
    L.w.unit = attn_unit(P.fmt, L.w.dim, L.w.nt, L.w.wide);
    L.w.divide = kv_divide_by(P.cache.page_size);
    const int size = P.fmt == COLI_KV_E4M3 ? 1 : 2;
    attn_steps(P.cache, P.kv_heads, size, L.w.off_shift);
    L.w.page_step = (uint32_t)(P.cache.page_stride * size >> L.w.off_shift);
    L.w.token_step = (uint32_t)(P.cache.token_stride * size >> L.w.off_shift);
    L.w.head_step = (uint32_t)(P.cache.head_stride * size >> L.w.off_shift);
    // no more CTAs than units that the page tables can name
    const int64_t held = (int64_t)P.table_width * P.cache.page_size;
    const int64_t seen = P.window > 0 && P.window < held ? P.window : held;
    const int64_t most = ((seen + L.w.unit - 1) / L.w.unit) * P.seqs * L.w.groups;
    const int64_t ctas = (int64_t)num_sms() * attn_ctas_per_sm(P.fmt, L.w.dim, L.w.nt, L.w.wide);
    L.units = most;
    L.grid = (int)(most < ctas ? most : ctas);
    const int64_t items = (int64_t)P.seqs * L.w.groups;
    L.w.times = attn_times(P.fmt, L.w.dim, L.w.nt, L.w.unit, (int64_t)L.w.unit * P.dim * 2 * size);
    L.w.ctas = L.grid;
    // certain for the longest items that the tables can name: no second launch; else the kernel decides by the lengths
    if (attn_whole(items, most / items, ctas, L.w.times)) L.w.whole = kAttnWhole;
    else if (items <= 16 * ctas && 5 * items >= 4 * ctas) L.w.whole = kAttnMaybe;
    if (L.w.whole == kAttnWhole) L.grid = (int)items;
    if (L.w.whole == kAttnMaybe && items > L.grid) L.grid = (int)items;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    L.ml = up((size_t)L.w.ctas * sizeof(AttnCut));
    L.o = L.ml + up((size_t)2 * L.w.ctas * 8 * L.w.nt * sizeof(float2));
    L.total = L.o + up((size_t)2 * L.w.ctas * 8 * L.w.nt * L.w.dim * 4);
    return L;
}

}  // namespace

bool attn_steps(const KvShape &c, int heads, int elem_bytes, uint32_t &shift) {
    // an axis of one entry takes no step
    const uint64_t page = c.pages > 1 ? (uint64_t)c.page_stride * elem_bytes : 0;
    const uint64_t token = c.page_size > 1 ? (uint64_t)c.token_stride * elem_bytes : 0;
    const uint64_t head = heads > 1 ? (uint64_t)c.head_stride * elem_bytes : 0;
    shift = 4;  // strides are multiples of 16 bytes
    while (shift < 20 && ((page | token | head) >> shift) % 2 == 0) shift++;
    // at most 2^40 * 2 bytes a step: the sum of the last row's offsets is formed without overflow
    const unsigned __int128 last = (unsigned __int128)page * (c.pages - 1) + (unsigned __int128)token * (c.page_size - 1) +
                                   (unsigned __int128)head * (heads - 1);
    return (last >> shift) >> 32 == 0;
}

size_t attn_workspace_bytes(const AttnParams &P) {
    const Layout L = layout_of(P);
    return L.units > INT32_MAX ? 0 : L.total;  // units are counted in 32 bits
}

cudaError_t launch_attn_decode(const AttnParams &P, cudaStream_t s) {
    Layout L = layout_of(P);
    char *ws = (char *)P.ws;
    L.w.cuts = (AttnCut *)ws;
    L.w.part_ml = (float2 *)(ws + L.ml);
    L.w.part_o = (float *)(ws + L.o);
    const cudaError_t e = P.fmt == COLI_KV_BF16  ? launch_attn_bf16(P, L.w, L.grid, s)
                          : P.fmt == COLI_KV_F16 ? launch_attn_f16(P, L.w, L.grid, s)
                                                 : launch_attn_e4m3(P, L.w, L.grid, s);
    if (e != cudaSuccess || L.w.whole == kAttnWhole || L.w.ctas == 1) return e;  // no borders
    // the join's blocks start while the streaming kernel runs and wait for its end
    const dim3 grid(L.w.ctas - 1, 8 * L.w.nt);
    const int shift = P.fmt == COLI_KV_BF16 ? 0 : 14;
    return L.w.dim == 64    ? launch_overlapped(attn_join_kernel<64>, grid, kJoinThreads, 0, s, P, L.w, shift)
           : L.w.dim == 128 ? launch_overlapped(attn_join_kernel<128>, grid, kJoinThreads, 0, s, P, L.w, shift)
                            : launch_overlapped(attn_join_kernel<256>, grid, kJoinThreads, 0, s, P, L.w, shift);
}

}  // namespace colimoe
