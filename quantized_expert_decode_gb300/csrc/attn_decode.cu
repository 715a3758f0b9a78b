// attn_decode.cu — coli_attn_decode: how a call is laid out, and the join of the items that a run's
// border cut (attn_kernel.cuh has the streaming kernel).
#include <cudaTypedefs.h>

#include "attn.h"
#include "host.h"

namespace colimoe {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // prefill.cu

namespace {

constexpr int kJoinThreads = 256;

// One block per (border between runs, head of the group): the block of an item's first border adds up
// the partial sums of all runs that hold units of the item, in the order of the runs. Everything is
// scaled to the largest m, by exact powers of two.
template <int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams P, const AttnWork W, int grid, int shift) {
    constexpr int kWarps = kJoinThreads / 32, kPer = DP / 32;
    __shared__ float red[kWarps][DP];
    __shared__ float2 red_ml[kWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = 8 * W.nt;
    const int64_t total = (int64_t)W.prefix[P.seqs] * W.groups;
    const int64_t n = min((int64_t)grid, total), c = (int64_t)blockIdx.x + 1;
    if (c >= n) return;
    const int64_t x = attn_run_start(c, total, n);
    int lo = 0, hi = P.seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((int64_t)W.prefix[mid] * W.groups <= x) lo = mid;
        else hi = mid;
    }
    const int b = lo, units = W.prefix[lo + 1] - W.prefix[lo];
    const int64_t base = (int64_t)W.prefix[lo] * W.groups;
    const int hv = (int)((x - base) / units);
    const int64_t i0 = base + (int64_t)hv * units, i1 = i0 + units;
    // this border cuts the item, and is the first that does
    if (i0 == x || attn_run_start(c - 1, total, n) > i0) return;
    const int64_t c0 = c - 1, c1 = attn_run_of(i1 - 1, total, n);
    const int kh = hv / W.chunks, group = P.q_heads / P.kv_heads, h0 = (hv - kh * W.chunks) * heads, h = blockIdx.y;
    if (h0 + h >= group) return;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    auto slot = [&](int64_t r) { return (2 * r + (r == c0 ? 1 : 0)) * heads + h; };
    float top = -INFINITY;
    for (int64_t r = c0 + lane; r <= c1; r += 32) top = fmaxf(top, W.part_ml[slot(r)].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float ref = top == -INFINITY ? 0.f : top;
    float o[kPer], l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; j++) o[j] = 0.f;
#pragma unroll 4
    for (int64_t r = c0 + w; r <= c1; r += kWarps) {
        const int64_t s = slot(r);
        const float2 e = W.part_ml[s];
        Run<float, kPer> v;
        v.load(W.part_o + s * DP + lane * kPer);
        const float f = exp2f(e.x - ref);
        l = fmaf(e.y, f, l);
#pragma unroll
        for (int j = 0; j < kPer; j++) o[j] = fmaf(v.e[j], f, o[j]);
    }
#pragma unroll
    for (int j = 0; j < kPer; j++) red[w][lane * kPer + j] = o[j];
    if (lane == 0) red_ml[w].y = l;
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; k++) sum += red_ml[k].y;
    const float vs = P.v_scale ? P.v_scale[kh] : 1.f;
    const int qh = kh * group + h0 + h;
    for (int d = threadIdx.x; d < P.dim; d += kJoinThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; k++) v += red[k][d];
        store_act(P.out, b * P.out_stride + (int64_t)qh * P.dim + d, sum == 0.f ? 0.f : v / sum * vs, P.act);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[(int64_t)b * P.q_heads + qh] = attn_lse(ref, sum, shift);
}

struct Layout {
    AttnWork w;
    int grid;
    size_t ml, o, total;
};

Layout layout_of(const AttnParams &P) {
    Layout L{};
    const int group = P.q_heads / P.kv_heads;
    L.w.dim = P.dim <= 64 ? 64 : P.dim <= 128 ? 128 : 256;
    L.w.nt = group <= 8 ? 1 : 2;
    // q in one part where the cache's type (f16 for e4m3, scaled) holds it
    L.w.wide = P.act == COLI_ACT_F32 || (P.act == COLI_ACT_F16 && P.fmt == COLI_KV_BF16);
    L.w.chunks = (group + 8 * L.w.nt - 1) / (8 * L.w.nt);
    L.w.groups = P.kv_heads * L.w.chunks;
    L.w.unit = attn_unit(P.fmt, L.w.dim);
    // the tallest box that divides a page, up to a tile
    const int tile = P.fmt == COLI_KV_E4M3 ? 32 : 16, size = P.fmt == COLI_KV_E4M3 ? 1 : 2;
    for (int r = tile; r >= 8 && !L.w.box_rows; r /= 2)
        if (P.cache.page_size % r == 0) L.w.box_rows = r;
    L.w.divide = kv_divide_by(P.cache.page_size);
    L.w.mask = L.w.box_rows ? L.w.box_rows - 1 : 0;
    // (a stage holds a span's rows one below the other for the whole tile)
    L.w.whole_rows = L.w.box_rows == tile && P.dim * size % (L.w.dim * size < 128 ? L.w.dim * size : 128) == 0;
    // no more CTAs than units that the page tables can name
    const int64_t seen = P.window > 0 ? P.window : (int64_t)P.table_width * P.cache.page_size;
    const int64_t most = ((seen + L.w.mask + L.w.unit - 1) / L.w.unit) * P.seqs * L.w.groups;
    const int64_t ctas = (int64_t)num_sms() * attn_ctas_per_sm(L.w.dim);
    L.grid = (int)(most < ctas ? most : ctas);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    L.ml = up((size_t)(P.seqs + 1) * 4);
    L.o = L.ml + up((size_t)2 * L.grid * 8 * L.w.nt * sizeof(float2));
    L.total = L.o + up((size_t)2 * L.grid * 8 * L.w.nt * L.w.dim * 4);
    return L;
}

// Maps for boxes of W.box_rows tokens; false where the strides are none that a tensor map takes. Rows whose
// size is whole spans of 128 bytes are a fifth axis, and a box takes them whole; other rows come span by
// span, the last one filled up with zeros.
bool make_maps(const AttnParams &P, const AttnWork &W, AttnMaps &M) {
    const int size = P.fmt == COLI_KV_E4M3 ? 1 : 2;
    const KvShape &c = P.cache;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const int row = W.dim * size, span = (row < 128 ? row : 128) / size;
    const cuuint64_t dims[5] = {(cuuint64_t)(W.whole_rows ? span : P.dim), (cuuint64_t)c.page_size,
                                (cuuint64_t)(W.whole_rows ? P.dim / span : 1), (cuuint64_t)P.kv_heads, (cuuint64_t)c.pages};
    cuuint64_t strides[4] = {(cuuint64_t)c.token_stride * size, (cuuint64_t)span * size, (cuuint64_t)c.head_stride * size,
                             (cuuint64_t)c.page_stride * size};
    for (int i = 0; i < 4; i++) {
        if (strides[i] >> 40) return false;
        if (strides[i] == 0) strides[i] = 16;  // an axis of one entry
    }
    const cuuint32_t box[5] = {(cuuint32_t)span, (cuuint32_t)W.box_rows, (cuuint32_t)(W.whole_rows ? W.dim / span : 1), 1, 1};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType type = size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    auto map = [&](CUtensorMap *m, const void *base) {
        return encode(m, type, 5, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      span * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(&M.k, P.k_cache) && map(&M.v, P.v_cache);
}

}  // namespace

size_t attn_workspace_bytes(const AttnParams &P) { return layout_of(P).total; }

cudaError_t launch_attn_decode(const AttnParams &P, cudaStream_t s) {
    Layout L = layout_of(P);
    char *ws = (char *)P.ws;
    L.w.prefix = (int32_t *)ws;
    L.w.part_ml = (float2 *)(ws + L.ml);
    L.w.part_o = (float *)(ws + L.o);
    AttnMaps M{};
    if (L.w.box_rows && !make_maps(P, L.w, M)) L.w.box_rows = 0;
    const cudaError_t e = P.fmt == COLI_KV_BF16  ? launch_attn_bf16(P, L.w, M, L.grid, s)
                          : P.fmt == COLI_KV_F16 ? launch_attn_f16(P, L.w, M, L.grid, s)
                                                 : launch_attn_e4m3(P, L.w, M, L.grid, s);
    if (e != cudaSuccess || L.grid == 1) return e;  // one run: no borders
    // the join's blocks start while the streaming kernel runs and wait for its end
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(L.grid - 1, 8 * L.w.nt);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int shift = P.fmt == COLI_KV_BF16 ? 0 : 14;
    return L.w.dim == 64    ? cudaLaunchKernelEx(&cfg, attn_join_kernel<64>, P, L.w, L.grid, shift)
           : L.w.dim == 128 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<128>, P, L.w, L.grid, shift)
                            : cudaLaunchKernelEx(&cfg, attn_join_kernel<256>, P, L.w, L.grid, shift);
}

}  // namespace colimoe
