// attn_tree.cu — coli_attn_tree: attention of drafted nodes over a paged cache.
//
// A CTA per node and query head; its warps take every fourth token, a lane holds 8 elements of the head, and each warp
// keeps a running maximum and sum; the warps' parts are joined at the end.
#include <cmath>

#include "act.cuh"
#include "attn.h"
#include "draft.h"
#include "host.h"
#include "pdl.cuh"

namespace colimoe {
namespace {

constexpr int kWarps = 4;

template <typename C>
__global__ void __launch_bounds__(kWarps * 32) attn_tree_kernel(const TreeParams P) {
    constexpr int kPer = 8;
    __shared__ uint32_t line[8];  // the node's ancestors and itself
    __shared__ int depth_of;
    __shared__ float red[kWarps][256], red_m[kWarps], red_l[kWarps];
    wait_for_previous();
    let_next_start();
    const int b = blockIdx.x / P.nodes, i = blockIdx.x % P.nodes, h = blockIdx.y, kh = h / (P.q_heads / P.kv_heads);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    int row, n, past, why, why2;
    draft_rows(P.first[b], P.first[b + 1], P.rows, P.nodes, row, n, why);
    draft_places(P.past[b], P.table_width, P.cache.page_size, past, n, why2);
    if ((why || why2) && i == 0 && h == 0 && threadIdx.x == 0 && P.err)
        atomicOr(P.err, (why ? COLI_LAYER_BAD_SEQUENCE : 0) | (why2 ? COLI_LAYER_BAD_POSITION : 0));
    if (i >= n) return;
    if (threadIdx.x < 8) line[threadIdx.x] = 0;
    __syncthreads();
    if (threadIdx.x == 0) {
        auto parent = [&](int x) {
            int p = P.parent ? P.parent[row + x] : x - 1;
            if (p < -1 || p >= x) {
                p = -1;
                if (P.err) atomicOr(P.err, COLI_DRAFT_BAD_NODE);
            }
            return p;
        };
        int d = 0;
        for (int x = i; x >= 0; x = parent(x), d++)
            if (P.window == 0 || d < P.window) line[x / 32] |= 1u << x % 32;
        depth_of = d - 1;
    }
    __syncthreads();
    const int depth = depth_of;
    const bool in = lane * kPer < P.dim;
    float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
    const int64_t at = (row + i) * P.q_stride + (int64_t)h * P.dim + lane * kPer;
    const float ks = (P.k_scale ? P.k_scale[kh] : 1.f) * P.scale, vs = P.v_scale ? P.v_scale[kh] : 1.f;
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        o[j] = 0.f;
        q[j] = !in ? 0.f
               : P.act == COLI_ACT_F32 ? ((const float *)P.q)[at + j]
               : P.act == COLI_ACT_BF16 ? to_f32(((const __nv_bfloat16 *)P.q)[at + j])
                                        : to_f32(((const __half *)P.q)[at + j]);
    }
    const int32_t *pages = P.table + (int64_t)b * P.table_width;
    for (int64_t t = (int64_t)draft_start(past, P.window) + w; t < (int64_t)past + n; t += kWarps) {
        const int j = (int)(t - past);
        if (t >= past ? !(line[j / 32] >> j % 32 & 1) : !draft_sees(past, depth, P.window, (int)t)) continue;
        int bad;
        const int64_t off = kv_row(P.cache, pages, P.table_width, (int)t, kh, bad);
        if (bad) {
            if (lane == 0 && P.err) atomicOr(P.err, COLI_LAYER_BAD_PAGE);
            continue;
        }
        Run<C, kPer> k, v;
        float s = 0.f;
        if (in) {
            k.load((const C *)P.k_cache + off + lane * kPer);
            v.load((const C *)P.v_cache + off + lane * kPer);
#pragma unroll
            for (int e = 0; e < kPer; e++) s = fmaf(q[e], to_f32(k.e[e]), s);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= ks;
        const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - top), p = expf(s - top);
        m = top;
        l = fmaf(l, f, p);
        if (in)
#pragma unroll
            for (int e = 0; e < kPer; e++) o[e] = fmaf(o[e], f, p * to_f32(v.e[e]));
    }
    if (in)
#pragma unroll
        for (int e = 0; e < kPer; e++) red[w][lane * kPer + e] = o[e];
    if (lane == 0) red_m[w] = m, red_l[w] = l;
    __syncthreads();
    float top = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
    for (int k = 0; k < kWarps; k++) top = fmaxf(top, red_m[k]);
#pragma unroll
    for (int k = 0; k < kWarps; k++) {
        f[k] = red_m[k] == -INFINITY ? 0.f : expf(red_m[k] - top);
        sum = fmaf(red_l[k], f[k], sum);
    }
    for (int d = threadIdx.x; d < P.dim; d += kWarps * 32) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; k++) v = fmaf(red[k][d], f[k], v);
        store_act(P.out, (row + i) * P.out_stride + (int64_t)h * P.dim + d, sum == 0.f ? 0.f : v / sum * vs, P.act);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[(int64_t)(row + i) * P.q_heads + h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

size_t tree_workspace_bytes(const TreeParams &P) { return 256; }

cudaError_t launch_attn_tree(const TreeParams &P, cudaStream_t s) {
    const dim3 grid((unsigned)P.seqs * P.nodes, P.q_heads);
    switch (P.fmt) {
    case COLI_KV_BF16: return launch_overlapped(attn_tree_kernel<__nv_bfloat16>, grid, kWarps * 32, 0, s, P);
    case COLI_KV_F16: return launch_overlapped(attn_tree_kernel<__half>, grid, kWarps * 32, 0, s, P);
    default: return launch_overlapped(attn_tree_kernel<__nv_fp8_e4m3>, grid, kWarps * 32, 0, s, P);
    }
}

}  // namespace colimoe
