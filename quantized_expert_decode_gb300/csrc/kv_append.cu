// kv_append.cu — new tokens' queries and keys rotated by their positions, keys and values written
// to the paged cache, in one launch.
//
// Mathematics: append.cuh has the angles and the rounding to the cache's type.
//
// What bounds it: bytes, each read and written once. A CTA owns a few tokens; its threads compute
// the tokens' cosines and sines once into shared memory and then walk all heads of q, k and v of
// those tokens, so that the angle work is shared by the heads. Every thread has several items' loads
// on their way before it touches the first, the first of them before the angles are computed.
#include "append.cuh"
#include "host.h"
#include "layer.h"
#include "pdl.cuh"

namespace colimoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;                // tokens of a CTA
constexpr int kFewRounds = 8, kCtasPerSm = 3;
constexpr int kMaxPairs = 128;               // rotary / 2 at most (dim <= 256)

// One item: 2 * V elements of one head of one token. Items below rotary / (2 V) rotate V pairs: V
// elements at i * V and V at rotary / 2 + i * V, or, interleaved, 2 V elements at i * 2 V. The rest
// copy 2 V elements. A thread keeps its item number within the rows and walks over rows, kBatch at a time.
template <typename A, typename C, int V>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams P, int tokens_per_cta,
                                                             int heads_per_cta) {
    constexpr int kBatch = V == 1 ? 2 : 32 / (V * (int)sizeof(A));  // 64 bytes
    __shared__ float2 cs[kMaxTokens * kMaxPairs];
    __shared__ long long row_k[kMaxTokens];  // offset of the token's row of kv head 0, or -1
    wait_for_previous();
    let_next_start();
    const int n0 = blockIdx.x * tokens_per_cta;
    const int nt = min(tokens_per_cta, P.tokens - n0);
    const int half = P.rotary / 2;
    const int per_row = P.dim / (2 * V), turned = half / V;
    const int h0 = blockIdx.y * heads_per_cta;
    const int heads = min(heads_per_cta, P.q_heads + 2 * P.kv_heads - h0);
    const int step = kThreads / per_row;  // rows that the CTA takes at once
    const int c = threadIdx.x % per_row;
    // two runs of V elements at o0, o1; adjacent unless the item rotates halves
    const bool in_turn = c < turned, split = in_turn && !P.interleaved;
    const int s0 = split ? c * V : c * 2 * V, s1 = split ? half + c * V : c * 2 * V + V;
    const int v0 = c * 2 * V, v1 = v0 + V;  // of a value
    // the thread's next row: token t, head h of the CTA's
    int t = 0, h = threadIdx.x / per_row;
    if (h >= step) t = nt;  // threads beyond whole rows
    auto settle = [&]() {
        while (h >= heads && t < nt) {
            h -= heads;
            t++;
        }
    };
    settle();
    struct Item {
        int t, h;  // t < 0: none; h counts q heads, k heads, v heads
        Run<A, V> a, b;
        float scale;
    };
    Item item[kBatch];
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            Item &x = item[i];
            x.t = t < nt ? t : -1;
            x.h = h0 + h;
            if (t < nt) {
                const int64_t n = n0 + t;
                const int kh = x.h - P.q_heads, vh = kh - P.kv_heads;
                const A *src = kh < 0   ? (const A *)P.q + n * P.q_stride + (int64_t)x.h * P.dim
                               : vh < 0 ? (const A *)P.k + n * P.k_stride + (int64_t)kh * P.dim
                                        : (const A *)P.v + n * P.v_stride + (int64_t)vh * P.dim;
                x.a.load(src + (vh < 0 ? s0 : v0));
                x.b.load(src + (vh < 0 ? s1 : v1));
                const float *sc = kh < 0 ? nullptr : vh < 0 ? P.k_scale : P.v_scale;
                x.scale = sizeof(C) == 1 && sc ? sc[vh < 0 ? kh : vh] : 1.f;
                h += step;
                settle();
            }
        }
    };
    fetch();
    if (threadIdx.x < nt) {
        const int n = n0 + threadIdx.x;
        const int b = P.seq ? P.seq[n] : n;
        const int p = P.pos[n];
        long long off = -1;
        int flag = 0;
        if (b >= 0 && b < P.seqs) {
            int why;
            off = kv_row(P.cache, P.table + (int64_t)b * P.table_width, P.table_width, p, 0, why);
            flag = why == kKvBadPage ? COLI_LAYER_BAD_PAGE : why == kKvBadPosition ? COLI_LAYER_BAD_POSITION : 0;
        } else if (b != -1) {
            flag = COLI_LAYER_BAD_SEQUENCE;
        }
        row_k[threadIdx.x] = off;
        if (flag && P.err) atomicOr(P.err, flag);
    }
    // pair c * V + j of a token at [j][c]: neighbouring threads read neighbouring words
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int u = i / half, j = i - u * half;
        cs[u * half + j % V * turned + j / V] = turn(P.pos[n0 + u], P.inv_freq[j]);
    }
    __syncthreads();
    while (item[0].t >= 0) {
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            Item &it = item[i];
            if (it.t < 0) continue;
            const int kh = it.h - P.q_heads, vh = kh - P.kv_heads;
            float x[V], y[V];
#pragma unroll
            for (int j = 0; j < V; j++) {
                x[j] = to_f32(it.a.e[j]);
                y[j] = to_f32(it.b.e[j]);
            }
            if (vh < 0 && in_turn) {
                const float2 *w = cs + it.t * half + c;
                if (split) {
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        const float2 e = w[j * turned];
                        const float u = x[j], v = y[j];
                        x[j] = fmaf(u, e.x, -(v * e.y));
                        y[j] = fmaf(v, e.x, u * e.y);
                    }
                } else {
                    // the 2 V elements x, y hold V adjacent pairs
                    float z[2 * V];
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        z[j] = x[j];
                        z[V + j] = y[j];
                    }
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        const float2 e = w[j * turned];
                        const float u = z[2 * j], v = z[2 * j + 1];
                        z[2 * j] = fmaf(u, e.x, -(v * e.y));
                        z[2 * j + 1] = fmaf(v, e.x, u * e.y);
                    }
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        x[j] = z[j];
                        y[j] = z[V + j];
                    }
                }
            }
            if (kh < 0) {
                A *dst = (A *)P.q_out + (int64_t)(n0 + it.t) * P.q_out_stride + (int64_t)it.h * P.dim;
                Run<A, V> a, b;
#pragma unroll
                for (int j = 0; j < V; j++) {
                    a.e[j] = from_f32<A>(x[j]);
                    b.e[j] = from_f32<A>(y[j]);
                }
                a.store(dst + s0);
                b.store(dst + s1);
            } else if (row_k[it.t] >= 0) {
                const int g = vh < 0 ? kh : vh;
                const Divisor by(it.scale);
                C *dst = (C *)(vh < 0 ? P.k_cache : P.v_cache) + row_k[it.t] + (int64_t)g * P.cache.head_stride;
                Run<C, V> a, b;
                to_cache(a.e, x, by);
                to_cache(b.e, y, by);
                a.store(dst + (vh < 0 ? s0 : v0));
                b.store(dst + (vh < 0 ? s1 : v1));
            }
        }
        fetch();
    }
}

template <typename A, typename C>
cudaError_t launch_typed(const AppendParams &P, cudaStream_t s) {
    // widest run that the rotated part, the rest, and the rows' alignment allow (the cache's rows
    // are 16-byte aligned with strides of 16 bytes, which the entry point has checked)
    const int half = P.rotary / 2, rest = P.dim - P.rotary;
    auto fits = [&](int v) {
        const int sz = (int)sizeof(A);
        return half % v == 0 && rest % (2 * v) == 0 && (!P.q_heads || (multiple(P.q, P.q_stride, sz, v) && multiple(P.q_out, P.q_out_stride, sz, v))) &&
               multiple(P.k, P.k_stride, sz, v) && multiple(P.v, P.v_stride, sz, v);
    };
    const int rows = P.q_heads + 2 * P.kv_heads;
    const int v = fits(8) ? 8 : fits(4) ? 4 : 1;
    const int step = kThreads / (P.dim / (2 * v));
    // few rows: one round of a CTA's threads each, for latency; many: whole tokens, several per CTA where
    // that still leaves some CTAs for every SM
    const bool few = (int64_t)P.tokens * rows <= (int64_t)step * kFewRounds * num_sms();
    int tp = 1;
    while (tp < kMaxTokens && (P.tokens + 2 * tp - 1) / (2 * tp) >= kCtasPerSm * num_sms()) tp *= 2;
    const int hp = few ? step : rows;
    const dim3 grid((P.tokens + tp - 1) / tp, (rows + hp - 1) / hp);
    if (v == 8) return launch_overlapped(kv_append_kernel<A, C, 8>, grid, kThreads, 0, s, P, tp, hp);
    if (v == 4) return launch_overlapped(kv_append_kernel<A, C, 4>, grid, kThreads, 0, s, P, tp, hp);
    return launch_overlapped(kv_append_kernel<A, C, 1>, grid, kThreads, 0, s, P, tp, hp);
}

template <typename A>
cudaError_t launch_act(const AppendParams &P, cudaStream_t s) {
    switch (P.fmt) {
    case COLI_KV_BF16: return launch_typed<A, __nv_bfloat16>(P, s);
    case COLI_KV_F16: return launch_typed<A, __half>(P, s);
    default: return launch_typed<A, __nv_fp8_e4m3>(P, s);
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &P, cudaStream_t s) {
    switch (P.act) {
    case COLI_ACT_F32: return launch_act<float>(P, s);
    case COLI_ACT_BF16: return launch_act<__nv_bfloat16>(P, s);
    default: return launch_act<__half>(P, s);
    }
}

}  // namespace colimoe
