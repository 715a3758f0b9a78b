// norm_append.cu — new tokens' queries and keys normalised per head and rotated by their positions, keys and values
// written to places of the paged cache, in one launch.
//
// Mathematics: x' = x * w / sqrt(mean x^2 + eps) over a head's elements, then the rotation (append.cuh). A head's row lies
// on a power of two of neighbouring lanes, which sum its squares by shuffles, so that the norm costs no exchange through
// shared memory and the row is read once.
//
// What bounds it: bytes, each read and written once; for a few sequences' nodes the launch and one round of loads.
// A CTA owns a few tokens; its threads compute the tokens' cosines and sines once into shared memory, the loads of
// the first rows on their way before that, and walk all heads of q, k and v of those tokens.
#include <type_traits>

#include "append.cuh"
#include "draft.h"
#include "host.h"
#include "pdl.cuh"

namespace colimoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of a CTA
constexpr int kFewRounds = 8, kCtasPerSm = 3;
constexpr int kMaxPairs = 128;  // rotary / 2 at most (dim <= 256)

// A row's items are 2 * V elements each: those below rotary / (2 V) rotate V pairs (V elements at i * V and V at
// rotary / 2 + i * V, or, interleaved, 2 V elements at i * 2 V), the rest hold 2 V adjacent elements. A lane has kN
// items, the row's `lanes` lanes a power of two. Which elements make a pair is known at compile time: 32 sequences' trees of
// 32 to 64 nodes, 48 + 2 x 8 bf16 heads to e4m3, 19.0 us against 19.9.
template <typename A, typename C, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_append_kernel(const NormAppendParams N, int tokens_per_cta, int heads_per_cta,
                                                               int lanes) {
    constexpr int kN = V == 1 ? 4 : 1;
    constexpr int kBatch = V == 1 ? 1 : 32 / (V * (int)sizeof(A));  // 64 bytes
    const AppendParams &P = N.a;
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
    const int step = kThreads / lanes, c = threadIdx.x % lanes, mine = threadIdx.x / lanes;
    // the two runs of V elements of an item, adjacent unless the item rotates halves
    auto place0 = [&](int i, bool apart) { return apart ? i * V : i * 2 * V; };
    auto place1 = [&](int i, bool apart) { return apart ? half + i * V : i * 2 * V + V; };
    struct Item {
        int t, h;  // t < 0: none; h counts q heads, k heads, v heads
        Run<A, V> a[kN], b[kN];
        float scale;
    };
    Item item[kBatch];
    const int total = nt * heads;
    auto fetch = [&](int from) {
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            Item &x = item[k];
            const int r = from + k * step + mine;
            x.t = -1;
            x.scale = 1.f;
            if (r >= total) continue;
            x.t = r / heads;
            x.h = h0 + r - x.t * heads;
            const int64_t n = n0 + x.t;
            const int kh = x.h - P.q_heads, vh = kh - P.kv_heads;
            const A *src = kh < 0   ? (const A *)P.q + n * P.q_stride + (int64_t)x.h * P.dim
                           : vh < 0 ? (const A *)P.k + n * P.k_stride + (int64_t)kh * P.dim
                                    : (const A *)P.v + n * P.v_stride + (int64_t)vh * P.dim;
#pragma unroll
            for (int j = 0; j < kN; j++) {
                const int i = c + j * lanes;
                if (i >= per_row) continue;
                const bool apart = !INTER && vh < 0 && i < turned;
                x.a[j].load(src + place0(i, apart));
                x.b[j].load(src + place1(i, apart));
            }
            const float *sc = kh < 0 ? nullptr : vh < 0 ? P.k_scale : P.v_scale;
            if (sizeof(C) == 1 && sc) x.scale = sc[vh < 0 ? kh : vh];
        }
    };
    fetch(0);
    if (threadIdx.x < nt) {
        const int n = n0 + threadIdx.x;
        const int b = P.seq ? P.seq[n] : n;
        const int p = N.place ? N.place[n] : P.pos[n];
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
    for (int from = 0; from < total; from += step * kBatch) {
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const Item &it = item[k];
            const bool real = it.t >= 0;
            const int kh = it.h - P.q_heads, vh = kh - P.kv_heads;
            const float *w = !real ? nullptr : kh < 0 ? N.q_norm : vh < 0 ? N.k_norm : nullptr;
            float x[kN][V], y[kN][V], ss = 0.f;
#pragma unroll
            for (int j = 0; j < kN; j++) {
                const bool in = real && c + j * lanes < per_row;
#pragma unroll
                for (int e = 0; e < V; e++) {
                    x[j][e] = in ? to_f32(it.a[j].e[e]) : 0.f;
                    y[j][e] = in ? to_f32(it.b[j].e[e]) : 0.f;
                    ss = fmaf(x[j][e], x[j][e], ss);
                    ss = fmaf(y[j][e], y[j][e], ss);
                }
            }
            // (every lane of the warp takes part)
            for (int o = lanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!real) continue;
            const float rs = w ? rsqrtf(ss / (float)P.dim + N.eps) : 1.f;
#pragma unroll
            for (int j = 0; j < kN; j++) {
                const int i = c + j * lanes;
                if (i >= per_row) continue;
                const bool in_turn = vh < 0 && i < turned, apart = !INTER && in_turn;
                const int s0 = place0(i, apart), s1 = place1(i, apart);
                if (w) {
                    Run<float, V> w0, w1;
                    w0.load(w + s0);
                    w1.load(w + s1);
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        x[j][e] *= rs * w0.e[e];
                        y[j][e] *= rs * w1.e[e];
                    }
                }
                if (in_turn) {
                    const float2 *f = cs + it.t * half + i;
                    auto turn_pair = [&](float &u, float &v, float2 r) {
                        const float p = fmaf(u, r.x, -(v * r.y));
                        v = fmaf(v, r.x, u * r.y);
                        u = p;
                    };
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        const float2 r = f[e * turned];
                        if constexpr (INTER && V > 1) {
                            // the 2 V elements x, y hold V adjacent pairs
                            if (e < V / 2) turn_pair(x[j][2 * e], x[j][2 * e + 1], r);
                            else turn_pair(y[j][2 * e - V], y[j][2 * e + 1 - V], r);
                        } else {
                            turn_pair(x[j][e], y[j][e], r);
                        }
                    }
                }
                if (kh < 0) {
                    A *dst = (A *)P.q_out + (int64_t)(n0 + it.t) * P.q_out_stride + (int64_t)it.h * P.dim;
                    Run<A, V> a, b;
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        a.e[e] = from_f32<A>(x[j][e]);
                        b.e[e] = from_f32<A>(y[j][e]);
                    }
                    a.store(dst + s0);
                    b.store(dst + s1);
                } else if (row_k[it.t] >= 0) {
                    const int g = vh < 0 ? kh : vh;
                    const Divisor by(it.scale);
                    C *dst = (C *)(vh < 0 ? P.k_cache : P.v_cache) + row_k[it.t] + (int64_t)g * P.cache.head_stride;
                    Run<C, V> a, b;
                    to_cache(a.e, x[j], by);
                    to_cache(b.e, y[j], by);
                    a.store(dst + s0);
                    b.store(dst + s1);
                }
            }
        }
        fetch(from + step * kBatch);
    }
}

template <typename A, typename C>
cudaError_t launch_typed(const NormAppendParams &N, cudaStream_t s) {
    const AppendParams &P = N.a;
    // widest run that the rotated part, the rest, and the rows' alignment allow (the cache's rows
    // are 16-byte aligned with strides of 16 bytes, which the entry point has checked)
    const int half = P.rotary / 2, rest = P.dim - P.rotary;
    auto fits = [&](int v) {
        const int sz = (int)sizeof(A);
        return half % v == 0 && rest % (2 * v) == 0 &&
               (!P.q_heads || (multiple(P.q, P.q_stride, sz, v) && multiple(P.q_out, P.q_out_stride, sz, v))) &&
               multiple(P.k, P.k_stride, sz, v) && multiple(P.v, P.v_stride, sz, v) && multiple(N.q_norm, 0, 4, v) &&
               multiple(N.k_norm, 0, 4, v);
    };
    const int rows = P.q_heads + 2 * P.kv_heads;
    const int v = fits(8) ? 8 : fits(4) ? 4 : 1;
    int lanes = 1;
    while (lanes < 32 && lanes < P.dim / (2 * v)) lanes *= 2;
    const int step = kThreads / lanes;
    // few rows: one round of a CTA's threads each, for latency; many: whole tokens, several per CTA where
    // that still leaves some CTAs for every SM
    const bool few = (int64_t)P.tokens * rows <= (int64_t)step * kFewRounds * num_sms();
    int tp = 1;
    while (tp < kMaxTokens && (P.tokens + 2 * tp - 1) / (2 * tp) >= kCtasPerSm * num_sms()) tp *= 2;
    const int hp = few ? step : rows;
    const dim3 grid((P.tokens + tp - 1) / tp, (rows + hp - 1) / hp);
    auto launch = [&](auto inter) {
        constexpr bool kInter = decltype(inter)::value;
        if (v == 8) return launch_overlapped(norm_append_kernel<A, C, 8, kInter>, grid, kThreads, 0, s, N, tp, hp, lanes);
        if (v == 4) return launch_overlapped(norm_append_kernel<A, C, 4, kInter>, grid, kThreads, 0, s, N, tp, hp, lanes);
        return launch_overlapped(norm_append_kernel<A, C, 1, kInter>, grid, kThreads, 0, s, N, tp, hp, lanes);
    };
    return P.interleaved ? launch(std::true_type{}) : launch(std::false_type{});
}

template <typename A>
cudaError_t launch_act(const NormAppendParams &N, cudaStream_t s) {
    switch (N.a.fmt) {
    case COLI_KV_BF16: return launch_typed<A, __nv_bfloat16>(N, s);
    case COLI_KV_F16: return launch_typed<A, __half>(N, s);
    default: return launch_typed<A, __nv_fp8_e4m3>(N, s);
    }
}

}  // namespace

cudaError_t launch_norm_append(const NormAppendParams &N, cudaStream_t s) {
    switch (N.a.act) {
    case COLI_ACT_F32: return launch_act<float>(N, s);
    case COLI_ACT_BF16: return launch_act<__nv_bfloat16>(N, s);
    default: return launch_act<__half>(N, s);
    }
}

}  // namespace colimoe
