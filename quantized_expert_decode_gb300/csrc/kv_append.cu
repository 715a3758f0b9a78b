// kv_append.cu — new tokens' queries and keys rotated by their positions, keys and values written
// to the paged cache, in one launch.
//
// Mathematics. Pair i of a head turns by p * inv_freq[i]. In units of a full turn that is
// p * (inv_freq[i] / 2 pi), and only its fraction counts. fp32 has no fraction left at far
// positions, so inv_freq / 2 pi is taken as a 64-bit fixed-point fraction of a turn (the 24-bit
// mantissa times 64 bits of 1 / 2 pi) and the product with the integer p wraps modulo one turn by
// itself: off by p * 2^-64 turns. sincospi then takes the fraction as a float.
//
// What bounds it: bytes, each read and written once. A CTA owns a few tokens; its threads compute
// the tokens' cosines and sines once into shared memory and then walk all heads of q, k and v of
// those tokens, so that the angle work is shared by the heads. Every thread has several items' loads
// on their way before it touches the first, the first of them before the angles are computed.
#include "act.cuh"
#include "host.h"
#include "layer.h"
#include "pdl.cuh"

namespace colimoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;                // tokens of a CTA
constexpr int kFewRounds = 8, kCtasPerSm = 3;
constexpr int kMaxPairs = 128;               // rotary / 2 at most (dim <= 256)

// f / 2 pi as a fraction of a turn in units of 2^-64, modulo one turn
__device__ __forceinline__ unsigned long long turns_per_step(float f) {
    constexpr unsigned long long kR = 0xa2f9836e4e441529ull;  // 2^66 / 2 pi
    const unsigned bits = __float_as_uint(f), e = (bits >> 23) & 0xff;
    const unsigned long long m = e ? (bits & 0x7fffff) | 0x800000 : 0;  // f = m * 2^(e - 150); below 2^-126: 0
    const unsigned long long hi = __umul64hi(m, kR), lo = m * kR;
    const int s = 152 - (int)e;
    unsigned long long c;
    if (s >= 128) c = 0;
    else if (s >= 64) c = hi >> (s - 64);
    else if (s > 0) c = (hi << (64 - s)) | (lo >> s);
    else c = s > -64 ? lo << -s : 0;
    return (bits >> 31) ? 0ull - c : c;
}

__device__ __forceinline__ float2 turn(int p, float f) {
    const long long t = (long long)((unsigned long long)(long long)p * turns_per_step(f));
    float s, c;
    sincospif((float)t * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    if (!isfinite(f)) s = c = __int_as_float(0x7fffffff);
    return make_float2(c, s);
}

// Division by an e4m3 scale: 1 / scale = r + rest, with r the largest float that is no larger in size, so that
// x * rest + x * r in one rounding is the quotient rounded to fp32, but for 2^-22 of its last bit. (The product with a
// rounded reciprocal puts some values next to a border between two e4m3 values on its other side.) r and rest have one
// sign and neither is 0, so infinities stay infinite. Scales far from 1, whose reciprocal would leave fp32's range, are
// brought nearer by a power of two, and x with them. Two packed instructions for two values, as many as the product
// alone took: 16,411 tokens of 64 + 2 x 8 bf16 heads 103.5 us against 105, 2048 of 32 + 2 x 32 heads 18.1 against 16.9
// (there each item's r and rest count); the plain division 105.7 and 21.8.
struct Divisor {
    float r, rest, shift;
    __device__ __forceinline__ explicit Divisor(float scale) {
        shift = fabsf(scale) < 0x1p-60f ? 0x1p100f : fabsf(scale) > 0x1p60f ? 0x1p-100f : 1.f;
        const float s = scale * shift;
        r = 1.f / s;
        float left = fmaf(-s, r, 1.f);
        if (left < 0.f) {
            r = __uint_as_float(__float_as_uint(r) - 1);
            left = fmaf(-s, r, 1.f);
        }
        rest = left > 0.f ? left * r : r * 0x1p-60f;
    }
};

// N values in the cache's type; e4m3 holds value / scale and is converted in pairs
template <typename C, int N>
__device__ __forceinline__ void to_cache(C (&to)[N], const float (&x)[N], const Divisor &by) {
#pragma unroll
    for (int j = 0; j < N; j++) to[j] = from_f32<C>(x[j]);
}
template <int N>
__device__ __forceinline__ void to_cache(__nv_fp8_e4m3 (&to)[N], const float (&v)[N], const Divisor &by) {
    float x[N];
#pragma unroll
    for (int j = 0; j < N; j++) x[j] = v[j];
    if (by.shift != 1.f) {
#pragma unroll
        for (int j = 0; j < N; j++) x[j] *= by.shift;
    }
    if constexpr (N % 2 == 0) {
        const float2 r = make_float2(by.r, by.r), rest = make_float2(by.rest, by.rest);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 a = make_float2(x[j], x[j + 1]);
            const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(__ffma2_rn(a, r, __fmul2_rn(a, rest)), __NV_SATFINITE, __NV_E4M3);
            to[j].__x = (__nv_fp8_storage_t)p;
            to[j + 1].__x = (__nv_fp8_storage_t)(p >> 8);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) to[j] = from_f32<__nv_fp8_e4m3>(fmaf(x[j], by.r, x[j] * by.rest));
    }
}

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

bool multiple(const void *p, int64_t stride, int act_bytes, int run) {
    const int64_t bytes = (int64_t)run * act_bytes;
    const int64_t a = bytes % 16 == 0 ? 16 : bytes;
    return reinterpret_cast<uintptr_t>(p) % a == 0 && (stride * act_bytes) % a == 0;
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
