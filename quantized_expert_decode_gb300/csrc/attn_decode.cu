// attn_decode.cu — attention of one new token per sequence over a paged cache.
//
// Mathematics: s_t = scale * q . k_t, p = softmax(s), out = sum_t p_t v_t, with a running maximum m
// and sum l: a later score above m scales what is summed so far by exp(m - m').
//
// One CTA per (sequence, query head); each warp takes every fourth token, its lanes share the
// head's elements, and the four warps' (m, l, sum) are joined in shared memory.
#include "act.cuh"
#include "layer.h"

namespace colimoe {
namespace {

constexpr int kWarps = 4;

template <typename A, typename C>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(const AttnParams P) {
    const int h = blockIdx.x, b = blockIdx.y, w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int kh = h / (P.q_heads / P.kv_heads);
    int first, end, why;
    kv_span(P.lens[b], P.table_width, P.cache.page_size, P.window, first, end, why);
    if (why && threadIdx.x == 0 && P.err) atomicOr(P.err, COLI_LAYER_BAD_POSITION);
    float q[8], o[8];
    const float ks = P.scale * (P.k_scale ? P.k_scale[kh] : 1.f);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int d = lane + 32 * j;
        q[j] = d < P.dim ? to_f32(((const A *)P.q)[b * P.q_stride + (int64_t)h * P.dim + d]) : 0.f;
        o[j] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int t = first + w; t < end; t += kWarps) {
        const int64_t off = kv_row(P.cache, P.table + (int64_t)b * P.table_width, P.table_width, t, kh, why);
        if (off < 0) {
            if (lane == 0 && P.err) atomicOr(P.err, COLI_LAYER_BAD_PAGE);
            continue;
        }
        const C *k = (const C *)P.k_cache + off, *v = (const C *)P.v_cache + off;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (lane + 32 * j < P.dim) s = fmaf(q[j], to_f32(k[lane + 32 * j]), s);
#pragma unroll
        for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        s *= ks;
        const float n = fmaxf(m, s), f = n == -INFINITY ? 0.f : expf(m - n), p = n == -INFINITY ? 0.f : expf(s - n);
        m = n;
        l = fmaf(l, f, p);
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (lane + 32 * j < P.dim) o[j] = fmaf(o[j], f, p * to_f32(v[lane + 32 * j]));
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
    if (lane == 0) {
        sm[w] = m;
        sl[w] = l;
    }
#pragma unroll
    for (int j = 0; j < 8; j++) so[w][lane + 32 * j] = o[j];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int i = 0; i < kWarps; i++) top = fmaxf(top, sm[i]);
    for (int i = 0; i < kWarps; i++) sum += sm[i] == -INFINITY ? 0.f : sl[i] * expf(sm[i] - top);
    const float vs = P.v_scale ? P.v_scale[kh] : 1.f;
    for (int d = threadIdx.x; d < P.dim; d += kWarps * 32) {
        float x = 0.f;
        for (int i = 0; i < kWarps; i++) x += sm[i] == -INFINITY ? 0.f : so[i][d] * expf(sm[i] - top);
        ((A *)P.out)[b * P.out_stride + (int64_t)h * P.dim + d] = from_f32<A>(sum == 0.f ? 0.f : x / sum * vs);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[(int64_t)b * P.q_heads + h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <typename A>
void launch_act(const AttnParams &P, cudaStream_t s) {
    const dim3 grid(P.q_heads, P.seqs);
    switch (P.fmt) {
    case COLI_KV_BF16: attn_decode_kernel<A, __nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(P); break;
    case COLI_KV_F16: attn_decode_kernel<A, __half><<<grid, kWarps * 32, 0, s>>>(P); break;
    default: attn_decode_kernel<A, __nv_fp8_e4m3><<<grid, kWarps * 32, 0, s>>>(P); break;
    }
}

}  // namespace

size_t attn_workspace_bytes(const AttnParams &P) { return 256; }

cudaError_t launch_attn_decode(const AttnParams &P, cudaStream_t s) {
    switch (P.act) {
    case COLI_ACT_F32: launch_act<float>(P, s); break;
    case COLI_ACT_BF16: launch_act<__nv_bfloat16>(P, s); break;
    default: launch_act<__half>(P, s); break;
    }
    return cudaGetLastError();
}

}  // namespace colimoe
