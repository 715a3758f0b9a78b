// attn.h — what the streaming and the join kernel of coli_attn_decode share. Internal to libcolimoe.
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "layer.h"

namespace colimoe {

constexpr int kAttnMaxSeqs = 2048;
constexpr int kAttnStages = 3;

// A stage is 64 bytes per head element and warp (K and V, 16 tokens of 2 bytes or 32 of 1), so three
// stages of eight warps fill the SM's shared memory at 128 elements; two such CTAs fit at 64, four
// warps at 256.
constexpr int attn_warps(int dim) { return dim == 256 ? 4 : 8; }
constexpr int attn_ctas_per_sm(int dim) { return dim == 64 ? 2 : 1; }
constexpr int attn_unit(int fmt, int dim) { return attn_warps(dim) * (fmt == COLI_KV_E4M3 ? 32 : 16); }

// How the launch is laid out, and the workspace
struct AttnWork {
    int32_t dim;     // head size rounded up: 64, 128 or 256
    int32_t nt;      // query heads of a CTA / 8
    int32_t wide;    // more parts of q and p
    int32_t chunks;  // head groups per kv head
    int32_t groups;  // head groups per sequence
    int32_t unit;    // tokens of a unit
    int32_t box_rows;    // K and V come as boxes of so many tokens through tensor maps; 0: row by row
    int32_t whole_rows;  // a box holds whole rows, not one span of 128 bytes
    KvDivide divide;     // by the page size
    int32_t mask;        // tiles begin at tokens that are 0 under it
    int32_t *prefix; // [seqs + 1] units (per head group) before each sequence
    float2 *part_ml; // [2 * CTAs][8 * nt] (m, l) of a run's first and last cut item
    float *part_o;   // [2 * CTAs][8 * nt][dim]
};

// first unit of run c of n on a line of `total` units
__host__ __device__ __forceinline__ int64_t attn_run_start(int64_t c, int64_t total, int64_t n) { return c * total / n; }
// the run that unit x lies in: the last c with attn_run_start(c) <= x
__host__ __device__ __forceinline__ int64_t attn_run_of(int64_t x, int64_t total, int64_t n) { return ((x + 1) * n - 1) / total; }

__device__ __forceinline__ void store_act(void *p, int64_t i, float x, int act) {
    if (act == COLI_ACT_F32) ((float *)p)[i] = x;
    else if (act == COLI_ACT_BF16) ((__nv_bfloat16 *)p)[i] = from_f32<__nv_bfloat16>(x);
    else ((__half *)p)[i] = from_f32<__half>(x);
}

// ln sum of exp(scores) from m and l = sum * 2^shift, both to base 2
__device__ __forceinline__ float attn_lse(float m, float l, int shift) {
    return l == 0.f ? -INFINITY : (m - (float)shift + log2f(l)) * 0.6931471805599453f;
}

// tensor maps of K and V: (element of a span, slot, span, head, page)
struct AttnMaps {
    CUtensorMap k, v;
};

cudaError_t launch_attn_bf16(const AttnParams &P, const AttnWork &W, const AttnMaps &M, int grid, cudaStream_t s);
cudaError_t launch_attn_f16(const AttnParams &P, const AttnWork &W, const AttnMaps &M, int grid, cudaStream_t s);
cudaError_t launch_attn_e4m3(const AttnParams &P, const AttnWork &W, const AttnMaps &M, int grid, cudaStream_t s);

}  // namespace colimoe
