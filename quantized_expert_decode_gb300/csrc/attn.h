// attn.h — what the streaming and the join kernel of coli_attn_decode share. Internal to libcolimoe.
#pragma once

#include "act.cuh"
#include "layer.h"

namespace colimoe {

constexpr int kAttnMaxSeqs = 2048;

// A slot is K or V of a tile: 16 rows of 256 bytes or more, or 32 shorter ones, 4 KB at 128 elements. Two CTAs
// share an SM, each with three slots per warp there, except where the sums of 16 heads take the
// registers of one, or the three parts of q at 256 elements too much shared memory: that one has as many
// slots as both would (at 256 elements and 16 heads, no room: three).
constexpr bool attn_alone(int fmt, int dim, int nt, bool wide) {
    return (nt == 2 && dim != 64) || (dim == 256 && wide && fmt == COLI_KV_BF16);
}
constexpr int attn_tile(int fmt, int dim) { return dim == 64 || fmt == COLI_KV_E4M3 ? 32 : 16; }
// 16 heads of 128 elements leave 168 registers a lane to 12 warps, which hide more of each other's waiting than 8 with
// 255 (32 sequences of 3051 tokens, 128 query heads on 8: 82.5 -> 77.3 us in bf16; 4000 tokens of 96 elements: 102 -> 92).
// The wide form on e4m3 spills too much there (123 us with 8, 136 with 12).
constexpr bool attn_twelve(int fmt, int dim, int nt, bool wide) {
    return dim == 128 && nt == 2 && !(wide && fmt == COLI_KV_E4M3);
}
constexpr int attn_warps(int fmt, int dim, int nt, bool wide) {
    return attn_twelve(fmt, dim, nt, wide) ? 12 : dim == 256 && nt == 1 ? 4 : 8;
}
constexpr int attn_ctas_per_sm(int fmt, int dim, int nt, bool wide) { return attn_alone(fmt, dim, nt, wide) ? 1 : 2; }
constexpr int attn_slots(int fmt, int dim, int nt, bool wide) {
    return attn_twelve(fmt, dim, nt, wide) ? 4
           : (dim == 64 && fmt == COLI_KV_E4M3) || (attn_alone(fmt, dim, nt, wide) && !(dim == 256 && nt == 2)) ? 6
                                                                                                              : 3;
}
constexpr int attn_unit(int fmt, int dim, int nt, bool wide) {
    return attn_warps(fmt, dim, nt, wide) * attn_tile(fmt, dim);
}

// Whether a CTA per item, none cut, is the faster way for items of u units, with room for `ctas` CTAs at once (the
// others start as those end). Measured on bf16 caches of 128 elements, 8 kv heads, groups of 8 heads (units of 128
// tokens), against runs that go on from item to item, or parts of items, and their join:
//   few short items: 333 tokens of one sequence 8.2 us against 6.8 on the device, but without the second launch
//     8.5 against 10.4 called from Python;
//   a quarter of the places: 16 sequences of 1000 tokens 17 us against 21, 32 of 500 16 against 20;
//   more items than places: 64 sequences of 500 tokens 29 us against 37, of 4000 156 against 171; 16 windows of 1024
//     on 32 heads 23 against 30; but 40 of 2000 (320 items, 304 places) 70 against 62.
// So where items fill the places the time of the waves is estimated, each the larger of its bytes' time and of
// one CTA's alone (1.25 us a unit), against the other way's: its bytes' and 15 us of starts, cuts and join. Items
// of more than 40 us alone (32 units) count only where all are as long: in a ragged batch the last of them would end
// alone (32 sequences of 1 to 8192 tokens 134 us against 95). Up to there ragged items fill the waves' gaps (40 sequences
// of 1 to 2000 tokens 35 us against 47, of 1 to 4000 64 against 72).
//   The 9 to 16 heads of 65 to 128 elements that a CTA takes alone on its SM (`big`, units of 192 to 384 tokens) take
// longer for a unit, and no less beside each other; and cutting short items finds more places free: one sequence of
// 576 bf16 tokens on 8 kv heads 11.7 us whole against 9.7, 5 of 1500 21.8 against 16.6, 8 of 1500 21.8 against 19.2; but
// 12 of 1500 22.0 against 25.9, 5 of 700 13.4 against 14.4; 20 of 3000 e4m3 tokens 58 against 44, in ragged batches 19
// of 1 to 4000 bf16 tokens 52 whole against 72, 16 of 1 to 6000 75 against 66.
constexpr int kAttnWhole = 1, kAttnMaybe = 2;
struct AttnTimes {  // us
    float bytes;  // of a unit's bytes at the memory's full rate
    float alone;  // of a unit on a CTA that has none beside it
    bool big;
    __host__ __device__ bool short_item(int64_t u) const { return (float)u * alone <= (big ? 50.f : 40.f); }
};
inline AttnTimes attn_times(int fmt, int dim, int nt, int unit, int64_t unit_bytes) {
    const bool big = dim == 128 && nt == 2;
    return {(float)unit_bytes / 7.2e6f, !big ? 1.25f : fmt == COLI_KV_E4M3 ? unit / 125.f : unit / 100.f, big};
}
__host__ __device__ inline bool attn_waves(float items, float u, float ctas, AttnTimes t) {
    const float alone = t.alone * u, full = floorf(items / ctas), rest = items - full * ctas;
    const float cut = items * u * (t.big ? fmaxf(t.bytes, t.alone / ctas) : t.bytes);
    return 6.f + full * fmaxf(ctas * u * t.bytes, alone) + (rest > 0.f ? fmaxf(rest * u * t.bytes, alone) : 0.f) < 15.f + 1.06f * cut;
}
__host__ __device__ inline bool attn_whole(int64_t items, int64_t u, int64_t ctas, AttnTimes t) {
    if (items > 16 * ctas) return false;
    if (t.big) {
        if (u <= 2 || (u <= 4 && 4 * items >= ctas) || (u <= 8 && 5 * items >= 3 * ctas && items <= ctas)) return true;
    } else if (u <= 3 || (u <= 8 && 4 * items >= ctas)) {
        return true;
    }
    return t.short_item(u) && 5 * items >= 4 * ctas && attn_waves((float)items, (float)u, (float)ctas, t);
}

// The same by the lengths themselves: `total` units, the longest item's u.
__device__ inline bool attn_whole_now(uint32_t total, int64_t items, int64_t u, int64_t ctas, AttnTimes t) {
    if (attn_whole(items, u, ctas, t)) return true;
    if (items > 16 * ctas || 5 * items < 4 * ctas) return false;
    const float full = (float)total / ((float)items * (float)u);  // 1: all as long
    return full >= 0.9f ? attn_waves((float)items, (float)u, (float)ctas, t) : full < 0.75f && t.short_item(u);
}

// The line of all units is cut into runs of equal length, the first ones one unit longer; one CTA each. (A
// second, shorter run per share as further CTAs, to even out the 20 % by which the SMs' bandwidths differ,
// costs as much in starts as it evens out.)
struct AttnRuns {
    uint32_t runs, each, more;  // `more` runs of each + 1 units
    __device__ __forceinline__ AttnRuns(uint32_t total, uint32_t ctas) {
        runs = total < ctas ? total : ctas;
        each = runs ? total / runs : 0;
        more = total - each * runs;
    }
    __device__ __forceinline__ uint32_t start(uint32_t r) const { return r * each + (r < more ? r : more); }
    __device__ __forceinline__ uint32_t of(uint32_t x) const {  // the run that unit x lies in
        const uint32_t y = more * (each + 1);
        return x < y ? x / (each + 1) : more + (x - y) / each;
    }
};

// The item whose units the border before a run cuts, told for its first cut only (b < 0: none): its sequence,
// head group and last run. The first entry tells how many runs there are.
struct AttnCut {
    int32_t b, hv, last, runs;
};

// How the launch is laid out, and the workspace
struct AttnWork {
    int32_t dim;     // head size rounded up: 64, 128 or 256
    int32_t use;     // of which the products take: dim, or 96 of 128
    int32_t nt;      // query heads of a CTA / 8
    int32_t wide;    // more parts of q and p
    int32_t chunks;  // head groups per kv head
    int32_t groups;  // head groups per sequence
    int32_t unit;    // tokens of a unit
    int32_t whole;   // kAttnWhole: no item is cut; kAttnMaybe: by the lengths; 0: items may be cut
    int32_t ctas;    // CTAs that share the units where items may be cut
    AttnTimes times;
    KvDivide divide;  // by the page size
    // the cache's strides in steps of 2^off_shift bytes, which divides them all
    uint32_t page_step, token_step, head_step, off_shift;
    AttnCut *cuts;   // [runs] at the border before a run
    float2 *part_ml; // [2 * runs][8 * nt] (m, l) of a run's first and last cut item
    float *part_o;   // [2 * runs][8 * nt][dim]
};

__device__ __forceinline__ void store_act(void *p, int64_t i, float x, int act) {
    if (act == COLI_ACT_F32) ((float *)p)[i] = x;
    else if (act == COLI_ACT_BF16) ((__nv_bfloat16 *)p)[i] = from_f32<__nv_bfloat16>(x);
    else ((__half *)p)[i] = from_f32<__half>(x);
}

// ln sum of exp(scores) from m and l = sum * 2^shift, both to base 2
__device__ __forceinline__ float attn_lse(float m, float l, int shift) {
    return l == 0.f ? -INFINITY : (m - (float)shift + log2f(l)) * 0.6931471805599453f;
}

cudaError_t launch_attn_bf16(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s);
cudaError_t launch_attn_f16(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s);
cudaError_t launch_attn_e4m3(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s);

// Whether 32 bits reach every row of the pool in steps of the strides' largest common power of two; then
// that step's shift.
bool attn_steps(const KvShape &c, int heads, int elem_bytes, uint32_t &shift);

}  // namespace colimoe
