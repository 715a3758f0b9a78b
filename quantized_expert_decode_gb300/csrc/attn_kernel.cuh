// attn_kernel.cuh — the streaming kernel of coli_attn_decode. Internal to libcolimoe; instantiated
// per cache type by attn_bf16.cu, attn_f16.cu and attn_e4m3.cu.
//
// Mathematics. With x_t = scale * log2(e) * q . k_t a running integer m >= max x_t is kept (the
// maximum rounded up), l = sum 2^(x_t - m) and o = sum 2^(x_t - m) v_t. A later, larger m' scales l
// and o by 2^(m - m'), which is exact because both are integers; so is every later join of parts.
//
// What bounds it: the bytes of K and V, read once for all query heads of a kv head up to 16 (4 * heads
// operations per pair of K and V elements: far below the tensor cores' rate). 64 sequences of 8000 tokens
// on 8 kv heads of 128 bf16 elements (2.1 GB) take 306 us, 6.9 TB/s; ragged and middling batches (0.2 to 0.6
// GB) reach 65 to 90 % of the copy's 6.8 TB/s: a start of some 4 us (launch, plan, page numbers, first rows), the
// spread of the SMs' bandwidths by 20 % and the join's 3 us are the rest. The instructions of a tile
// (about 350 for 16 tokens of 128 bf16 elements, 600 beside fp32 queries, 700 for 32 e4m3 tokens) keep an SM's
// issue slots 40 to 55 % busy; e4m3 and 16 heads come near being bound by them.
//
// Work. An item is the cached tokens of a (sequence, kv head, group of query heads), cut into units of
// kWarps tiles of kTile tokens. attn_whole() says when a CTA takes a whole item; otherwise every item is cut
// into parts by itself where that gives equal parts for all CTAs, or all units form one line that is cut into
// equal runs, one per CTA, so that a CTA's share does not depend on how the lengths are spread. An item
// that is cut leaves partial sums in the workspace, which the join kernel adds up in a fixed order. (The last
// CTA to end adding them up in this kernel takes registers from its loop: 107 us against 88 for one sequence of
// 131071 tokens. Rows by tensor copies, boxes of 8 to 32 tokens, were 4 to 8 % slower than 16-byte copies.)
//
// Within a unit each warp owns one tile: it copies the tile's K rows and V rows to its own ring of kSlots
// slots with 16-byte asynchronous copies, K and V of a tile apart, so that a slot is copied into as
// soon as its half is used up, and no warp waits for another until the item ends. Page numbers are
// loaded one tile ahead of the copies that need them.
//
// Products. Tokens are the rows of the matrix instruction and the query heads its 8 columns, so a
// group of up to 8 heads fills it: S^T [16 tokens x 8 heads] = K q^T, then O^T [16 dims x 8 heads] +=
// V^T P^T, where P^T comes from S^T's registers by an 8x8 transposition. K and V enter in the cache's
// own type (e4m3 widened to f16, exactly). q and p are sums of parts in that type: a bf16 or f16 q
// that the type holds is one part; an fp32 q is three bf16 parts or two f16 parts (scaled by a power of
// two per head); p is two parts, or three in bf16 beside an fp32 q (two bf16 parts leave 2^-17 of p, against the
// 2^-9 or 2^-12 of the 16-bit output they are for; l is summed from p before it is split). Each tile's O is summed
// from zero and added in fp32, so that the matrix unit's truncating accumulation never runs over more than a tile.
#pragma once

#include <atomic>

#include "act.cuh"
#include "attn.h"
#include "attn_parts.cuh"
#include "pdl.cuh"
#include "ptx.cuh"  // smem_u32

namespace colimoe {

namespace attn {

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// d = a b (+ d)
template <int FMT, bool ADD>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    const float c0 = ADD ? d[0] : 0.f, c1 = ADD ? d[1] : 0.f, c2 = ADD ? d[2] : 0.f, c3 = ADD ? d[3] : 0.f;
    if (FMT == COLI_KV_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void add_scaled(float4 &x, const float4 &y, float f) {
    x.x = fmaf(y.x, f, x.x);
    x.y = fmaf(y.y, f, x.y);
    x.z = fmaf(y.z, f, x.z);
    x.w = fmaf(y.w, f, x.w);
}

// a place on the line of units
struct Cursor {
    int b, hv, u, units;  // sequence, head group, unit of the item, units of the item
};

}  // namespace attn

// FMT the cache type, DP the head size rounded up to 64, 128 or 256, USE the elements of it that the products
// take (96 of 128 for heads of up to 96), NT groups of 8 query heads per CTA,
// WIDE: q (and p in bf16) in more parts
template <int FMT, int DP, int USE, int NT, bool WIDE>
struct AttnTraits {
    static constexpr int kFmt = FMT, kDim = DP, kNT = NT;
    static constexpr int kSize = FMT == COLI_KV_E4M3 ? 1 : 2;
    static constexpr int kRow = DP * kSize;                       // bytes of a row in shared memory
    static constexpr int kTile = attn_tile(FMT, DP);              // tokens of a warp's tile
    static constexpr int kMT = kTile / 16;
    static constexpr int kWarps = attn_warps(FMT, DP, NT, WIDE);
    static constexpr int kCtas = attn_ctas_per_sm(FMT, DP, NT, WIDE), kSlots = attn_slots(FMT, DP, NT, WIDE);
    static constexpr int kSlotBytes = kTile * kRow;               // K or V of a tile
    static constexpr int kHeads = 8 * NT;
    static constexpr int kQParts = !WIDE ? 1 : FMT == COLI_KV_BF16 ? 3 : 2;
    static constexpr int kPParts = WIDE && FMT == COLI_KV_BF16 ? 3 : 2;
    static constexpr int kUse = USE, kKS = USE / 16;              // products of 16 along the head
    static constexpr int kQWords = kQParts * NT * kKS / 2 * 32;   // uint4
    // p is kept times 2^kShift, so that the second f16 part of a small p is still above f16's smallest step
    static constexpr int kShift = FMT == COLI_KV_BF16 ? 0 : 14;
    static_assert(8 * DP * 4 <= kSlotBytes, "a warp's sums of 8 heads fit its free slot");
    static_assert(kWarps * kTile == attn_unit(FMT, DP, NT, WIDE), "unit");
    static constexpr size_t smem(int seqs) {
        return (size_t)kWarps * kSlots * kSlotBytes + (size_t)kQWords * 16 + kWarps * kHeads * 8 + kHeads * 4 +
               kWarps * 4 * 4 + ((size_t)seqs + 1) * 4 + 336;
    }
    static_assert(kWarps * kSlots * kSlotBytes + kQWords * 16 + kWarps * kHeads * 8 + kHeads * 4 + kWarps * 16 +
                          (kAttnMaxSeqs + 1) * 4 + 336 <=
                      (228 << 10) / kCtas - 1024,
                  "shared memory of an SM");
};

template <typename T>
__global__ void __launch_bounds__(T::kWarps * 32, T::kCtas) attn_stream_kernel(const AttnParams P, const AttnWork W) {
    using namespace attn;
    constexpr int DP = T::kDim, NT = T::kNT, kThreads = T::kWarps * 32, FMT = T::kFmt;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *ring = sm;
    uint4 *qf = reinterpret_cast<uint4 *>(ring + T::kWarps * T::kSlots * T::kSlotBytes);
    float2 *ml = reinterpret_cast<float2 *>(qf + T::kQWords);          // [warp][head] (m, l)
    float *qs = reinterpret_cast<float *>(ml + T::kWarps * T::kHeads);  // [head] factor of the products
    uint32_t *seen = reinterpret_cast<uint32_t *>(qs + T::kHeads);     // [warp][tile % 4] rows that hold a token
    int *pre = reinterpret_cast<int *>(seen + T::kWarps * 4);          // [seqs + 1] units before a sequence
    int *scan = pre + P.seqs + 1;                                      // [83]
    const int tid = threadIdx.x, w = tid / 32, lane = tid % 32, g = lane >> 2, c = lane & 3;

    wait_for_previous();
    let_next_start();  // the join's blocks may wait beside this

    // ---- units before each sequence (per head group)
    auto units_of = [&](int b) {
        int first, end, why;
        kv_span(P.lens[b], P.table_width, P.cache.page_size, P.window, first, end, why);
        if (why && blockIdx.x == 0 && P.err) atomicOr(P.err, COLI_LAYER_BAD_POSITION);
        return kv_units(end - first, W.unit);
    };
    const int per = (P.seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, P.seqs), b1 = min(b0 + per, P.seqs);
    int mine = 0, longest = 0;
    for (int b = b0; b < b1; b++) {
        const int u = units_of(b);
        pre[b + 1] = u;
        mine += u;
        longest = max(longest, u);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) {
        scan[w] = incl;
        scan[16 + w] = longest;
    }
    __syncthreads();
    int before = incl - mine;
    for (int i = 0; i < w; i++) before += scan[i];
    for (int b = b0; b < b1; b++) {
        const int u = pre[b + 1];
        before += u;
        pre[b + 1] = before;
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const uint32_t total = (uint32_t)pre[P.seqs] * W.groups;

    // ---- sequences with nothing to see
    for (int b = blockIdx.x; b < P.seqs; b += gridDim.x) {
        if (pre[b + 1] != pre[b]) continue;
        for (int i = tid; i < P.q_heads * P.dim; i += kThreads)
            store_act(P.out, b * P.out_stride + i, 0.f, P.act);
        if (P.lse)
            for (int i = tid; i < P.q_heads; i += kThreads) P.lse[(int64_t)b * P.q_heads + i] = -INFINITY;
    }

    bool whole_mode = W.whole == kAttnWhole;
    if (W.whole == kAttnMaybe) {
        int u = 0;
#pragma unroll
        for (int i = 0; i < T::kWarps; i++) u = max(u, scan[16 + i]);
        whole_mode = attn_whole_now(total, P.seqs * W.groups, u, W.ctas, W.times);
        if (whole_mode && blockIdx.x == 0 && tid == 0) W.cuts[0].runs = 0;  // nothing for the join
    }

    // ---- this CTA's run: an item; or a part of an item, every item cut by itself into parts of at most c units, if
    // that makes no more runs than there are CTAs and none much longer than the others; or a run of as many units
    // as any other's, which may go on from item to item (of one unit where there are CTAs enough).
    const uint32_t run = blockIdx.x;
    Cursor at{0, 0, 0, 0};
    int n_units = 0;
    AttnCut cut{-1, 0, 0, 0};  // for the join
    if (whole_mode) {
        if (run >= (uint32_t)(P.seqs * W.groups)) return;
        at.b = run / W.groups;
        at.hv = run - at.b * W.groups;
        at.units = n_units = pre[at.b + 1] - pre[at.b];
        if (n_units == 0) return;
    }
    const uint32_t ctas = W.ctas;
    if (!whole_mode && total > ctas) {
        const uint32_t c0 = (total + ctas - 1) / ctas;
        const uint32_t c[3] = {c0, c0 + 1, c0 + 2 + c0 / 8};
        uint32_t sum[3] = {0, 0, 0}, run_to[3];
        for (int b = b0; b < b1; b++) {
            const uint32_t u = pre[b + 1] - pre[b];
#pragma unroll
            for (int k = 0; k < 3; k++) sum[k] += (u + c[k] - 1) / c[k];
        }
#pragma unroll
        for (int k = 0; k < 3; k++) {
            run_to[k] = sum[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, run_to[k], o);
                if (lane >= o) run_to[k] += v;
            }
            if (lane == 31) scan[16 * (k + 2) + w] = run_to[k];
        }
        __syncthreads();
        uint32_t all[3], mine_from[3];
#pragma unroll
        for (int k = 0; k < 3; k++) {
            all[k] = 0;
            mine_from[k] = run_to[k] - sum[k];
#pragma unroll
            for (int i = 0; i < T::kWarps; i++) {
                const uint32_t v = scan[16 * (k + 2) + i];
                if (i < w) mine_from[k] += v;
                all[k] += v;
            }
        }
        const int k = (uint64_t)all[0] * W.groups <= ctas ? 0 : (uint64_t)all[1] * W.groups <= ctas ? 1 : 2;
        const uint32_t parts = k == 0 ? all[0] : k == 1 ? all[1] : all[2], cap = k == 0 ? c[0] : k == 1 ? c[1] : c[2];
        if ((uint64_t)parts * W.groups <= ctas) {
            cut.runs = parts * W.groups;
            if (run < (uint32_t)cut.runs) {
                // the thread whose sequences the run is among tells which one it is
                uint32_t from = (k == 0 ? mine_from[0] : k == 1 ? mine_from[1] : mine_from[2]) * W.groups;
                for (int b = b0; b < b1; b++) {
                    const uint32_t p = ((uint32_t)(pre[b + 1] - pre[b]) + cap - 1) / cap;
                    if (run >= from && run < from + p * W.groups) {
                        scan[80] = b;
                        scan[81] = run - from;
                        scan[82] = p;
                    }
                    from += p * W.groups;
                }
            }
            __syncthreads();
            if (run >= (uint32_t)cut.runs) {
                if (run == 0 && tid == 0) W.cuts[0] = cut;
                return;
            }
            const int p = scan[82], part = scan[81] % p;
            at.b = scan[80];
            at.hv = scan[81] / p;
            at.units = pre[at.b + 1] - pre[at.b];
            at.u = part * (at.units / p) + min(part, at.units % p);
            n_units = at.units / p + (part < at.units % p ? 1 : 0);
            if (part == 1) {
                cut.b = at.b;
                cut.hv = at.hv;
                cut.last = run + p - 2;
            }
        }
    }
    if (!whole_mode && n_units == 0) {
        const AttnRuns R(total, ctas);
        cut.runs = R.runs;
        if (run >= R.runs) {
            if (run == 0 && tid == 0) W.cuts[0] = cut;
            return;
        }
        const uint32_t x0 = R.start(run);
        n_units = R.start(run + 1) - x0;
        // the last sequence whose units begin at or before x0
        int lo = 0, hi = P.seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if ((uint32_t)pre[mid] * W.groups <= x0) lo = mid;
            else hi = mid;
        }
        at.b = lo;
        at.units = pre[lo + 1] - pre[lo];
        const uint32_t r = x0 - (uint32_t)pre[lo] * W.groups;
        at.hv = (int)(r / (uint32_t)at.units);
        at.u = (int)r - at.hv * at.units;
        const uint32_t i0 = x0 - at.u;
        if (at.u > 0 && R.start(run - 1) <= i0) {
            cut.b = at.b;
            cut.hv = at.hv;
            cut.last = (int)R.of(i0 + at.units - 1);
        }
    }
    auto advance = [&](Cursor &k) {
        if (++k.u < k.units) return;
        k.u = 0;
        if (++k.hv < W.groups) return;
        k.hv = 0;
        do {
            k.b++;
        } while (k.b < P.seqs && pre[k.b + 1] == pre[k.b]);
        if (k.b < P.seqs) k.units = pre[k.b + 1] - pre[k.b];
    };

    // ---- q of an item: read early, turned into parts when the item begins. A warp has the heads w, w + kWarps, ..,
    // a lane the pairs of elements 2 * lane + 64 * i.
    constexpr int kMyHeads = (T::kHeads + T::kWarps - 1) / T::kWarps;
    const int group = P.q_heads / P.kv_heads;
    float qx[kMyHeads][DP / 32];
    auto load_q = [&](const Cursor &k) {
        const int kh = k.hv / W.chunks, h0 = (k.hv - kh * W.chunks) * T::kHeads;
#pragma unroll
        for (int a = 0; a < kMyHeads; a++) {
            const int h = w + a * T::kWarps < T::kHeads ? h0 + w + a * T::kWarps : group;  // group: none
            const int64_t src = k.b * P.q_stride + (int64_t)(kh * group + h) * P.dim;
#pragma unroll
            for (int i = 0; i < DP / 32; i++) {
                const int d = 64 * (i >> 1) + 2 * lane + (i & 1);
                qx[a][i] = h < group && d < P.dim ? load_act(P.q, src + d, P.act) : 0.f;
            }
        }
    };
    load_q(at);

    // ---- copies
    unsigned char *my_ring = ring + w * T::kSlots * T::kSlotBytes;
    const uint32_t my_ring_a = smem_u32(my_ring);
    // 16-byte chunks of a 128-byte line are exchanged so that 8 rows' same chunk lie in 8 bank groups. A chunk's
    // number is only ever or'ed or xor'ed into an address, whose bits from 4 up it then owns (rows start at
    // multiples of 128 bytes): place(row, c ^ d) = place(row, c) ^ (d << 4).
    auto place = [](int row, int chunk) -> uint32_t {
        if (T::kRow >= 128) return row * T::kRow + ((chunk ^ (row & 7)) << 4);
        const int line = row >> 1;
        return line * 128 + (((((row & 1) << 2) | chunk) ^ (line & 3)) << 4);
    };
    constexpr uint32_t kAll = T::kTile == 32 ? 0xffffffffu : 0xffffu;
    constexpr int kChunks = T::kRow / 16, kRowsPer = 32 / kChunks;
    const int ch = lane % kChunks, sub = lane / kChunks;
    // chunks behind the head's elements are zeros, and behind those that are used nothing
    const bool in_row = ch * 16 < P.dim * T::kSize, in_use = ch * 16 < T::kUse * T::kSize;
    const uint32_t ch_bytes = in_row ? 16 : 0;
    const char *kbase = (const char *)P.k_cache + (in_row ? ch * 16 : 0), *vbase = (const char *)P.v_cache + (in_row ? ch * 16 : 0);
    const uint32_t off_step = 1u << W.off_shift, my_place = place(sub, ch);
    Cursor ld = at;
    int ld_first = 0, ld_end = 0, ld_head = 0;
    const int32_t *ld_pages = P.table;
    auto enter = [&]() {  // an item
        int why;
        kv_span(P.lens[ld.b], P.table_width, P.cache.page_size, P.window, ld_first, ld_end, why);
        ld_pages = P.table + (int64_t)ld.b * P.table_width;
        ld_head = ld.hv / W.chunks;
    };
    // lane r has row r of a tile; the page number is not looked at before the copy, so that its load is not
    // waited for
    struct Look {
        int32_t page, slot, head;
        bool real;
    };
    auto look_up = [&](int left) {  // of how many units
        Look k{0, 0, ld_head, false};
        if (left <= 0) return k;
        int t;
        if (kv_unit_token(ld_first, ld_end, W.unit, ld.u, w * T::kTile + lane, t) && lane < T::kTile) {
            const int i = kv_quotient(W.divide, t);
            k.slot = t - i * P.cache.page_size;
            k.page = ld_pages[i];
            k.real = true;
        }
        if (left > 1) {
            advance(ld);
            if (ld.u == 0) enter();
        }
        return k;
    };
    uint32_t cp_rows = 0, cp_off = 0;  // of the tile whose halves are copied
    auto copy_rows = [&](uint32_t dst, const char *base) {
        // row i * kRowsPer + sub: its place differs from row sub's by a distance and, within 8 rows, by an xor
        auto to = [&](int i) {
            const int row = i * kRowsPer;  // of sub 0
            if (T::kRow >= 128) return (dst + row * T::kRow) + (my_place ^ ((row & 7) << 4));
            return (dst + row * T::kRow) + (my_place ^ (((row >> 1) & 3) << 4));
        };
        if (cp_rows == kAll) {
#pragma unroll
            for (int i = 0; i < T::kTile / kRowsPer; i++) {
                const uint32_t o = __shfl_sync(0xffffffffu, cp_off, i * kRowsPer + sub);
                if (T::kUse == DP || in_use) copy16(to(i), base + (uint64_t)o * off_step, ch_bytes);
            }
        } else if (cp_rows) {
#pragma unroll
            for (int i = 0; i < T::kTile / kRowsPer; i++) {
                const int row = i * kRowsPer + sub;
                const uint32_t o = __shfl_sync(0xffffffffu, cp_off, row);
                const bool ok = (cp_rows >> row) & 1;
                if (T::kUse == DP || in_use) copy16(to(i), base + (uint64_t)(ok ? o : 0) * off_step, ok ? ch_bytes : 0);
            }
        }
        copy_commit();
    };
    auto next_slot = [](int &s) { s = s + 1 == T::kSlots ? 0 : s + 1; };
    auto copy_k = [&](Look k, int tile, int into) {
        if (k.real && (uint32_t)k.page >= (uint32_t)P.cache.pages) {
            k.real = false;
            if (P.err) atomicOr(P.err, COLI_LAYER_BAD_PAGE);
        }
        cp_rows = __ballot_sync(0xffffffffu, k.real);
        cp_off = k.page * W.page_step + k.slot * W.token_step + k.head * W.head_step;
        if (lane == 0) seen[w * 4 + (tile & 3)] = cp_rows;
        copy_rows(my_ring_a + into * T::kSlotBytes, kbase);
    };
    auto copy_v = [&](int into) { copy_rows(my_ring_a + into * T::kSlotBytes, vbase); };

    enter();
    Look next;  // the tile whose K is copied next
    {
        constexpr int kFirst = (T::kSlots + 1) / 2;  // K and V in turn
        Look k[kFirst];
#pragma unroll
        for (int i = 0; i < kFirst; i++) k[i] = look_up(n_units - i);
        next = look_up(n_units - kFirst);
#pragma unroll
        for (int i = 0; i < T::kSlots; i++) {
            if (i % 2 == 0) copy_k(k[i / 2], i / 2, i);
            else copy_v(i);
        }
    }

    // ---- for the join: the item that this run's first border cuts, told by the run behind its first cut
    if (tid == 0 && !whole_mode) W.cuts[run] = cut;

    float o[T::kKS][NT][4], m[NT][2], l[NT][2], sc[NT][2];
    int slot = 0;
    bool fresh = true;
    int seg0 = 0;  // first unit of the current segment
    for (int it = 0; it < n_units; it++) {
        if (fresh) {
            // ---- q of the item: parts in the order the matrix instruction takes them
            fresh = false;
            seg0 = at.u;
            const float ks = P.scale * 1.4426950408889634f * (P.k_scale ? P.k_scale[at.hv / W.chunks] : 1.f);
#pragma unroll
            for (int hh = 0; hh < kMyHeads; hh++) {
                const int h = w + hh * T::kWarps;
                if (h >= T::kHeads) continue;
                float (&x)[DP / 32] = qx[hh];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < DP / 32; i++) top = fmaxf(top, fabsf(x[i]));
                float up = 1.f, down = 1.f;
                if (FMT != COLI_KV_BF16) {
                    // the largest element of the head at 2^14..2^15
#pragma unroll
                    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                    int e = (int)((__float_as_uint(top) >> 23) & 0xff) - 127;
                    e = max(e, -100);
                    if (top > 0.f && e < 128) {
                        up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
                        down = __uint_as_float((unsigned)(127 - 14 + e) << 23);
                    }
                }
                if (lane == 0) qs[h] = ks * down;
#pragma unroll
                for (int i = 0; i < DP / 64; i++) {
                    float a = x[2 * i] * up, b = x[2 * i + 1] * up;
                    const int d = 64 * i + 2 * lane;  // even
                    if (d >= T::kUse) continue;
                    // which 16-product, lane of the group and register of the fragment hold (d, d + 1)
                    const int k = d & 15;
                    const int cc = FMT == COLI_KV_E4M3 ? k >> 2 : (k & 7) >> 1;
                    const int rr = FMT == COLI_KV_E4M3 ? (k >> 1) & 1 : k >> 3;
#pragma unroll
                    for (int p = 0; p < T::kQParts; p++) {
                        const uint32_t v = take_part<FMT>(a, b);
                        uint32_t *to = reinterpret_cast<uint32_t *>(
                            qf + ((p * NT + h / 8) * (T::kKS / 2) + (d >> 5)) * 32 + (h & 7) * 4 + cc);
                        to[((d >> 4) & 1) * 2 + rr] = v;
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NT; n++) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    m[n][j] = -INFINITY;
                    l[n][j] = 0.f;
                    sc[n][j] = qs[n * 8 + 2 * c + j];
                    if (sc[n][j] == 0.f) sc[n][j] = 1.175494351e-38f;  // so that it keeps an infinity one
                }
#pragma unroll
                for (int i = 0; i < T::kKS; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) o[i][n][j] = 0.f;
            }
        }

        copy_wait<T::kSlots - 1>();
        __syncwarp();
        const uint32_t rows = seen[w * 4 + (it & 3)];
        const int k_slot = slot;
        const uint32_t kt = my_ring_a + k_slot * T::kSlotBytes;
        next_slot(slot);
        const int v_slot = slot;
        const uint32_t vt = my_ring_a + v_slot * T::kSlotBytes;
        next_slot(slot);
        const int lr = lane & 7, li = lane >> 3;
        float s[T::kMT][NT][4];
        if (rows) {
            // ---- S^T = K q^T; the leading part in two chains, the others in one, added at the end
#pragma unroll
            for (int i = 0; i < T::kMT; i++) {
                // (one chain where two 16-row blocks follow each other: the second's registers spill there, 94 us
                // against 78 on an 8-bit cache of 128 elements beside fp32 queries)
                constexpr int kLead = T::kMT > 1 && FMT == COLI_KV_E4M3 ? 1 : 2, kChains = kLead + (T::kQParts > 1 ? 1 : 0);
                float acc[kChains][NT][4];
                const uint32_t at_row = kt + place(i * 16 + lr + (li & 1) * 8, li >> 1);
                // two products of 16 along the head
                auto product = [&](const uint32_t (&a0)[4], const uint32_t (&a1)[4], int k2) {
#pragma unroll
                    for (int p = 0; p < T::kQParts; p++)
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            const uint4 q = qf[((p * NT + n) * (T::kKS / 2) + k2) * 32 + lane];
                            float (&first)[4] = acc[p ? kChains - 1 : 0][n], (&second)[4] = acc[p ? kChains - 1 : kLead - 1][n];
                            if (k2 == 0 && p < 2) mma<FMT, false>(first, a0, q.x, q.y);
                            else mma<FMT, true>(first, a0, q.x, q.y);
                            if (k2 == 0 && p == 0 && kLead == 2) mma<FMT, false>(second, a1, q.z, q.w);
                            else mma<FMT, true>(second, a1, q.z, q.w);
                        }
                };
#pragma unroll
                for (int k2 = 0; k2 < T::kKS / 2; k2++) {
                    if (FMT != COLI_KV_E4M3) {
                        uint32_t a0[4], a1[4];
                        ldm4(a0, at_row ^ ((4 * k2) << 4));
                        ldm4(a1, at_row ^ ((4 * k2 + 2) << 4));
                        product(a0, a1, k2);
                    } else {
                        uint32_t raw[4];
                        ldm4(raw, at_row ^ ((2 * k2) << 4));
                        const uint32_t a0[4] = {widen(raw[0]), widen(raw[1]), widen_hi(raw[0]), widen_hi(raw[1])};
                        const uint32_t a1[4] = {widen(raw[2]), widen(raw[3]), widen_hi(raw[2]), widen_hi(raw[3])};
                        product(a0, a1, k2);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float x = acc[kChains - 1][n][j];
#pragma unroll
                        for (int k = kChains - 2; k >= 0; k--) x += acc[k][n][j];
                        s[i][n][j] = x;
                    }
            }
            if (rows != kAll) {  // a score of -inf where there is no token
#pragma unroll
                for (int i = 0; i < T::kMT; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (!((rows >> (i * 16 + (j >> 1) * 8 + g)) & 1))
#pragma unroll
                            for (int n = 0; n < NT; n++) s[i][n][j] = sc[n][j & 1] > 0.f ? -INFINITY : INFINITY;
            }
        }
        __syncwarp();
        // the half that is kSlots behind K takes its slot
        if (T::kSlots % 2) {
            copy_v(k_slot);
        } else {
            copy_k(next, it + T::kSlots / 2, k_slot);
            next = look_up(n_units - it - (T::kSlots / 2 + 1));
        }
        copy_wait<T::kSlots - 1>();
        __syncwarp();
        if (rows) {
            // ---- softmax over the tile's tokens, head by head
            uint32_t pf[T::kPParts][T::kMT][NT][2];
            float f[NT][2];
#pragma unroll
            for (int n = 0; n < NT; n++) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < T::kMT; i++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            top = fmaxf(top, s[i][n][2 * r + j] * sc[n][j]);
                        }
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float mn = fmaxf(m[n][j], ceilf(top));
                    const float ref = mn == -INFINITY ? 0.f : mn;
                    f[n][j] = exp2_fast(m[n][j] - ref);  // exact: an integer power; 0 from -inf
                    m[n][j] = mn;
                    // One rounding for the exponent, of the exact product, small where p is large. But the maximum is of
                    // rounded products, from 2^23 on steps of 1 and more away from the exact ones (p would pass f16's
                    // range, or be 0 for every token): there the exponents are of those too. (64 sequences of 24,576
                    // e4m3 tokens 497 -> 500 us; by a vote and a branch other forms pay up to 6 % through the registers.)
                    const float off = __fsub_rd((float)T::kShift, ref);
                    float sum = 0.f, by = sc[n][j];
                    if (!(fabsf(mn) < 0x1p23f)) {
#pragma unroll
                        for (int i = 0; i < T::kMT; i++)
#pragma unroll
                            for (int r = 0; r < 2; r++) s[i][n][2 * r + j] = __fmul_rn(s[i][n][2 * r + j], by);
                        by = 1.f;
                    }
#pragma unroll
                    for (int i = 0; i < T::kMT; i++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            const float p = exp2_fast(fmaf(s[i][n][2 * r + j], by, off));
                            s[i][n][2 * r + j] = p;
                            sum += p;
                        }
                    l[n][j] = fmaf(l[n][j], f[n][j], sum);
                }
#pragma unroll
                for (int i = 0; i < T::kMT; i++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        float a = s[i][n][2 * r], b = s[i][n][2 * r + 1];
#pragma unroll
                        for (int p = 0; p < T::kPParts; p++) pf[p][i][n][r] = transpose8(take_part<FMT>(a, b));
                    }
            }
            // ---- O^T += V^T P^T
            if (FMT != COLI_KV_E4M3) {
                const uint32_t at_row = vt + place(lr + (li >> 1) * 8, li & 1);
#pragma unroll
                for (int d = 0; d < T::kKS; d++) {
                    float t[NT][4];
#pragma unroll
                    for (int i = 0; i < T::kMT; i++) {
                        uint32_t a[4];
                        ldm4t(a, (at_row ^ ((2 * d) << 4)) + i * 16 * T::kRow);
#pragma unroll
                        for (int p = T::kPParts - 1; p >= 0; p--)
#pragma unroll
                            for (int n = 0; n < NT; n++) {
                                if (i == 0 && p == T::kPParts - 1) mma<FMT, false>(t[n], a, pf[p][i][n][0], pf[p][i][n][1]);
                                else mma<FMT, true>(t[n], a, pf[p][i][n][0], pf[p][i][n][1]);
                            }
                    }
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int j = 0; j < 4; j++) o[d][n][j] = fmaf(o[d][n][j], f[n][j & 1], t[n][j]);
                }
            } else {
                const uint32_t at_row = vt + place(lr + (li & 1) * 8, li >> 1);
#pragma unroll
                for (int d2 = 0; d2 < T::kKS / 2; d2++) {
                    float t[2][NT][4];
#pragma unroll
                    for (int i = 0; i < T::kMT; i++) {
                        uint32_t raw[4];
                        ldm4t(raw, (at_row ^ ((2 * d2) << 4)) + i * 16 * T::kRow);
#pragma unroll
                        for (int hf = 0; hf < 2; hf++) {
                            // bytes (token, dim): 00 01 10 11 -> even dim's two tokens, odd dim's two tokens
                            const uint32_t x = __byte_perm(raw[2 * hf], 0, 0x3120), y = __byte_perm(raw[2 * hf + 1], 0, 0x3120);
                            const uint32_t a[4] = {widen(x), widen_hi(x), widen(y), widen_hi(y)};
#pragma unroll
                            for (int p = T::kPParts - 1; p >= 0; p--)
#pragma unroll
                                for (int n = 0; n < NT; n++) {
                                    if (i == 0 && p == T::kPParts - 1) mma<FMT, false>(t[hf][n], a, pf[p][i][n][0], pf[p][i][n][1]);
                                    else mma<FMT, true>(t[hf][n], a, pf[p][i][n][0], pf[p][i][n][1]);
                                }
                        }
                    }
#pragma unroll
                    for (int hf = 0; hf < 2; hf++)
#pragma unroll
                        for (int n = 0; n < NT; n++)
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                o[2 * d2 + hf][n][j] = fmaf(o[2 * d2 + hf][n][j], f[n][j & 1], t[hf][n][j]);
                }
            }
            __syncwarp();
        }

        if (at.u + 1 == at.units || it + 1 == n_units) {
            // ---- the segment ends: the warps' sums through their free slots, 8 heads at a time
            if (it + 1 < n_units) {
                Cursor k = at;
                advance(k);
                load_q(k);
            }
            float *mo = reinterpret_cast<float *>(my_ring + v_slot * T::kSlotBytes);
            const int kh = at.hv / W.chunks, h0 = (at.hv - kh * W.chunks) * T::kHeads;
            const bool whole = seg0 == 0 && at.u + 1 == at.units;
            const float vs = P.v_scale ? P.v_scale[kh] : 1.f;
            const int64_t part = (int64_t)(2 * run + (seg0 == 0 ? 1 : 0)) * T::kHeads;
#pragma unroll
            for (int n = 0; n < NT; n++) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float x = l[n][j];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    if (g == 0) ml[w * T::kHeads + n * 8 + 2 * c + j] = make_float2(m[n][j], x);
                }
#pragma unroll
                for (int i = 0; i < T::kKS; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int head = 2 * c + (j & 1);
                        const int d = 16 * i + (FMT == COLI_KV_E4M3 ? 2 * g + (j >> 1) : g + 8 * (j >> 1));
                        mo[head * DP + (d ^ (c << 3))] = o[i][n][j];
                    }
                __syncthreads();
                for (int i = tid; i < 8 * DP / 4; i += kThreads) {
                    const int h = i / (DP / 4), d = i % (DP / 4) * 4;
                    if (h0 + n * 8 + h >= group) break;
                    float top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < T::kWarps; k++) top = fmaxf(top, ml[k * T::kHeads + n * 8 + h].x);
                    const float ref = top == -INFINITY ? 0.f : top;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.f;
#pragma unroll
                    for (int k = 0; k < T::kWarps; k++) {
                        const float2 e = ml[k * T::kHeads + n * 8 + h];
                        const float e2 = exp2_fast(e.x - ref);
                        const float4 y = *reinterpret_cast<const float4 *>(ring + (k * T::kSlots + v_slot) * T::kSlotBytes +
                                                                           (h * DP + (d ^ ((h >> 1) << 3))) * 4);
                        add_scaled(x, y, e2);
                        sum = fmaf(e.y, e2, sum);
                    }
                    if (whole) {
                        const int qh = kh * group + h0 + n * 8 + h;
                        const float y[4] = {x.x, x.y, x.z, x.w}, f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            if (d + j < P.dim) store_act(P.out, at.b * P.out_stride + (int64_t)qh * P.dim + d + j, y[j] * f * vs, P.act);
                        if (d == 0 && P.lse) P.lse[(int64_t)at.b * P.q_heads + qh] = attn_lse(ref, sum, T::kShift);
                    } else {
                        *reinterpret_cast<float4 *>(W.part_o + (part + n * 8 + h) * DP + d) = x;
                        if (d == 0) W.part_ml[part + n * 8 + h] = make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
            fresh = true;
        }
        if (T::kSlots % 2) {
            copy_k(next, it + T::kSlots / 2 + 1, v_slot);
            next = look_up(n_units - it - (T::kSlots / 2 + 2));
        } else {
            copy_v(v_slot);
        }
        advance(at);
    }
    copy_wait<0>();
}

template <typename T>
cudaError_t launch_stream(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s) {
    static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(attn_stream_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)T::smem(kAttnMaxSeqs));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_overlapped(attn_stream_kernel<T>, dim3(grid), T::kWarps * 32, T::smem(P.seqs), s, P, W);
}

template <int FMT, int DP, int USE>
cudaError_t launch_heads(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s) {
    if (W.nt == 1)
        return W.wide ? launch_stream<AttnTraits<FMT, DP, USE, 1, true>>(P, W, grid, s)
                      : launch_stream<AttnTraits<FMT, DP, USE, 1, false>>(P, W, grid, s);
    return W.wide ? launch_stream<AttnTraits<FMT, DP, USE, 2, true>>(P, W, grid, s)
                  : launch_stream<AttnTraits<FMT, DP, USE, 2, false>>(P, W, grid, s);
}

template <int FMT>
cudaError_t launch_dims(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s) {
    return W.dim == 64    ? launch_heads<FMT, 64, 64>(P, W, grid, s)
           : W.use == 96  ? launch_heads<FMT, 128, 96>(P, W, grid, s)
           : W.dim == 128 ? launch_heads<FMT, 128, 128>(P, W, grid, s)
                          : launch_heads<FMT, 256, 256>(P, W, grid, s);
}

}  // namespace colimoe
