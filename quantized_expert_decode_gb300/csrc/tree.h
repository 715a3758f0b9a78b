// tree.h — what the streaming and the join kernel of coli_attn_tree share. Internal to libcolimoe.
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "attn.h"
#include "draft.h"

namespace colimoe {

constexpr int kTreeMaxSeqs = 1024, kTreeMaxNodes = 256;
constexpr int kTreeRows = 128;  // rows of a tile of the products: (node, head of the group)

// Head sizes are rounded up to 64, 128 or 256 (DP); at 256 a CTA takes half of V's columns, so that 128 columns of sums
// stay in registers. WIDE: more parts of q and p.
template <int FMT, int DP, bool WIDE>
struct TreeTraits {
    static constexpr int kFmt = FMT, kDim = DP;
    static constexpr bool kWide = WIDE, kRaw = FMT == COLI_KV_E4M3;
    static constexpr int kCols = DP < 128 ? DP : 128;  // of V
    static constexpr int kHalves = DP / kCols;
    static constexpr int kQParts = !WIDE ? 1 : FMT == COLI_KV_BF16 ? 3 : 2;
    static constexpr int kPParts = WIDE && FMT == COLI_KV_BF16 ? 3 : 2;
    static constexpr int kTile = DP == 256 ? (WIDE ? 32 : 64) : 128;  // tokens
    // p is kept times 2^kShift, so that the second f16 part of a small p is still above f16's smallest step
    static constexpr int kShift = FMT == COLI_KV_BF16 ? 0 : 14;
    static constexpr int kQBytes = kQParts * kTreeRows * DP * 2;
    static constexpr int kSlotBytes = kTile * DP * 2;  // K or V of a tile, 16-bit
    static constexpr int kRawSlots = kRaw ? 4 : 0;     // K or V of a tile on its way in 8 bits
    static constexpr int kRawBytes = kTile * DP;
    static constexpr int kMiscBytes = 16896;
    static constexpr int kRoom = (227 << 10) - kMiscBytes - kQBytes - kRawSlots * kRawBytes;
    static constexpr int kSlots = kRoom / kSlotBytes < 8 ? kRoom / kSlotBytes : 8;
    static_assert(kSlots >= 1, "shared memory of an SM");
    static constexpr int kSmem = kQBytes + kSlots * kSlotBytes + kRawSlots * kRawBytes + kMiscBytes;
    // tensor memory: two buffers of scores, over which the parts of p are written, and two of a tile's sums; one where
    // two do not fit (beside three parts of p; the scores' products of 128 places then run while the sums are read. Tiles of
    // 64 places with two buffers: products with 64 columns take as long as with 128, 32 sequences of up to 8192 tokens
    // with 21 nodes 289 us)
    static constexpr int kScoreCols = kPParts == 3 ? (kTile + kTile / 2 + 31) / 32 * 32 : kTile;
    static constexpr int kSumBuffers = 2 * kScoreCols + 2 * kCols <= 512 ? 2 : 1;
    static_assert(2 * kScoreCols + kSumBuffers * kCols <= 512, "tensor memory of an SM");
};

// The item whose units the border before a run cuts, told for its first cut only (else it has no rows): its rows are
// [first, first + rows) of the (node, head) pairs of a sequence whose nodes begin at `row`
struct alignas(16) TreeCut {
    int32_t rows, last, row, runs, first, kh, half;
    int32_t side;  // the runs of an item are so far apart
};

// How the launch is laid out, and the workspace
struct TreeWork {
    int32_t dim, cols, tile, halves;
    int32_t wide, ctas;
    KvDivide divide, group;  // by the page size, by the query heads of a kv head
    // the cache's strides in steps of 2^off_shift bytes, which divides them all
    uint32_t page_step, token_step, head_step, off_shift;
    int32_t box;             // places of a box of the tensor maps: a power of two that divides the page size; 0: none
    int32_t q_vec, out_vec;  // rows of q and out may be moved 16 bytes at a time
    TreeCut *cuts;           // [ctas] at the border before a run
    float2 *part_ml;         // [2 * ctas][128] (m, l) of a run's first and last cut item
    float4 *part_o;          // [2 * ctas][cols / 4][128]
};

// K and V pools as (element, slot, head, page)
struct TreeMaps {
    CUtensorMap k, v;
};

// What an item is: rows [row0, row0 + rows) of a sequence's (node, head) pairs on one kv head, and a half of V
struct TreeItem {
    int32_t kh, half, tile;
};
__host__ __device__ __forceinline__ TreeItem tree_item(int32_t item, int32_t row_tiles, int32_t halves) {
    // row tiles beside each other, so that they find each other's K and V in L2
    TreeItem t;
    t.tile = item % row_tiles;
    item /= row_tiles;
    t.half = item % halves;
    t.kh = item / halves;
    return t;
}

cudaError_t launch_tree_bf16(const TreeParams &P, const TreeWork &W, const TreeMaps &maps, int grid, cudaStream_t s);
cudaError_t launch_tree_f16(const TreeParams &P, const TreeWork &W, const TreeMaps &maps, int grid, cudaStream_t s);
cudaError_t launch_tree_e4m3(const TreeParams &P, const TreeWork &W, const TreeMaps &maps, int grid, cudaStream_t s);

}  // namespace colimoe
