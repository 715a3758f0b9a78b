// draft_index.h — which rows and places a sequence's nodes have. Plain C++ with no CUDA header, so that the
// arithmetic is the same on the device and in the host tests. Internal to libcolimoe.
#pragma once

#include "kv_index.h"

namespace colimoe {

enum DraftWhy : int { kDraftOk = 0, kDraftBadSequence = 1, kDraftBadPosition = 2 };

// The rows [row, row + n) of a sequence whose first row and the next sequence's are r0 and r1, clamped to the `rows`
// that there are and to `nodes`.
COLI_HD void draft_rows(int32_t r0, int32_t r1, int32_t rows, int32_t nodes, int32_t &row, int32_t &n, int &why) {
    const int32_t a = r0 < 0 ? 0 : r0 > rows ? rows : r0, e = r1 < a ? a : r1 > rows ? rows : r1;
    row = a;
    n = e - a < nodes ? e - a : nodes;
    why = a != r0 || e != r1 || n != e - a ? kDraftBadSequence : kDraftOk;
}

// Committed tokens and nodes, clamped to the places that the page table names: past + n <= width * page_size.
COLI_HD void draft_places(int32_t given, int32_t width, int32_t page_size, int32_t &past, int32_t &n, int &why) {
    const int64_t most = (int64_t)width * page_size;
    why = kDraftOk;
    if (n > most) {
        n = (int32_t)most;
        why = kDraftBadPosition;
    }
    past = given < 0 ? 0 : given > most - n ? (int32_t)(most - n) : given;
    if (past != given && n > 0) why = kDraftBadPosition;
}

// The first place that any node sees: those of depth 0 reach back furthest.
COLI_HD int32_t draft_start(int32_t past, int32_t window) {
    return window > 0 && past >= window ? past - window + 1 : 0;
}

// Whether a node at `depth` sees the cached place t < past.
COLI_HD bool draft_sees(int32_t past, int32_t depth, int32_t window, int32_t t) {
    return window == 0 || (int64_t)t > (int64_t)past + depth - window;
}

}  // namespace colimoe
