// layer_check.h — what the entry points around a paged cache check alike. Internal to libcolimoe.
#pragma once

#include "host.h"
#include "layer.h"

namespace colimoe {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadDim = 256;
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // keeps row * stride in 64 bits

inline int act_bytes(int act) { return act == COLI_ACT_F32 ? 4 : 2; }
inline bool act_ok(int act) { return act == COLI_ACT_F32 || act == COLI_ACT_BF16 || act == COLI_ACT_F16; }

inline int check_cache(const coli_kv_cache *c) {
    if (!c || !c->k || !c->v || c->reserved != 0) return COLI_MOE_EINVAL;
    if (c->fmt != COLI_KV_BF16 && c->fmt != COLI_KV_F16 && c->fmt != COLI_KV_E4M3) return COLI_MOE_EINVAL;
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->heads > kMaxHeads || c->dim < 1) return COLI_MOE_EINVAL;
    const int bytes = c->fmt == COLI_KV_E4M3 ? 1 : 2;
    if (c->dim > kMaxHeadDim || c->dim % (16 / bytes)) return COLI_MOE_ENOTSUP;
    // an axis of one entry needs no stride; the others must not overlap within a row
    const int64_t st[3] = {c->page_stride, c->token_stride, c->head_stride};
    const int32_t n[3] = {c->pages, c->page_size, c->heads};
    for (int i = 0; i < 3; i++) {
        if (st[i] < 0 || st[i] > kMaxStride || (n[i] > 1 && st[i] < c->dim)) return COLI_MOE_EINVAL;
        if (st[i] * bytes % 16) return COLI_MOE_EALIGN;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return COLI_MOE_EALIGN;
    return COLI_MOE_OK;
}

inline KvShape shape_of(const coli_kv_cache &c) {
    KvShape s;
    s.page_stride = c.page_stride;
    s.token_stride = c.token_stride;
    s.head_stride = c.head_stride;
    s.pages = c.pages;
    s.page_size = c.page_size;
    return s;
}

// 0 stands for `row`; a stride below it is an overlap
inline int stride_of(int64_t given, int64_t row, int64_t &out) {
    out = given == 0 ? row : given;
    return given < 0 || given > kMaxStride || out < row ? COLI_MOE_EINVAL : COLI_MOE_OK;
}

}  // namespace colimoe
