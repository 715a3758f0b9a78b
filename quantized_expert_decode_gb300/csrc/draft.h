// draft.h — host-side launchers of the kernels of a step on drafted tokens (internal, not part of the ABI).
#pragma once

#include "colidraft.h"
#include "draft_index.h"
#include "layer.h"

namespace colimoe {

struct NormAppendParams {
    AppendParams a;
    const float *q_norm, *k_norm;
    const int32_t *place;
    float eps;
};
cudaError_t launch_norm_append(const NormAppendParams &p, cudaStream_t s);

struct TreeParams {
    const void *q, *k_cache, *v_cache;
    void *out;
    float *lse;
    const float *k_scale, *v_scale;
    const int32_t *first, *past, *parent, *table;
    int32_t *err;
    KvShape cache;
    int64_t q_stride, out_stride;
    float scale;
    int32_t seqs, rows, nodes, q_heads, kv_heads, dim, table_width, window;
    int32_t act, fmt;
    void *ws;
};
size_t tree_workspace_bytes(const TreeParams &p);
cudaError_t launch_attn_tree(const TreeParams &p, cudaStream_t s);

struct VerifyParams {
    const void *target, *draft;
    const int32_t *tokens, *parent, *first;
    const float *uniform;
    int32_t *path, *count, *next, *err;
    int64_t target_stride, draft_stride;
    int32_t seqs, rows, nodes, vocab, act, mode;
};
cudaError_t launch_draft_verify(const VerifyParams &p, cudaStream_t s);

// Pools of the layers that one launch takes
constexpr int kPoolLayers = 64;
struct Pools {
    void *k[kPoolLayers], *v[kPoolLayers];
};
struct CompactParams {
    KvShape cache;
    const int32_t *past, *path, *count, *table;
    int32_t *err;
    int32_t seqs, nodes, table_width, layers, heads, row_bytes, elem_bytes;
};
cudaError_t launch_kv_compact(const CompactParams &p, const Pools &pools, cudaStream_t s);

struct CopyParams {
    KvShape cache;
    const int32_t *src, *dst;
    int32_t *err;
    int32_t n, layers, heads, row_bytes, elem_bytes;
};
cudaError_t launch_kv_copy(const CopyParams &p, const Pools &pools, cudaStream_t s);

}  // namespace colimoe
