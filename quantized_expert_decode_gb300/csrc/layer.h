// layer.h — host-side launchers of the layer operators' kernels (internal, not part of the ABI).
#pragma once

#include "colilayer.h"
#include "kv_index.h"

#include <cuda_runtime.h>

namespace colimoe {

struct AppendParams {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    const float *inv_freq, *k_scale, *v_scale;
    const int32_t *seq, *pos, *table;
    int32_t *err;
    KvShape cache;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int32_t tokens, q_heads, kv_heads, dim, rotary, interleaved, seqs, table_width;
    int32_t act, fmt;
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t s);

struct AttnParams {
    const void *q, *k_cache, *v_cache;
    void *out;
    float *lse;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    int32_t *err;
    KvShape cache;
    int64_t q_stride, out_stride;
    float scale;
    int32_t seqs, q_heads, kv_heads, dim, table_width, window;
    int32_t act, fmt;
    void *ws;
};
size_t attn_workspace_bytes(const AttnParams &p);
cudaError_t launch_attn_decode(const AttnParams &p, cudaStream_t s);

struct NormsParams {
    const void *y, *resid, *gate;
    const float *post_w, *pre_w;
    void *resid_out, *xn;
    int64_t y_stride, resid_stride, gate_stride, resid_out_stride, xn_stride;
    float post_eps, pre_eps, resid_scale;
    int32_t rows, width, act, gate_kind;
};
cudaError_t launch_block_norms(const NormsParams &p, cudaStream_t s);

}  // namespace colimoe
