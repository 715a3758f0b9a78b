// draft_api.cu — the C ABI of a step on drafted tokens (include/colidraft.h): argument validation and launches.
// No allocation, no synchronisation.
#include <cmath>

#include "attn.h"
#include "draft.h"
#include "layer_check.h"

using namespace colimoe;

namespace {

constexpr int kTreeSeqs = 1024, kTreeNodes = 256;
constexpr int kVerifyNodes = 1024, kMaxVocab = 1 << 20;
constexpr int kMaxLayers = 4096, kMostSeqs = 65535;

int check_tree(const coli_tree_desc *d, const coli_kv_cache *c) {
    if (!d) return COLI_MOE_EINVAL;
    if (int rc = check_cache(c)) return rc;
    if (d->seqs < 1 || d->seqs > kTreeSeqs || d->rows < 1 || d->nodes < 1 || d->nodes > kTreeNodes || d->q_heads < 1 ||
        d->q_heads > kMaxHeads || d->q_heads % c->heads || d->table_width < 1 ||
        (int64_t)d->table_width * c->page_size > INT32_MAX || !act_ok(d->act) || d->window < 0 || !std::isfinite(d->scale))
        return COLI_MOE_EINVAL;
    uint32_t shift;
    if (!attn_steps(shape_of(*c), c->heads, c->fmt == COLI_KV_E4M3 ? 1 : 2, shift)) return COLI_MOE_ENOTSUP;
    int64_t s;
    const int64_t row = (int64_t)d->q_heads * c->dim;
    if (stride_of(d->q_stride, row, s) || stride_of(d->out_stride, row, s)) return COLI_MOE_EINVAL;
    return COLI_MOE_OK;
}

TreeParams tree_params(const coli_tree_desc *d, const coli_kv_cache *c) {
    TreeParams p{};
    p.k_cache = c->k;
    p.v_cache = c->v;
    p.k_scale = c->fmt == COLI_KV_E4M3 ? c->k_scale : nullptr;
    p.v_scale = c->fmt == COLI_KV_E4M3 ? c->v_scale : nullptr;
    p.cache = shape_of(*c);
    stride_of(d->q_stride, (int64_t)d->q_heads * c->dim, p.q_stride);
    stride_of(d->out_stride, (int64_t)d->q_heads * c->dim, p.out_stride);
    p.scale = d->scale;
    p.seqs = d->seqs;
    p.rows = d->rows;
    p.nodes = d->nodes;
    p.q_heads = d->q_heads;
    p.kv_heads = c->heads;
    p.dim = c->dim;
    p.table_width = d->table_width;
    // no place is further from a node than the table is wide and the nodes are deep
    p.window = (int64_t)d->window > (int64_t)d->table_width * c->page_size ? 0 : d->window;
    p.act = d->act;
    p.fmt = c->fmt;
    return p;
}

// pools of one type, shape and strides
int check_pools(const coli_kv_cache *c, int layers) {
    if (!c || layers < 1 || layers > kMaxLayers) return COLI_MOE_EINVAL;
    for (int i = 0; i < layers; i++) {
        if (int rc = check_cache(c + i)) return rc;
        if (c[i].fmt != c->fmt || c[i].pages != c->pages || c[i].page_size != c->page_size || c[i].heads != c->heads ||
            c[i].dim != c->dim || c[i].page_stride != c->page_stride || c[i].token_stride != c->token_stride ||
            c[i].head_stride != c->head_stride)
            return COLI_MOE_EINVAL;
    }
    return COLI_MOE_OK;
}

// `launch` for every kPoolLayers layers
template <typename P, typename F>
int each_pools(const coli_kv_cache *c, int layers, P &p, F launch) {
    for (int at = 0; at < layers; at += kPoolLayers) {
        Pools pools{};
        p.layers = layers - at < kPoolLayers ? layers - at : kPoolLayers;
        for (int i = 0; i < p.layers; i++) {
            pools.k[i] = c[at + i].k;
            pools.v[i] = c[at + i].v;
        }
        const cudaError_t e = launch(p, pools);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return COLI_MOE_OK;
}

}  // namespace

extern "C" {

int coli_norm_append(const coli_norm_append_desc *d, const coli_kv_cache *c, const void *q, const void *k, const void *v,
                     const float *q_norm, const float *k_norm, const float *inv_freq, const int32_t *seq, const int32_t *pos,
                     const int32_t *place, const int32_t *table, void *q_out, int32_t *err, coli_stream_t stream) {
    if (!d) return COLI_MOE_EINVAL;
    if (int rc = check_cache(c)) return rc;
    if (d->tokens < 1 || d->q_heads < 0 || d->q_heads > kMaxHeads || d->seqs < 1 || d->table_width < 1 ||
        (int64_t)d->table_width * c->page_size > INT32_MAX || !act_ok(d->act) || d->rotary < 0 || d->rotary > c->dim ||
        d->rotary % 2 || (d->interleaved != 0 && d->interleaved != 1) || !(d->eps >= 0.f) || !std::isfinite(d->eps))
        return COLI_MOE_EINVAL;
    if (!k || !v || !pos || !table || (d->rotary > 0 && !inv_freq) || (d->q_heads > 0) != (q != nullptr) ||
        (d->q_heads > 0) != (q_out != nullptr) || (!seq && d->tokens > d->seqs) || (q_norm && !q))
        return COLI_MOE_EINVAL;
    NormAppendParams p{};
    AppendParams &a = p.a;
    const int64_t qrow = (int64_t)d->q_heads * c->dim, krow = (int64_t)c->heads * c->dim;
    if (stride_of(d->q_stride, qrow, a.q_stride) || stride_of(d->q_out_stride, qrow, a.q_out_stride) ||
        stride_of(d->k_stride, krow, a.k_stride) || stride_of(d->v_stride, krow, a.v_stride))
        return COLI_MOE_EINVAL;
    const int ab = act_bytes(d->act);
    if (!aligned(q, ab) || !aligned(k, ab) || !aligned(v, ab) || !aligned(q_out, ab) || !aligned(inv_freq, 4) ||
        !aligned(seq, 4) || !aligned(pos, 4) || !aligned(place, 4) || !aligned(table, 4) || !aligned(err, 4) ||
        !aligned(q_norm, 4) || !aligned(k_norm, 4))
        return COLI_MOE_EALIGN;
    // a rotation in place needs the same rows
    if (q && q == q_out && a.q_stride != a.q_out_stride) return COLI_MOE_EINVAL;
    if (int rc = check_device()) return rc;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_cache = c->k;
    a.v_cache = c->v;
    a.inv_freq = inv_freq;
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.seq = seq;
    a.pos = pos;
    a.table = table;
    a.err = err;
    a.cache = shape_of(*c);
    a.tokens = d->tokens;
    a.q_heads = d->q_heads;
    a.kv_heads = c->heads;
    a.dim = c->dim;
    a.rotary = d->rotary;
    a.interleaved = d->interleaved;
    a.seqs = d->seqs;
    a.table_width = d->table_width;
    a.act = d->act;
    a.fmt = c->fmt;
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.place = place;
    p.eps = d->eps;
    const cudaError_t e = launch_norm_append(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? COLI_MOE_OK : cuda_fail(e);
}

size_t coli_tree_workspace_bytes(const coli_tree_desc *d, const coli_kv_cache *c) {
    if (check_tree(d, c)) return 0;
    return tree_workspace_bytes(tree_params(d, c));
}

int coli_attn_tree(const coli_tree_desc *d, const coli_kv_cache *c, const void *q, const int32_t *first, const int32_t *past,
                   const int32_t *parent, const int32_t *table, void *out, float *lse, int32_t *err, void *ws,
                   size_t ws_bytes, coli_stream_t stream) {
    if (int rc = check_tree(d, c)) return rc;
    if (!q || !first || !past || !table || !out || q == out) return COLI_MOE_EINVAL;
    const int ab = act_bytes(d->act);
    if (!aligned(q, ab) || !aligned(out, ab) || !aligned(first, 4) || !aligned(past, 4) || !aligned(parent, 4) ||
        !aligned(table, 4) || !aligned(lse, 4) || !aligned(err, 4))
        return COLI_MOE_EALIGN;
    TreeParams p = tree_params(d, c);
    const size_t need = tree_workspace_bytes(p);
    if (need == 0) return COLI_MOE_ENOTSUP;
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return COLI_MOE_EWORKSPACE;
    if (int rc = check_device()) return rc;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.first = first;
    p.past = past;
    p.parent = parent;
    p.table = table;
    p.err = err;
    p.ws = ws;
    const cudaError_t e = launch_attn_tree(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? COLI_MOE_OK : cuda_fail(e);
}

int coli_draft_verify(const coli_verify_desc *d, const void *target, const void *draft, const int32_t *tokens,
                      const int32_t *parent, const float *uniform, const int32_t *first, int32_t *path, int32_t *count,
                      int32_t *next, int32_t *err, coli_stream_t stream) {
    if (!d) return COLI_MOE_EINVAL;
    if (d->seqs < 1 || d->seqs > kMostSeqs || d->rows < 1 || d->nodes < 1 || d->nodes > kVerifyNodes || d->vocab < 1 ||
        d->vocab > kMaxVocab || !act_ok(d->act) || (d->mode != COLI_VERIFY_SAMPLE && d->mode != COLI_VERIFY_GREEDY))
        return COLI_MOE_EINVAL;
    if (!target || !tokens || !first || !path || !count || !next) return COLI_MOE_EINVAL;
    if (d->mode == COLI_VERIFY_GREEDY ? (draft || uniform) : !uniform) return COLI_MOE_EINVAL;
    VerifyParams p{};
    if (stride_of(d->target_stride, d->vocab, p.target_stride) || stride_of(d->draft_stride, d->vocab, p.draft_stride))
        return COLI_MOE_EINVAL;
    const int ab = act_bytes(d->act);
    if (!aligned(target, ab) || !aligned(draft, ab) || !aligned(tokens, 4) || !aligned(parent, 4) || !aligned(uniform, 4) ||
        !aligned(first, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(next, 4) || !aligned(err, 4))
        return COLI_MOE_EALIGN;
    if (int rc = check_device()) return rc;
    p.target = target;
    p.draft = draft;
    p.tokens = tokens;
    p.parent = parent;
    p.first = first;
    p.uniform = uniform;
    p.path = path;
    p.count = count;
    p.next = next;
    p.err = err;
    p.seqs = d->seqs;
    p.rows = d->rows;
    p.nodes = d->nodes;
    p.vocab = d->vocab;
    p.act = d->act;
    p.mode = d->mode;
    const cudaError_t e = launch_draft_verify(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? COLI_MOE_OK : cuda_fail(e);
}

int coli_kv_compact(const coli_compact_desc *d, const coli_kv_cache *caches, const int32_t *past, const int32_t *path,
                    const int32_t *count, const int32_t *table, int32_t *err, coli_stream_t stream) {
    if (!d) return COLI_MOE_EINVAL;
    if (int rc = check_pools(caches, d->layers)) return rc;
    if (d->seqs < 1 || d->seqs > kMostSeqs || d->nodes < 1 || d->table_width < 1 ||
        (int64_t)d->table_width * caches->page_size > INT32_MAX)
        return COLI_MOE_EINVAL;
    if (!past || !path || !count || !table) return COLI_MOE_EINVAL;
    if (!aligned(past, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(table, 4) || !aligned(err, 4))
        return COLI_MOE_EALIGN;
    if (int rc = check_device()) return rc;
    CompactParams p{};
    p.cache = shape_of(*caches);
    p.past = past;
    p.path = path;
    p.count = count;
    p.table = table;
    p.err = err;
    p.seqs = d->seqs;
    p.nodes = d->nodes;
    p.table_width = d->table_width;
    p.heads = caches->heads;
    p.elem_bytes = caches->fmt == COLI_KV_E4M3 ? 1 : 2;
    p.row_bytes = caches->dim * p.elem_bytes;
    return each_pools(caches, d->layers, p, [&](const CompactParams &part, const Pools &pools) {
        return launch_kv_compact(part, pools, reinterpret_cast<cudaStream_t>(stream));
    });
}

int coli_kv_copy_pages(const coli_kv_cache *caches, int32_t layers, int32_t n, const int32_t *src, const int32_t *dst,
                       int32_t *err, coli_stream_t stream) {
    if (int rc = check_pools(caches, layers)) return rc;
    if (n < 1 || !src || !dst) return COLI_MOE_EINVAL;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(err, 4)) return COLI_MOE_EALIGN;
    if (int rc = check_device()) return rc;
    CopyParams p{};
    p.cache = shape_of(*caches);
    p.src = src;
    p.dst = dst;
    p.err = err;
    p.n = n;
    p.heads = caches->heads;
    p.elem_bytes = caches->fmt == COLI_KV_E4M3 ? 1 : 2;
    p.row_bytes = caches->dim * p.elem_bytes;
    return each_pools(caches, layers, p, [&](const CopyParams &part, const Pools &pools) {
        return launch_kv_copy(part, pools, reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
