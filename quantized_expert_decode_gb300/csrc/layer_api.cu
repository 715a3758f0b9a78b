// layer_api.cu — the C ABI of the layer operators (include/colilayer.h): argument validation and
// launches. No allocation, no synchronisation.
#include <cmath>

#include "attn.h"
#include "host.h"
#include "layer_check.h"

using namespace colimoe;

namespace {

int check_attn(const coli_attn_desc *d, const coli_kv_cache *c) {
    if (!d) return COLI_MOE_EINVAL;
    if (int rc = check_cache(c)) return rc;
    if (d->seqs < 1 || d->seqs > kAttnMaxSeqs || d->q_heads < 1 || d->q_heads > kMaxHeads || d->q_heads % c->heads ||
        d->table_width < 1 || (int64_t)d->table_width * c->page_size > INT32_MAX || !act_ok(d->act) || d->window < 0 ||
        !std::isfinite(d->scale))
        return COLI_MOE_EINVAL;
    uint32_t shift;
    if (!attn_steps(shape_of(*c), c->heads, c->fmt == COLI_KV_E4M3 ? 1 : 2, shift)) return COLI_MOE_ENOTSUP;
    int64_t s;
    const int64_t row = (int64_t)d->q_heads * c->dim;
    if (stride_of(d->q_stride, row, s) || stride_of(d->out_stride, row, s)) return COLI_MOE_EINVAL;
    return COLI_MOE_OK;
}

AttnParams attn_params(const coli_attn_desc *d, const coli_kv_cache *c) {
    AttnParams p{};
    p.k_cache = c->k;
    p.v_cache = c->v;
    p.k_scale = c->fmt == COLI_KV_E4M3 ? c->k_scale : nullptr;
    p.v_scale = c->fmt == COLI_KV_E4M3 ? c->v_scale : nullptr;
    p.cache = shape_of(*c);
    stride_of(d->q_stride, (int64_t)d->q_heads * c->dim, p.q_stride);
    stride_of(d->out_stride, (int64_t)d->q_heads * c->dim, p.out_stride);
    p.scale = d->scale;
    p.seqs = d->seqs;
    p.q_heads = d->q_heads;
    p.kv_heads = c->heads;
    p.dim = c->dim;
    p.table_width = d->table_width;
    p.window = d->window;
    p.act = d->act;
    p.fmt = c->fmt;
    return p;
}

}  // namespace

extern "C" {

int coli_kv_append(const coli_append_desc *d, const coli_kv_cache *c, const void *q, const void *k, const void *v,
                   const float *inv_freq, const int32_t *seq, const int32_t *pos, const int32_t *table, void *q_out,
                   int32_t *err, coli_stream_t stream) {
    if (!d || d->reserved != 0) return COLI_MOE_EINVAL;
    if (int rc = check_cache(c)) return rc;
    if (d->tokens < 1 || d->q_heads < 0 || d->q_heads > kMaxHeads || d->seqs < 1 || d->table_width < 1 ||
        (int64_t)d->table_width * c->page_size > INT32_MAX || !act_ok(d->act) || d->rotary < 0 || d->rotary > c->dim ||
        d->rotary % 2 || (d->interleaved != 0 && d->interleaved != 1))
        return COLI_MOE_EINVAL;
    if (!k || !v || !pos || !table || (d->rotary > 0 && !inv_freq) || (d->q_heads > 0) != (q != nullptr) ||
        (d->q_heads > 0) != (q_out != nullptr) || (!seq && d->tokens > d->seqs))
        return COLI_MOE_EINVAL;
    AppendParams p{};
    const int64_t qrow = (int64_t)d->q_heads * c->dim, krow = (int64_t)c->heads * c->dim;
    if (stride_of(d->q_stride, qrow, p.q_stride) || stride_of(d->q_out_stride, qrow, p.q_out_stride) ||
        stride_of(d->k_stride, krow, p.k_stride) || stride_of(d->v_stride, krow, p.v_stride))
        return COLI_MOE_EINVAL;
    const int ab = act_bytes(d->act);
    if (!aligned(q, ab) || !aligned(k, ab) || !aligned(v, ab) || !aligned(q_out, ab) || !aligned(inv_freq, 4) ||
        !aligned(seq, 4) || !aligned(pos, 4) || !aligned(table, 4) || !aligned(err, 4))
        return COLI_MOE_EALIGN;
    // a rotation in place needs the same rows
    if (q && q == q_out && p.q_stride != p.q_out_stride) return COLI_MOE_EINVAL;
    if (int rc = check_device()) return rc;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_cache = c->k;
    p.v_cache = c->v;
    p.inv_freq = inv_freq;
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.seq = seq;
    p.pos = pos;
    p.table = table;
    p.err = err;
    p.cache = shape_of(*c);
    p.tokens = d->tokens;
    p.q_heads = d->q_heads;
    p.kv_heads = c->heads;
    p.dim = c->dim;
    p.rotary = d->rotary;
    p.interleaved = d->interleaved;
    p.seqs = d->seqs;
    p.table_width = d->table_width;
    p.act = d->act;
    p.fmt = c->fmt;
    const cudaError_t e = launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? COLI_MOE_OK : cuda_fail(e);
}

size_t coli_attn_workspace_bytes(const coli_attn_desc *d, const coli_kv_cache *c) {
    if (check_attn(d, c)) return 0;
    return attn_workspace_bytes(attn_params(d, c));
}

int coli_attn_decode(const coli_attn_desc *d, const coli_kv_cache *c, const void *q, const int32_t *table,
                     const int32_t *lens, void *out, float *lse, int32_t *err, void *ws, size_t ws_bytes,
                     coli_stream_t stream) {
    if (int rc = check_attn(d, c)) return rc;
    if (!q || !table || !lens || !out) return COLI_MOE_EINVAL;
    const int ab = act_bytes(d->act);
    if (!aligned(q, ab) || !aligned(out, ab) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4) ||
        !aligned(err, 4))
        return COLI_MOE_EALIGN;
    AttnParams p = attn_params(d, c);
    const size_t need = attn_workspace_bytes(p);
    if (need == 0) return COLI_MOE_ENOTSUP;
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return COLI_MOE_EWORKSPACE;
    if (int rc = check_device()) return rc;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.table = table;
    p.lens = lens;
    p.err = err;
    p.ws = ws;
    const cudaError_t e = launch_attn_decode(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? COLI_MOE_OK : cuda_fail(e);
}

int coli_block_norms(const coli_norms_desc *d, const void *y, const void *resid, const float *post_w, const void *gate,
                     const float *pre_w, void *resid_out, void *xn, coli_stream_t stream) {
    if (!d || d->reserved != 0) return COLI_MOE_EINVAL;
    if (d->rows < 1 || d->width < 1 || d->width > 65536 || !act_ok(d->act) || d->gate < COLI_GATE_NONE ||
        d->gate > COLI_GATE_ELEMENT || !(d->post_eps >= 0.f) || !(d->pre_eps >= 0.f) || !std::isfinite(d->post_eps) ||
        !std::isfinite(d->pre_eps) || !std::isfinite(d->resid_scale))
        return COLI_MOE_EINVAL;
    if (!y || !resid || !resid_out || (d->gate != COLI_GATE_NONE) != (gate != nullptr) || (pre_w && !xn))
        return COLI_MOE_EINVAL;
    NormsParams p{};
    if (stride_of(d->y_stride, d->width, p.y_stride) || stride_of(d->resid_stride, d->width, p.resid_stride) ||
        stride_of(d->gate_stride, d->width, p.gate_stride) ||
        stride_of(d->resid_out_stride, d->width, p.resid_out_stride) || stride_of(d->xn_stride, d->width, p.xn_stride))
        return COLI_MOE_EINVAL;
    // outputs written over an input take its place row by row
    if ((resid_out == resid && p.resid_out_stride != p.resid_stride) || (resid_out == y && p.resid_out_stride != p.y_stride) ||
        (pre_w && ((xn == y && p.xn_stride != p.y_stride) || (xn == resid && p.xn_stride != p.resid_stride) ||
                   (xn == resid_out) || (xn == gate && (d->gate != COLI_GATE_ELEMENT || p.xn_stride != p.gate_stride)))) ||
        (gate && resid_out == gate))
        return COLI_MOE_EINVAL;
    const int ab = act_bytes(d->act);
    if (!aligned(y, ab) || !aligned(resid, ab) || !aligned(gate, ab) || !aligned(resid_out, ab) ||
        (pre_w && !aligned(xn, ab)) || !aligned(post_w, 4) || !aligned(pre_w, 4))
        return COLI_MOE_EALIGN;
    if (int rc = check_device()) return rc;
    p.y = y;
    p.resid = resid;
    p.post_w = post_w;
    p.gate = gate;
    p.pre_w = pre_w;
    p.resid_out = resid_out;
    p.xn = xn;
    p.post_eps = d->post_eps;
    p.pre_eps = d->pre_eps;
    p.resid_scale = d->resid_scale;
    p.rows = d->rows;
    p.width = d->width;
    p.act = d->act;
    p.gate_kind = d->gate;
    const cudaError_t e = launch_block_norms(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? COLI_MOE_OK : cuda_fail(e);
}

}  // extern "C"
