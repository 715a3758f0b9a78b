/* colilayer.h — C ABI of libcolimoe, second part: the operators around the MoE block that a
 * decoder layer needs besides it, computed by hand-written CUDA kernels for GB300 (sm_103a).
 *
 *   coli_kv_append    rotates new tokens' queries and keys by their positions and appends keys and
 *                     values to a paged cache
 *   coli_attn_decode  attention of one new token per sequence over that cache
 *   coli_block_norms  the norms before and after a block, its gate and the scaled residual
 *
 * Conventions are those of colimoe.h: tensors live in DEVICE memory, the caller owns every buffer,
 * nothing is allocated, freed or synchronised inside a call, work is enqueued on `stream` on the
 * current device (so every call can be captured into a graph), arguments are validated on the host
 * before anything is launched, and the return value is COLI_MOE_OK or a COLI_MOE_E* code. The
 * tensors must be ready on `stream`.
 *
 * Conditions that only the device can see (a page number outside the pool, a position beyond the
 * page table, a sequence number out of range) never lead to an access: the entry is skipped, or
 * attends to what is left, and a bit is set in the error word `err` (device int32, may be NULL;
 * zeroed by the caller once). coli_moe_check(err, stream) reads and clears it.
 */
#ifndef COLILAYER_H
#define COLILAYER_H

#include "colimoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* activation types */
#define COLI_ACT_F32 0
#define COLI_ACT_BF16 1
#define COLI_ACT_F16 2

/* cache types */
#define COLI_KV_BF16 1
#define COLI_KV_F16 2
#define COLI_KV_E4M3 3 /* 8-bit floats, one fp32 scale per kv head */

/* bits of the error word */
#define COLI_LAYER_BAD_PAGE 1     /* a page number outside [0, pages) */
#define COLI_LAYER_BAD_POSITION 2 /* a position or length beyond table_width * page_size, or below 0 */
#define COLI_LAYER_BAD_SEQUENCE 4 /* a sequence number outside [0, seqs) */

/* A paged cache: `pages` pages of `page_size` tokens, for keys and (with the same strides) for
 * values. The row of `dim` contiguous elements of page p, slot s, kv head h starts
 * p * page_stride + s * token_stride + h * head_stride elements behind k (or v). Any order of the
 * three axes is taken; offsets are computed in 64 bits. Strides are multiples of 16 bytes and k, v
 * 16-byte aligned (COLI_MOE_EALIGN). dim: a multiple of 16 bytes of elements, at most 256
 * (COLI_MOE_ENOTSUP). The attention reaches rows by 32-bit multiples of the strides' largest common power of
 * two, which is at least 16 bytes: 64 GB of keys at that least, 1 TB at rows of 256 bytes; beyond, it
 * answers COLI_MOE_ENOTSUP. COLI_KV_E4M3 stores value / scale[head] (the quotient rounded to fp32, then to
 * e4m3), saturated to +-448 (NaN stays NaN); a NULL scale stands for 1. The scales are ignored for the other types. */
typedef struct {
    void *k, *v;
    const float *k_scale, *v_scale; /* [heads] each */
    int32_t fmt;
    int32_t pages;
    int32_t page_size;
    int32_t heads; /* kv heads, <= 1024 */
    int32_t dim;
    int32_t reserved; /* 0 */
    int64_t page_stride, token_stride, head_stride;
} coli_kv_cache;

/* Append: `tokens` new tokens. Row n of q, k, v and q_out starts n * *_stride elements behind the
 * pointer and holds its heads one after another, dim elements each (so q, k and v may be slices of
 * one projection's output). A stride of 0 stands for heads * dim. */
typedef struct {
    int32_t tokens;      /* >= 1 */
    int32_t q_heads;     /* heads of q; 0: no q */
    int32_t seqs;        /* rows of the page table */
    int32_t table_width; /* entries per row of the page table */
    int32_t act;         /* COLI_ACT_* of q, k, v and q_out */
    int32_t rotary;      /* leading elements of each head that are rotated: even, 0..dim */
    int32_t interleaved; /* 1: pairs (2i, 2i+1); 0: pairs (i, i + rotary/2) */
    int32_t reserved;    /* 0 */
    int64_t q_stride, k_stride, v_stride, q_out_stride;
} coli_append_desc;

/* For every token n, with b = seq[n] (seq NULL: b = n) and p = pos[n] (its position in its
 * sequence, counted from 0, which is also its place in the cache):
 *   the first `rotary` elements of each head of q and k are rotated pairwise by the angle
 *     p * inv_freq[i], i < rotary/2:  (a, b) -> (a cos - b sin, b cos + a sin)
 *     (angles reduced to a fraction of a turn in 64-bit fixed point, so far positions keep their
 *     angle; the rest is fp32)
 *   q_out[n] = rotated q[n], in q's type (q_out may be q itself)
 *   page table[b][p / page_size], slot p % page_size of the cache = rotated k[n] and v[n], rounded
 *     once to the cache's type.
 * A token with seq[n] = -1 is padding: its q is rotated, nothing is cached and no error is flagged. Two tokens
 * must not name the same place. q and q_out are NULL iff q_heads is 0; inv_freq [rotary/2] fp32 may
 * be NULL iff rotary is 0; table [seqs][table_width] int32, pos and seq [tokens] int32. */
int coli_kv_append(const coli_append_desc *desc, const coli_kv_cache *cache, const void *q, const void *k,
                   const void *v, const float *inv_freq, const int32_t *seq, const int32_t *pos,
                   const int32_t *table, void *q_out, int32_t *err, coli_stream_t stream);

/* Attention of one new token per sequence. */
typedef struct {
    int32_t seqs;        /* 1..2048 */
    int32_t q_heads;     /* a multiple of cache->heads, <= 1024; head h reads kv head h / (q_heads / heads) */
    int32_t table_width; /* entries per row of the page table; table_width * page_size < 2^31 */
    int32_t act;         /* COLI_ACT_* of q and out */
    int32_t window;      /* > 0: only the last `window` cached tokens are seen; 0: all */
    float scale;         /* factor of q . k, usually 1 / sqrt(dim); finite */
    int64_t q_stride, out_stride; /* elements from one sequence's row to the next; 0: q_heads * dim */
} coli_attn_desc;

/* Bytes of device workspace (256-byte aligned) coli_attn_decode needs; 0 if a description is
 * invalid. The workspace needs no preparation and may be shared with other calls on one stream. */
size_t coli_attn_workspace_bytes(const coli_attn_desc *desc, const coli_kv_cache *cache);

/* For sequence b with n = lens[b] cached tokens (the new token's own among them) and head h:
 *   s_t = scale * q . k_t  for t in [max(0, n - window), n),   p = softmax(s)
 *   out[b][h] = sum_t p_t v_t, rounded once to q's type;  lse[b][h] = ln(sum_t exp(s_t))
 * A sequence of no tokens gives out = 0 and lse = -inf. Tokens whose page number is outside the pool
 * are left out (and flagged); a length outside [0, table_width * page_size] is clamped (and flagged).
 * What the pages hold behind a sequence's end, before its window, or on pages that no table names
 * is never used, whatever its bits. The products of q and k and the sums are fp32 (q and p enter the
 * tensor cores as sums of 16-bit parts, so that fp32 activations keep 22 bits or more; beside 16-bit activations
 * p keeps 16 bits on a bf16 cache, 22 on the others); scores, maxima and sums of the softmax are fp32.
 * Keys and values that are seen should be finite: an infinity among them may give NaN where the formula has
 * an infinity or leaves a token out (the parts make it 0 times infinity).
 *   q [seqs][q_heads][dim], out alike, lse [seqs][q_heads] fp32 or NULL, lens [seqs] int32,
 *   table [seqs][table_width] int32 (entries behind a sequence's end are not read).
 * The same call gives the same bits: the split over the length and the order of its join are fixed
 * by the lengths. */
int coli_attn_decode(const coli_attn_desc *desc, const coli_kv_cache *cache, const void *q, const int32_t *table,
                     const int32_t *lens, void *out, float *lse, int32_t *err, void *ws, size_t ws_bytes,
                     coli_stream_t stream);

/* what a gate multiplies */
#define COLI_GATE_NONE 0
#define COLI_GATE_CHANNEL 1 /* gate [width]: one factor per channel */
#define COLI_GATE_ROW 2     /* gate [rows]: one factor per token */
#define COLI_GATE_ELEMENT 3 /* gate [rows][width] */

/* Norms around a block. Strides are elements from one row to the next; 0 stands for width. */
typedef struct {
    int32_t rows;  /* >= 1 */
    int32_t width; /* 1..65536 */
    int32_t act;   /* COLI_ACT_* of y, resid, gate, resid_out and xn */
    int32_t gate;  /* COLI_GATE_* */
    float post_eps, pre_eps; /* >= 0 */
    float resid_scale;
    int32_t reserved; /* 0 */
    int64_t y_stride, resid_stride, gate_stride, resid_out_stride, xn_stride;
} coli_norms_desc;

/* For every row, y the block's output and resid the residual stream before it:
 *   z = y * post_w / sqrt(mean(y^2) + post_eps)          (post_w NULL: z = y)
 *   r = resid_scale * resid + gate * z                   -> resid_out
 *   xn = r * pre_w / sqrt(mean(r^2) + pre_eps)           (pre_w NULL: not written, xn may be NULL)
 * xn is the input of the next block. Everything is fp32 and rounded once, on the way to resid_out
 * and xn; the second norm uses r before that rounding. post_w, pre_w [width] fp32. resid_out may be
 * resid or y, and xn may be y, resid or the element gate (rows are read whole before they are
 * written; the strides of the two must then be the same). Any width, alignment and stride is taken;
 * the 16-byte path needs width, strides and pointers in multiples of 16 bytes. */
int coli_block_norms(const coli_norms_desc *desc, const void *y, const void *resid, const float *post_w,
                     const void *gate, const float *pre_w, void *resid_out, void *xn, coli_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* COLILAYER_H */
