/* lean_cache.h -- the paged cache of lean_step.h beyond one new token per
 * sequence: tokens read back out of it, and attention where many sequences begin
 * with one prefix whose keys and values the cache holds once.
 *
 * Conventions: those of lean_step.h.  Caches may be LEAN_BF16, LEAN_F16 or
 * LEAN_I8 (whole numbers with a scale for each token and kv head).
 */
#ifndef LEAN_CACHE_H
#define LEAN_CACHE_H

#include <stdint.h>

#include "lean_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens read back: k_out[t], v_out[t] are what the caches hold at slots[t] =
 * page * page_size + place, for t in 0..n_tokens-1, in out_dtype (LEAN_I8: c * s
 * in fp32, rounded once).  A prompt's earlier tokens come back so as contiguous
 * rows for its next chunk; a slot may be read any number of times.  A negative
 * slot gives zeros (padding).  A slot at or past n_pages * page_size gives NaN
 * and sets bit 64 of the device error word.
 * Either cache may be left out together with its output.  Outputs overlap nothing.
 * LEAN_ERR_SHAPE: n_tokens, n_kv_heads or head_dim <= 0, above 2^31 - 1 tokens,
 * 65536 heads or head_dim 512, a negative stride, page_size or n_pages <= 0 or
 * more than 2^31 - 1 slots.  LEAN_ERR_NULL: a part missing, or both caches.
 * LEAN_ERR_FORMAT: an unknown type.  LEAN_ERR_ALIGN: a pointer off its element
 * (rows on 16 bytes are read fastest). */
typedef struct {
    int64_t n_tokens, n_kv_heads, head_dim;
    int64_t out_dtype;
    int64_t cache_dtype;
    const void *k_cache;      /* [page][place][kv head][head_dim] by strides   */
    const void *v_cache;      /* the same strides                              */
    int64_t n_pages, page_size;
    int64_t page_stride, place_stride, cache_head_stride;
    const float *k_scales, *v_scales; /* LEAN_I8: [page][place][kv head] by strides */
    int64_t scale_page_stride, scale_place_stride, scale_head_stride;
    const int32_t *slots;     /* int32[n_tokens]                               */
    void *k_out;              /* [token][head][head_dim]                       */
    int64_t k_out_stride, k_out_head_stride;
    void *v_out;
    int64_t v_out_stride, v_out_head_stride;
    int64_t flags;
} lean_kv_read_args;
lean_status lean_kv_read(const lean_kv_read_args *args, void *stream);

/* Attention of one new token per sequence, where sequences share prefixes:
 * sequences seq_starts[p] .. seq_starts[p + 1] - 1 begin with the prefix_lens[p]
 * tokens in the pages of row p of prefix_table, and go on with seq_lens[s] tokens
 * of their own in the pages of row s of block_table (the new token's k and v
 * among them, or among the prefix's):
 *   out[s][h] = sum_j p_j v_j,  p = softmax_j(scale * q[s][h] . k_j)
 * over both.  A prefix's keys and values are read once for up to 128 rows (query
 * heads that share a kv head, of its sequences), not once for each sequence; once
 * for 256 where q and p are in one part (below) and the sequences' rows, shared out
 * evenly, come to more than 128 a prefix.
 * Sequences before seq_starts[0] or from seq_starts[n_prefixes] on have no
 * prefix.  seq_starts ascends, from 0 on, to n_seqs at most; where it does not,
 * what comes out for the sequences concerned is unspecified (numbers outside
 * 0..n_seqs count as the nearest of these, a descent as no sequences).  A
 * sequence of no tokens at all gives out 0 and lse -inf.
 * Lengths, pages, what is not finite, lse, and what lies past a length: as for
 * lean_paged_attention, a prefix's like a sequence's.
 * Precision: of the prefix, 16-bit out takes p in one part of the operands' type
 * (that of the cache; f16 for LEAN_I8), which errs by 2^-8 of sum p |v| at most
 * (bf16; f16 2^-11 and, for each key, 2^-34 of the largest p, LEAN_I8: of the largest
 * p times the largest of the v_scales), and is summed in fp32: less exact than
 * lean_paged_attention over a joined table, which takes two.  fp32 out, and f16 out
 * of a bf16 cache, takes q and p in three parts, which leave nothing of fp32's
 * precision behind but what f16 operands do there.  Sequences' own tokens, and how large
 * values may be, are as for lean_paged_attention.
 * q, out: 16-byte aligned, strides multiples of 8 elements; caches: 16-byte
 * aligned, strides multiples of 16 bytes.  workspace:
 * lean_prefix_attention_workspace_bytes() bytes, 256-byte aligned, any contents.
 * Calls that may run at the same time must not share one.  Results do not depend
 * on timing.
 * LEAN_ERR_SHAPE: as for lean_paged_attention, of both tables, with head_dim at
 * most 128 (LEAN_I8: a multiple of 16), prefixes whose pages can hold more than
 * 2^31 - 129 tokens, n_prefixes <= 0 or above n_seqs, query
 * heads and prefixes x tokens that a prefix's pages can hold / 2^14 near 2^32 or
 * above, or a workspace too small. */
typedef struct {
    int64_t n_seqs, n_q_heads, n_kv_heads, head_dim;
    int64_t act_dtype;         /* of q and out                                 */
    int64_t cache_dtype;
    const void *q;             /* [seq][head][head_dim]                        */
    int64_t q_stride, q_head_stride;
    const void *k_cache, *v_cache;
    int64_t n_pages, page_size;
    int64_t page_stride, place_stride, cache_head_stride;
    const float *k_scales, *v_scales; /* LEAN_I8                               */
    int64_t scale_page_stride, scale_place_stride, scale_head_stride;
    int64_t n_prefixes;
    const int32_t *prefix_table; /* int32[n_prefixes][prefix_stride]           */
    int64_t prefix_width, prefix_stride;
    const int32_t *prefix_lens; /* int32[n_prefixes]                           */
    const int32_t *seq_starts; /* int32[n_prefixes + 1]                        */
    const int32_t *block_table; /* int32[n_seqs][table_stride]                 */
    int64_t table_width, table_stride;
    const int32_t *seq_lens;   /* int32[n_seqs]                                */
    void *out;                 /* [seq][head][head_dim]                        */
    int64_t out_stride, out_head_stride;
    float *lse;                /* float[n_seqs][n_q_heads], or NULL            */
    double scale;
    void *workspace;
    int64_t workspace_bytes;
    int64_t flags;
} lean_prefix_args;
lean_status lean_prefix_attention(const lean_prefix_args *args, void *stream);
/* -1 for sizes that lean_prefix_attention refuses. */
int64_t lean_prefix_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                              int64_t head_dim, int64_t n_prefixes);

#ifdef __cplusplus
}
#endif

#endif /* LEAN_CACHE_H */
