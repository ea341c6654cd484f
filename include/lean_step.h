/* lean_step.h -- the operators of a serving step around the quantized linears
 * of lean_qmatmul.h: residual sums with their norms, rotary positions with the
 * append to a paged key-value cache, the cache's page bookkeeping, attention of
 * one new token per sequence over that cache, and what is read off the lm_head's
 * logits (log probabilities, entropy, top alternatives).
 *
 * Pages: the "wgpu-llm" README, Architecture at a Glance, runs a decode step as
 * N x (attention + FFN) over a paged KV cache; the linears alone do not make
 * one.  The pages give no interface for the rest; this one is the library's own.
 *
 * Conventions (besides those of lean_qmatmul.h: nothing is allocated, nothing
 * synchronises, calls run on `stream` and may be captured into a CUDA graph,
 * argument errors are returned before anything is queued):
 *   - A call takes its arguments in a struct, read during the call only.  Zero
 *     it first (lean_norm_args a = {0}): optional parts are off when 0 or NULL.
 *   - Every field is 8 bytes wide.  Strides count elements, not bytes, and are
 *     >= 0; the innermost dimension is contiguous.
 *   - Every pointer is device memory unless it says host, aligned to its element
 *     unless it says more.
 *   - Arithmetic is fp32 (or wider) whatever the buffers hold; results are
 *     rounded once, to nearest even, when they are stored.
 *   - flags: 0 or LEAN_FLAG_EARLY_WEIGHTS (the kernel may be scheduled before
 *     the preceding kernel on `stream` has finished; it waits for it before it
 *     touches anything).  Others: LEAN_ERR_FORMAT.
 *   - What only the device can see is reported in outputs, as each call says, and
 *     in the device error word (lean_device_error): bit 64, a page or slot
 *     outside the cache, bit 256, a token id outside the vocabulary.
 */
#ifndef LEAN_STEP_H
#define LEAN_STEP_H

#include <stdint.h>

#include "lean_qmatmul.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations, residuals and caches.  LEAN_I8: of caches only
 * (lean_rope_append, lean_paged_attention and the calls of lean_cache.h), whole
 * numbers c in -127..127 with one fp32 scale s, 0 or above, for each token and kv
 * head, which stand for c * s.  The scales lie in two arrays beside the caches, at page *
 * scale_page_stride + place * scale_place_stride + kv head * scale_head_stride
 * (a head's places beside one another are read fastest: scale_place_stride 1).
 * Their fields end the structs and are read for such caches only. */
typedef enum { LEAN_F32 = 0, LEAN_BF16 = 1, LEAN_F16 = 2, LEAN_I8 = 3 } lean_dtype;

/* Residual sum with the norms before and after a block, for each of `rows`
 * rows of `width` elements:
 *   u  = post_w ? post_w * x / sqrt(mean(x^2) + eps) : x
 *   h' = h + res_scale * (gate ? gate * u : u)
 *   y  = (w ? w : 1) * h' / sqrt(mean(h'^2) + eps)
 * x is a block's output, h the residual stream, y the next block's input.  x =
 * NULL: h' = h (the norm before the first block); h = NULL: no residual (h' is
 * the branch alone).  y is computed from h' before h' is rounded for h_out.
 * h_out and y may be NULL (not stored), and may be the buffers of h and x with
 * the same strides; otherwise outputs overlap nothing.
 * LEAN_ERR_SHAPE: rows or width <= 0 or above 2^30 - 1, a negative stride, or an output's stride
 * below width with more than one row.  LEAN_ERR_NULL: x and h both NULL, h_out
 * and y both NULL, or a gate or post_w without x.  LEAN_ERR_FORMAT: an unknown
 * type, or a residual type that is neither LEAN_F32 nor act_dtype. */
typedef struct {
    int64_t rows, width;
    int64_t act_dtype;       /* of x, gate and y                              */
    int64_t res_dtype;       /* of h and h_out: LEAN_F32 or act_dtype         */
    const void *x;
    int64_t x_stride;        /* elements from one row to the next             */
    const void *h;
    int64_t h_stride;
    const void *gate;        /* multiplied as it is                           */
    int64_t gate_stride;     /* 0: one row for all                            */
    const float *post_w;     /* float[width]                                  */
    const float *w;          /* float[width]                                  */
    void *h_out;
    int64_t h_out_stride;
    void *y;
    int64_t y_stride;
    double eps, res_scale;
    int64_t flags;
} lean_norm_args;
lean_status lean_residual_norm(const lean_norm_args *args, void *stream);

/* Rotary frequencies as whole numbers: turns[i] = 2^64 * freq[i] / (2 pi) mod
 * 2^64, the turns that pair i makes per position in units of 2^-64.  The upper
 * half of position * turns[i] in 64-bit arithmetic is then the angle, exact at
 * any position: whole turns drop out by themselves.  Host; freq[i] in radians
 * per position, finite and >= 0.  LEAN_ERR_SHAPE otherwise or for n <= 0. */
lean_status lean_rope_turns(const double *freq, int64_t n, uint64_t *turns);

/* How lean_rope_frequencies scales the frequencies base^(-2i / rot_dim) for
 * contexts longer than the trained one (s = factor, L = trained_len):
 *   LEAN_ROPE_PLAIN   not at all
 *   LEAN_ROPE_LINEAR  freq / s (positions interpolated)
 *   LEAN_ROPE_BASE    base replaced by base * s^(rot_dim / (rot_dim - 2))
 *   LEAN_ROPE_RAMP    freq * (1 - r + r / s) with r linear in the pair's index i,
 *                     from 0 where a pair makes `fast` turns within L to 1 where
 *                     it makes `slow`: r = (i - lo) / max(hi - lo, 0.001) held to
 *                     0..1, lo = max(0, floor c(fast)), hi = min(rot_dim - 1,
 *                     ceil c(slow)), c(t) = rot_dim ln(L / (2 pi t)) / (2 ln base)
 *   LEAN_ROPE_BANDS   the same with r linear in the pair's own turns within L, t =
 *                     L freq / (2 pi): r = 1 - (t - slow) / (fast - slow) held to
 *                     0..1 */
enum {
    LEAN_ROPE_PLAIN = 0,
    LEAN_ROPE_LINEAR = 1,
    LEAN_ROPE_BASE = 2,
    LEAN_ROPE_RAMP = 3,
    LEAN_ROPE_BANDS = 4
};
/* freq[rot_dim / 2], host.  base > 1, rot_dim even and > 0 (LEAN_ROPE_BASE: >
 * 2), factor >= 1; LEAN_ROPE_RAMP and LEAN_ROPE_BANDS also trained_len > 0 and
 * fast > slow > 0.  LEAN_ERR_SHAPE otherwise, LEAN_ERR_FORMAT for an unknown
 * kind.  (The length-dependent scale of the rotated vectors that goes with some
 * of these is rot_scale below.) */
lean_status lean_rope_frequencies(int kind, int64_t rot_dim, double base, double factor,
                                  double trained_len, double slow, double fast, double *freq);

/* Rotary positions of new tokens' q and k, and the append of k and v to the
 * paged cache.  The first rot_dim elements of each head of q and k are rotated,
 * the others copied: pair i is (x[i], x[i + rot_dim/2]), or (x[2i], x[2i+1])
 * when interleaved, and with angle a = positions[t] * freq[i]
 *   (u, v) -> rot_scale * (u cos a - v sin a, u sin a + v cos a).
 * Token t's k and v go to the cache at slots[t] = page * page_size + place; a
 * negative slot stores nothing (padding).  A slot at or past n_pages *
 * page_size stores nothing and sets bit 64 of the device error word.  Two tokens
 * of a call must not share a slot.
 * Negative positions turn backwards.  q and q_out may be NULL together (n_q_heads
 * 0), and so may k, v and both caches (n_kv_heads 0).  k_out, optional, receives
 * the rotated k as well.  q_out may be q and k_out may be k, with the same
 * strides; otherwise outputs overlap nothing.
 * LEAN_I8 caches: a head's elements x (of k as rotated in fp32, before k_out's
 * rounding) are stored as s = max |x| / 127, rounded to fp32, and c = the whole
 * number nearest to x / s, halves away from 0; s = 0 and c = 0 where all x are
 * 0, s = NaN and c = 0 where one is not finite.  k_scales and v_scales hold s.
 * LEAN_ERR_SHAPE: n_tokens <= 0, negative head counts or both 0, head_dim odd
 * or not in 2..512, rot_dim odd, < 0 or > head_dim, a negative stride, page_size or
 * n_pages <= 0 or more than 2^31 - 1 slots (caches given).  LEAN_ERR_NULL: a
 * part missing.  LEAN_ERR_FORMAT: an unknown type or a cache_dtype that is none
 * of LEAN_BF16, LEAN_F16 and LEAN_I8. */
typedef struct {
    int64_t n_tokens, n_q_heads, n_kv_heads, head_dim;
    int64_t rot_dim;
    int64_t interleaved;      /* 0: halves, 1: neighbours                      */
    int64_t act_dtype;        /* of q, k, v, q_out, k_out                      */
    int64_t cache_dtype;
    const void *q;            /* [token][head][head_dim]                       */
    int64_t q_stride, q_head_stride;
    const void *k;
    int64_t k_stride, k_head_stride;
    const void *v;
    int64_t v_stride, v_head_stride;
    void *q_out;
    int64_t q_out_stride, q_out_head_stride;
    void *k_out;
    int64_t k_out_stride, k_out_head_stride;
    const int32_t *positions; /* int32[n_tokens]                               */
    const int32_t *slots;     /* int32[n_tokens]                               */
    const uint64_t *turns;    /* uint64[rot_dim / 2], 8-byte aligned           */
    void *k_cache;            /* [page][place][kv head][head_dim] by strides   */
    void *v_cache;            /* the same strides                              */
    int64_t n_pages, page_size;
    int64_t page_stride, place_stride, cache_head_stride;
    double rot_scale;
    int64_t flags;
    float *k_scales, *v_scales; /* LEAN_I8: float[page][place][kv head] by strides */
    int64_t scale_page_stride, scale_place_stride, scale_head_stride;
} lean_rope_args;
lean_status lean_rope_append(const lean_rope_args *args, void *stream);

/* Page bookkeeping of the cache: block tables, slot maps and the pool of free
 * pages follow from the sequences' lengths, on the device.  Sequence s holds
 * lens[s] tokens in ceil(lens[s] / page_size) pages, the first entries of its
 * row of block_table, and goes to targets[s] tokens: it grows (pages are taken
 * from the free ring), shrinks (they go back; 0 ends the sequence) or stays.
 * The new tokens of all sequences, in order, are one packed batch:
 *   token_starts[s]   where sequence s's new tokens begin; token_starts[n_seqs]
 *                     is how many there are (counts past 2^31 - 1 stay there)
 *   slots[i], positions[i], token_seqs[i]  token i's place in the cache (for
 *                     lean_rope_append), its position, and its sequence; entries
 *                     from token_starts[n_seqs] to max_tokens - 1 are -1, 0, -1
 * The free ring holds ring_state[1] pages from place ring_state[0] on, around a
 * buffer of ring_size entries (at least as many as there are pages).  Pages are
 * taken from its front in the order of the sequences and their pages, and pages
 * given back are appended in that order; those given back in a call are not
 * taken in the same call.  Table entries that a shorter sequence no longer
 * needs keep their old values.
 * A page in the ring or the table that is negative, or whose slots pass 2^31 - 2,
 * is handed on as it is, but its tokens get slot -1 and bit 64 of the device error
 * word is set.
 * status[s] (0: done).  Otherwise the sequence stays at lens[s], and its new
 * tokens get slot -1:
 *   1  the ring ran out (then every later sequence that needs pages fails too)
 *   2  more pages than a row of the table has
 *   3  its tokens end past max_tokens (those past it are not written), also when
 *      no map is wanted (2^31 - 1 then sets no limit)
 *   4  a negative length, a ring_state outside the ring, or more pages given back
 *      than the ring has room for (then every later one that gives any fails too)
 * lens_out and ring_state_out must not overlap lens, targets or ring_state (use
 * two sets in turn); all other outputs overlap nothing.
 * LEAN_ERR_SHAPE: n_seqs, page_size, table_width or ring_size <= 0, max_tokens <
 * 0, table_stride < table_width, n_seqs above 2^30 - 1, another of these above
 * 2^31 - 1, lens_out that is lens or targets, or ring_state_out that is
 * ring_state.  LEAN_ERR_NULL: a missing pointer (slots, positions and token_seqs
 * may be NULL: not wanted). */
typedef struct {
    int64_t n_seqs, page_size, max_tokens;
    const int32_t *lens;      /* int32[n_seqs]                                 */
    const int32_t *targets;   /* int32[n_seqs]                                 */
    int32_t *block_table;     /* int32[n_seqs][table_stride], updated          */
    int64_t table_width, table_stride;
    int32_t *free_ring;       /* int32[ring_size], updated                     */
    int64_t ring_size;
    const int32_t *ring_state; /* int32[2]: first place, pages                 */
    int32_t *lens_out;        /* int32[n_seqs]                                 */
    int32_t *ring_state_out;  /* int32[2]                                      */
    int32_t *status;          /* int32[n_seqs]                                 */
    int32_t *token_starts;    /* int32[n_seqs + 1]                             */
    int32_t *slots, *positions, *token_seqs; /* int32[max_tokens]              */
    int64_t flags;
} lean_kv_pages_args;
lean_status lean_kv_pages(const lean_kv_pages_args *args, void *stream);

/* Attention of one new token per sequence over the paged cache:
 *   out[s][h] = sum_j p_j v_j,  p = softmax_j(scale * q[s][h] . k_j),
 * j over the last `window` of the seq_lens[s] cached tokens (0: all of them; the
 * new token's own k and v are among them, appended before).  n_q_heads is a
 * multiple of n_kv_heads; query heads h share kv head h / (n_q_heads /
 * n_kv_heads).  lse, optional: ln sum_j exp(scale * q . k_j), with which results
 * over several caches can be joined.  A sequence of no tokens gives out 0 and
 * lse -inf.  What the cache holds past a sequence's length, or before its
 * window, is never used, whatever it is.  A page outside 0..n_pages-1 among
 * those needed gives NaN for its sequence and sets bit 64 of the device error
 * word; a length below 0 counts as 0, one past table_width * page_size as that.
 * What is not finite among the attended keys and values gives NaN or infinities
 * in the outputs that it reaches.
 * LEAN_I8 caches: k_j = c s of k_scales, v_j of v_scales; a scale that is not
 * finite counts as a key or value that is not.
 * q and p are split in parts of the cache's type, three for fp32 q and out and
 * two for 16-bit ones, and sums are fp32, so that fp32 q keeps its precision: out
 * errs by about 2^-17 of sum p |v|, and by fp32's rounding of the scores.  With an
 * f16 cache each p errs by up to 2^-38 of the sequence's largest one as well, and
 * each element of q by 2^-38 of its head's largest (f16 has no smaller steps);
 * with a LEAN_I8 cache p times its token's v_scales is so held, to 2^-38 of the
 * largest p times the largest of the v_scales.  Sums of p v are held in fp32, with p
 * up to 2^8: values above 2^120 / keys in size may give infinities.
 * q, out and the caches: 16-byte aligned, strides multiples of 8 elements
 * (LEAN_I8 caches: of 16, and head_dim as well).
 * workspace: lean_paged_attention_workspace_bytes() bytes, 256-byte aligned,
 * any contents.  Calls that may run at the same time must not share one.
 * Results do not depend on timing.
 * LEAN_ERR_SHAPE: a size <= 0, heads that do not divide, head_dim not a multiple
 * of 8 or above 256, window < 0, table_width * page_size above 2^31 - 1, more
 * than 2^31 - 1 sequences x heads, sequences x kv heads x table_width x page_size
 * / 16 near 2^32 or above, or a workspace too small.  LEAN_ERR_ALIGN,
 * LEAN_ERR_NULL, LEAN_ERR_FORMAT as for the other calls (cache_dtype: LEAN_BF16,
 * LEAN_F16 or LEAN_I8). */
typedef struct {
    int64_t n_seqs, n_q_heads, n_kv_heads, head_dim;
    int64_t act_dtype;         /* of q and out                                 */
    int64_t cache_dtype;
    const void *q;             /* [seq][head][head_dim]                        */
    int64_t q_stride, q_head_stride;
    const void *k_cache, *v_cache; /* as for lean_rope_append                  */
    int64_t n_pages, page_size;
    int64_t page_stride, place_stride, cache_head_stride;
    const int32_t *block_table; /* int32[n_seqs][table_stride]                 */
    int64_t table_width, table_stride;
    const int32_t *seq_lens;   /* int32[n_seqs]                                */
    void *out;                 /* [seq][head][head_dim]                        */
    int64_t out_stride, out_head_stride;
    float *lse;                /* float[n_seqs][n_q_heads]                     */
    double scale;
    int64_t window;
    void *workspace;
    int64_t workspace_bytes;
    int64_t flags;
    const float *k_scales, *v_scales; /* LEAN_I8: as for lean_rope_append      */
    int64_t scale_page_stride, scale_place_stride, scale_head_stride;
} lean_attention_args;
lean_status lean_paged_attention(const lean_attention_args *args, void *stream);
/* -1 for sizes that lean_paged_attention refuses. */
int64_t lean_paged_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                             int64_t head_dim);

/* What is read off rows of logits, in one pass over them.  With z = scale * x
 * (scale: one over the temperature, > 0):
 *   logprobs[r] = z[ids[r]] - ln sum_j exp z[j]
 *   ranks[r]    = how many logits are larger than x[ids[r]]
 *   entropy[r]  = - sum_j p_j ln p_j
 *   top_ids[r][i], top_logprobs[r][i], i < top_k: the largest logits in
 *                 descending order, equal ones by ascending id
 * A logit of -inf is a masked token: it has probability 0 and is never among the
 * top ones (places left over hold id -1 and -inf).  A row that is all -inf has
 * logprobs -inf and entropy 0.  A row with a NaN or +inf gives NaN (its top_ids
 * are the largest logits that are not NaN).  An id outside 0..vocab-1 gives NaN
 * and rank -1 and sets bit 256 of the device error word.
 * ids may be NULL (then logprobs and ranks are not computed); each output may be
 * NULL.  logits: aligned to their element; rows that start on 16 bytes are read
 * fastest.  workspace: lean_token_logprobs_workspace_bytes() bytes (with
 * alternatives, a 64th of the logits in fp32), 256-byte aligned, any contents;
 * calls that may run at the same time must not share one.
 * LEAN_ERR_SHAPE: rows <= 0, vocab not in 1..2^20, stride < vocab with more than
 * one row, rows x vocab past about 2^40, top_k not in 0..LEAN_MAX_TOP, scale not
 * finite or <= 0, or a workspace too small.  LEAN_ERR_NULL: no logits, no
 * workspace, logprobs or ranks without ids, or top_k > 0 without top_ids and
 * top_logprobs. */
#define LEAN_MAX_TOP 64
typedef struct {
    int64_t rows, vocab;
    int64_t dtype;
    const void *logits;
    int64_t stride;
    const int32_t *ids;        /* int32[rows]                                  */
    double scale;
    int64_t top_k;
    float *logprobs;           /* float[rows]                                  */
    int32_t *ranks;            /* int32[rows]                                  */
    float *entropy;            /* float[rows]                                  */
    int32_t *top_ids;          /* int32[rows][top_k]                           */
    float *top_logprobs;       /* float[rows][top_k]                           */
    void *workspace;
    int64_t workspace_bytes;
    int64_t flags;
} lean_logprobs_args;
lean_status lean_token_logprobs(const lean_logprobs_args *args, void *stream);
/* -1 for sizes that lean_token_logprobs refuses. */
int64_t lean_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top_k);

#ifdef __cplusplus
}
#endif

#endif /* LEAN_STEP_H */
