/* lean_cache.h -- the paged cache of lean_step.h beyond one new token per
 * sequence: tokens read back out of it.
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

#ifdef __cplusplus
}
#endif

#endif /* LEAN_CACHE_H */
