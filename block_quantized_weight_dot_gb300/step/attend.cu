// attend.cu -- lean_paged_attention: attention of one new token per sequence
// over the paged cache.
//
// One block per (sequence, query head): each warp takes every eighth token,
// a lane holds its share of the head dimension, and running maximum, sum and
// weighted values are joined over the warps at the end.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kAttThreads = 256, kAttWarps = kAttThreads / 32;
constexpr int kAttMaxDim = 256, kAttPer = kAttMaxDim / 32;

struct AttArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    int64_t qs, qhs, os, ohs, page_stride, place_stride, cache_hs, table_stride, n_pages;
    int n_seqs, hq, hkv, dim, page, width, window;
    int act, cache_bf16;
    float scale;
    unsigned *err;
};

__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype) {
    if (dtype == LEAN_F32) return static_cast<const float *>(p)[i];
    if (dtype == LEAN_BF16) return to_f(static_cast<const __nv_bfloat16 *>(p)[i]);
    return to_f(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, float v, int dtype) {
    if (dtype == LEAN_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == LEAN_BF16) static_cast<__nv_bfloat16 *>(p)[i] = from_f<__nv_bfloat16>(v);
    else static_cast<__half *>(p)[i] = from_f<__half>(v);
}

__global__ void __launch_bounds__(kAttThreads) attend_kernel(const AttArgs p) {
    step_begin();
    __shared__ float ms[kAttWarps], ls[kAttWarps], acc_s[kAttWarps][kAttMaxDim];
    __shared__ int bad;
    const int s = blockIdx.x / p.hq, h = blockIdx.x % p.hq, kvh = h / (p.hq / p.hkv);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int len = p.lens[s];
    len = len < 0 ? 0 : len;
    len = (int64_t)len > (int64_t)p.width * p.page ? p.width * p.page : len;
    const int start = p.window > 0 && len > p.window ? len - p.window : 0;
    const int cdt = p.cache_bf16 ? LEAN_BF16 : LEAN_F16;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    float q[kAttPer], acc[kAttPer];
#pragma unroll
    for (int i = 0; i < kAttPer; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < p.dim ? load_any(p.q, s * p.qs + h * p.qhs + d, p.act) * p.scale : 0.f;
        acc[i] = 0.f;
    }
    float m = -CUDART_INF_F, l = 0.f;
    for (int j = start + warp; j < len; j += kAttWarps) {
        const int page = p.table[s * p.table_stride + j / p.page];
        if (page < 0 || page >= p.n_pages) {
            bad = 1;
            continue;
        }
        const int64_t at = page * p.page_stride + (j % p.page) * p.place_stride + kvh * p.cache_hs;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kAttPer; ++i)
            if (lane + 32 * i < p.dim) dot = fmaf(q[i], load_any(p.k, at + lane + 32 * i, cdt), dot);
        dot = warp_sum(dot);
        const float mn = fmaxf(m, dot), c = __expf(m - mn), e = __expf(dot - mn);
        l = l * c + e;
#pragma unroll
        for (int i = 0; i < kAttPer; ++i)
            if (lane + 32 * i < p.dim) acc[i] = fmaf(e, load_any(p.v, at + lane + 32 * i, cdt), acc[i] * c);
        m = mn;
    }
    if (lane == 0) {
        ms[warp] = m;
        ls[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < kAttPer; ++i) acc_s[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    float top = -CUDART_INF_F, sum = 0.f;
    for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, ms[w]);
    for (int w = 0; w < kAttWarps; ++w) sum += ls[w] > 0.f ? ls[w] * __expf(ms[w] - top) : ls[w];
    if (bad) sum = CUDART_NAN_F;
    if (threadIdx.x == 0) {
        if (bad) atomicOr(p.err, kErrSlot);
        if (p.lse) p.lse[(int64_t)s * p.hq + h] = sum == 0.f ? -CUDART_INF_F : top + logf(sum);
    }
    for (int d = threadIdx.x; d < p.dim; d += kAttThreads) {
        float o = 0.f;
        for (int w = 0; w < kAttWarps; ++w)
            if (ls[w] != 0.f) o += acc_s[w][d] * __expf(ms[w] - top);
        store_any(p.out, s * p.os + h * p.ohs + d, sum == 0.f ? 0.f : o / sum, p.act);
    }
}

bool att_sizes_ok(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim) {
    return n_seqs > 0 && hkv > 0 && hq > 0 && hq <= 65536 && hq % hkv == 0 && dim > 0 && dim % 8 == 0 &&
           dim <= kAttMaxDim && n_seqs <= INT32_MAX / hq;
}

}  // namespace

extern "C" int64_t lean_paged_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                                        int64_t head_dim) {
    return att_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim) ? 256 : -1;
}

extern "C" lean_status lean_paged_attention(const lean_attention_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!known_dtype(a->act_dtype) || (a->cache_dtype != LEAN_BF16 && a->cache_dtype != LEAN_F16) ||
        !step_flags_ok(a->flags))
        return LEAN_ERR_FORMAT;
    if (!att_sizes_ok(a->n_seqs, a->n_q_heads, a->n_kv_heads, a->head_dim) || a->window < 0 || a->n_pages <= 0 ||
        a->n_pages > INT32_MAX || a->page_size <= 0 || a->table_width <= 0 ||
        a->table_width > INT32_MAX / a->page_size || a->table_stride < a->table_width)
        return LEAN_ERR_SHAPE;
    if (!a->q || !a->k_cache || !a->v_cache || !a->block_table || !a->seq_lens || !a->out || !a->workspace)
        return LEAN_ERR_NULL;
    const int64_t strides[] = {a->q_stride, a->q_head_stride, a->out_stride, a->out_head_stride, a->page_stride,
                               a->place_stride, a->cache_head_stride};
    for (int64_t s : strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        if (s % 8) return LEAN_ERR_ALIGN;
    }
    if (!step_aligned(a->q, 16) || !step_aligned(a->k_cache, 16) || !step_aligned(a->v_cache, 16) ||
        !step_aligned(a->out, 16) || !step_aligned(a->block_table, 4) || !step_aligned(a->seq_lens, 4) ||
        !step_aligned(a->lse, 4) || !step_aligned(a->workspace, 256))
        return LEAN_ERR_ALIGN;
    if (a->workspace_bytes <
        lean_paged_attention_workspace_bytes(a->n_seqs, a->n_q_heads, a->n_kv_heads, a->head_dim))
        return LEAN_ERR_SHAPE;
    AttArgs p = {};
    p.q = a->q;
    p.k = a->k_cache;
    p.v = a->v_cache;
    p.out = a->out;
    p.lse = a->lse;
    p.table = a->block_table;
    p.lens = a->seq_lens;
    p.qs = a->q_stride;
    p.qhs = a->q_head_stride;
    p.os = a->out_stride;
    p.ohs = a->out_head_stride;
    p.page_stride = a->page_stride;
    p.place_stride = a->place_stride;
    p.cache_hs = a->cache_head_stride;
    p.table_stride = a->table_stride;
    p.n_pages = a->n_pages;
    p.n_seqs = (int)a->n_seqs;
    p.hq = (int)a->n_q_heads;
    p.hkv = (int)a->n_kv_heads;
    p.dim = (int)a->head_dim;
    p.page = (int)a->page_size;
    p.width = (int)a->table_width;
    p.window = (int)std::min<int64_t>(a->window, INT32_MAX);
    p.act = (int)a->act_dtype;
    p.cache_bf16 = a->cache_dtype == LEAN_BF16;
    p.scale = (float)a->scale;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    return step_launch(attend_kernel, a->n_seqs * a->n_q_heads, kAttThreads, 0, a->flags, stream, p);
}
