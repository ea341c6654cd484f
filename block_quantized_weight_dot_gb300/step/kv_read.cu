// kv_read.cu -- lean_kv_read: tokens of the paged cache as contiguous rows.
//
// Values are c * s (caches in 8 bits) or the cache's own.  Every byte moves once,
// so HBM bounds the call.  A thread writes 16 bytes of a row at a time (V
// elements) and reads the V elements they come from; consecutive threads follow a
// token's row through its heads, U pieces of a thread are under way at once.
#include "../../include/lean_cache.h"
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kReadThreads = 256;

struct ReadArgs {
    const void *k, *v;
    const float *k_scales, *v_scales;
    void *k_out, *v_out;
    const int32_t *slots;
    int64_t page_stride, place_stride, cache_hs, scale_page, scale_place, scale_hs;
    int64_t kos, kohs, vos, vohs;
    int64_t n_tokens, n_slots;
    int64_t cache_end, scale_end, k_end, v_end;  // elements, for the checked build
    int hkv, dim, page, pieces, row, tokens;  // pieces: of a head; row: of a token; tokens: of a block
    unsigned *err;
};

template <typename C>
__device__ __forceinline__ float cached(C v) { return to_f(v); }
template <>
__device__ __forceinline__ float cached(int8_t v) {  // exact: 2^23 + (c + 128) has c + 128 in its low bits
    return __uint_as_float(0x4b000000u | ((uint32_t)(uint8_t)v ^ 0x80u)) - 8388736.f;
}

// C: of the cache, A: of the output.  Blocks of gridDim.y = 1 read values, of 0 keys (or the one there is).
template <typename C, typename A, int V>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs p) {
    constexpr int U = 4;
    constexpr bool IN8 = sizeof(C) == 1;
    step_begin();
    const bool is_k = p.k && blockIdx.y == 0;
    const C *cache = static_cast<const C *>(is_k ? p.k : p.v);
    const float *scales = is_k ? p.k_scales : p.v_scales;
    A *out = static_cast<A *>(is_k ? p.k_out : p.v_out);
    const int64_t os = is_k ? p.kos : p.vos, ohs = is_k ? p.kohs : p.vohs, out_end = is_k ? p.k_end : p.v_end;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)min((int64_t)p.tokens, p.n_tokens - t0), n = nt * p.row;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * kReadThreads) {
        Vec<C, V> x[U];
        float s[U];
        int64_t to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kReadThreads;
            s[u] = 1.f;
            x[u] = Vec<C, V>{};
            if (i >= n) continue;
            const int t = i / p.row, j = i - t * p.row, head = j / p.pieces, d = (j - head * p.pieces) * V;
            to[u] = (t0 + t) * os + head * ohs + d;
            const int32_t slot = LEAN_IN(t0 + t, p.n_tokens, p.err) ? p.slots[t0 + t] : -1;
            if (slot >= p.n_slots) {
                s[u] = CUDART_NAN_F;
                if (j == 0) atomicOr(p.err, kErrSlot);
            } else if (slot >= 0) {
                const int64_t page = slot / p.page, place = slot - (int)page * p.page;
                const int64_t at = page * p.page_stride + place * p.place_stride + head * p.cache_hs + d;
                if (LEAN_SPAN(at, V, p.cache_end, p.err)) x[u] = load_vec<C, V>(cache + at);
                const int64_t at_s = page * p.scale_page + place * p.scale_place + head * p.scale_hs;
                if (IN8 && LEAN_IN(at_s, p.scale_end, p.err)) s[u] = scales[at_s];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * kReadThreads >= n) break;
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = cached(x[u].v[e]) * s[u];
            if (LEAN_SPAN(to[u], V, out_end, p.err)) store_vec<A, V>(out + to[u], f);
        }
    }
}

template <typename C, typename A, int V>
lean_status launch_read(ReadArgs p, int64_t flags, void *stream) {
    p.pieces = p.dim / V;
    p.row = p.hkv * p.pieces;
    // about two rounds of U pieces a thread, but no fewer blocks than two for an SM while there are tokens for them
    int64_t tokens = std::max<int64_t>(1, 8 * kReadThreads / p.row);
    tokens = std::min(tokens, std::max<int64_t>(1, p.n_tokens / (2 * step_sm_count())));
    p.tokens = (int)tokens;
    const int64_t grid = (p.n_tokens + tokens - 1) / tokens;
    if (grid > INT32_MAX) return LEAN_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid, p.k && p.v ? 2 : 1, 1);
    cfg.blockDim = dim3(kReadThreads, 1, 1);
    cfg.stream = (cudaStream_t)stream;
    if (flags & LEAN_FLAG_EARLY_WEIGHTS) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    cudaGetLastError();
    return cudaLaunchKernelEx(&cfg, kv_read_kernel<C, A, V>, p) == cudaSuccess ? LEAN_OK : LEAN_ERR_CUDA;
}
// Pieces of 16 bytes of the output where every row lies so that they and what they come from are whole accesses.
template <typename C, typename A>
lean_status pick_read(const ReadArgs &p, bool whole, int64_t flags, void *stream) {
    return whole ? launch_read<C, A, 16 / sizeof(A)>(p, flags, stream) : launch_read<C, A, 1>(p, flags, stream);
}
template <typename C>
lean_status pick_out(const ReadArgs &p, int64_t out, bool whole, int64_t flags, void *stream) {
    if (out == LEAN_F32) return pick_read<C, float>(p, whole, flags, stream);
    if (out == LEAN_BF16) return pick_read<C, __nv_bfloat16>(p, whole, flags, stream);
    return pick_read<C, __half>(p, whole, flags, stream);
}

}  // namespace

extern "C" lean_status lean_kv_read(const lean_kv_read_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    const bool in8 = a->cache_dtype == LEAN_I8;
    if (!known_dtype(a->out_dtype) || (!in8 && a->cache_dtype != LEAN_BF16 && a->cache_dtype != LEAN_F16) ||
        !step_flags_ok(a->flags))
        return LEAN_ERR_FORMAT;
    if (a->n_tokens <= 0 || a->n_tokens > INT32_MAX || a->n_kv_heads <= 0 || a->n_kv_heads > 65536 || a->head_dim <= 0 ||
        a->head_dim > 512 || a->page_size <= 0 || a->n_pages <= 0 || a->n_pages > INT32_MAX / a->page_size)
        return LEAN_ERR_SHAPE;
    const int64_t cache_strides[] = {a->page_stride, a->place_stride, a->cache_head_stride};
    const int64_t out_strides[] = {a->k_out_stride, a->k_out_head_stride, a->v_out_stride, a->v_out_head_stride};
    const int64_t scale_strides[] = {a->scale_page_stride, a->scale_place_stride, a->scale_head_stride};
    int64_t any = a->head_dim;
    for (int64_t s : cache_strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        any |= s;
    }
    for (int64_t s : out_strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        any |= s;
    }
    for (int64_t s : scale_strides)
        if (in8 && s < 0) return LEAN_ERR_SHAPE;
    if ((!a->k_cache && !a->v_cache) || !a->k_cache != !a->k_out || !a->v_cache != !a->v_out || !a->slots ||
        (in8 && ((a->k_cache && !a->k_scales) || (a->v_cache && !a->v_scales))))
        return LEAN_ERR_NULL;
    const int64_t size = in8 ? 1 : 2, out_size = dtype_size(a->out_dtype), v = 16 / out_size;
    if (!step_aligned(a->k_cache, size) || !step_aligned(a->v_cache, size) || !step_aligned(a->k_out, out_size) ||
        !step_aligned(a->v_out, out_size) || !step_aligned(a->slots, 4) ||
        (in8 && (!step_aligned(a->k_scales, 4) || !step_aligned(a->v_scales, 4))))
        return LEAN_ERR_ALIGN;
    const bool whole = any % v == 0 && step_aligned(a->k_cache, size * v) && step_aligned(a->v_cache, size * v) &&
                       step_aligned(a->k_out, 16) && step_aligned(a->v_out, 16);
    ReadArgs p = {};
    p.k = a->k_cache;
    p.v = a->v_cache;
    if (in8) {
        p.k_scales = a->k_scales;
        p.v_scales = a->v_scales;
        p.scale_page = a->scale_page_stride;
        p.scale_place = a->scale_place_stride;
        p.scale_hs = a->scale_head_stride;
    }
    p.k_out = a->k_out;
    p.v_out = a->v_out;
    p.slots = a->slots;
    p.page_stride = a->page_stride;
    p.place_stride = a->place_stride;
    p.cache_hs = a->cache_head_stride;
    p.kos = a->k_out_stride;
    p.kohs = a->k_out_head_stride;
    p.vos = a->v_out_stride;
    p.vohs = a->v_out_head_stride;
    p.n_tokens = a->n_tokens;
    p.n_slots = a->n_pages * a->page_size;
    p.cache_end = (a->n_pages - 1) * a->page_stride + (a->page_size - 1) * a->place_stride +
                  (a->n_kv_heads - 1) * a->cache_head_stride + a->head_dim;
    p.scale_end = (a->n_pages - 1) * a->scale_page_stride + (a->page_size - 1) * a->scale_place_stride +
                  (a->n_kv_heads - 1) * a->scale_head_stride + 1;
    p.k_end = (a->n_tokens - 1) * a->k_out_stride + (a->n_kv_heads - 1) * a->k_out_head_stride + a->head_dim;
    p.v_end = (a->n_tokens - 1) * a->v_out_stride + (a->n_kv_heads - 1) * a->v_out_head_stride + a->head_dim;
    p.hkv = (int)a->n_kv_heads;
    p.dim = (int)a->head_dim;
    p.page = (int)a->page_size;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    if (in8) return pick_out<int8_t>(p, a->out_dtype, whole, a->flags, stream);
    if (a->cache_dtype == LEAN_BF16) return pick_out<__nv_bfloat16>(p, a->out_dtype, whole, a->flags, stream);
    return pick_out<__half>(p, a->out_dtype, whole, a->flags, stream);
}
