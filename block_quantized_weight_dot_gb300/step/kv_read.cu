// kv_read.cu -- lean_kv_read: tokens of the paged cache as contiguous rows.
//
// Values are c * s (caches in 8 bits) or the cache's own.  Every byte moves once,
// so HBM bounds the call.  A thread has one piece of a token's row, V elements,
// which are 16 bytes of the output, for all tokens of its block: addresses then
// only step by the tokens' places, which the block looks up once, in shared memory.
// What is under way at once comes from the number of threads, not from a thread's
// own loads: with one token's key and value each, 131072 tokens of 8 heads of 128
// in 8 bits to bf16 take 132 us (92% of a copy's rate), with two tokens' 142, four
// 152, eight 175.  (Pieces numbered through, each with its own divisions and its own
// slot: 292.)
#include "../../include/lean_cache.h"
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 256;  // of a block, at most

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

// V elements of a cache as they lie there, and as fp32.
template <typename C, int V>
struct alignas(sizeof(C) * V >= 16 ? 16 : sizeof(C) * V) Cached {
    C v[V];
    __device__ __forceinline__ void values(float, float *f) const {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f(v[i]);
    }
};
template <int V>
struct alignas(V) Cached<int8_t, V> {  // c * s: 2^23 + (c + 128) has c + 128 in its low bits, and the difference is exact
    int8_t v[V];
    __device__ __forceinline__ void values(float s, float *f) const {
        if constexpr (V == 1) {
            f[0] = (float)v[0] * s;
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const uint32_t u = reinterpret_cast<const uint32_t *>(v)[i] ^ 0x80808080u;
#pragma unroll
                for (int k = 0; k < 4; ++k) f[4 * i + k] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + k)) - 8388736.f) * s;
            }
        }
    }
};

// C: of the cache, A: of the output.
template <typename C, typename A, int V>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs p) {
    constexpr bool IN8 = sizeof(C) == 1;
    __shared__ int64_t place[kReadTokens], scale_place[kReadTokens];  // -1: zeros, -2: NaN
    step_begin();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)min((int64_t)p.tokens, p.n_tokens - t0);
    for (int t = threadIdx.x; t < nt; t += kReadThreads) {
        const int32_t slot = LEAN_IN(t0 + t, p.n_tokens, p.err) ? p.slots[t0 + t] : -1;
        int64_t at = -1, at_scale = 0;
        if (slot >= p.n_slots) {
            at = -2;
            atomicOr(p.err, kErrSlot);
        } else if (slot >= 0) {
            const int page = slot / p.page, in = slot - page * p.page;
            at = page * p.page_stride + in * p.place_stride;
            at_scale = page * p.scale_page + in * p.scale_place;
        }
        place[t] = at;
        scale_place[t] = at_scale;
    }
    __syncthreads();
    // tokens side by side, where a token has few pieces
    const int sub = max(1, kReadThreads / p.row), first = p.row <= kReadThreads ? (int)threadIdx.x / p.row : 0;
    if (first >= sub) return;
    for (int j = p.row <= kReadThreads ? (int)threadIdx.x - first * p.row : threadIdx.x; j < p.row; j += kReadThreads) {
        const int head = j / p.pieces, d = (j - head * p.pieces) * V;
        const int64_t in_row = head * p.cache_hs + d, in_scales = head * p.scale_hs;
        for (int t = first; t < nt; t += sub) {
            const int64_t at = place[t], at_scale = scale_place[t] + in_scales;
            Cached<C, V> x[2];
            float s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const C *cache = static_cast<const C *>(i ? p.v : p.k);
                x[i] = Cached<C, V>{};
                s[i] = at == -2 ? CUDART_NAN_F : 1.f;
                if (cache && at >= 0) {
                    if (LEAN_SPAN(at + in_row, V, p.cache_end, p.err)) x[i] = *reinterpret_cast<const Cached<C, V> *>(cache + at + in_row);
                    if (IN8 && LEAN_IN(at_scale, p.scale_end, p.err)) s[i] = (i ? p.v_scales : p.k_scales)[at_scale];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                A *out = static_cast<A *>(i ? p.v_out : p.k_out);
                if (!out) continue;
                float f[V];
                x[i].values(s[i], f);
                if (!IN8 && at == -2) {
#pragma unroll
                    for (int e = 0; e < V; ++e) f[e] = CUDART_NAN_F;
                }
                const int64_t to = (t0 + t) * (i ? p.vos : p.kos) + head * (i ? p.vohs : p.kohs) + d;
                if (LEAN_SPAN(to, V, i ? p.v_end : p.k_end, p.err)) store_vec<A, V>(out + to, f);
            }
        }
    }
}

template <typename C, typename A, int V>
lean_status launch_read(ReadArgs p, int64_t flags, void *stream) {
    p.pieces = p.dim / V;
    p.row = p.hkv * p.pieces;
    // eight tokens a thread, but no fewer blocks than four for an SM while there are tokens for them
    int64_t tokens = 8 * std::max(1, kReadThreads / p.row);
    tokens = std::min(tokens, std::max<int64_t>(1, p.n_tokens / (4 * step_sm_count())));
    p.tokens = (int)std::min<int64_t>(tokens, kReadTokens);
    return step_launch(kv_read_kernel<C, A, V>, (p.n_tokens + p.tokens - 1) / p.tokens, kReadThreads, 0, flags, stream, p);
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
