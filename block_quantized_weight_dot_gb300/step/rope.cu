// rope.cu -- lean_rope_append: rotary positions of q and k, and the append of
// k and v to the paged cache.
//
// The angle of pair i at position p is p * turns[i] / 2^64 turns: the upper 32
// bits of a 64-bit product, two integer instructions, with every whole turn
// already gone.  (In fp32, p * freq alone is off by 0.004 radians at position
// 100000.)  sincospif takes the fraction of a turn as it is.
//
// A block takes a few tokens: its threads first compute the tokens' cosines and
// sines into shared memory, once for all heads, then run over (token, head,
// piece), where a piece is V pairs: two runs of V elements (halves) or one of
// 2 V (neighbours and the unrotated rest).  All traffic is 16-byte accesses at
// V = 8 (4 for fp32) and every element moves once, so HBM bounds it.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;
constexpr int kRopeMaxTokens = 16;  // of a block

struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out, *k_cache, *v_cache;
    const int32_t *positions, *slots;
    const uint64_t *turns;
    int64_t qs, qhs, ks, khs, vs, vhs, qos, qohs, kos, kohs;
    int64_t page_stride, place_stride, cache_hs;
    int64_t n_tokens, n_slots;
    int hq, hkv, hv, dim, rot, page; // hv: heads of v, 0 without caches
    int tokens;            // of a block
    int pieces, rot_pieces; // of a head; the rotated ones come first
    int cache_bf16;
    float scale;
    unsigned *err;
};

template <typename A, int V>
__device__ __forceinline__ void load_f(const A *p, float *f) {
    const Vec<A, V> v = load_vec<A, V>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f(v.v[i]);
}
template <int V>
__device__ __forceinline__ void store_cache(void *base, int64_t at, const float *f, int bf16) {
    if (bf16) store_vec<__nv_bfloat16, V>(static_cast<__nv_bfloat16 *>(base) + at, f);
    else store_vec<__half, V>(static_cast<__half *>(base) + at, f);
}

// V: pairs of a piece; INTER: pairs are neighbours.
template <typename A, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs p) {
    step_begin();
    extern __shared__ float2 cs[];  // [token][pair]: cosine, sine
    __shared__ int64_t place[kRopeMaxTokens];  // in the caches, or -1
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)(p.n_tokens - t0 < p.tokens ? p.n_tokens - t0 : p.tokens);
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half, j = i - t * half;
        const int32_t pos = p.positions[t0 + t];
        const uint64_t f = p.turns[j];
        // upper half of pos * f mod 2^64, pos signed
        const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32), u = (uint32_t)pos;
        const uint32_t turn = __umulhi(u, lo) + u * hi - (pos < 0 ? lo : 0u);
        float s, c;
        sincospif((float)(int32_t)turn * (1.f / 2147483648.f), &s, &c);
        cs[i] = make_float2(c * p.scale, s * p.scale);
    }
    if (p.k_cache && threadIdx.x < nt) {
        const int32_t slot = p.slots[t0 + threadIdx.x];
        int64_t at = -1;
        if (slot >= p.n_slots) atomicOr(p.err, kErrSlot);
        else if (slot >= 0) at = (int64_t)(slot / p.page) * p.page_stride + (int64_t)(slot % p.page) * p.place_stride;
        place[threadIdx.x] = at;
    }
    __syncthreads();

    const int per_token = (p.hq + p.hkv + p.hv) * p.pieces;
    const int64_t cache_end = (p.n_slots / p.page - 1) * p.page_stride + (p.page - 1) * p.place_stride +
                              (p.hkv - 1) * p.cache_hs + p.dim;
#pragma unroll 2
    for (int i = threadIdx.x; i < nt * per_token; i += kRopeThreads) {
        const int t = i / per_token, hp = i - t * per_token, head = hp / p.pieces, piece = hp - head * p.pieces;
        const bool rotated = piece < p.rot_pieces;
        const int64_t tok = t0 + t;
        // where the piece's two runs of V elements begin
        const bool apart = !INTER && rotated;
        const int a = apart ? piece * V : piece * 2 * V, b = apart ? a + half : a + V;
        const bool is_q = head < p.hq, is_k = !is_q && head < p.hq + p.hkv;
        const int kvh = head - p.hq - (is_k ? 0 : p.hkv);
        const A *src = is_q ? static_cast<const A *>(p.q) + tok * p.qs + head * p.qhs
                     : is_k ? static_cast<const A *>(p.k) + tok * p.ks + kvh * p.khs
                            : static_cast<const A *>(p.v) + tok * p.vs + kvh * p.vhs;
        float x[2 * V];
        load_f<A, V>(src + a, x);
        load_f<A, V>(src + b, x + V);
        if (rotated && (is_q || is_k)) {
            const float2 *w = cs + t * half + piece * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float &u = INTER ? x[2 * j] : x[j], &v = INTER ? x[2 * j + 1] : x[V + j];
                const float2 c = w[j];
                const float nu = u * c.x - v * c.y, nv = fmaf(u, c.y, v * c.x);
                u = nu;
                v = nv;
            }
        }
        if (is_q || (is_k && p.k_out)) {
            A *dst = is_q ? static_cast<A *>(p.q_out) + tok * p.qos + head * p.qohs
                          : static_cast<A *>(p.k_out) + tok * p.kos + kvh * p.kohs;
            store_vec<A, V>(dst + a, x);
            store_vec<A, V>(dst + b, x + V);
        }
        if (!is_q && p.k_cache && place[t] >= 0) {
            void *cache = is_k ? p.k_cache : p.v_cache;
            const int64_t at = place[t] + kvh * p.cache_hs;
            if (LEAN_SPAN(at + a, V, cache_end, p.err)) store_cache<V>(cache, at + a, x, p.cache_bf16);
            if (LEAN_SPAN(at + b, V, cache_end, p.err)) store_cache<V>(cache, at + b, x + V, p.cache_bf16);
        }
    }
}

template <typename A, int V>
lean_status launch_rope(RopeArgs p, bool inter, int64_t flags, void *stream) {
    p.pieces = p.dim / (2 * V);
    p.rot_pieces = p.rot / (2 * V);
    const int64_t items = (int64_t)(p.hq + p.hkv + p.hv) * p.pieces;
    // about eight pieces a thread, but no fewer blocks than SMs while there are tokens for them
    int64_t tokens = std::max<int64_t>(1, 8 * kRopeThreads / items);
    tokens = std::min(tokens, std::max<int64_t>(1, p.n_tokens / (2 * step_sm_count())));
    p.tokens = (int)std::min<int64_t>(tokens, kRopeMaxTokens);
    const size_t smem = sizeof(float2) * p.tokens * std::max(p.rot / 2, 1);  // 32 KB at most
    const int64_t grid = (p.n_tokens + p.tokens - 1) / p.tokens;
    if (inter) return step_launch(rope_kernel<A, V, true>, grid, kRopeThreads, smem, flags, stream, p);
    return step_launch(rope_kernel<A, V, false>, grid, kRopeThreads, smem, flags, stream, p);
}

// Pairs per piece: the most for which every run of elements is a whole number
// of them and lies on 16 bytes (8 or 4 elements), else one.
template <typename A>
lean_status pick_rope(const RopeArgs &p, bool inter, int64_t any_stride, bool on16, int64_t flags, void *stream) {
    constexpr int V = 16 / sizeof(A);
    if (on16 && any_stride % V == 0 && p.rot / 2 % V == 0 && p.dim % (2 * V) == 0 && p.rot % (2 * V) == 0)
        return launch_rope<A, V>(p, inter, flags, stream);
    return launch_rope<A, 1>(p, inter, flags, stream);
}

}  // namespace

extern "C" lean_status lean_rope_append(const lean_rope_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!known_dtype(a->act_dtype) || !step_flags_ok(a->flags)) return LEAN_ERR_FORMAT;
    const bool cached = a->k_cache || a->v_cache;
    if (cached && a->cache_dtype != LEAN_BF16 && a->cache_dtype != LEAN_F16) return LEAN_ERR_FORMAT;
    const int64_t strides[] = {a->q_stride, a->q_head_stride, a->k_stride, a->k_head_stride, a->v_stride,
                               a->v_head_stride, a->q_out_stride, a->q_out_head_stride, a->k_out_stride,
                               a->k_out_head_stride};
    const int64_t cache_strides[] = {a->page_stride, a->place_stride, a->cache_head_stride};
    int64_t any = 0;
    for (int64_t s : strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        any |= s;
    }
    if (a->n_tokens <= 0 || a->n_q_heads < 0 || a->n_kv_heads < 0 || a->n_q_heads > 65536 ||
        a->n_kv_heads > 65536 || a->n_q_heads + a->n_kv_heads == 0 || a->head_dim < 2 ||
        a->head_dim > kRopeMaxDim || a->head_dim % 2 || a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2)
        return LEAN_ERR_SHAPE;
    if (a->n_tokens > INT32_MAX) return LEAN_ERR_SHAPE;
    if (cached) {
        for (int64_t s : cache_strides) {
            if (s < 0) return LEAN_ERR_SHAPE;
            any |= s;
        }
        if (a->page_size <= 0 || a->n_pages <= 0 || a->n_pages > INT32_MAX / a->page_size) return LEAN_ERR_SHAPE;
    }
    if ((a->n_q_heads > 0) != (a->q != nullptr) || !a->q != !a->q_out || (a->n_kv_heads > 0) != (a->k != nullptr) ||
        (a->k_cache && !a->v_cache) || (a->v_cache && !a->k_cache) || (cached && (!a->k || !a->v || !a->slots)) ||
        (a->k && !cached && !a->k_out) || (a->k_out && !a->k) || !a->positions || (a->rot_dim > 0 && !a->turns))
        return LEAN_ERR_NULL;
    const int64_t size = dtype_size(a->act_dtype);
    const void *acts[] = {a->q, a->k, a->v, a->q_out, a->k_out};
    bool on16 = step_aligned(a->k_cache, 16) && step_aligned(a->v_cache, 16);
    for (const void *q : acts) {
        if (!step_aligned(q, size)) return LEAN_ERR_ALIGN;
        on16 = on16 && step_aligned(q, 16);
    }
    if (!step_aligned(a->k_cache, 2) || !step_aligned(a->v_cache, 2) || !step_aligned(a->positions, 4) ||
        !step_aligned(a->slots, 4) || !step_aligned(a->turns, 8))
        return LEAN_ERR_ALIGN;
    RopeArgs p = {};
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.q_out = a->q_out;
    p.k_out = a->k_out;
    p.k_cache = a->k_cache;
    p.v_cache = a->v_cache;
    p.positions = a->positions;
    p.slots = a->slots;
    p.turns = a->turns;
    p.qs = a->q_stride;
    p.qhs = a->q_head_stride;
    p.ks = a->k_stride;
    p.khs = a->k_head_stride;
    p.vs = a->v_stride;
    p.vhs = a->v_head_stride;
    p.qos = a->q_out_stride;
    p.qohs = a->q_out_head_stride;
    p.kos = a->k_out_stride;
    p.kohs = a->k_out_head_stride;
    p.page_stride = a->page_stride;
    p.place_stride = a->place_stride;
    p.cache_hs = a->cache_head_stride;
    p.n_tokens = a->n_tokens;
    p.hq = (int)a->n_q_heads;
    p.hkv = (int)a->n_kv_heads;
    p.hv = cached ? p.hkv : 0;
    p.dim = (int)a->head_dim;
    p.rot = (int)a->rot_dim;
    p.page = cached ? (int)a->page_size : 1;
    p.n_slots = cached ? a->n_pages * a->page_size : 1;
    p.cache_bf16 = a->cache_dtype == LEAN_BF16;
    p.scale = (float)a->rot_scale;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    const bool inter = a->interleaved != 0;
    switch (a->act_dtype) {
    case LEAN_F32: return pick_rope<float>(p, inter, any, on16, a->flags, stream);
    case LEAN_BF16: return pick_rope<__nv_bfloat16>(p, inter, any, on16, a->flags, stream);
    default: return pick_rope<__half>(p, inter, any, on16, a->flags, stream);
    }
}
