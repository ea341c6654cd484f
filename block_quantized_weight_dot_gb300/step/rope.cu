// rope.cu -- lean_rope_append: rotary positions of q and k, and the append of
// k and v to the paged cache.
//
// The angle of pair i at position p is p * turns[i] / 2^64 turns: the upper 32
// bits of a 64-bit product, two integer instructions, with every whole turn
// already gone.  (In fp32, p * freq alone is off by 0.004 radians at position
// 100000.)  sincospif takes the fraction of a turn as it is.
//
// A block takes a few tokens: their cosines and sines go to shared memory, once
// for all heads.  A thread has one piece of one head, for all of the block's
// tokens (its addresses then only step by the tokens' strides), where a piece is
// two runs of V elements: the two sides of V pairs (halves), or V / 2 pairs each
// (neighbours) or none (the unrotated rest) from the two halves of what there is,
// so that neighbouring threads read neighbouring 16 bytes (runs of 2 V elements a
// thread read every other 16: 34.1 us in place of 30.1 at the sizes below).  All
// traffic is 16-byte accesses at V = 8 (4 for fp32), four tokens' loads at a time,
// the first ones before the angles are computed; every element moves once, so HBM
// bounds it.  (Tokens staged in shared memory by asynchronous copies: 41 us.)
//
// Measured (GB300, calls in a graph): 16384 tokens of 16 query and 2 kv heads of
// 128 (half of them rotated, neighbours) 30.4 us in bf16 (5.5 TB/s), 51.4 in fp32
// (6.2 TB/s; a copy reaches 6.78); pairs of halves in bf16 34.1, over the whole head
// 37.0, in fp32 52.2; 2000 tokens 5.3 us; four tokens of 15/5 heads of 64 2.6 us.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kRopeMaxThreads = 384;
constexpr int kRopeMaxDim = 512;
constexpr int kRopeMaxTokens = 64;  // of a block

struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out, *k_cache, *v_cache;
    const int32_t *positions, *slots;
    const uint64_t *turns;
    int64_t qs, qhs, ks, khs, vs, vhs, qos, qohs, kos, kohs;
    int64_t page_stride, place_stride, cache_hs;
    int64_t n_tokens, n_slots;
    int64_t q_end, k_end, v_end, qo_end, ko_end;  // elements, for the checked build
    int hq, hkv, hv, dim, rot, page; // hv: heads of v, 0 without caches
    int tokens;            // of a block
    int pieces, rot_pieces; // of a head; the rotated ones come first
    int cache_bf16;
    float scale;
    unsigned *err;
};

template <int V>
__device__ __forceinline__ void store_cache(void *base, int64_t at, const float *f, int bf16) {
    if (bf16) store_vec<__nv_bfloat16, V>(static_cast<__nv_bfloat16 *>(base) + at, f);
    else store_vec<__half, V>(static_cast<__half *>(base) + at, f);
}

// V elements as they lie in memory, in registers.
template <typename A, int V>
struct alignas(sizeof(A) * V) Piece {
    uint32_t w[sizeof(A) * V / 4];
};
template <>
struct Piece<__nv_bfloat16, 1> {
    __nv_bfloat16 w;
};
template <>
struct Piece<__half, 1> {
    __half w;
};
__device__ __forceinline__ void unpack_piece(const Piece<float, 4> &x, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x.w[i]);
}
__device__ __forceinline__ void unpack_piece(const Piece<float, 1> &x, float *f) { f[0] = __uint_as_float(x.w[0]); }
template <int V>
__device__ __forceinline__ void unpack_piece(const Piece<__nv_bfloat16, V> &x, float *f) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = __uint_as_float(x.w[i] << 16);
        f[2 * i + 1] = __uint_as_float(x.w[i] & 0xffff0000u);
    }
}
template <int V>
__device__ __forceinline__ void unpack_piece(const Piece<__half, V> &x, float *f) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&x.w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
__device__ __forceinline__ void unpack_piece(const Piece<__nv_bfloat16, 1> &x, float *f) { f[0] = to_f(x.w); }
__device__ __forceinline__ void unpack_piece(const Piece<__half, 1> &x, float *f) { f[0] = to_f(x.w); }

// Two pairs of neighbours.
template <typename F>
__device__ __forceinline__ void turn2(const float2 *w, float *f, F turn) {
    const float4 c = *reinterpret_cast<const float4 *>(w);
    turn(f[0], f[1], make_float2(c.x, c.y));
    turn(f[2], f[3], make_float2(c.z, c.w));
}

// V: elements of a run; INTER: pairs are neighbours.
template <typename A, int V, bool INTER>
__global__ void __launch_bounds__(kRopeMaxThreads, 2) rope_kernel(const RopeArgs p) {
    step_begin();
    constexpr int U = 4;  // tokens of a thread at a time
    extern __shared__ __align__(16) float2 cs[];  // [token][pair]: cosine, sine
    __shared__ int64_t place[kRopeMaxTokens];  // in the caches, or -1
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)(p.n_tokens - t0 < p.tokens ? p.n_tokens - t0 : p.tokens);
    const int half = p.rot / 2;
    const int per_token = (p.hq + p.hkv + p.hv) * p.pieces;
    // tokens side by side, where a token has few pieces; a thread's first piece and first token
    const int T = blockDim.x, sub = max(1, T / per_token);
    const int first = per_token <= T ? (int)threadIdx.x / per_token : 0;
    const int64_t cache_end = (p.n_slots / p.page - 1) * p.page_stride + (p.page - 1) * p.place_stride +
                              (p.hkv - 1) * p.cache_hs + p.dim;

    Piece<A, V> x[U][2];
    struct Run {  // a thread's piece of a head: where its two runs of V elements begin in token t0's row, and go to
        const A *src;
        A *dst;
        void *cache;
        int64_t step, to_step, cache_at;
        int64_t at, end, to, to_end;  // the same places as offsets, and what there is (checked build)
        int b, pair_a, pair_b;  // the second run's distance; the runs' first pairs, -1: not rotated
    };
    auto open = [&](int slot) {
        Run q;
        const int head = slot / p.pieces, piece = slot - head * p.pieces;
        const bool rotated = piece < p.rot_pieces;
        int a;
        if (INTER && V > 1) {  // runs of whole pairs
            a = piece * V;
            q.b = p.dim / 2;
        } else if (INTER) {
            a = 2 * piece;
            q.b = 1;
        } else if (rotated) {
            a = piece * V;
            q.b = half;
        } else {
            a = p.rot + (piece - p.rot_pieces) * V;
            q.b = (p.dim - p.rot) / 2;
        }
        const bool is_q = head < p.hq, is_k = !is_q && head < p.hq + p.hkv;
        const int kvh = head - p.hq - (is_k ? 0 : p.hkv);
        if (INTER && V > 1) {
            q.pair_a = (is_q || is_k) && a < p.rot ? a / 2 : -1;
            q.pair_b = (is_q || is_k) && a + q.b < p.rot ? (a + q.b) / 2 : -1;
        } else {
            q.pair_a = q.pair_b = (is_q || is_k) && rotated ? piece * V : -1;
        }
        q.step = is_q ? p.qs : is_k ? p.ks : p.vs;
        q.to_step = is_q ? p.qos : p.kos;
        q.src = (is_q ? static_cast<const A *>(p.q) + head * p.qhs
                 : is_k ? static_cast<const A *>(p.k) + kvh * p.khs
                        : static_cast<const A *>(p.v) + kvh * p.vhs) + t0 * q.step + a;
        q.dst = is_q ? static_cast<A *>(p.q_out) + head * p.qohs + t0 * q.to_step + a
                : is_k && p.k_out ? static_cast<A *>(p.k_out) + kvh * p.kohs + t0 * q.to_step + a
                                  : nullptr;
        q.at = (is_q ? head * p.qhs : kvh * (is_k ? p.khs : p.vhs)) + t0 * q.step + a;
        q.end = is_q ? p.q_end : is_k ? p.k_end : p.v_end;
        q.to = (is_q ? head * p.qohs : kvh * p.kohs) + t0 * q.to_step + a;
        q.to_end = is_q ? p.qo_end : p.ko_end;
        q.cache = is_q || !p.k_cache ? nullptr : is_k ? p.k_cache : p.v_cache;
        q.cache_at = kvh * p.cache_hs + a;
        return q;
    };
    auto load = [&](const Run &q, int t1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t1 + u * sub;
            if (t < nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (LEAN_SPAN(q.at + t * q.step + i * q.b, V, q.end, p.err))
                        x[u][i] = *reinterpret_cast<const Piece<A, V> *>(q.src + t * q.step + i * q.b);
                    else x[u][i] = Piece<A, V>{};
            }
        }
    };
    auto finish = [&](const Run &q, int t1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t1 + u * sub;
            if (t >= nt) break;
            float f[2 * V];
            unpack_piece(x[u][0], f);
            unpack_piece(x[u][1], f + V);
            auto turn = [&](float &e0, float &e1, float2 c) {
                const float n0 = e0 * c.x - e1 * c.y, n1 = fmaf(e0, c.y, e1 * c.x);
                e0 = n0;
                e1 = n1;
            };
            const float2 *w = cs + t * half;
            if (INTER && V > 1) {
                if (q.pair_a >= 0)
#pragma unroll
                    for (int j = 0; j < V; j += 4) turn2(w + q.pair_a + j / 2, f + j, turn);
                if (q.pair_b >= 0)
#pragma unroll
                    for (int j = 0; j < V; j += 4) turn2(w + q.pair_b + j / 2, f + V + j, turn);
            } else if (q.pair_a >= 0) {
                if (V > 1) {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float4 c = *reinterpret_cast<const float4 *>(w + q.pair_a + j);
                        turn(f[j], f[V + j], make_float2(c.x, c.y));
                        turn(f[j + 1], f[V + j + 1], make_float2(c.z, c.w));
                    }
                } else {
                    turn(f[0], f[V], w[q.pair_a]);
                }
            }
            if (q.dst) {
                const int64_t to = q.to + t * q.to_step;
                if (LEAN_SPAN(to, V, q.to_end, p.err)) store_vec<A, V>(q.dst + t * q.to_step, f);
                if (LEAN_SPAN(to + q.b, V, q.to_end, p.err)) store_vec<A, V>(q.dst + t * q.to_step + q.b, f + V);
            }
            if (q.cache && place[t] >= 0) {
                const int64_t at = place[t] + q.cache_at;
                if (LEAN_SPAN(at, V, cache_end, p.err)) store_cache<V>(q.cache, at, f, p.cache_bf16);
                if (LEAN_SPAN(at + q.b, V, cache_end, p.err)) store_cache<V>(q.cache, at + q.b, f + V, p.cache_bf16);
            }
        }
    };

    int slot = per_token <= T ? threadIdx.x - first * per_token : threadIdx.x;
    const bool live = first < sub && slot < per_token;
    Run run;
    if (live) {
        run = open(slot);
        load(run, first);  // under way while the angles are computed
    }
    for (int i = threadIdx.x; i < nt * half; i += T) {
        const int t = i / half, j = i - t * half;
        const int32_t pos = LEAN_IN(t0 + t, p.n_tokens, p.err) ? p.positions[t0 + t] : 0;
        const uint64_t f = LEAN_IN(j, p.rot / 2, p.err) ? p.turns[j] : 0;
        // upper half of pos * f mod 2^64, pos signed
        const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32), u = (uint32_t)pos;
        const uint32_t turn = __umulhi(u, lo) + u * hi - (pos < 0 ? lo : 0u);
        float s, c;
        sincospif((float)(int32_t)turn * (1.f / 2147483648.f), &s, &c);
        cs[i] = make_float2(c * p.scale, s * p.scale);
    }
    if (p.k_cache && threadIdx.x < nt) {
        const int32_t s = LEAN_IN(t0 + threadIdx.x, p.n_tokens, p.err) ? p.slots[t0 + threadIdx.x] : -1;
        int64_t at = -1;
        if (s >= p.n_slots) atomicOr(p.err, kErrSlot);
        else if (s >= 0) at = (int64_t)(s / p.page) * p.page_stride + (int64_t)(s % p.page) * p.place_stride;
        place[threadIdx.x] = at;
    }
    __syncthreads();
    if (!live) return;
    for (int t1 = first;;) {
        finish(run, t1);
        t1 += U * sub;
        if (t1 >= nt) {  // on to the thread's next piece
            slot += T;
            if (per_token <= T || slot >= per_token) return;
            run = open(slot);
            t1 = first;
        }
        load(run, t1);
    }
}

template <typename A, int V>
lean_status launch_rope(RopeArgs p, bool inter, int64_t flags, void *stream) {
    p.pieces = p.dim / (2 * V);
    p.rot_pieces = p.rot / (2 * V);
    const int64_t items = (int64_t)(p.hq + p.hkv + p.hv) * p.pieces;
    // A thread for each piece of a token, or of several tokens side by side, and no more threads than that: idle ones
    // cost resident blocks.  (At 16384 tokens of 16/2 bf16 heads of 128, 80 registers: 160 threads and eight tokens a
    // block 30.1 us, four tokens 33.7, twelve 31.7, two tokens side by side in 320 threads 31.4; 64 registers
    // 33.8; two tokens' loads at a time 38.7.  At 80 registers the 16-bit kernels spill 5 to 22 words, at 64 more.)
    const int64_t sub = std::max<int64_t>(1, 256 / items);
    const int64_t passes = (items + kRopeMaxThreads - 1) / kRopeMaxThreads;
    const int threads = (int)(((sub * items + passes - 1) / passes + 31) / 32 * 32);
    // eight tokens a thread, but no fewer blocks than SMs while there are tokens for them
    int64_t tokens = std::min<int64_t>(8 * sub, std::max<int64_t>(1, p.n_tokens / (2 * step_sm_count())));
    tokens = std::min<int64_t>(tokens, std::max(1, 4096 / std::max(p.rot / 2, 1)));  // angles: 32 KB at most
    p.tokens = (int)std::min<int64_t>(tokens, kRopeMaxTokens);
    const size_t smem = sizeof(float2) * p.tokens * std::max(p.rot / 2, 1);
    const int64_t grid = (p.n_tokens + p.tokens - 1) / p.tokens;
    if (inter) return step_launch(rope_kernel<A, V, true>, grid, threads, smem, flags, stream, p);
    return step_launch(rope_kernel<A, V, false>, grid, threads, smem, flags, stream, p);
}

// Elements of a run: as many as 16 bytes have where every run is a whole number of
// them and lies on 16 bytes, of 16-bit types else half as many, else one (2000
// tokens of 32/8 bf16 heads of 80, 40 of them rotated: pairs of neighbours 7.6 us by
// eight and 19.3 by one, of halves 7.8 by four and 20.1 by one).
template <typename A>
lean_status pick_rope(const RopeArgs &p, bool inter, int64_t any_stride, bool on16, int64_t flags, void *stream) {
    constexpr int V = 16 / sizeof(A);
    auto fits = [&](int v) {
        return on16 && any_stride % v == 0 && p.dim % (2 * v) == 0 && p.rot % (inter ? v : 2 * v) == 0;
    };
    if (fits(V)) return launch_rope<A, V>(p, inter, flags, stream);
    if (V == 8 && fits(4)) return launch_rope<A, 4>(p, inter, flags, stream);
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
    auto end = [&](int64_t stride, int64_t heads, int64_t head_stride) {
        return (a->n_tokens - 1) * stride + (heads - 1) * head_stride + a->head_dim;
    };
    p.q_end = end(a->q_stride, a->n_q_heads, a->q_head_stride);
    p.k_end = end(a->k_stride, a->n_kv_heads, a->k_head_stride);
    p.v_end = end(a->v_stride, a->n_kv_heads, a->v_head_stride);
    p.qo_end = end(a->q_out_stride, a->n_q_heads, a->q_out_head_stride);
    p.ko_end = end(a->k_out_stride, a->n_kv_heads, a->k_out_head_stride);
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
