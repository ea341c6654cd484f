// logprobs.cu -- lean_token_logprobs: log probabilities of given tokens, with
// ranks, entropy and the top alternatives.
//
// With t_j = (x_j - m) c, c = scale log2 e and m the row's largest logit,
//   S = sum 2^t_j,  W = sum t_j 2^t_j,
//   logprob = ln 2 (t - log2 S),  entropy = ln 2 (log2 S - W / S),
// all from one reading of the logits, which is what bounds the call (HBM; 16-bit
// logits come near the rate of exponentials, 16 a clock and SM).
//
//   - Units of 2 KB of a row; every warp of the GPU takes an equal run of them,
//     whatever rows they belong to, and walks it without barriers, the next
//     unit's loads under way while one is computed.  Maxima and sums are kept
//     per lane and joined where a row ends.
//   - Top alternatives: of every half unit the largest logit is kept, and of
//     every lane the largest of each half.  The k-th largest of those 64 is a
//     value that k logits of the row reach, so that only half units that reach
//     it are read again (from L2) when the row ends; what reaches it there, a
//     few more than k, is ranked by counting.  Cost does not depend on the order
//     of the logits; ties go by the token id.
//   - Rows shared by warps join through shared memory, rows shared by blocks
//     through the workspace and a second kernel, launched early.
#include <type_traits>

#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kLpWarps = 8, kLpThreads = kLpWarps * 32, kLpCtas = 3;  // blocks an SM
constexpr int kLpMaxCtas = 160 * kLpCtas;
constexpr int kVecs = 4;            // 16-byte pieces of a lane in a unit
constexpr int kUnitVecs = 32 * kVecs;
constexpr int kHalves = 128;        // half units whose maxima a warp keeps before it takes their top logits
constexpr int kList = 256;          // candidates of a warp
constexpr int kTop = LEAN_MAX_TOP;
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = 1e30f;       // a power of two of minus this is 0, and it is far from overflow
constexpr int64_t kLpSharedBytes = 4096;  // what blocks share, per block

struct Entry {  // a logit and its token
    float v;
    int id;
};
__device__ __forceinline__ bool beats(const Entry &a, const Entry &b) { return a.v > b.v || (a.v == b.v && a.id < b.id); }

struct Stats {  // largest logit, sums relative to it, logits above the given token's
    float m, s, w;
    int above;
};
struct Part {  // of a row: its first token's place does not matter, ids are the row's
    Stats st;
    int n;  // entries
    int pad[3];
    Entry top[kTop];
};
struct LpShared {  // a row that begins in a block and goes on in others (-1: none), and how many blocks it has
    int row, parts;
};

struct LpArgs {
    const void *x;
    const int32_t *ids;
    float *logprobs, *entropy, *top_lp;
    int32_t *ranks, *top_ids;
    LpShared *shared;
    Part *parts;
    int64_t stride;
    int rows, vocab, top_k;
    int row_units, units;
    float scale, c;  // c = scale * log2 e
    float far;       // a reference m up to here has m c <= kFar
    float low;       // and one from here on (to far) makes 0 of what pair<CLAMP> makes of -inf
    unsigned *err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// Where logit x lies relative to the reference m, in powers of two: x c - (m c as rounded), one rounding, or for
// references near the ends of fp32 (x - m) c.
__device__ __forceinline__ float place_of(const LpArgs &p, float x, float m) {
    return fabsf(m) <= p.far ? fmaf(x, p.c, -(m * p.c)) : (x - m) * p.c;
}
// From the reference a.m to a larger one (the products rounded as add_words has them, never fused with the
// difference).
__device__ __forceinline__ void move_to(const LpArgs &p, Stats &a, float m) {
    float d = fabsf(a.m) <= p.far && fabsf(m) <= p.far ? __fsub_rn(__fmul_rn(a.m, p.c), __fmul_rn(m, p.c))
                                                      : (a.m - m) * p.c;
    d = max_nan(d, -kFar);
    const float f = ex2(d);
    a.w = f * fmaf(d, a.s, a.w);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void join(const LpArgs &p, Stats &a, Stats b) {
    const float m = fmaxf(a.m, b.m);
    move_to(p, a, m);
    move_to(p, b, m);
    a.s += b.s;
    a.w += b.w;
    a.above += b.above;
}
__device__ __forceinline__ Stats shuffle(const Stats &a, int o) {
    return Stats{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                 __shfl_xor_sync(0xffffffffu, a.w, o), __shfl_xor_sync(0xffffffffu, a.above, o)};
}

// Order of floats as whole numbers, -inf the least that is not NaN.
__device__ __forceinline__ int ordered(float f) {
    const int b = __float_as_int(f + 0.f);  // -0 is 0
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7fffffff)); }

// ---- a lane's words of logits --------------------------------------------------------

template <typename T>
struct Lane;
template <>
struct Lane<float> {
    static constexpr int kPer = 4;  // of 16 bytes
    __device__ static float largest(const uint32_t *w, int n) {
        float m = __uint_as_float(w[0]);
        for (int i = 1; i < n; ++i) m = fmaxf(m, __uint_as_float(w[i]));
        return m;
    }
    __device__ static int above(const uint32_t *w, int n, float x, uint32_t) {
        int c = 0;
        for (int i = 0; i < n; ++i) c += __uint_as_float(w[i]) > x;
        return c;
    }
    // words i and i + 1 (i even) as a pair; CLAMP: no less than -kFar
    template <bool CLAMP>
    __device__ static float2 pair(const uint32_t *w, int i) {
        const float a = __uint_as_float(w[i]), b = __uint_as_float(w[i + 1]);
        return CLAMP ? make_float2(max_nan(a, -kFar), max_nan(b, -kFar)) : make_float2(a, b);
    }
    static constexpr int kPairWords = 2;
    __device__ static float get(uint32_t w, int) { return __uint_as_float(w); }
    __device__ static uint32_t twice(float) { return 0; }
    static constexpr uint32_t kMasked = 0xff800000u;
};
template <>
struct Lane<__nv_bfloat16> {
    static constexpr int kPer = 8;
    __device__ static __nv_bfloat162 as(uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); }
    __device__ static float largest(const uint32_t *w, int n) {
        __nv_bfloat162 m = as(w[0]);
        for (int i = 1; i < n; ++i) m = __hmax2(m, as(w[i]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ static int above(const uint32_t *w, int n, float, uint32_t x2) {
        __nv_bfloat162 c = __hgt2(as(w[0]), as(x2));  // 1 or 0 each; up to 256 are exact
        for (int i = 1; i < n; ++i) c = __hadd2(c, __hgt2(as(w[i]), as(x2)));
        return (int)(__low2float(c) + __high2float(c));
    }
    template <bool CLAMP>
    __device__ static float2 pair(const uint32_t *w, int i) {
        uint32_t u = w[i];
        if (CLAMP) {
            const __nv_bfloat162 v = __hmax2_nan(as(u), as(0xf149f149u));  // -9.98e29 twice
            u = *reinterpret_cast<const uint32_t *>(&v);
        }
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static constexpr int kPairWords = 1;
    __device__ static float get(uint32_t w, int half) { return __uint_as_float(half ? w & 0xffff0000u : w << 16); }
    __device__ static uint32_t twice(float x) {
        const __nv_bfloat162 v = __float2bfloat162_rn(x);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static constexpr uint32_t kMasked = 0xff80ff80u;
};
template <>
struct Lane<__half> {
    static constexpr int kPer = 8;
    __device__ static __half2 as(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }
    __device__ static float largest(const uint32_t *w, int n) {
        __half2 m = as(w[0]);
        for (int i = 1; i < n; ++i) m = __hmax2(m, as(w[i]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ static int above(const uint32_t *w, int n, float, uint32_t x2) {
        __half2 c = __hgt2(as(w[0]), as(x2));
        for (int i = 1; i < n; ++i) c = __hadd2(c, __hgt2(as(w[i]), as(x2)));
        return (int)(__low2float(c) + __high2float(c));
    }
    template <bool CLAMP>
    __device__ static float2 pair(const uint32_t *w, int i) {
        return CLAMP ? __half22float2(__hmax2_nan(as(w[i]), as(0xfbfffbffu))) : __half22float2(as(w[i]));
    }
    static constexpr int kPairWords = 1;
    __device__ static float get(uint32_t w, int half) { return half ? __high2float(as(w)) : __low2float(as(w)); }
    __device__ static uint32_t twice(float x) {
        const __half2 v = __float2half2_rn(x);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static constexpr uint32_t kMasked = 0xfc00fc00u;
};

// A row as 16-byte pieces from the one that holds its first logit; `before` elements of that one are not the row's.
template <typename T>
struct Row {
    const uint8_t *base;
    int before;
    __device__ Row(const LpArgs &p, int row) {
        const uint8_t *at = static_cast<const uint8_t *>(p.x) + (int64_t)row * p.stride * sizeof(T);
        const int off = (int)((uintptr_t)at & 15);
        base = at - off;
        before = off / (int)sizeof(T);
    }
    // piece v as words; what is not the row's is -inf
    __device__ uint4 load(const LpArgs &p, int v) const {
        constexpr int E = Lane<T>::kPer;
        const int first = v * E - before;
        if (first >= 0 && first + E <= p.vocab) return __ldg(reinterpret_cast<const uint4 *>(base) + v);
        uint32_t w[4] = {Lane<T>::kMasked, Lane<T>::kMasked, Lane<T>::kMasked, Lane<T>::kMasked};
        if (first + E > 0 && first < p.vocab) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (first + i < 0 || first + i >= p.vocab) continue;
                if (sizeof(T) == 4) {
                    w[i % 4] = reinterpret_cast<const uint32_t *>(base)[(int64_t)v * E + i];
                } else {
                    const uint32_t u = reinterpret_cast<const uint16_t *>(base)[(int64_t)v * E + i];
                    w[i / 2 % 4] = i & 1 ? (w[i / 2 % 4] & 0xffffu) | u << 16 : (w[i / 2 % 4] & 0xffff0000u) | u;
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// ---- a warp's candidates ---------------------------------------------------------------

struct Candidates {
    Entry *list, *best;  // kList, and kTop in order
    int n, k;
    float reach;  // candidates have to reach it,
    float kth;    // and where k are known already (full), to exceed the last of them
    bool full;

    // the k largest of the list, in order, to best; *kept: how many
    __device__ int rank(int lane) {
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
            const Entry mine = list[i];
            int r = 0;
            for (int j = 0; j < n; ++j) r += beats(list[j], mine);
            if (r < k) best[r] = mine;
        }
        __syncwarp();
        return n < k ? n : k;
    }
    __device__ void shrink(int lane) {
        n = rank(lane);
        for (int i = lane; i < n; i += 32) list[i] = best[i];
        __syncwarp();
        if (n == k) {
            full = true;
            kth = list[k - 1].v;
        }
    }
    // candidates come in rising order of their ids, so that one equal to the k-th already known loses to it
    __device__ bool wants(float v) const { return v >= reach && v > (full ? kth : -CUDART_INF_F); }
    __device__ void push(int lane, bool mine, float v, int id) {
        unsigned m = __ballot_sync(0xffffffffu, mine);
        if (m == 0) return;
        if (n + 32 > kList) {
            shrink(lane);
            mine = mine && wants(v);
            m = __ballot_sync(0xffffffffu, mine);
        }
        if (mine) list[n + __popc(m & ((1u << lane) - 1))] = Entry{v, id};
        n += __popc(m);
    }
};

__device__ __forceinline__ float log_prob(const LpArgs &p, float x, const Stats &a) {
    const float t = place_of(p, x, a.m);
    // (a logit near the lowest of fp32: beyond it in powers of two, not in powers of e)
    return fabsf(t) <= 3e38f || isnan(a.s) ? 0.69314718056f * (t - log2f(a.s)) : (x - a.m) * p.scale;
}
__device__ __forceinline__ void write_row(const LpArgs &p, int row, const Stats &a, const Entry *top, int n, int t, int step) {
    const float log_s = log2f(a.s), ln2 = 0.69314718056f;
    if (t == 0) {
        const int id = p.ids ? p.ids[row] : -1;
        const bool ok = id >= 0 && id < p.vocab;
        // (the mark of an id outside the vocabulary was left where its logit was looked up)
        if (p.ranks) p.ranks[row] = ok ? a.above : -1;
        if (p.entropy) p.entropy[row] = a.s == 0.f ? 0.f : ln2 * (log_s - a.w / a.s);
    }
    for (int i = t; i < p.top_k; i += step) {
        p.top_ids[(int64_t)row * p.top_k + i] = i < n ? top[i].id : -1;
        p.top_lp[(int64_t)row * p.top_k + i] = i < n ? log_prob(p, top[i].v, a) : -CUDART_INF_F;
    }
}
template <typename T>
__device__ __forceinline__ void write_given(const LpArgs &p, int row, const Stats &a) {
    if (!p.logprobs) return;
    const int id = p.ids[row];
    float lp = CUDART_NAN_F;
    if (id >= 0 && id < p.vocab) {
        const float x = to_f(static_cast<const T *>(p.x)[(int64_t)row * p.stride + id]);
        lp = a.s == 0.f ? -CUDART_INF_F : log_prob(p, x, a);
    }
    p.logprobs[row] = lp;
}

// A unit's share of a lane, relative to the lane's reference.  FAR: some lane's reference, or the scale, is near the
// ends of fp32 (rows masked with the type's lowest value).
template <typename T, bool FAR>
__device__ __forceinline__ void add_words(const LpArgs &p, const uint32_t (&w)[4 * kVecs], Stats &a) {
    const bool near_ = fabsf(a.m) <= p.far;
    const float off = near_ ? 0.f : -a.m, ref = near_ ? -(a.m * p.c) : 0.f;
    const f32x2 c2 = pack2(p.c, p.c), off2 = pack2(off, off), ref2 = pack2(ref, ref);
    f32x2 s2 = pack2(0.f, 0.f), w2 = s2;
#pragma unroll
    for (int i = 0; i < 4 * kVecs; i += Lane<T>::kPairWords) {
        const float2 x = Lane<T>::template pair<!FAR>(w, i);
        f32x2 t2;
        if (FAR) {
            const float2 d = unpack2(fma2(add2(pack2(x.x, x.y), off2), c2, ref2));
            t2 = pack2(max_nan(d.x, -kFar), max_nan(d.y, -kFar));
        } else {
            t2 = fma2(pack2(x.x, x.y), c2, ref2);
        }
        const float2 t = unpack2(t2);
        const f32x2 e2 = pack2(ex2(t.x), ex2(t.y));
        s2 = add2(s2, e2);
        w2 = fma2(e2, t2, w2);
    }
    const float2 s = unpack2(s2), v = unpack2(w2);
    a.s += s.x + s.y;
    a.w += v.x + v.y;
}

struct LpRecord {
    int row, first;  // row (-1: none), and its first unit counted from the block's first one
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) logprobs_kernel(const LpArgs p, int blocks) {
    constexpr int E = Lane<T>::kPer, WORDS = 4 * kVecs;
    __shared__ Entry lists[kLpWarps][kList];
    __shared__ Entry bests[kLpWarps][kTop];
    __shared__ int halves[kLpWarps][kHalves];
    __shared__ Part part_s[2 * kLpWarps];
    __shared__ LpRecord rec[2 * kLpWarps];
    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x < 2 * kLpWarps) rec[threadIdx.x].row = -1;
    __syncthreads();
    // equal runs of units
    const unsigned q = (unsigned)p.units / blocks, rest = (unsigned)p.units - q * blocks;
    const unsigned b_lo = q * blockIdx.x + min(blockIdx.x, rest);
    const int b_n = (int)(q + (blockIdx.x < rest));
    const int u_lo = (int)((int64_t)b_n * warp / kLpWarps), u_hi = (int)((int64_t)b_n * (warp + 1) / kLpWarps);
    const bool tops = p.top_k > 0;

    if (u_lo < u_hi) {
        int row = (int)((b_lo + u_lo) / p.row_units), c = (int)((b_lo + u_lo) - (unsigned)row * p.row_units);
        Row<T> at(p, row);
        auto load = [&](const Row<T> &from, int unit, uint4 (&v)[kVecs]) {
            const int v0 = unit * kUnitVecs + lane;
            // (all of a unit inside the row: no piece needs a look)
            if (v0 - lane > 0 && (v0 - lane + kUnitVecs) * E - from.before <= p.vocab) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    if (LEAN_SPAN((int64_t)(v0 + 32 * j) * E - from.before, E, p.vocab, p.err))
                        v[j] = __ldg(reinterpret_cast<const uint4 *>(from.base) + v0 + 32 * j);
            } else {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) v[j] = from.load(p, v0 + 32 * j);
            }
        };
        uint4 next[kVecs];
        load(at, c, next);
        Stats a;
        float given = 0.f, lane_max[2];
        uint32_t given2 = 0;
        Candidates cand;
        cand.list = lists[warp];
        cand.best = bests[warp];
        cand.k = p.top_k;
        int taken = 0;  // unit of the row from which half maxima are kept
        bool fresh = true;
        for (int u = u_lo; u < u_hi; ++u) {
            if (fresh) {
                fresh = false;
                a = Stats{kLowest, 0.f, 0.f, 0};
                lane_max[0] = lane_max[1] = -CUDART_INF_F;
                cand.n = 0;
                cand.full = false;
                cand.reach = -CUDART_INF_F;
                taken = c;
                given = CUDART_INF_F;  // nothing is above it
                if (p.ids) {
                    const int id = p.ids[row];
                    if (id >= 0 && id < p.vocab) given = to_f(static_cast<const T *>(p.x)[(int64_t)row * p.stride + id]);
                    else if (lane == 0) atomicOr(p.err, kErrTokenId);
                }
                given2 = Lane<T>::twice(given);
            }
            uint32_t w[WORDS];
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                w[4 * j] = next[j].x;
                w[4 * j + 1] = next[j].y;
                w[4 * j + 2] = next[j].z;
                w[4 * j + 3] = next[j].w;
            }
            const bool row_end = c == p.row_units - 1, at_end = u == u_hi - 1;
            if (!at_end) {
                if (row_end) at = Row<T>(p, row + 1);
                load(at, row_end ? 0 : c + 1, next);
            }
            const float top0 = Lane<T>::largest(w, WORDS / 2), top1 = Lane<T>::largest(w + WORDS / 2, WORDS / 2);
            const float m = fmaxf(a.m, fmaxf(top0, top1));
            if (p.ranks) a.above += Lane<T>::above(w, WORDS, given, given2);
            move_to(p, a, m);
            if (__any_sync(0xffffffffu, !(m >= p.low && m <= p.far))) add_words<T, true>(p, w, a);
            else add_words<T, false>(p, w, a);
            if (tops) {
                lane_max[0] = fmaxf(lane_max[0], top0);
                lane_max[1] = fmaxf(lane_max[1], top1);
                const int h0 = __reduce_max_sync(0xffffffffu, ordered(top0)), h1 = __reduce_max_sync(0xffffffffu, ordered(top1));
                if (lane < 2) halves[warp][2 * (c - taken) + lane] = lane ? h1 : h0;
                if (row_end || at_end || c - taken == kHalves / 2 - 1) {
                    // the k-th largest of the lanes' 64 maxima, bit by bit; -inf where fewer lanes have any
                    const int o0 = ordered(lane_max[0]), o1 = ordered(lane_max[1]), none = ordered(-CUDART_INF_F);
                    unsigned t = 0;  // order of unsigned numbers: the sign turned round
#pragma unroll 1
                    for (unsigned bit = 1u << 31; bit; bit >>= 1) {
                        const unsigned try_ = t | bit;
                        const int n = __popc(__ballot_sync(0xffffffffu, ((unsigned)o0 ^ 0x80000000u) >= try_)) +
                                      __popc(__ballot_sync(0xffffffffu, ((unsigned)o1 ^ 0x80000000u) >= try_));
                        if (n >= p.top_k) t = try_;
                    }
                    const int reach = max((int)(t ^ 0x80000000u), none);
                    cand.reach = fmaxf(cand.reach, unordered(reach));
                    __syncwarp();
                    // the half units that reach it, again, in their order
                    const int n_half = 2 * (c - taken + 1);
                    const Row<T> self(p, row);
                    for (int i0 = 0; i0 < n_half; i0 += 32) {
                        const int hm = i0 + lane < n_half ? halves[warp][i0 + lane] : none;
                        unsigned todo = __ballot_sync(0xffffffffu, hm > none && hm >= ordered(cand.reach));
                        while (todo) {
                            const int i = i0 + __ffs(todo) - 1;
                            todo &= todo - 1;
                            const int v0 = taken * kUnitVecs + i * (kUnitVecs / 2) + lane;
                            uint4 r[kVecs / 2];
#pragma unroll
                            for (int j = 0; j < kVecs / 2; ++j) r[j] = self.load(p, v0 + 32 * j);
#pragma unroll
                            for (int j = 0; j < kVecs / 2; ++j) {
                                const uint32_t x[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
                                // whether any lane has a candidate among its pieces at all
                                if (!__any_sync(0xffffffffu, cand.wants(Lane<T>::largest(x, 4)))) continue;
                                // ids rise from lane to lane and within a lane, so a lane's all go in before the next's
                                int mine = 0;
#pragma unroll
                                for (int e = 0; e < E; ++e) mine |= (int)cand.wants(Lane<T>::get(x[e * 4 / E], e & 1)) << e;
                                for (unsigned lanes = __ballot_sync(0xffffffffu, mine != 0); lanes; lanes &= lanes - 1) {
                                    const int l = __ffs(lanes) - 1;
                                    const int its = __shfl_sync(0xffffffffu, mine, l);
#pragma unroll
                                    for (int e = 0; e < E; ++e) {
                                        if (!(its >> e & 1)) continue;
                                        const float v = Lane<T>::get(x[e * 4 / E], e & 1);
                                        cand.push(lane, lane == l && cand.wants(v), v, (v0 + 32 * j) * E - self.before + e);
                                    }
                                }
                            }
                        }
                    }
                    taken = c + 1;
                    cand.shrink(lane);
                }
            }
            if (row_end || at_end) {
                fresh = true;
#pragma unroll
                for (int o = 16; o; o >>= 1) join(p, a, shuffle(a, o));
                const int first = u - c;
                const int n = tops ? cand.n : 0;
                if (first >= u_lo && row_end) {
                    write_row(p, row, a, cand.list, n, lane, 32);
                    if (lane == 0) write_given<T>(p, row, a);
                } else {
                    Part &x = part_s[2 * warp + at_end];
                    for (int i = lane; i < n; i += 32) x.top[i] = cand.list[i];
                    if (lane == 0) {
                        x.st = a;
                        x.n = n;
                        rec[2 * warp + at_end] = LpRecord{row, first};
                    }
                }
                __syncwarp();
            }
            c = row_end ? 0 : c + 1;
            row += row_end;
        }
    }
    __syncthreads();

    // ---- rows shared by warps: record by record, the whole block on each row
    Entry *all = lists[0];  // 2048 entries
    static_assert(kLpWarps * kList >= 2 * kLpWarps * kTop, "room for all records' entries");
    LpShared goes_on = {-1, 0};
    for (int i = 0; i < 2 * kLpWarps;) {
        const LpRecord head = rec[i];
        if (head.row < 0) {
            ++i;
            continue;
        }
        int end = i + 1;
        while (end < 2 * kLpWarps && (rec[end].row < 0 || rec[end].row == head.row)) ++end;
        Stats a = part_s[i].st;
        int n = 0;
        for (int k = i; k < end; ++k) {
            if (rec[k].row < 0) continue;
            if (k > i) join(p, a, part_s[k].st);
            const int more = part_s[k].n;
            for (int e = threadIdx.x; e < more; e += kLpThreads) all[n + e] = part_s[k].top[e];
            n += more;
        }
        __syncthreads();
        Entry *best = bests[0];
        for (int e = threadIdx.x; e < n; e += kLpThreads) {
            const Entry mine = all[e];
            int r = 0;
            for (int k = 0; k < n; ++k) r += beats(all[k], mine);
            if (r < p.top_k) best[r] = mine;
        }
        __syncthreads();
        n = min(n, p.top_k);
        const bool whole = head.first >= 0 && head.first + p.row_units <= b_n;
        if (whole) {
            write_row(p, head.row, a, best, n, threadIdx.x, kLpThreads);
            if (threadIdx.x == 0) write_given<T>(p, head.row, a);
        } else {
            Part &x = p.parts[blockIdx.x * 2 + (head.first < 0 ? 0 : 1)];
            for (int e = threadIdx.x; e < n; e += kLpThreads) x.top[e] = best[e];
            if (threadIdx.x == 0) {
                x.st = a;
                x.n = n;
            }
            if (head.first >= 0) {
                const unsigned last = b_lo + head.first + p.row_units - 1;
                const unsigned b = last < rest * (q + 1) ? last / (q + 1) : rest + (last - rest * (q + 1)) / q;
                goes_on = LpShared{head.row, (int)(b - blockIdx.x) + 1};
            }
        }
        __syncthreads();
        i = end;
    }
    if (threadIdx.x == 0) p.shared[blockIdx.x] = goes_on;
}

// Rows shared by blocks: a block for each row that begins in block blockIdx.x of the kernel before and goes on.
constexpr int kMostCand = 4096;  // k parts' entries at most, see below
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_sum_kernel(const LpArgs p) {
    __shared__ Entry list[kMostCand];
    __shared__ Entry best[kTop], firsts[kLpMaxCtas];
    __shared__ Stats stats[kLpWarps];
    __shared__ Entry least_s;
    __shared__ int n_s;
    step_begin();
    const LpShared x = p.shared[blockIdx.x];
    if (x.row < 0) return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto part = [&](int k) -> const Part & { return p.parts[(blockIdx.x + k) * 2 + (k == 0)]; };
    if (threadIdx.x == 0) {
        least_s = Entry{-CUDART_INF_F, INT32_MAX};
        n_s = 0;
    }
    Stats a = {kLowest, 0.f, 0.f, 0};
    for (int k = threadIdx.x; k < x.parts; k += kLpThreads) {
        const Part &y = part(k);
        const int n = y.n;
        firsts[k] = n > 0 && p.top_k > 0 ? y.top[0] : Entry{-CUDART_INF_F, INT32_MAX};
        join(p, a, y.st);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) join(p, a, shuffle(a, o));
    if (lane == 0) stats[warp] = a;
    __syncthreads();
    a = stats[0];
    for (int i = 1; i < kLpWarps; ++i) join(p, a, stats[i]);
    int n = 0;
    if (p.top_k > 0) {
        // the k-th of the parts' first entries: k entries are as good, so no other one counts (at most the k parts
        // that are as good have any: k * k entries)
        for (int k = threadIdx.x; k < x.parts; k += kLpThreads) {
            const Entry mine = firsts[k];
            int r = 0;
            for (int j = 0; j < x.parts; ++j) r += beats(firsts[j], mine);
            if (r == p.top_k - 1 && mine.id != INT32_MAX) least_s = mine;
        }
        __syncthreads();
        const Entry least = least_s;
        for (int e = threadIdx.x; e < x.parts * p.top_k; e += kLpThreads) {
            const int k = e / p.top_k, i = e - k * p.top_k;
            if (beats(least, firsts[k]) || firsts[k].id == INT32_MAX) continue;
            const Part &y = part(k);
            if (i >= y.n) continue;
            const Entry mine = y.top[i];
            if (!beats(least, mine)) {
                const int to = atomicAdd(&n_s, 1);
                if (to < kMostCand) list[to] = mine;
            }
        }
        __syncthreads();
        n = min(n_s, kMostCand);
        for (int e = threadIdx.x; e < n; e += kLpThreads) {
            const Entry mine = list[e];
            int r = 0;
            for (int k = 0; k < n && r < p.top_k; ++k) r += beats(list[k], mine);
            if (r < p.top_k) best[r] = mine;
        }
        __syncthreads();
        n = min(n, p.top_k);
    }
    write_row(p, x.row, a, best, n, threadIdx.x, kLpThreads);
    if (threadIdx.x == 0) write_given<T>(p, x.row, a);
}

template <typename T>
lean_status launch_logprobs(LpArgs p, int64_t flags, void *stream) {
    // pieces of a row that begins anywhere in one
    const int64_t vecs = ((int64_t)p.vocab + 2 * Lane<T>::kPer - 2) / Lane<T>::kPer;
    const bool aligned = (p.stride * sizeof(T)) % 16 == 0 && (uintptr_t)p.x % 16 == 0;
    p.row_units = (int)(((aligned ? ((int64_t)p.vocab + Lane<T>::kPer - 1) / Lane<T>::kPer : vecs) + kUnitVecs - 1) / kUnitVecs);
    const int64_t units = (int64_t)p.rows * p.row_units;
    if (units > INT32_MAX) return LEAN_ERR_SHAPE;
    p.units = (int)units;
    // a unit a warp at least
    const int64_t grid = std::min<int64_t>(std::min(step_sm_count() * kLpCtas, kLpMaxCtas), (units + kLpWarps - 1) / kLpWarps);
    // (the largest scales go by the far path always)
    const float clamp = sizeof(T) == 2 && std::is_same<T, __half>::value ? -65504.f : -9.9e29f;
    p.low = p.c > 1e6f ? 3.4e38f : std::max(-p.far, clamp + 160.f / p.c);
    const lean_status st = step_launch(logprobs_kernel<T>, grid, kLpThreads, 0, flags, stream, p, (int)grid);
    if (st != LEAN_OK || grid == 1) return st;
    return step_launch(logprobs_sum_kernel<T>, grid, kLpThreads, 0, LEAN_FLAG_EARLY_WEIGHTS, stream, p);
}

}  // namespace

extern "C" int64_t lean_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top_k) {
    if (rows <= 0 || rows > INT32_MAX || vocab < 1 || vocab > (1 << 20) || top_k < 0 || top_k > LEAN_MAX_TOP) return -1;
    return kLpSharedBytes + (int64_t)kLpMaxCtas * 2 * sizeof(Part);
}

extern "C" lean_status lean_token_logprobs(const lean_logprobs_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!known_dtype(a->dtype) || !step_flags_ok(a->flags)) return LEAN_ERR_FORMAT;
    const int64_t need = lean_token_logprobs_workspace_bytes(a->rows, a->vocab, a->top_k);
    if (need < 0 || a->stride < 0 || (a->rows > 1 && a->stride < a->vocab) || !(a->scale > 0) || a->scale > 3e38)
        return LEAN_ERR_SHAPE;
    if (!a->logits || !a->workspace || (!a->ids && (a->logprobs || a->ranks)) ||
        (a->top_k > 0 && (!a->top_ids || !a->top_logprobs)))
        return LEAN_ERR_NULL;
    if (!step_aligned(a->logits, dtype_size(a->dtype)) || !step_aligned(a->ids, 4) || !step_aligned(a->logprobs, 4) ||
        !step_aligned(a->ranks, 4) || !step_aligned(a->entropy, 4) || !step_aligned(a->top_ids, 4) ||
        !step_aligned(a->top_logprobs, 4) || !step_aligned(a->workspace, 256))
        return LEAN_ERR_ALIGN;
    if (a->workspace_bytes < need) return LEAN_ERR_SHAPE;
    LpArgs p = {};
    p.x = a->logits;
    p.ids = a->ids;
    p.logprobs = a->logprobs;
    p.entropy = a->entropy;
    p.top_lp = a->top_logprobs;
    p.ranks = a->ranks;
    p.top_ids = a->top_ids;
    p.shared = static_cast<LpShared *>(a->workspace);
    p.parts = reinterpret_cast<Part *>(static_cast<uint8_t *>(a->workspace) + kLpSharedBytes);
    p.stride = a->stride;
    p.rows = (int)a->rows;
    p.vocab = (int)a->vocab;
    p.top_k = (int)a->top_k;
    p.scale = (float)a->scale;
    p.c = (float)std::min(a->scale * 1.4426950408889634, 3.4e38);
    p.far = p.c > 1.f ? kFar / p.c : kFar;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    switch (a->dtype) {
    case LEAN_F32: return launch_logprobs<float>(p, a->flags, stream);
    case LEAN_BF16: return launch_logprobs<__nv_bfloat16>(p, a->flags, stream);
    default: return launch_logprobs<__half>(p, a->flags, stream);
    }
}
