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
//     whatever rows they belong to, and walks it alone, the next unit's loads
//     under way while one is computed.  Maxima and sums are kept per lane and
//     joined where a row or the run ends; what a warp has of a row goes to the
//     workspace.
//   - A second kernel, launched early, finishes the rows.  For the top
//     alternatives the first one leaves every half unit's largest logit: the k
//     half units with the largest ones (ties: the first) hold the row's k
//     largest logits, so only they are read again, 1 KB each, and what reaches
//     the k-th of the threads' largest is ranked by counting.  The cost does not
//     depend on the order of the logits; ties go by the token id.
//
// Measured (GB300, calls in a graph): 2048 x 151936 bf16, 8 alternatives, 119 us
// (104 without, 6.0 TB/s of the 6.78 that a copy reaches; 74% of issue slots);
// fp32 229 (203 without); one row of 151936 fp32, 20 alternatives, 12.3 us (5.1
// without); 37 x 32003 fp32, 5 alternatives, 9.6 us; 90 x 18478 f16, 5: 10.4 us.
// Many rows of small vocabularies, or with many alternatives, are bound by the second
// kernel, which reads as many half units again: 6000 x 5843 fp32, 20 alternatives, 115
// us (a copy of the logits 21), 6000 x 32000 bf16, 20: 178 (57); 2885 x 2638 f16, 5: 22.
#include <type_traits>

#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kLpWarps = 8, kLpThreads = kLpWarps * 32, kLpCtas = 3;  // blocks an SM
constexpr int kLpMaxWarps = 160 * kLpCtas * kLpWarps;
constexpr int kVecs = 4;  // 16-byte pieces of a lane in a unit
constexpr int kUnitVecs = 32 * kVecs, kHalfVecs = kUnitVecs / 2;
constexpr int kTop = LEAN_MAX_TOP;
constexpr int kEndThreads = 128;  // of the second kernel
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = 1e30f;  // a power of two of minus this is 0, and it is far from overflow

struct Entry {  // a logit and its token
    float v;
    int id;
};
__device__ __forceinline__ bool beats(const Entry &a, const Entry &b) { return a.v > b.v || (a.v == b.v && a.id < b.id); }

struct Stats {  // largest logit, sums relative to it, logits above the given token's
    float m, s, w;
    int above;
};
#define LP_NONE (Entry{-CUDART_INF_F, INT32_MAX})  // no entry: beaten by every one

struct LpArgs {
    const void *x;
    const int32_t *ids;
    float *logprobs, *entropy, *top_lp;
    int32_t *ranks, *top_ids;
    Stats *runs;   // of a warp: of the row that began before it, and of the one that goes on after it
    Stats *whole;  // of a row that lies in one warp's run
    int *halves;   // [row][half unit]: largest logits, as ordered()
    int64_t n_runs, n_whole, n_halves;  // entries there are, for the checked build
    int64_t stride;
    int rows, vocab, top_k;
    int row_units;
    unsigned units, warps, q, rest;  // a warp has q units, the first `rest` warps one more
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
// Order of floats as whole numbers, -inf the least that is not NaN.
__device__ __forceinline__ int ordered(float f) {
    const int b = __float_as_int(f + 0.f);  // -0 is 0
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7fffffff)); }

// The lanes' sums as one, in all lanes.
__device__ __forceinline__ void join_lanes(const LpArgs &p, Stats &a) {
    move_to(p, a, unordered(__reduce_max_sync(0xffffffffu, ordered(a.m))));
    a.s = warp_sum(a.s);
    a.w = warp_sum(a.w);
    a.above = __reduce_add_sync(0xffffffffu, a.above);
}

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

// Entries of the workspace (what is outside it is not there in the checked build).
__device__ __forceinline__ Stats load_stats(const LpArgs &p, const Stats *v, int64_t i, int64_t n) {
    return LEAN_IN(i, n, p.err) ? v[i] : Stats{kLowest, 0.f, 0.f, 0};
}
__device__ __forceinline__ Stats load_run(const LpArgs &p, unsigned i) { return load_stats(p, p.runs, i, p.n_runs); }
__device__ __forceinline__ Stats load_whole(const LpArgs &p, int64_t row) { return load_stats(p, p.whole, row, p.n_whole); }
__device__ __forceinline__ int load_half(const LpArgs &p, const int *of_row, int i) {
    return LEAN_IN(of_row - p.halves + i, p.n_halves, p.err) ? of_row[i] : ordered(-CUDART_INF_F);
}
// A row's given token (-1: none, or outside the vocabulary) and its logit.
__device__ __forceinline__ int given_id(const LpArgs &p, int row) {
    const int id = p.ids && LEAN_IN(row, p.rows, p.err) ? p.ids[row] : -1;
    return id >= 0 && id < p.vocab ? id : -1;
}
template <typename T>
__device__ __forceinline__ float logit_of(const LpArgs &p, int row, int id) {
    const int64_t at = (int64_t)row * p.stride + id;
    return LEAN_IN(at, (p.rows - 1) * p.stride + p.vocab, p.err) ? to_f(static_cast<const T *>(p.x)[at]) : 0.f;
}

// A row as 16-byte pieces from the one that holds its first logit; `before` elements of that one are not the row's.
template <typename T>
struct Row {
    const uint8_t *base;
    int before;
    __device__ Row(const LpArgs &p, int row) {
        if (!LEAN_IN(row, p.rows, p.err)) row = 0;
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

__device__ __forceinline__ float log_prob(const LpArgs &p, float x, const Stats &a) {
    const float t = place_of(p, x, a.m);
    // (a logit near the lowest of fp32: beyond it in powers of two, not in powers of e)
    return fabsf(t) <= 3e38f || isnan(a.s) ? 0.69314718056f * (t - log2f(a.s)) : (x - a.m) * p.scale;
}
__device__ __forceinline__ void write_row(const LpArgs &p, int row, const Stats &a, const Entry *top, int n, int t, int step) {
    const float log_s = log2f(a.s), ln2 = 0.69314718056f;
    if (!LEAN_IN(row, p.rows, p.err)) return;
    if (t == 0) {
        const bool ok = given_id(p, row) >= 0;
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
    if (!p.logprobs || !LEAN_IN(row, p.rows, p.err)) return;
    const int id = p.ids[row];
    float lp = CUDART_NAN_F;
    if (id >= 0 && id < p.vocab) {
        const float x = logit_of<T>(p, row, id);
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

// first unit of warp g, and the warp that has unit u
__device__ __forceinline__ unsigned first_unit(const LpArgs &p, unsigned g) { return p.q * g + min(g, p.rest); }
__device__ __forceinline__ unsigned warp_of(const LpArgs &p, unsigned u) {
    const unsigned more = p.rest * (p.q + 1);
    return u < more ? u / (p.q + 1) : p.rest + (u - more) / p.q;
}

template <typename T, bool TOPS>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) logprobs_kernel(const LpArgs p) {
    constexpr int E = Lane<T>::kPer, WORDS = 4 * kVecs;
    step_begin();
    const int lane = threadIdx.x % 32;
    const unsigned g = blockIdx.x * kLpWarps + threadIdx.x / 32;
    if (g >= p.warps) return;
    const unsigned lo = first_unit(p, g);
    const int n = (int)(first_unit(p, g + 1) - lo);
    int row = (int)(lo / p.row_units), c = (int)(lo - (unsigned)row * p.row_units);
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
    float given = 0.f;
    uint32_t given2 = 0;
    bool fresh = true, began_here = c == 0;
    for (int i = 0; i < n; ++i) {
        if (fresh) {
            fresh = false;
            a = Stats{kLowest, 0.f, 0.f, 0};
            given = CUDART_INF_F;  // nothing is above it
            if (p.ids) {
                const int id = given_id(p, row);
                if (id >= 0) given = logit_of<T>(p, row, id);
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
        const bool row_end = c == p.row_units - 1, at_end = i == n - 1;
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
        if (TOPS) {
            // (a lane that has only NaN: -inf)
            const int h0 = __reduce_max_sync(0xffffffffu, ordered(fmaxf(top0, -CUDART_INF_F)));
            const int h1 = __reduce_max_sync(0xffffffffu, ordered(fmaxf(top1, -CUDART_INF_F)));
            const int64_t at_half = ((int64_t)row * p.row_units + c) * 2;
            if (lane == 0 && LEAN_SPAN(at_half, 2, p.n_halves, p.err))
                *reinterpret_cast<int2 *>(p.halves + at_half) = make_int2(h0, h1);
        }
        if (row_end || at_end) {
            fresh = true;
            join_lanes(p, a);
            if (lane == 0) {
                if (!began_here || !row_end) {
                    const unsigned run = 2 * g + began_here;
                    if (LEAN_IN(run, p.n_runs, p.err)) p.runs[run] = a;
                } else if (TOPS) {
                    if (LEAN_IN(row, p.n_whole, p.err)) p.whole[row] = a;
                } else {
                    write_row(p, row, a, nullptr, 0, 0, 1);
                    write_given<T>(p, row, a);
                }
            }
            began_here = true;
        }
        c = row_end ? 0 : c + 1;
        row += row_end;
    }
}

// The order of entries as one number: the greater beats.
__device__ __forceinline__ unsigned long long key_of(const Entry &e) {
    return (unsigned long long)((unsigned)ordered(e.v) ^ 0x80000000u) << 32 | (unsigned)(INT32_MAX - e.id);
}

// The k best of all threads' entries, in order, to best; how many there are.  `mine`: the thread's best; each(t, f)
// calls f with all of its entries that reach t, and may call it with more.  Entries at -inf are none.  k threads' bests
// are as good as the k-th of them, so that only entries that it does not beat count, and only k threads have any.
// list: room for n entries that are there already, and all of k threads.
struct Pick {
    alignas(16) int values[kEndThreads], ids[kEndThreads];
    unsigned long long least;
    int kth, n, ties;
};
template <typename F>
__device__ __forceinline__ int pick_best(Pick &sh, Entry *list, int n, Entry *best, int k, const Entry &mine, F each) {
    const int none = ordered(-CUDART_INF_F), v = ordered(mine.v);
    sh.values[threadIdx.x] = v;
    if (threadIdx.x == 0) {
        sh.n = n;
        sh.ties = 0;
        sh.kth = INT32_MAX;
    }
    __syncthreads();
    int r = 0;  // threads whose best is larger
#pragma unroll 8
    for (int i = 0; i < kEndThreads; i += 4) {
        const int4 q = *reinterpret_cast<const int4 *>(sh.values + i);
        r += (q.x > v) + (q.y > v) + (q.z > v) + (q.w > v);
    }
    if (r < k) atomicMin(&sh.kth, v);
    const int as_good = __syncthreads_count(r < k);
    const int t = max(sh.kth, none + 1);  // (the k-th largest; of what is not -inf, the least)
    // the lowest key that counts: all that reach t, unless more than k threads do
    unsigned long long least = (unsigned long long)((unsigned)t ^ 0x80000000u) << 32;
    if (as_good > k && sh.kth > none) {
        // of equal bests the lowest ids count; their threads come after r others (a rare path: short code, which
        // is not in the instruction cache)
        if (v == t) sh.ids[atomicAdd(&sh.ties, 1)] = mine.id;
        __syncthreads();
        if (v == t) {
#pragma unroll 1
            for (int i = sh.ties; --i >= 0;) r += sh.ids[i] < mine.id;
            if (r == k - 1) sh.least = key_of(mine);
        }
        __syncthreads();
        least = sh.least;
    }
    if (v >= t)
        each(unordered(t), [&](const Entry &e) {
            if (key_of(e) >= least && e.v <= CUDART_INF_F) list[atomicAdd(&sh.n, 1)] = e;  // (NaN is none either)
        });
    __syncthreads();
    n = sh.n;
    for (int i = threadIdx.x; i < n; i += kEndThreads) {
        const Entry e = list[i];
        int q = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) q += beats(list[j], e);
        if (q < k) best[q] = e;
    }
    __syncthreads();
    return n < k ? n : k;
}

struct EndShared {
    Entry best[kTop];
    int picked[kTop];
    Stats stats[kEndThreads / 32];
    Pick pick;
};

// The rows' ends: sums joined, top logits found.  TOPS: a block per row; else a block per warp of the kernel before,
// for the row that begins in its run and goes on after it.
template <typename T, bool TOPS, int PIECES>
__global__ void __launch_bounds__(kEndThreads) logprobs_end_kernel(const LpArgs p) {
    constexpr int E = Lane<T>::kPer;
    extern __shared__ __align__(16) uint8_t list_raw[];  // candidates: of k threads at most, and the k so far
    Entry *list = reinterpret_cast<Entry *>(list_raw);
    __shared__ EndShared sh;
    Entry *const best = sh.best;
    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n_half = 2 * p.row_units, k = p.top_k;
    int row = blockIdx.x;
    unsigned u0 = (unsigned)row * p.row_units;
    if (!TOPS) {
        const unsigned lo = first_unit(p, blockIdx.x), hi = first_unit(p, blockIdx.x + 1);
        row = (int)((hi - 1) / p.row_units);
        u0 = (unsigned)row * p.row_units;
        if (u0 < lo || u0 + p.row_units <= hi) return;
    }
    const unsigned g0 = warp_of(p, u0), g1 = warp_of(p, u0 + p.row_units - 1);
    Stats a = {kLowest, 0.f, 0.f, 0};
    if (g0 == g1) {
        a = load_whole(p, row);
    } else {
        for (unsigned i = g0 + threadIdx.x; i <= g1; i += kEndThreads) join(p, a, load_run(p, 2 * i + (i == g0)));
        join_lanes(p, a);
        if (lane == 0) sh.stats[warp] = a;
    }
    __syncthreads();
    if (g0 != g1) {
        a = sh.stats[0];
        for (int i = 1; i < kEndThreads / 32; ++i) join(p, a, sh.stats[i]);
    }
    int n = 0;
    if (TOPS) {
        // the k half units with the largest maxima, equal ones in their order
        const int *halves = p.halves + (int64_t)row * n_half;
        Entry mine = LP_NONE;
        for (int i = threadIdx.x; i < n_half; i += kEndThreads) {
            const float v = unordered(load_half(p, halves, i));
            if (v > mine.v) mine = Entry{v, i};
        }
        const int n_picked = pick_best(sh.pick, list, 0, best, k, mine, [&](float, auto f) {
            for (int i = threadIdx.x; i < n_half; i += kEndThreads) f(Entry{unordered(load_half(p, halves, i)), i});
        });
        if (threadIdx.x < n_picked) sh.picked[threadIdx.x] = best[threadIdx.x].id;
        __syncthreads();
        // their logits, in rounds of PIECES pieces a thread, the best so far carried on
        const int pieces = n_picked * kHalfVecs;
        const Row<T> at(p, row);
        for (int from = 0; from < pieces; from += PIECES * kEndThreads) {
            uint4 v[PIECES];
            int id[PIECES];
            mine = LP_NONE;
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const int i = from + j * kEndThreads + threadIdx.x;
                if (i >= pieces) break;
                const int piece = sh.picked[i / kHalfVecs] * kHalfVecs + i % kHalfVecs;
                id[j] = piece * E - at.before;
                v[j] = at.load(p, piece);
            }
            auto each = [&](float t, auto f) {
#pragma unroll
                for (int j = 0; j < PIECES; ++j) {
                    if (from + j * kEndThreads + (int)threadIdx.x >= pieces) break;
                    const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                    if (!(Lane<T>::largest(x, 4) >= t)) continue;
#pragma unroll
                    for (int e = 0; e < E; ++e) f(Entry{Lane<T>::get(x[e * 4 / E], e & 1), id[j] + e});
                }
            };
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                if (from + j * kEndThreads + (int)threadIdx.x >= pieces) break;
                const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                const float top = Lane<T>::largest(x, 4);
                if (top > mine.v) {
                    mine.v = top;
#pragma unroll
                    for (int e = E - 1; e >= 0; --e)
                        if (Lane<T>::get(x[e * 4 / E], e & 1) == top) mine.id = id[j] + e;
                } else if (top == mine.v) {  // (picked half units are in the order of their maxima: ids do not rise)
#pragma unroll
                    for (int e = E - 1; e >= 0; --e)
                        if (Lane<T>::get(x[e * 4 / E], e & 1) == top) mine.id = min(mine.id, id[j] + e);
                }
            }
            for (int i = threadIdx.x; i < n; i += kEndThreads) list[i] = best[i];
            n = pick_best(sh.pick, list, n, best, k, mine, each);
        }
    }
    write_row(p, row, a, best, n, threadIdx.x, kEndThreads);
    if (threadIdx.x == 0) write_given<T>(p, row, a);
}

// The same with a warp per row, for many rows: no barriers, a sixth of the instructions.  k <= 32.
constexpr int kRowWarps = 4, kRowList = 32 + 32 * 8 + 32;  // candidates: the best so far and a step's
// The k best of a warp's list of n, in order, to its front; how many they are.  (A call: it is rare, and its state must
// not make the list's live in memory.)
__device__ __noinline__ int rank_list(Entry *list, Entry *best, int n, int k) {
    const int lane = threadIdx.x % 32;
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
        const Entry e = list[i];
        int q = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) q += beats(list[j], e);
        if (q < k) best[q] = e;
    }
    __syncwarp();
    n = min(n, k);
    if (lane < n) list[lane] = best[lane];
    __syncwarp();
    return n;
}
struct WarpList {
    Entry *list, *best;
    int *count;  // entries in the list
    int most;    // and how many there may be
    int n, k;    // after rank(): entries
    bool full;   // k are known: others have to beat the last of them
    Entry kth;

    __device__ __forceinline__ void clear() {
        __syncwarp();
        if (threadIdx.x % 32 == 0) *count = 0;
        __syncwarp();
        most = 0;
        full = false;
    }
    __device__ __forceinline__ void rank() {
        __syncwarp();
        n = rank_list(list, best, *count, k);
        if (threadIdx.x % 32 == 0) *count = n;
        __syncwarp();
        most = n;
        full = n == k;
        if (full) kth = list[k - 1];
    }
    // What a logit has to reach to count: not less than the k-th, and more than -inf.
    __device__ __forceinline__ float reach(float least) const {
        return fmaxf(full ? fmaxf(least, kth.v) : least, kLowest);
    }
    // One lane's entry.  (Few lanes have one: their turns cost less than a vote of all lanes for every logit.)
    __device__ __forceinline__ void add(const Entry &e) {
        if (!(full && beats(kth, e))) list[atomicAdd(count, 1)] = e;
    }
    __device__ __forceinline__ void room(int more) {
        if (most + more > kRowList) rank();
        most += more;
    }
};
// The k-th largest of the lanes' values (none where fewer lanes have more than none): k of them reach it.
__device__ __forceinline__ int kth_of_lanes(int *values, int v, int k) {
    const int lane = threadIdx.x % 32;
    __syncwarp();
    values[lane] = v;
    __syncwarp();
    int r = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const int4 q = *reinterpret_cast<const int4 *>(values + i);
        r += (q.x > v) + (q.y > v) + (q.z > v) + (q.w > v);
    }
    return __reduce_min_sync(0xffffffffu, r < k ? v : INT32_MAX);
}

struct RowsShared {
    Entry lists[kRowWarps][kRowList], bests[kRowWarps][32];
    alignas(16) int values[kRowWarps][32];
    int counts[kRowWarps];
};

template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32) logprobs_rows_kernel(const LpArgs p) {
    constexpr int E = Lane<T>::kPer, PIECES = 8;  // a lane's in a round
    __shared__ RowsShared sh;
    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n_half = 2 * p.row_units, k = p.top_k;
    const int64_t row64 = (int64_t)blockIdx.x * kRowWarps + warp;
    if (row64 >= p.rows) return;
    const int row = (int)row64;
    const unsigned u0 = (unsigned)row * p.row_units, g0 = warp_of(p, u0), g1 = warp_of(p, u0 + p.row_units - 1);
    // the half units with the largest maxima
    const int *halves = p.halves + (int64_t)row * n_half;
    int most = ordered(-CUDART_INF_F);
    for (int i = lane; i < n_half; i += 32) most = max(most, load_half(p, halves, i));
    Stats a = load_whole(p, row);
    if (g0 != g1) {
        a = load_run(p, 2 * g0 + 1);
        if (g1 - g0 < 8) {
            for (unsigned g = g0 + 1; g <= g1; ++g) join(p, a, load_run(p, 2 * g));
        } else {
            if (lane > 0) a = Stats{kLowest, 0.f, 0.f, 0};
            for (unsigned g = g0 + 1 + lane; g <= g1; g += 32) join(p, a, load_run(p, 2 * g));
            join_lanes(p, a);
        }
    }
    WarpList w;
    w.list = sh.lists[warp];
    w.best = sh.bests[warp];
    w.count = &sh.counts[warp];
    w.k = k;
    w.clear();
    float least = unordered(kth_of_lanes(sh.values[warp], most, k));
    for (int i0 = 0; i0 < n_half; i0 += 32) {
        const int i = i0 + lane;
        const float v = i < n_half ? unordered(load_half(p, halves, i)) : -CUDART_INF_F;
        w.room(32);
        if (v >= w.reach(least)) w.add(Entry{v, i});
    }
    w.rank();
    const int n_picked = w.n, picked = lane < n_picked ? w.list[lane].id : 0;
    w.clear();
    // their logits
    const int pieces = n_picked * kHalfVecs;
    const Row<T> at(p, row);
    for (int from = 0; from < pieces; from += PIECES * 32) {
        uint4 v[PIECES];
        int id[PIECES];
        float top[PIECES], mine = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int i = from + j * 32 + lane;  // (a half unit is two steps of the warp)
            const int piece = __shfl_sync(0xffffffffu, picked, min(i / kHalfVecs, 31)) * kHalfVecs + i % kHalfVecs;
            id[j] = piece * E - at.before;
            v[j] = make_uint4(Lane<T>::kMasked, Lane<T>::kMasked, Lane<T>::kMasked, Lane<T>::kMasked);
            if (i < pieces) v[j] = at.load(p, piece);
        }
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            top[j] = fmaxf(Lane<T>::largest(x, 4), -CUDART_INF_F);
            mine = fmaxf(mine, top[j]);
        }
        least = unordered(kth_of_lanes(sh.values[warp], ordered(mine), k));
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const float t = w.reach(least);
            const unsigned lanes = __ballot_sync(0xffffffffu, top[j] >= t);
            if (!lanes) continue;
            w.room(__popc(lanes) * E);
            if (top[j] >= t) {
                const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const Entry it = {Lane<T>::get(x[e * 4 / E], e & 1), id[j] + e};
                    if (it.v >= t) w.add(it);
                }
            }
        }
        w.rank();
    }
    write_row(p, row, a, w.list, w.n, lane, 32);
    if (lane == 0) write_given<T>(p, row, a);
}

// units of a row of 16-byte pieces, which may begin anywhere in one
int64_t lp_row_units(int64_t vocab, int64_t size, bool aligned) {
    const int64_t per = 16 / size;
    return ((vocab + (aligned ? 0 : per - 1) + per - 1) / per + kUnitVecs - 1) / kUnitVecs;
}

template <typename T>
lean_status launch_logprobs(LpArgs p, int64_t flags, void *stream) {
    p.row_units = (int)lp_row_units(p.vocab, sizeof(T), (p.stride * sizeof(T)) % 16 == 0 && (uintptr_t)p.x % 16 == 0);
    const int64_t units = (int64_t)p.rows * p.row_units;
    if (units > INT32_MAX) return LEAN_ERR_SHAPE;
    p.units = (unsigned)units;
    // a unit a warp at least
    const int64_t grid = std::min<int64_t>(std::min(step_sm_count(), 160) * kLpCtas, (units + kLpWarps - 1) / kLpWarps);
    p.warps = (unsigned)std::min<int64_t>(grid * kLpWarps, units);
    p.q = p.units / p.warps;
    p.rest = p.units % p.warps;
    // (the largest scales go by the far path always)
    const float clamp = std::is_same<T, __half>::value ? -65504.f : -9.9e29f;
    p.low = p.c > 1e6f ? 3.4e38f : std::max(-p.far, clamp + 160.f / p.c);
    // The second kernel's blocks come while the first one's end, which takes the same amount of shared memory from L1
    // for both: what the blocks of the second that an SM gets need, its registers allow five.  (Left to the driver, 90
    // x 18478 f16, 5 alternatives, took 16.0 us in place of 10.7: an SM changes its amount when it is idle.  Too little
    // costs blocks at a time: 2885 x 2638 f16 45 us with 18 KB in place of 33.7, 37 x 32003 fp32 10.6 with 9 in place of
    // 9.5.  Too much leaves no L1 to load into: 2048 x 151936 bf16 130 with all of it in place of 119.)
    auto launch = [&](auto first, auto second, int64_t blocks, int threads, size_t fixed, size_t list) {
        const int64_t of_sm = std::min<int64_t>(5, (blocks + step_sm_count() - 1) / step_sm_count());
        const int64_t need = std::max<int64_t>(of_sm * (int64_t)(fixed + list + 1024) + kLpCtas * 2048, 13 << 10);
        const int shared = (int)std::min<int64_t>(100, (100 * need + 228 * 1024 - 1) / (228 * 1024));
        const lean_status st = step_launch_with(shared, first, grid, kLpThreads, 0, flags, stream, p);
        if (st != LEAN_OK || blocks == 0) return st;
        return step_launch_with(shared, second, blocks, threads, list, LEAN_FLAG_EARLY_WEIGHTS, stream, p);
    };
    if (p.top_k == 0)  // (no row is shared by warps if there is one)
        return launch(logprobs_kernel<T, false>, logprobs_end_kernel<T, false, 1>, p.warps == 1 ? 0 : p.warps, kEndThreads,
                      sizeof(EndShared), 0);
    // A warp per row where there are so many that a barrier's wait counts more than a row's own time, which grows with
    // the half units that it reads.  Measured, us a call, block and warp per row: 16-bit 2048 x 151936, 8 alternatives
    // 134 119; 780 x 32000, 5: 22.1 21.3; 600 x 32000, 1: 17.9 15.6; 6000 x 32000, 20: 202 179; 3040 x 151936, 20: 228
    // 229; 512 x 151936, 8: 41.6 43.9; fp32 500 x 32000, 1: 24.1 21.4; 8000 x 32000, 5: 234 222; 1000 x 32000, 5: 36.8
    // 37.9; 6000 x 5843, 20: 119 151.
    const int64_t reads = std::min(p.top_k, 2 * p.row_units);
    const bool wide = sizeof(T) == 4;
    if (p.top_k <= 32 && p.rows >= (wide ? 2 : 1) * reads * step_sm_count() && (!wide || reads <= 8))
        return launch(logprobs_kernel<T, true>, logprobs_rows_kernel<T>, ((int64_t)p.rows + kRowWarps - 1) / kRowWarps,
                      kRowWarps * 32, sizeof(RowsShared), 0);
    // pieces of a thread in a round: 4 take 8 half units at once, 10 take 20
    auto end = [&](auto kern, int pieces) {
        const int per_thread = std::max(pieces * Lane<T>::kPer, (2 * p.row_units + kEndThreads - 1) / kEndThreads);
        return launch(logprobs_kernel<T, true>, kern, p.rows, kEndThreads, sizeof(EndShared),
                      sizeof(Entry) * p.top_k * (per_thread + 1));
    };
    return p.top_k <= 8 ? end(logprobs_end_kernel<T, true, 4>, 4) : end(logprobs_end_kernel<T, true, 10>, 10);
}

}  // namespace

extern "C" int64_t lean_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top_k) {
    if (rows <= 0 || rows > INT32_MAX || vocab < 1 || vocab > (1 << 20) || top_k < 0 || top_k > LEAN_MAX_TOP) return -1;
    // sums of the warps' runs; with top logits, sums of every row and the largest logits of its half units (of 16-bit
    // logits there are half as many)
    const int64_t runs = (int64_t)kLpMaxWarps * 2 * sizeof(Stats);
    return top_k == 0 ? runs : runs + rows * (int64_t)sizeof(Stats) + rows * lp_row_units(vocab, 4, false) * 2 * (int64_t)sizeof(int);
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
    p.runs = static_cast<Stats *>(a->workspace);
    p.whole = p.runs + 2 * kLpMaxWarps;
    p.halves = reinterpret_cast<int *>(p.whole + a->rows);
    p.n_runs = 2 * kLpMaxWarps;
    p.n_whole = a->top_k ? a->rows : 0;
    p.n_halves = a->top_k ? a->rows * lp_row_units(a->vocab, 4, false) * 2 : 0;
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
