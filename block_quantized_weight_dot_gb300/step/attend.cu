// attend.cu -- lean_paged_attention: attention of one new token per sequence
// over the paged cache.
//
//   z_j = scale q . k_j,  p_j = e^(z_j - m),  m = max z_j,
//   out = sum p_j v_j / sum p_j,  lse = m + ln sum p_j
//
// Every key and value of the cache is needed once per kv head, whatever the
// number of query heads that share it: HBM bounds the call, 2 * dim * 2 bytes a
// token and kv head.  So the design is about keeping loads in flight:
//
//   - The work is a list of units: 16 tokens of one (sequence, kv head, group of
//     query heads).  Every warp of the GPU takes an equal run of units, whatever
//     the lengths are, and walks it alone: no barrier between its first load
//     and its last.
//   - A lane copies with cp.async exactly the 16-byte pieces that it will itself
//     read, in the order in which the matrix instruction wants them: K as 8
//     elements of one token (the contraction over the head dimension may take
//     the elements in any order, as long as q has the same), V as 8 elements of
//     four tokens (whose pairs are then interleaved in registers).  Shared memory
//     is a queue of registers: no swizzle, no conflicts, and cp.async.wait_group
//     is the only synchronisation.
//   - Scores and outputs come from mma.sync m16n8k16 with the query heads as
//     rows: 16 tokens take dim / 4 of them for 64 * dim bytes, a fraction of the
//     time the bytes take (tcgen05 wants 64 rows or more; a group has 1 to 16).
//     With up to 8 heads in a group, rows 0-7 hold the first part of q (or p) and
//     rows 8-15 the second, so that one instruction serves both.
//   - Running maximum and sum per warp; a warp's first and last group may be
//     shared with its neighbours: the warps of a block join through shared
//     memory, blocks through the workspace, where the block that arrives last
//     adds the parts up in their order (results do not depend on timing).
//
// q and p are split into parts of the cache's type, x = x0 + x1 (+ x2), 8 (bf16)
// or 11 bits each: three parts for fp32 q and out, which leave nothing of fp32's
// 24 bits behind; two for 16-bit ones, whose rounding of out is larger.  q is
// first scaled by a power of two so that no part can overflow or vanish.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kAttMaxDim = 256;
constexpr int kAttMaxCtas = 160;  // of a launch: at most one per SM
constexpr int kUnit = 16;         // tokens
constexpr int64_t kCounterBytes = 1024;  // an arrival counter per block

struct AttArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    unsigned *counters;
    float *warp_parts, *cta_parts;
    int64_t qs, qhs, os, ohs, page_stride, place_stride, cache_hs, table_stride, n_pages;
    int n_seqs, hq, hkv, group, tiles, dim, page, width, window;
    int act;
    float scale_log2;
    int64_t cache_extent, q_extent, out_extent;  // elements, for the checked build
    unsigned *err;
};

// Warps of a block, stages of a warp's queue: 128-192 KB of loads an SM can have
// under way.
template <int DP>
struct AttShape {
    static constexpr int kWarps = DP == 256 ? 4 : 8;
    static constexpr int kStages = DP == 64 ? 5 : DP == 128 ? 3 : 2;
    static constexpr int kStageBytes = kUnit * DP * 4;  // K and V
    // at 256 the warps' q as well (up to 12 registers per 16 elements)
    static constexpr int kSmem = kWarps * (kStages * kStageBytes + (DP == 256 ? DP / 16 * 12 * 128 : 0));
};
// A part: maxima, sums and outputs of a group of H heads.
__host__ __device__ constexpr int part_floats(int heads, int dp) { return heads * (dp + 8); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename C>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two values as one part each (nearest), with what is left of them; a in the low half.
template <typename C>
__device__ __forceinline__ uint32_t take_part(float &a, float &b);
template <>
__device__ __forceinline__ uint32_t take_part<__nv_bfloat16>(float &a, float &b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&h);
    a -= __uint_as_float(u << 16);
    b -= __uint_as_float(u & 0xffff0000u);
    return u;
}
template <>
__device__ __forceinline__ uint32_t take_part<__half>(float &a, float &b) {
    const __half2 h = __floats2half2_rn(a, b);
    a -= __low2float(h);
    b -= __high2float(h);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename A>
__device__ __forceinline__ void load8_as(const void *p, int64_t i, float *f) {
    const Vec<A, 8> v = load_vec<A, 8>(static_cast<const A *>(p) + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_f(v.v[j]);
}
__device__ __forceinline__ void load8(const void *p, int64_t i, int act, float *f) {
    if (act == LEAN_F32) load8_as<float>(p, i, f);
    else if (act == LEAN_BF16) load8_as<__nv_bfloat16>(p, i, f);
    else load8_as<__half>(p, i, f);
}
__device__ __forceinline__ void store8(void *p, int64_t i, int act, const float *f) {
    if (act == LEAN_F32) store_vec<float, 8>(static_cast<float *>(p) + i, f);
    else if (act == LEAN_BF16) store_vec<__nv_bfloat16, 8>(static_cast<__nv_bfloat16 *>(p) + i, f);
    else store_vec<__half, 8>(static_cast<__half *>(p) + i, f);
}
__device__ __forceinline__ void store4(void *p, int64_t i, int act, const float *f) {
    if (act == LEAN_F32) store_vec<float, 4>(static_cast<float *>(p) + i, f);
    else if (act == LEAN_BF16) store_vec<__nv_bfloat16, 4>(static_cast<__nv_bfloat16 *>(p) + i, f);
    else store_vec<__half, 4>(static_cast<__half *>(p) + i, f);
}

// What of a sequence is attended: tokens start..len-1, in n units from base on.
struct Span {
    int len, start, base, n;
};
__device__ __forceinline__ Span open_span(const AttArgs &p, int s) {
    Span x;
    const int64_t most = (int64_t)p.width * p.page;
    int len = p.lens[s];
    len = len < 0 ? 0 : len;
    x.len = len > most ? (int)most : len;
    x.start = p.window > 0 && x.len > p.window ? x.len - p.window : 0;
    x.base = x.start & ~(kUnit - 1);
    x.n = (x.len - x.base + kUnit - 1) / kUnit;
    x.n = x.n < 1 ? 1 : x.n;  // an empty sequence is one unit in which nothing is attended
    return x;
}

// A place in the list of units.
struct Place {
    int s, g, c;  // sequence, kv head and group of its heads (h * tiles + tile), unit of it
    Span x;
};
__device__ __forceinline__ void advance(const AttArgs &p, Place &at) {
    if (++at.c < at.x.n) return;
    at.c = 0;
    if (++at.g < p.hkv * p.tiles) return;
    at.g = 0;
    if (++at.s < p.n_seqs) at.x = open_span(p, at.s);
}

// A joined record of the warps of a block, and where its group lies.
struct Record {
    int item;           // -1: none
    int n;              // units of the item
    int64_t first;      // its first unit
    const float *part;  // maxima, sums, outputs
};

// WIDE: 9 to 16 query heads in a group, one per row; else up to 8, two rows each.
template <typename C, int DP, int PARTS, bool WIDE>
__global__ void __launch_bounds__(AttShape<DP>::kWarps * 32, 1) attend_kernel(const AttArgs p) {
    constexpr int W = AttShape<DP>::kWarps, S = AttShape<DP>::kStages, T = W * 32;
    constexpr int H = WIDE ? 16 : 8, NH = WIDE ? 2 : 1;  // heads of a group, of a thread
    constexpr int KX = DP / 32, VX = DP / 64;
    constexpr int AREGS = WIDE ? 4 * PARTS : 4 + (PARTS > 2 ? 2 : 0);  // of q per 16 elements
    constexpr bool QSMEM = DP == 256;                                  // no registers left for q
    constexpr int PF = part_floats(H, DP), PO = 8 + DP;                // a head's row of a part: m, l, -, out
    extern __shared__ __align__(16) uint8_t queue[];
    __shared__ int64_t scan[W];
    __shared__ struct {
        int s, g, c;
    } start_at[W];
    __shared__ Record rec[2 * W];
    __shared__ float total_m[H], total_l[H];
    __shared__ int last_block;

    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r = lane / 4, c4 = lane % 4;
    const int groups = p.hkv * p.tiles;

    // ---- the list of units, and this block's and warp's run of it
    const int per = (p.n_seqs + T - 1) / T;  // sequences a thread sums up
    const int s_lo = min(p.n_seqs, (int)threadIdx.x * per), s_hi = min(p.n_seqs, s_lo + per);
    int64_t mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += (int64_t)open_span(p, s).n * groups;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) scan[warp] = incl;
    if (threadIdx.x < 2 * W) rec[threadIdx.x].item = -1;
    __syncthreads();
    int64_t before = incl - mine, units = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (i < warp) before += scan[i];
        units += scan[i];
    }
    // blocks that get work: a unit a warp at least
    const int blocks = (int)min((int64_t)gridDim.x, (units + W - 1) / W);
    if ((int)blockIdx.x >= blocks) return;
    auto bound = [&](int64_t w) { return units * w / ((int64_t)blocks * W); };  // first unit of warp w of the grid
    const int64_t wg = (int64_t)blockIdx.x * W + warp;
    const int64_t u_lo = bound(wg), u_hi = bound(wg + 1);
    for (int i = 0; i < W; ++i) {
        const int64_t b = bound((int64_t)blockIdx.x * W + i);
        if (b < before || b >= before + mine) continue;
        int64_t at = before;
        for (int s = s_lo; s < s_hi; ++s) {
            const int n = open_span(p, s).n;
            if (b < at + (int64_t)n * groups) {
                const int in = (int)(b - at);
                start_at[i].s = s;
                start_at[i].g = in / n;
                start_at[i].c = in % n;
                break;
            }
            at += (int64_t)n * groups;
        }
    }
    __syncthreads();

    const uint32_t my_queue = smem_addr(queue) + warp * (S * AttShape<DP>::kStageBytes);
    if (u_lo < u_hi) {
        Place next;  // to be loaded
        next.s = start_at[warp].s;
        next.g = start_at[warp].g;
        next.c = start_at[warp].c;
        next.x = open_span(p, next.s);
        Place cur = next;  // to be computed
        int64_t u_next = u_lo;

        // the page of token lane % 16 of the unit to be loaded next, fetched one unit ahead
        auto fetch_page = [&]() {
            const int tok = next.x.base + next.c * kUnit + lane % kUnit;
            const bool in = tok >= next.x.start && tok < next.x.len;
            const int64_t e = (int64_t)next.s * p.table_stride + tok / p.page;
            return in && LEAN_IN(e, (int64_t)(p.n_seqs - 1) * p.table_stride + p.width, p.err) ? p.table[e] : 0;
        };
        int page_id = fetch_page();

        auto load_unit = [&](int stage) {
            if (u_next < u_hi) {
                const int tok = next.x.base + next.c * kUnit + lane % kUnit;
                int64_t off = -1;  // of the token's row; -1: not attended, -2: outside the cache
                if (tok >= next.x.start && tok < next.x.len) {
                    off = (int64_t)page_id * p.page_stride + (int64_t)(tok % p.page) * p.place_stride +
                          (int64_t)(next.g / p.tiles) * p.cache_hs;
                    if (page_id < 0 || page_id >= p.n_pages) off = -2;
                    else if (!LEAN_SPAN(off, p.dim, p.cache_extent, p.err)) off = -1;
                }
                if (__any_sync(0xffffffffu, off == -2) && lane == 0) atomicOr(p.err, kErrSlot);
                const uint32_t ks = my_queue + stage * AttShape<DP>::kStageBytes + lane * 16;
                const C *kb = static_cast<const C *>(p.k), *vb = static_cast<const C *>(p.v);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, 8 * j + r);
#pragma unroll
                    for (int x = 0; x < KX; ++x) {
                        const int d = 32 * x + 8 * c4;
                        const uint32_t dst = ks + (x * 2 + j) * 512;
                        const bool real = o >= 0 && d < p.dim;
                        if (o != -2)
                            cp_async16(dst, real ? kb + o + d : kb, real);
                        else  // keys that are not there: NaN, which reaches out and lse by itself
                            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0x7fff7fff) : "memory");
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, 2 * c4 + (i & 1) + 8 * (i >> 1));
#pragma unroll
                    for (int x = 0; x < VX; ++x) {
                        const int d = 64 * x + 8 * r;
                        const bool real = o >= 0 && d < p.dim;
                        cp_async16(ks + kUnit * DP * 2 + (x * 4 + i) * 512, real ? vb + o + d : vb, real);
                    }
                }
                if (++u_next < u_hi) {
                    advance(p, next);
                    page_id = fetch_page();
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < S - 1; ++i) load_unit(i);

        // q as rows of the matrix instruction, part by part
        uint32_t qa[QSMEM ? 1 : 2 * KX][AREGS];
        uint32_t *q_shared = reinterpret_cast<uint32_t *>(queue + W * S * AttShape<DP>::kStageBytes) + warp * (2 * KX * AREGS * 32);
        float acc[8 * VX][4], m[NH], l[NH], zs[NH];
        bool fresh = true;
        int stage = 0;
        for (int64_t u = u_lo; u < u_hi; ++u) {
            load_unit(stage == 0 ? S - 1 : stage - 1);
            const int kvh = cur.g / p.tiles, tile = cur.g - kvh * p.tiles;
            const int h0 = kvh * p.group + tile * H, nh = min(H, p.group - tile * H);
            if (fresh) {
                fresh = false;
                // (read twice, the second time from L1: fewer registers than keeping it)
                auto load_q = [&](int h, int x, float *f) {
                    const int d = 32 * x + 8 * c4;
                    const int64_t at = (int64_t)cur.s * p.qs + (int64_t)(h0 + r + 8 * h) * p.qhs + d;
                    if (r + 8 * h < nh && d < p.dim && LEAN_SPAN(at, 8, p.q_extent, p.err)) {
                        load8(p.q, at, p.act, f);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = 0.f;
                    }
                };
                float f[NH][8], up[NH];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float top = 0.f;
#pragma unroll
                    for (int x = 0; x < KX; ++x) {
                        load_q(h, x, f[h]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[h][i]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // a power of two that brings the largest element near 1 (1 where there is none)
                    const int e = (int)(__float_as_uint(top) >> 23);
                    const int fe = e == 0 || e == 255 ? 127 : max(1, 254 - e);
                    up[h] = __uint_as_float((uint32_t)fe << 23);
                    zs[h] = p.scale_log2 * __uint_as_float((uint32_t)(254 - fe) << 23);
                    m[h] = -CUDART_INF_F;
                    l[h] = 0.f;
                }
                // element pairs (0,1) and (2,3) are the two halves of k of one instruction, (4,5) and (6,7) of the next
#pragma unroll
                for (int x = 0; x < KX; ++x) {
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        load_q(h, x, f[h]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[h][i] *= up[h];
                    }
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        uint32_t a[AREGS];
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            const uint32_t lo = take_part<C>(f[0][4 * st], f[0][4 * st + 1]);
                            const uint32_t hi = take_part<C>(f[0][4 * st + 2], f[0][4 * st + 3]);
                            if (WIDE) {
                                a[4 * part] = lo;
                                a[4 * part + 2] = hi;
                                a[4 * part + 1] = take_part<C>(f[NH - 1][4 * st], f[NH - 1][4 * st + 1]);
                                a[4 * part + 3] = take_part<C>(f[NH - 1][4 * st + 2], f[NH - 1][4 * st + 3]);
                            } else if (part < 2) {
                                a[part] = lo;
                                a[2 + part] = hi;
                            } else {
                                a[4] = lo;
                                a[AREGS - 1] = hi;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < AREGS; ++i) {
                            if (QSMEM) q_shared[((2 * x + st) * AREGS + i) * 32 + lane] = a[i];
                            else qa[QSMEM ? 0 : 2 * x + st][i] = a[i];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8 * VX; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
            }
            cp_async_wait<S - 1>();

            // ---- scores of 16 tokens: two tiles of 8
            const uint32_t ks = my_queue + stage * AttShape<DP>::kStageBytes + lane * 16;
            float sc[2][4] = {};
#pragma unroll
            for (int x = 0; x < KX; ++x)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 w = lds128(ks + (x * 2 + j) * 512);
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        uint32_t a[AREGS];
#pragma unroll
                        for (int i = 0; i < AREGS; ++i)
                            a[i] = QSMEM ? q_shared[((2 * x + st) * AREGS + i) * 32 + lane] : qa[QSMEM ? 0 : 2 * x + st][i];
                        const uint32_t b0 = st ? w.z : w.x, b1 = st ? w.w : w.y;
                        if (WIDE) {
#pragma unroll
                            for (int part = 0; part < PARTS; ++part)
                                mma<C>(sc[j], a[4 * part], a[4 * part + 1], a[4 * part + 2], a[4 * part + 3], b0, b1);
                        } else {
                            mma<C>(sc[j], a[0], a[1], a[2], a[3], b0, b1);
                            if (PARTS > 2) mma<C>(sc[j], a[4], 0u, a[AREGS - 1], 0u, b0, b1);
                        }
                    }
                }
            // ---- running maximum and sum; p as rows of the next instruction
            const int t0 = cur.x.base + cur.c * kUnit + 2 * c4;
            float e[NH][4];
            bool moved = false;
            float fall[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float top = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = i >> 1, tok = t0 + 8 * j + (i & 1);
                    const float raw = WIDE ? sc[j][2 * h + (i & 1)] : sc[j][i & 1] + sc[j][2 + (i & 1)];
                    e[h][i] = tok >= cur.x.start && tok < cur.x.len ? raw * zs[h] : -CUDART_INF_F;
                    top = fmaxf(top, e[h][i]);
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[h], top), ms = mn == -CUDART_INF_F ? 0.f : mn;
                moved |= mn > m[h];
                fall[h] = ex2(m[h] - ms);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[h][i] = ex2(e[h][i] - ms);
                    sum += e[h][i];
                }
                l[h] = fmaf(l[h], fall[h], sum);
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int j = 0; j < 8 * VX; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] *= fall[WIDE ? i >> 1 : 0];
            }
            uint32_t pa[PARTS][4];
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    pa[part][h] = take_part<C>(e[h][0], e[h][1]);
                    pa[part][2 + h] = take_part<C>(e[h][2], e[h][3]);
                }
            // ---- values: tokens (2c, 2c+1) and (2c+8, 2c+9) are the two halves of k
#pragma unroll
            for (int x = 0; x < VX; ++x) {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = lds128(ks + kUnit * DP * 2 + (x * 4 + i) * 512);
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    auto word = [&](const uint4 &q4) { return jj < 2 ? q4.x : jj < 4 ? q4.y : jj < 6 ? q4.z : q4.w; };
                    const uint32_t sel = jj & 1 ? 0x7632 : 0x5410;
                    const uint32_t b0 = __byte_perm(word(v[0]), word(v[1]), sel);
                    const uint32_t b1 = __byte_perm(word(v[2]), word(v[3]), sel);
                    float(&d)[4] = acc[8 * x + jj];
                    if (WIDE) {
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            mma<C>(d, pa[part][0], pa[part][1], pa[part][2], pa[part][3], b0, b1);
                    } else {
                        mma<C>(d, pa[0][0], pa[1][0], pa[0][2], pa[1][2], b0, b1);
                        if (PARTS > 2) mma<C>(d, pa[PARTS - 1][0], 0u, pa[PARTS - 1][2], 0u, b0, b1);
                    }
                }
            }

            // ---- the end of a group, or of the run
            if (cur.c == cur.x.n - 1 || u == u_hi - 1) {
                fresh = true;
                const int64_t first = u - cur.c;
                const bool whole = first >= u_lo && cur.c == cur.x.n - 1;
                const bool at_end = u == u_hi - 1;
                const int slot = at_end ? 1 : 0;
                // a part that others continue: the run's last in this warp's own queue (nothing is under way to
                // it any more), an earlier one in the workspace
                float *part = at_end ? reinterpret_cast<float *>(queue + warp * (S * AttShape<DP>::kStageBytes))
                                     : p.warp_parts + wg * PF;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float sum = l[h];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    const int row = r + 8 * h;
                    if (whole) {
                        if (row < nh) {
                            const float inv = sum == 0.f ? 0.f : 1.f / sum;
                            if (p.lse && c4 == 0)
                                p.lse[(int64_t)cur.s * p.hq + h0 + row] =
                                    sum == 0.f ? -CUDART_INF_F : (m[h] + log2f(sum)) * 0.69314718056f;
#pragma unroll
                            for (int x = 0; x < VX; ++x)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int d = 64 * x + 16 * c4 + 8 * i;
                                    float o[8];
#pragma unroll
                                    for (int jj = 0; jj < 8; ++jj)
                                        o[jj] = (WIDE ? acc[8 * x + jj][2 * h + i]
                                                      : acc[8 * x + jj][i] + acc[8 * x + jj][2 + i]) * inv;
                                    const int64_t at = (int64_t)cur.s * p.os + (int64_t)(h0 + row) * p.ohs + d;
                                    if (d < p.dim && LEAN_SPAN(at, 8, p.out_extent, p.err)) store8(p.out, at, p.act, o);
                                }
                        }
                    } else {
                        if (c4 == 0) {
                            part[row * PO] = m[h];
                            part[row * PO + 1] = sum;
                        }
#pragma unroll
                        for (int x = 0; x < VX; ++x)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float o[8];
#pragma unroll
                                for (int jj = 0; jj < 8; ++jj)
                                    o[jj] = WIDE ? acc[8 * x + jj][2 * h + i] : acc[8 * x + jj][i] + acc[8 * x + jj][2 + i];
                                store_vec<float, 8>(part + row * PO + 8 + 64 * x + 16 * c4 + 8 * i, o);
                            }
                    }
                }
                if (!whole && lane == 0) {
                    Record &q = rec[2 * warp + slot];
                    q.item = cur.s * groups + cur.g;
                    q.n = cur.x.n;
                    q.first = first;
                    q.part = part;
                }
            }
            advance(p, cur);
            stage = stage + 1 == S ? 0 : stage + 1;
        }
        cp_async_wait<0>();
    }
    __syncthreads();

    // ---- groups shared by warps of this block, and with other blocks
    // (the parts' weights lie behind the first warp's part, in its own queue)
    static_assert((PF + kAttMaxCtas * H) * 4 <= S * AttShape<DP>::kStageBytes, "room for the weights");
    float(*weight)[H] = reinterpret_cast<float(*)[H]>(queue + PF * 4);
    const int64_t b_lo = bound((int64_t)blockIdx.x * W), b_hi = bound((int64_t)blockIdx.x * W + W);
    auto finish = [&](int item) {  // total_m and total_l are set; out = weighted sum of `parts` / total
        const int s = item / groups, g = item % groups, kvh = g / p.tiles, tile = g % p.tiles;
        const int nh = min(H, p.group - tile * H);
        return make_int4(s, kvh * p.group + tile * H, nh, 0);
    };
    for (int i = 0; i < 2 * W;) {
        if (rec[i].item < 0) {
            ++i;
            continue;
        }
        const Record head = rec[i];
        int end = i + 1, parts = 1;  // the group's records: the item's next ones
        while (end < 2 * W && (rec[end].item < 0 || rec[end].item == head.item)) {
            parts += rec[end].item >= 0;
            ++end;
        }
        for (int h = threadIdx.x; h < H; h += T) {
            float top = -CUDART_INF_F, sum = 0.f;
            for (int k = i; k < end; ++k)
                if (rec[k].item >= 0) top = fmaxf(top, rec[k].part[h * PO]);
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            for (int k = i; k < end; ++k) {
                if (rec[k].item < 0) continue;
                const float w = ex2(rec[k].part[h * PO] - ref);
                weight[k][h] = w;
                sum = fmaf(w, rec[k].part[h * PO + 1], sum);
            }
            total_m[h] = top;
            total_l[h] = sum;
        }
        __syncthreads();
        const bool whole = head.first >= b_lo && head.first + head.n <= b_hi;
        const int slot = head.first < b_lo ? 0 : 1;
        float *part = p.cta_parts + ((int64_t)blockIdx.x * 2 + slot) * PF;
        const int4 f = finish(head.item);
        for (int k = threadIdx.x; k < H * DP / 4; k += T) {
            const int h = k / (DP / 4), d = k % (DP / 4) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q = i; q < end; ++q) {
                if (rec[q].item < 0) continue;
                const float w = weight[q][h];
                const float4 v = *reinterpret_cast<const float4 *>(rec[q].part + h * PO + 8 + d);
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            }
            if (!whole) {
                *reinterpret_cast<float4 *>(part + h * PO + 8 + d) = o;
            } else if (h < f.z && d < p.dim) {
                const float sum = total_l[h], inv = sum == 0.f ? 0.f : 1.f / sum;
                const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
                const int64_t at = (int64_t)f.x * p.os + (int64_t)(f.y + h) * p.ohs + d;
                if (LEAN_SPAN(at, 4, p.out_extent, p.err)) store4(p.out, at, p.act, v);
            }
        }
        for (int h = threadIdx.x; h < H; h += T) {
            if (!whole) {
                part[h * PO] = total_m[h];
                part[h * PO + 1] = total_l[h];
            } else if (h < f.z && p.lse) {
                p.lse[(int64_t)f.x * p.hq + f.y + h] =
                    total_l[h] == 0.f ? -CUDART_INF_F : (total_m[h] + log2f(total_l[h])) * 0.69314718056f;
            }
        }
        if (!whole) {
            // the blocks of the item: first_b .. last_b; the last of them to arrive adds the parts up
            auto block_of = [&](int64_t u) { return (int)(((u + 1) * blocks - 1) / units); };
            const int first_b = block_of(head.first), last_b = block_of(head.first + head.n - 1), np = last_b - first_b + 1;
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const bool last = atomicAdd(p.counters + first_b, 1u) == (unsigned)(np - 1);
                if (last) p.counters[first_b] = 0;
                last_block = last;
            }
            __syncthreads();
            if (last_block) {
                __threadfence();
                // (the item is not its first block's first, but every later block's first part)
                auto part_of = [&](int k) { return p.cta_parts + ((int64_t)(first_b + k) * 2 + (k == 0 ? 1 : 0)) * PF; };
                for (int h = threadIdx.x; h < H; h += T) {
                    float top = -CUDART_INF_F, sum = 0.f;
                    for (int k = 0; k < np; ++k) top = fmaxf(top, __ldcg(part_of(k) + h * PO));
                    const float ref = top == -CUDART_INF_F ? 0.f : top;
                    for (int k = 0; k < np; ++k) {
                        const float w = ex2(__ldcg(part_of(k) + h * PO) - ref);
                        weight[k][h] = w;
                        sum = fmaf(w, __ldcg(part_of(k) + h * PO + 1), sum);
                    }
                    total_l[h] = sum;
                    if (h < f.z && p.lse)
                        p.lse[(int64_t)f.x * p.hq + f.y + h] =
                            sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718056f;
                }
                __syncthreads();
                for (int k = threadIdx.x; k < H * DP / 4; k += T) {
                    const int h = k / (DP / 4), d = k % (DP / 4) * 4;
                    if (h >= f.z || d >= p.dim) continue;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int q = 0; q < np; ++q) {
                        const float w = weight[q][h];
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part_of(q) + h * PO + 8 + d));
                        o.x = fmaf(w, v.x, o.x);
                        o.y = fmaf(w, v.y, o.y);
                        o.z = fmaf(w, v.z, o.z);
                        o.w = fmaf(w, v.w, o.w);
                    }
                    const float sum = total_l[h], inv = sum == 0.f ? 0.f : 1.f / sum;
                    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
                    const int64_t at = (int64_t)f.x * p.os + (int64_t)(f.y + h) * p.ohs + d;
                    if (LEAN_SPAN(at, 4, p.out_extent, p.err)) store4(p.out, at, p.act, v);
                }
            }
        }
        __syncthreads();
        i = end;
    }
}

template <typename C, int DP, int PARTS, bool WIDE>
lean_status launch_attend(const AttArgs &p, int64_t flags, void *stream) {
    static std::atomic<uint64_t> done{0};
    auto kern = attend_kernel<C, DP, PARTS, WIDE>;
    if (!step_ensure_smem(kern, AttShape<DP>::kSmem, done)) return LEAN_ERR_CUDA;
    // no more blocks than there can be units for
    constexpr int W = AttShape<DP>::kWarps;
    const int64_t units = ((int64_t)p.width * p.page + 2 * kUnit) / kUnit * p.n_seqs * p.hkv * p.tiles;
    const int64_t grid = std::min<int64_t>(std::min(step_sm_count(), kAttMaxCtas), std::max<int64_t>(1, units / W));
    return step_launch(kern, grid, W * 32, AttShape<DP>::kSmem, flags, stream, p);
}
template <typename C, int DP>
lean_status pick_attend(const AttArgs &p, int64_t flags, void *stream) {
    const bool wide = p.group > 8;
    if (p.act == LEAN_F32)
        return wide ? launch_attend<C, DP, 3, true>(p, flags, stream) : launch_attend<C, DP, 3, false>(p, flags, stream);
    return wide ? launch_attend<C, DP, 2, true>(p, flags, stream) : launch_attend<C, DP, 2, false>(p, flags, stream);
}
template <typename C>
lean_status pick_dim(const AttArgs &p, int64_t flags, void *stream) {
    if (p.dim <= 64) return pick_attend<C, 64>(p, flags, stream);
    if (p.dim <= 128) return pick_attend<C, 128>(p, flags, stream);
    return pick_attend<C, 256>(p, flags, stream);
}

int64_t att_part_bytes(int64_t hq, int64_t hkv, int64_t dim) {
    return 4 * part_floats(hq / hkv > 8 ? 16 : 8, dim <= 64 ? 64 : dim <= 128 ? 128 : 256);
}

bool att_sizes_ok(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim) {
    return n_seqs > 0 && hkv > 0 && hq > 0 && hq <= 65536 && hq % hkv == 0 && dim > 0 && dim % 8 == 0 &&
           dim <= kAttMaxDim && n_seqs <= INT32_MAX / hq;
}

}  // namespace

extern "C" int64_t lean_paged_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                                        int64_t head_dim) {
    if (!att_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim)) return -1;
    // counters, a part per warp and two per block, of the largest grid
    return kCounterBytes + kAttMaxCtas * (8 + 2) * att_part_bytes(n_q_heads, n_kv_heads, head_dim);
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
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    p.counters = reinterpret_cast<unsigned *>(ws);
    p.warp_parts = reinterpret_cast<float *>(ws + kCounterBytes);
    p.cta_parts = p.warp_parts + kAttMaxCtas * 8 * att_part_bytes(a->n_q_heads, a->n_kv_heads, a->head_dim) / 4;
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
    p.group = p.hq / p.hkv;
    p.tiles = p.group > 8 ? (p.group + 15) / 16 : 1;
    p.dim = (int)a->head_dim;
    p.page = (int)a->page_size;
    p.width = (int)a->table_width;
    p.window = (int)std::min<int64_t>(a->window, INT32_MAX);
    p.act = (int)a->act_dtype;
    p.scale_log2 = (float)(a->scale * 1.4426950408889634);
    p.cache_extent = (a->n_pages - 1) * a->page_stride + (a->page_size - 1) * a->place_stride +
                     (a->n_kv_heads - 1) * a->cache_head_stride + a->head_dim;
    p.q_extent = (a->n_seqs - 1) * a->q_stride + (a->n_q_heads - 1) * a->q_head_stride + a->head_dim;
    p.out_extent = (a->n_seqs - 1) * a->out_stride + (a->n_q_heads - 1) * a->out_head_stride + a->head_dim;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    return a->cache_dtype == LEAN_BF16 ? pick_dim<__nv_bfloat16>(p, a->flags, stream)
                                       : pick_dim<__half>(p, a->flags, stream);
}
