// attend.cu -- lean_paged_attention: attention of one new token per sequence
// over the paged cache.
//
//   z_j = scale q . k_j,  p_j = e^(z_j - m),  m = max z_j,
//   out = sum p_j v_j / sum p_j,  lse = m + ln sum p_j
//
// Every key and value of the cache is read once for up to 16 query heads that
// share its kv head (for more, once per 16 of them: 239 us at 48 heads of 128 where
// 12 take 98): HBM bounds the call, 2 * dim * 2 bytes a token and kv head.  So the
// design is about keeping loads in flight:
//
//   - The work is a list of units: 16 tokens of one (sequence, kv head, group of
//     query heads).  Every warp of the GPU takes an equal run of units, whatever
//     the lengths are, and walks it alone: no barrier between its first load
//     and its last.
//   - A warp copies its units into a queue of its own with cp.async, consecutive
//     lanes along a token's row (a copy in the order of the matrix fragments, 64
//     bytes of eight rows at a time, needs no exchange between lanes but stops at
//     5.2 TB/s; rows reach 6.6-7.0).  16-byte pieces are stored at their place XOR
//     the row's number, where ldmatrix reads them without conflicts: K as it is,
//     V transposed.
//   - Scores and outputs come from mma.sync m16n8k16 with the query heads as
//     rows: 16 tokens take dim / 4 of them for 64 * dim bytes, a fraction of the
//     time the bytes take (tcgen05 wants 64 rows or more; a group has 1 to 16).
//     With up to 8 heads in a group, rows 0-7 hold the first part of q (or p) and
//     rows 8-15 the second, so that one instruction serves both.
//   - Running maximum and sum per warp, the sums folded every 64 units so that long
//     runs keep fp32's precision; a warp's first and last group may be
//     shared with its neighbours: the warps of a block join through shared
//     memory, blocks through the workspace and a second kernel, launched early,
//     that adds the parts up in their order.
//
// q and p are split into parts of the cache's type, x = x0 + x1 (+ x2), 8 (bf16)
// or 11 bits each: three parts for fp32 q and out, which leave nothing of fp32's
// 24 bits behind; two for 16-bit ones, whose rounding of out is larger.  (p in f16:
// of probabilities near the largest; small ones are held to 2^-38 of it.)  q is
// first scaled by a power of two so that no part can overflow or vanish (f16: none
// above 2^-38 of the largest element).
//
// Measured (GB300, calls in a graph): 384 sequences of 1 to 8192 tokens, 32 query
// and 4 kv heads of 64, bf16: 68 us, 5.4 TB/s of the 6.78 that a copy reaches, with
// fp32 q 72.6; one sequence of 131072, 16/2 heads of 128, fp32 q: 33.7 us, 4.0 TB/s
// (5.8 at 524288): the stream itself runs at 6 TB/s and more, 3 us pass before the
// first keys arrive (lengths, table, keys, one after the other) and 8 after the last
// (joins, the second kernel, the launch); 613 tokens of 15/5 heads of 64: 9.2 us.
// What bounds the rest is a warp's time for a unit, not HBM: 192 sequences as above
// with heads of 128 and fp32 q, 8 query heads a group 73 us, 12 98 (floor 54); 96
// sequences with heads of 256, 88 and 131.
// Pages of 16 tokens or more hold a unit in one page or two, and two pages cost
// little (384 sequences as above: 69 us with pages of 24, 72 of 20).  In smaller
// pages every token is looked up: 90 us with pages of 8, 99 of one.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kAttMaxDim = 256;
constexpr int kAttMaxCtas = 160;  // of a launch: at most one per SM
constexpr int kUnit = 16;         // tokens
constexpr int64_t kSharedBytes = 2048;  // a Shared for each block

struct Shared {  // an item that begins in a block and goes on in others (-1: none), and how many blocks it has
    int item, parts;
};

struct AttArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *table, *lens;
    Shared *shared;
    float *warp_parts, *cta_parts;
    f32x2 *folds;  // a warp's: the sums of its item up to the last fold
    int64_t qs, qhs, os, ohs, page_stride, place_stride, cache_hs, table_stride, n_pages;
    int n_seqs, hq, hkv, group, tiles, dim, page, paged, whole, width, window;
    int act;
    float scale_log2;
    int64_t cache_extent, q_extent, out_extent;  // elements, for the checked build
    int64_t warp_extent, part_extent, fold_extent;
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
    static constexpr int kSmem = 512 + kWarps * (kStages * kStageBytes + (DP == 256 ? DP / 16 * 12 * 128 : 0));
};
// A part: maxima, sums and outputs of a group of H heads.
__host__ __device__ constexpr int part_floats(int heads, int dp) { return heads * (dp + 4); }
// What a warp folds: each lane's outputs, references and sums.
__host__ __device__ constexpr int fold_floats(int heads, int dp) { return heads * (dp + 8); }
// Shared memory of a block: queues; q at 256 (above); and, where it fits, a part per warp.
constexpr int kMaxSmem = 232448 - 1536;  // of 227 KB, less static variables
template <int DP>
__host__ __device__ constexpr bool parts_in_smem(int heads) {
    return AttShape<DP>::kSmem + AttShape<DP>::kWarps * part_floats(heads, DP) * 4 <= kMaxSmem;
}
template <int DP>
__host__ __device__ constexpr int att_smem(int heads) {
    return AttShape<DP>::kSmem + (parts_in_smem<DP>(heads) ? AttShape<DP>::kWarps * part_floats(heads, DP) * 4 : 0);
}

// 16 bytes of which `real` (16 or 0) are copied and the rest zero
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&v)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&v)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
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

// Two neighbouring elements of q as they were read (nothing waits for them until they are used) and as fp32; two or
// four of out.
template <bool F32>
struct RawPair;
template <>
struct RawPair<true> {
    float2 v;
    __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        v = *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i);
    }
    __device__ __forceinline__ float2 get(int) const { return v; }
};
template <>
struct RawPair<false> {
    uint32_t v;
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        v = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i);
    }
    __device__ __forceinline__ float2 get(int act) const {
        if (act == LEAN_BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
};
template <int N>
__device__ __forceinline__ void store_out(void *p, int64_t i, int act, const float *f) {
    if (act == LEAN_F32) store_vec<float, N>(static_cast<float *>(p) + i, f);
    else if (act == LEAN_BF16) store_vec<__nv_bfloat16, N>(static_cast<__nv_bfloat16 *>(p) + i, f);
    else store_vec<__half, N>(static_cast<__half *>(p) + i, f);
}
__device__ __forceinline__ int nth_bit(unsigned m, int n) {  // place of the n-th (from 0) bit that is set
    for (; n > 0; --n) m &= m - 1;
    return __ffs(m) - 1;
}
__device__ __forceinline__ float natural_lse(float m, float sum) {
    return sum == 0.f ? -CUDART_INF_F : (m + log2f(sum)) * 0.69314718056f;
}

// What of a sequence is attended: tokens start..len-1, in n units from base on.
struct Span {
    int len, start, base, n;
};
__device__ __forceinline__ Span open_span(const AttArgs &p, int s) {
    Span x;
    const int64_t most = (int64_t)p.width * p.page;
    int len = LEAN_IN(s, p.n_seqs, p.err) ? p.lens[s] : 0;
    len = len < 0 ? 0 : len;
    x.len = len > most ? (int)most : len;
    x.start = p.window > 0 && x.len > p.window ? x.len - p.window : 0;
    x.base = x.start & ~(kUnit - 1);
    x.n = (x.len - x.base) / kUnit + ((x.len - x.base) % kUnit != 0);
    x.n = x.n < 1 ? 1 : x.n;  // an empty sequence is one unit in which nothing is attended
    return x;
}

// A place in the list of units: sequence, kv head, tile of its query heads, unit.
// Where units lie in one page or two (p.paged: pages of 16 tokens or more), also
// the place of the unit's first token in its page.
struct Place {
    int s, kvh, tile, c;
    unsigned in_page;
    Span x;
};
__device__ __forceinline__ void to_page(const AttArgs &p, Place &at) {
    at.in_page = (at.x.base + at.c * kUnit) % p.page;
}
__device__ __forceinline__ bool advance(const AttArgs &p, Place &at) {  // true: to another item
    if (++at.c < at.x.n) {
        at.in_page += kUnit;
        if (at.in_page >= (unsigned)p.page) at.in_page -= p.page;
        return false;
    }
    at.c = 0;
    if (++at.tile == p.tiles) {
        at.tile = 0;
        if (++at.kvh == p.hkv) {
            at.kvh = 0;
            if (++at.s < p.n_seqs) at.x = open_span(p, at.s);
        }
    }
    to_page(p, at);
    return true;
}

// What a warp leaves of a group that it does not finish, or a block of one that
// it does not: where the group lies and its maxima, sums and outputs.
struct Record {
    int item;           // -1: none
    int n;              // units of the item
    int first;          // its first unit, counted from the block's first one
};

// The most that running scores may exceed the reference of their exponentials by
// before it moves, as a power of two: the sums are rescaled (a rounding each) a few
// times a run instead of in every unit with a new maximum.  And what probabilities
// are multiplied by before they are split: bf16 has fp32's range, f16 ends at 2^-24
// below and 2^16 above, so there they lie as high as they can, up to 2^15, and what
// is lost of one is 2^-38 of the reference at most (without: one below 2^-25 left
// nothing, 8192 keys 17 nats below one 2.3e-4 of the output).  The same for q, whose
// largest element is brought to 2^kLiftQ.
template <typename C>
struct PartRange {
    static constexpr float kSlack = 8.f, kLift = 1.f;
    static constexpr int kLiftQ = 0;
};
template <>
struct PartRange<__half> {
    static constexpr float kSlack = 2.f, kLift = 8192.f;
    static constexpr int kLiftQ = 14;
};
// Units after which a warp's sums of an item go to the workspace and begin again: sums of N units err by (kFold + N /
// kFold) U in place of N U (U = 2^-24), for 2% of the traffic, in L2.
constexpr int kFold = 64;
// Units of a warp's time that joining blocks costs, and that an item costs beside its
// units (q, the first maximum, the result): that many empty ones are counted to it
// when the runs are cut.
constexpr int kJoinUnits = 8;
constexpr int kItemUnits = 4;

// Parts added up: maximum, sum and outputs.
struct Sums {
    float top, sum;
    float4 o;
    __device__ __forceinline__ void clear() {
        top = -CUDART_INF_F;
        sum = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void add(float2 ml, float4 v) {
        const float now = fmaxf(top, ml.x), ref = now == -CUDART_INF_F ? 0.f : now;
        const float old = ex2(top - ref), w = ex2(ml.x - ref);
        top = now;
        sum = fmaf(sum, old, w * ml.y);
        o.x = fmaf(o.x, old, w * v.x);
        o.y = fmaf(o.y, old, w * v.y);
        o.z = fmaf(o.z, old, w * v.z);
        o.w = fmaf(o.w, old, w * v.w);
    }
};
struct Head {  // of an item: its sequence, first query head and number of heads
    int s, h0, nh;
};
__device__ __forceinline__ Head open_item(const AttArgs &p, int item, int heads) {
    const int groups = p.hkv * p.tiles, g = item % groups, tile = g % p.tiles;
    return Head{item / groups, g / p.tiles * p.group + tile * heads, min(heads, p.group - tile * heads)};
}
__device__ __forceinline__ void store_result(const AttArgs &p, const Head &f, int h, int d, float4 o, float top,
                                             float sum) {
    if (h >= f.nh || d >= p.dim) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    const int64_t at = (int64_t)f.s * p.os + (int64_t)(f.h0 + h) * p.ohs + d;
    if (LEAN_SPAN(at, 4, p.out_extent, p.err)) store_out<4>(p.out, at, p.act, v);
    const int64_t at_lse = (int64_t)f.s * p.hq + f.h0 + h;
    if (d == 0 && p.lse && LEAN_IN(at_lse, (int64_t)p.n_seqs * p.hq, p.err)) p.lse[at_lse] = natural_lse(top, sum);
}

// WIDE: 9 to 16 query heads in a group, one per row; else up to 8, two rows each.
template <typename C, int DP, int PARTS, bool WIDE>
__global__ void __launch_bounds__(AttShape<DP>::kWarps * 32, 1) attend_kernel(const AttArgs p) {
    constexpr int W = AttShape<DP>::kWarps, S = AttShape<DP>::kStages, T = W * 32, STAGE = AttShape<DP>::kStageBytes;
    constexpr int H = WIDE ? 16 : 8, NH = WIDE ? 2 : 1;  // heads of a group, of a thread
    constexpr int RB = DP * 2, LPR = RB / 16, RPI = 32 / LPR;  // a row's bytes and lanes, rows of a copy instruction
    constexpr int KS = DP / 16;                                // steps of the contraction, and pairs of output tiles
    constexpr int AREGS = WIDE ? 4 * PARTS : 4 + (PARTS > 2 ? 2 : 0);  // of q per step
    constexpr bool QSMEM = DP == 256;                                  // no registers left for q
    constexpr int PF = part_floats(H, DP), PO = 4 + DP;                // a head's row of a part: m, l, -, out
    constexpr bool PSMEM = parts_in_smem<DP>(H);
    // registers for q as it was read: beside the accumulators, and all through the item before
    constexpr bool EARLY_Q = !WIDE && DP <= 128, AHEAD_Q = !WIDE && DP == 64;
    static_assert(PF * 4 <= S * STAGE, "a part fits a queue");
    constexpr int AT = 2;  // steps of the values whose products are under way at once (more spill)
    extern __shared__ uint8_t queue_raw[];
    uint8_t *queue = queue_raw + (512 - smem_addr(queue_raw) % 512) % 512;
    __shared__ unsigned scan[W];
    __shared__ int longest[W];
    __shared__ unsigned units_before[T];
    __shared__ Record rec[2 * W];

    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r = lane / 4, c4 = lane % 4;
    const int groups = p.hkv * p.tiles;

    // ---- the list of units, and this block's and warp's run of it
    const int per = (p.n_seqs + T - 1) / T;  // sequences a thread sums up
    const int s_lo = min(p.n_seqs, (int)threadIdx.x * per), s_hi = min(p.n_seqs, s_lo + per);
    unsigned mine = 0;
    int most = 0;
    for (int s = s_lo; s < s_hi; ++s) {
        const int n = open_span(p, s).n;
        mine += (unsigned)(n + kItemUnits) * groups;
        most = max(most, n);
    }
    unsigned incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) {
        scan[warp] = incl;
        longest[warp] = most;
    }
    if (threadIdx.x < 2 * W) rec[threadIdx.x].item = -1;
    __syncthreads();
    unsigned before = incl - mine, units = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (i < warp) before += scan[i];
        units += scan[i];
        most = max(most, longest[i]);
    }
    // Equal runs for all blocks (a unit a warp at least) have to be joined across blocks; where there are few
    // items and none is long, a block for each is done sooner.
    const int64_t items = (int64_t)p.n_seqs * groups;
    const bool by_item = items <= gridDim.x && (unsigned)((most + W - 1) / W) <= units / (gridDim.x * W) + kJoinUnits;
    const int blocks = by_item ? (int)items : (int)min(gridDim.x, units / W + (units % W != 0));
    if ((int)blockIdx.x >= blocks) {
        if (threadIdx.x == 0 && LEAN_IN(blockIdx.x, kAttMaxCtas, p.err)) p.shared[blockIdx.x] = Shared{-1, 0};
        return;
    }
    units_before[threadIdx.x] = before;
    __syncthreads();
    unsigned b_lo = 0;
    int b_n;  // first unit of the block, and how many (unit numbers below count from b_lo)
    if (by_item) {
        b_n = open_span(p, blockIdx.x / groups).n;
    } else {
        const unsigned q = units / blocks, rest = units - q * blocks;  // the first `rest` blocks have one more
        b_lo = q * blockIdx.x + min(blockIdx.x, rest);
        b_n = (int)(q + (blockIdx.x < rest));
    }
    int u_lo = (int)((int64_t)b_n * warp / W);
    const int u_hi = (int)((int64_t)b_n * (warp + 1) / W);
    Place next;  // to be loaded
    if (u_lo < u_hi) {
        int at = 0;  // kv head and tile
        if (by_item) {
            next.s = blockIdx.x / groups;
            at = blockIdx.x - next.s * groups;
            next.c = u_lo;
            next.x = open_span(p, next.s);
        } else {
            // the thread whose sequences have the run's first unit, and among them the one that has it
            const unsigned b = b_lo + u_lo;
            int begun = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) begun += units_before[i * 32 + lane] <= b;
            const int t = __reduce_add_sync(0xffffffffu, begun) - 1;
            unsigned in = b - units_before[t];
            next.s = t * per;
            next.x = open_span(p, next.s);
            while (in >= (unsigned)(next.x.n + kItemUnits) * groups) {
                in -= (unsigned)(next.x.n + kItemUnits) * groups;
                next.x = open_span(p, ++next.s);
            }
            at = (int)(in / (next.x.n + kItemUnits));
            next.c = (int)(in - (unsigned)at * (next.x.n + kItemUnits));
        }
        next.kvh = at / p.tiles;
        next.tile = at - next.kvh * p.tiles;
        if (next.c >= next.x.n) {  // in the item's empty units: on to the next item
            u_lo += next.x.n + kItemUnits - next.c;
            next.c = next.x.n - 1;
            advance(p, next);
        } else {
            to_page(p, next);
        }
    }
    uint8_t *const tail_part = queue + warp * (S * STAGE);  // where a warp's last part goes, and an earlier one
    uint8_t *const head_part = PSMEM ? queue + AttShape<DP>::kSmem - 512 + warp * (PF * 4)
                                     : reinterpret_cast<uint8_t *>(p.warp_parts + ((int64_t)blockIdx.x * W + warp) * PF);

    if (u_lo < u_hi) {
        const uint32_t my_queue = smem_addr(queue) + warp * (S * STAGE);
        Place cur = next;  // to be computed
        int u_next = u_lo;

        // Pages, fetched before they are needed: (paged) those of the first and the last attended token of units
        // pages_from + lane of the item, 32 at a time, else those of token lane % 16 of the unit to be loaded next.
        int pages_from = next.c;
        auto fetch_page = [&](unsigned tok) {
            const bool in = tok >= (unsigned)next.x.start && tok < (unsigned)next.x.len;
            const int64_t e = (int64_t)next.s * p.table_stride + tok / (unsigned)p.page;
            return in && LEAN_IN(e, (int64_t)(p.n_seqs - 1) * p.table_stride + p.width, p.err) ? p.table[e] : 0;
        };
        int pages, last_pages = 0;
        auto fetch_pages = [&]() {
            if (p.paged) {
                const unsigned tok = next.x.base + (pages_from + lane) * kUnit;
                pages = fetch_page(max(tok, (unsigned)next.x.start));
                if (!p.whole) last_pages = fetch_page(min(tok + kUnit, (unsigned)next.x.len) - 1);
            } else {
                pages = fetch_page(next.x.base + next.c * kUnit + lane % kUnit);
            }
        };
        fetch_pages();
        // a lane's piece of a row: its place in the caches, in a stage, and whether the head has it at all
        const int lr = lane / LPR, col = lane % LPR;
        const C *k_lane = static_cast<const C *>(p.k) + 8 * col, *v_lane = static_cast<const C *>(p.v) + 8 * col;
        const uint32_t to_lane = my_queue + lr * RB + ((col ^ lr) * 16);
        const int real = 8 * col < p.dim ? 16 : 0;

        auto load_unit = [&](int stage) {
            if (u_next < u_hi) {
                const uint32_t dst = to_lane + stage * STAGE;
                const int t0 = next.x.base + next.c * kUnit;
                const int page_id = p.paged ? __shfl_sync(0xffffffffu, pages, next.c - pages_from) : pages;
                const bool page_ok = page_id >= 0 && page_id < p.n_pages;
                const unsigned in_first = p.page - next.in_page;  // the unit's tokens in its first page, 16 or more: all
                const int64_t unit_off = (int64_t)page_id * p.page_stride + (int64_t)next.in_page * p.place_stride +
                                         (int64_t)next.kvh * p.cache_hs;
                if (p.paged && in_first >= kUnit && page_ok && t0 >= next.x.start && t0 <= next.x.len - kUnit &&
                    LEAN_SPAN(unit_off, (kUnit - 1) * p.place_stride + p.dim, p.cache_extent, p.err)) {
                    // all of 16 tokens, one after the other
                    int64_t off = unit_off + lr * p.place_stride;
#pragma unroll
                    for (int i = 0; i < kUnit / RPI; ++i) {
                        const uint32_t to = i * RPI * RB + (dst ^ ((i * RPI & 7) * 16));
                        cp_async16(to, k_lane + off, real);
                        cp_async16(to + kUnit * RB, v_lane + off, real);
                        off += RPI * p.place_stride;
                    }
                } else {
                    const int in_unit = lane % kUnit;
                    const int last_id = __shfl_sync(0xffffffffu, last_pages, next.c - pages_from);
                    int64_t off = -1;  // of the token's row; -1: not attended, -2: outside the cache
                    if (in_unit >= next.x.start - t0 && in_unit < next.x.len - t0) {
                        const bool first = !p.paged || in_unit < in_first;
                        const int id = first ? page_id : last_id;
                        const int64_t place = !p.paged ? (t0 + in_unit) % p.page
                                                       : (int64_t)next.in_page + in_unit - (first ? 0 : p.page);
                        off = (int64_t)id * p.page_stride + place * p.place_stride + (int64_t)next.kvh * p.cache_hs;
                        if (id < 0 || id >= p.n_pages) off = -2;
                        else if (!LEAN_SPAN(off, p.dim, p.cache_extent, p.err)) off = -1;
                    }
                    if (__all_sync(0xffffffffu, off >= 0)) {
#pragma unroll
                        for (int i = 0; i < kUnit / RPI; ++i) {
                            const int64_t o = __shfl_sync(0xffffffffu, off, i * RPI + lr);
                            const uint32_t to = i * RPI * RB + (dst ^ ((i * RPI & 7) * 16));
                            cp_async16(to, k_lane + o, real);
                            cp_async16(to + kUnit * RB, v_lane + o, real);
                        }
                    } else {
                        if (__any_sync(0xffffffffu, off == -2) && lane == 0) atomicOr(p.err, kErrSlot);
#pragma unroll
                        for (int i = 0; i < kUnit / RPI; ++i) {
                            const int64_t o = __shfl_sync(0xffffffffu, off, i * RPI + lr);
                            const uint32_t to = i * RPI * RB + (dst ^ ((i * RPI & 7) * 16));
                            if (o != -2)
                                cp_async16(to, o >= 0 ? k_lane + o : static_cast<const C *>(p.k), o >= 0 ? real : 0);
                            else  // keys that are not there: NaN, which reaches out and lse by itself
                                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to), "r"(0x7fff7fff) : "memory");
                            cp_async16(to + kUnit * RB, o >= 0 ? v_lane + o : static_cast<const C *>(p.v), o >= 0 ? real : 0);
                        }
                    }
                }
                u_next += next.c == next.x.n - 1 ? 1 + kItemUnits : 1;
                if (u_next < u_hi) {
                    const bool other = advance(p, next);
                    if (!p.paged || other || next.c == pages_from + 32) {
                        pages_from = next.c;
                        fetch_pages();
                    }
                }
            }
            cp_async_commit();
        };
        // q of the current item, asked for before its first keys (after them it would wait for them)
        RawPair<(PARTS > 2)> raw[NH][2 * KS];
        auto load_q = [&](int s, int kvh, int tile) {
            const int h0 = kvh * p.group + tile * H, nh = min(H, p.group - tile * H);
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int i = 0; i < 2 * KS; ++i) {
                    const int d = 8 * i + 2 * c4;
                    const int64_t at = (int64_t)s * p.qs + (int64_t)(h0 + r + 8 * h) * p.qhs + d;
                    if (r + 8 * h < nh && d < p.dim && LEAN_SPAN(at, 2, p.q_extent, p.err)) raw[h][i].load(p.q, at);
                    else raw[h][i].zero();
                }
        };
        if (EARLY_Q) load_q(cur.s, cur.kvh, cur.tile);
#pragma unroll 1
        for (int i = 0; i < S - 1; ++i) load_unit(i);

        // ldmatrix rows of a lane: K, tokens 0-7 (8-15 from lane 16 on) and the even (odd) piece of a step; V,
        // tokens 0-7 (8-15) and the even (odd) output tile of a pair
        const uint32_t k_row = my_queue + ((lane >> 4) * 8 + (lane & 7)) * RB + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
        const uint32_t v_row =
            my_queue + kUnit * RB + (((lane >> 3) & 1) * 8 + (lane & 7)) * RB + (((lane >> 4) ^ (lane & 7)) * 16);
        // q as rows of the matrix instruction, part by part
        uint32_t qa[QSMEM ? 1 : KS][AREGS];
        uint32_t *q_shared = reinterpret_cast<uint32_t *>(queue + W * S * STAGE) + warp * (KS * AREGS * 32);
        // outputs and sums of the item since its last fold, with reference m
        f32x2 acc[2 * KS][NH];
        float m[NH], l[NH], zs[NH];
        const bool can_leave = PSMEM || LEAN_SPAN(((int64_t)blockIdx.x * W + warp) * PF, PF, p.warp_extent, p.err);
        const bool can_fold = LEAN_SPAN(((int64_t)blockIdx.x * W + warp) * fold_floats(H, DP), fold_floats(H, DP), p.fold_extent,
                                        p.err);
        f32x2 *const folded = p.folds + ((int64_t)blockIdx.x * W + warp) * (fold_floats(H, DP) / 2) + lane;
        int done = 0;  // units of the item so far
        bool fresh = true;
        int stage = 0;
        for (int u = u_lo; u < u_hi;) {
            load_unit(stage == 0 ? S - 1 : stage - 1);
            const int h0 = cur.kvh * p.group + cur.tile * H, nh = min(H, p.group - cur.tile * H);
            if (fresh) {
                fresh = false;
                if (!EARLY_Q) load_q(cur.s, cur.kvh, cur.tile);
                float2 f[NH][2 * KS];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < 2 * KS; ++i) f[h][i] = raw[h][i].get(p.act);
#pragma unroll
                    for (int i = 0; i < 2 * KS; ++i) top = fmaxf(top, fmaxf(fabsf(f[h][i].x), fabsf(f[h][i].y)));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // a power of two that brings the largest element near 1, or as high as f16 takes it, so that its
                    // steps below are small next to the others as well (1 where there is no largest element)
                    const int e = (int)(__float_as_uint(top) >> 23);
                    const int fe = e == 0 || e == 255 ? 127 : min(253, max(1, 254 + PartRange<C>::kLiftQ - e));
                    const float up = __uint_as_float((uint32_t)fe << 23);
                    zs[h] = p.scale_log2 * __uint_as_float((uint32_t)(254 - fe) << 23);
                    m[h] = -CUDART_INF_F;
                    l[h] = 0.f;
#pragma unroll
                    for (int i = 0; i < 2 * KS; ++i) {
                        f[h][i].x *= up;
                        f[h][i].y *= up;
                    }
                }
                // pieces 2 st and 2 st + 1 are the two halves of k of step st
#pragma unroll
                for (int st = 0; st < KS; ++st) {
                    uint32_t a[AREGS];
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t lo = take_part<C>(f[0][2 * st].x, f[0][2 * st].y);
                        const uint32_t hi = take_part<C>(f[0][2 * st + 1].x, f[0][2 * st + 1].y);
                        if (WIDE) {
                            a[4 * part] = lo;
                            a[4 * part + 2] = hi;
                            a[4 * part + 1] = take_part<C>(f[NH - 1][2 * st].x, f[NH - 1][2 * st].y);
                            a[4 * part + 3] = take_part<C>(f[NH - 1][2 * st + 1].x, f[NH - 1][2 * st + 1].y);
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
                        if (QSMEM) q_shared[(st * AREGS + i) * 32 + lane] = a[i];
                        else qa[QSMEM ? 0 : st][i] = a[i];
                    }
                }
#pragma unroll
                for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
                    for (int h = 0; h < NH; ++h) acc[j][h] = 0;
                done = 0;
                if (AHEAD_Q && u + cur.x.n - cur.c + kItemUnits < u_hi) {  // another item follows
                    const bool other_tile = cur.tile + 1 < p.tiles, other_head = other_tile || cur.kvh + 1 < p.hkv;
                    load_q(other_head ? cur.s : cur.s + 1, other_tile ? cur.kvh : other_head ? cur.kvh + 1 : 0,
                           other_tile ? cur.tile + 1 : 0);
                }
            }
            cp_async_wait<S - 1>();
            __syncwarp();

            // ---- scores of 16 tokens: two tiles of 8
            float sc[2][4] = {}, sd[2][4] = {};  // each in two sums: half as many instructions wait for one another
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                uint32_t b[4], a[AREGS];
                ldmatrix4(b, (k_row + stage * STAGE) ^ (32 * st));
#pragma unroll
                for (int i = 0; i < AREGS; ++i)
                    a[i] = QSMEM ? q_shared[(st * AREGS + i) * 32 + lane] : qa[QSMEM ? 0 : st][i];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (WIDE) {
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            mma<C>(st & 1 ? sd[j] : sc[j], a[4 * part], a[4 * part + 1], a[4 * part + 2], a[4 * part + 3],
                                   b[2 * j], b[2 * j + 1]);
                    } else {
                        mma<C>(sc[j], a[0], a[1], a[2], a[3], b[2 * j], b[2 * j + 1]);
                        if (PARTS > 2) mma<C>(sd[j], a[AREGS - 2], 0u, a[AREGS - 1], 0u, b[2 * j], b[2 * j + 1]);
                    }
                }
            }
            // ---- running maximum and sum; p as rows of the next instruction (tokens are looked at one by one where
            // not all of the unit is attended; always with two heads a thread, whose registers a branch would spill)
            const int u0 = cur.x.base + cur.c * kUnit, t0 = u0 + 2 * c4;
            const bool inside = u0 >= cur.x.start && u0 <= cur.x.len - kUnit;
            float e[NH][4];
            f32x2 fall2[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float top = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = i >> 1;
                    const float raw = WIDE ? sc[j][2 * h + (i & 1)] + sd[j][2 * h + (i & 1)]
                                           : sc[j][i & 1] + (sc[j][2 + (i & 1)] + sd[j][i & 1]);
                    e[h][i] = raw * zs[h];
                }
                if (WIDE || !inside) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = t0 + 8 * (i >> 1) + (i & 1);
                        if (tok < cur.x.start || tok >= cur.x.len) e[h][i] = -CUDART_INF_F;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, e[h][i]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // m: the reference of the exponentials, within kSlack of the largest score so far (the difference of
                // neighbours is exact; from -inf, infinite or NaN)
                const float mn = top - m[h] <= PartRange<C>::kSlack ? m[h] : top;
                const float ms = mn == -CUDART_INF_F ? 0.f : mn;
                const float fall = ex2(m[h] - ms);
                fall2[h] = pack2(fall, fall);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[h][i] = ex2(e[h][i] - ms) * PartRange<C>::kLift;
                    sum += e[h][i];
                }
                l[h] = fmaf(l[h], fall, sum);
            }
            uint32_t pa[PARTS][4];
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    pa[part][h] = take_part<C>(e[h][0], e[h][1]);
                    pa[part][2 + h] = take_part<C>(e[h][2], e[h][3]);
                }
            // ---- values: a unit's products summed from 0, then one addition in fp32 (the instruction cuts off what is
            // small next to its accumulator: 8192 keys 17 nats below one left nothing there, 2.3e-4 of the output)
#pragma unroll
            for (int st = 0; st < KS; st += AT) {
                uint32_t b[AT][4];
                float d[2 * AT][4] = {};
#pragma unroll
                for (int i = 0; i < AT; ++i) ldmatrix4_trans(b[i], (v_row + stage * STAGE) ^ (32 * (st + i)));
#pragma unroll
                for (int part = 0; part < (WIDE ? PARTS : PARTS - 1); ++part)
#pragma unroll
                    for (int i = 0; i < 2 * AT; ++i) {
                        const uint32_t b0 = b[i / 2][2 * (i & 1)], b1 = b[i / 2][2 * (i & 1) + 1];
                        if (WIDE) mma<C>(d[i], pa[part][0], pa[part][1], pa[part][2], pa[part][3], b0, b1);
                        else if (part == 0) mma<C>(d[i], pa[0][0], pa[1][0], pa[0][2], pa[1][2], b0, b1);
                        else mma<C>(d[i], pa[PARTS - 1][0], 0u, pa[PARTS - 1][2], 0u, b0, b1);
                    }
#pragma unroll
                for (int i = 0; i < 2 * AT; ++i) {
                    f32x2(&a)[NH] = acc[2 * st + i];
                    const f32x2 lo = pack2(d[i][0], d[i][1]), hi = pack2(d[i][2], d[i][3]);
                    a[0] = fma2(a[0], fall2[0], WIDE ? lo : add2(lo, hi));
                    if (WIDE) a[NH - 1] = fma2(a[NH - 1], fall2[NH - 1], hi);
                }
            }
            // ---- what was folded of the item, added with the present reference
            auto unfold = [&]() {
                f32x2 f2[NH];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float2 ml = unpack2(folded[(2 * KS * NH + h) * 32]);
                    const float f = ex2(ml.x - (m[h] == -CUDART_INF_F ? 0.f : m[h]));
                    l[h] = fmaf(ml.y, f, l[h]);
                    f2[h] = pack2(f, f);
                }
#pragma unroll
                for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
                    for (int h = 0; h < NH; ++h) acc[j][h] = fma2(folded[(j * NH + h) * 32], f2[h], acc[j][h]);
            };
            if (++done % kFold == 0 && can_fold) {
                if (done > kFold) unfold();
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    folded[(2 * KS * NH + h) * 32] = pack2(m[h], l[h]);
                    l[h] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        folded[(j * NH + h) * 32] = acc[j][h];
                        acc[j][h] = 0;
                    }
            }

            // ---- the end of a group, or of the run
            const bool item_end = cur.c == cur.x.n - 1;
            const int u_then = u + (item_end ? 1 + kItemUnits : 1);
            if (item_end || u_then >= u_hi) {
                fresh = true;
                const int first = u - cur.c;
                const bool whole = first >= u_lo && item_end, at_end = u_then >= u_hi;
                const bool leaves = !whole && (at_end || can_leave);
                // a part that others continue: the run's last in this warp's own queue (nothing is under way to
                // it any more)
                float *part = reinterpret_cast<float *>(at_end ? tail_part : head_part);
                if (done >= kFold && can_fold) unfold();
                __syncwarp();
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float sum = l[h];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    const int row = r + 8 * h;
                    if (whole && row >= nh) continue;
                    const float inv = !whole ? 1.f / PartRange<C>::kLift : sum == 0.f ? 0.f : 1.f / sum;
                    sum *= 1.f / PartRange<C>::kLift;
                    const int64_t at = (int64_t)cur.s * p.os + (int64_t)(h0 + row) * p.ohs + 2 * c4;
                    if (c4 == 0) {
                        if (leaves) *reinterpret_cast<float2 *>(part + row * PO) = make_float2(m[h], sum);
                        else if (whole && p.lse && LEAN_IN((int64_t)cur.s * p.hq + h0 + row, (int64_t)p.n_seqs * p.hq, p.err))
                            p.lse[(int64_t)cur.s * p.hq + h0 + row] = natural_lse(m[h], sum);
                    }
#pragma unroll
                    for (int j = 0; j < 2 * KS; ++j) {
                        const float2 a = unpack2(acc[j][h]);
                        const float o[2] = {a.x * inv, a.y * inv};
                        if (leaves) *reinterpret_cast<float2 *>(part + row * PO + 4 + 8 * j + 2 * c4) = make_float2(o[0], o[1]);
                        else if (whole && 8 * j < p.dim && LEAN_SPAN(at + 8 * j, 2, p.out_extent, p.err))
                            store_out<2>(p.out, at + 8 * j, p.act, o);
                    }
                }
                if (leaves && lane == 0) {
                    Record &q = rec[2 * warp + at_end];
                    q.item = cur.s * groups + cur.kvh * p.tiles + cur.tile;
                    q.n = cur.x.n;
                    q.first = first;
                }
                advance(p, cur);
                if (EARLY_Q && !AHEAD_Q && !at_end) load_q(cur.s, cur.kvh, cur.tile);
            } else {
                advance(p, cur);
            }
            u = u_then;
            stage = stage + 1 == S ? 0 : stage + 1;
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- groups shared by the warps of this block: each 32 x 4 outputs of one are added up by a warp
    // lane k knows record k; a group begins where the item changes
    const bool has = lane < 2 * W && rec[lane].item >= 0;
    const unsigned have = __ballot_sync(0xffffffffu, has);
    const unsigned below = have & ((1u << lane) - 1);
    const bool leads = has && (below == 0 || rec[31 - __clz(below)].item != rec[lane].item);
    const unsigned leaders = __ballot_sync(0xffffffffu, leads);
    constexpr int JOBS = H * DP / 128;
    const int n_groups = __popc(leaders);
    for (int job = warp; job < n_groups * JOBS; job += W) {
        const int i = nth_bit(leaders, job / JOBS), j = job % JOBS;
        const unsigned later = leaders & ~((2u << i) - 1);
        unsigned members = have & ~((1u << i) - 1) & (later ? (later & -later) - 1 : 0xffffffffu);
        const Record head = rec[i];
        const Head f = open_item(p, head.item, H);
        const int h = (j * 32 + lane) * 4 / DP, d = (j * 32 + lane) * 4 % DP;
        Sums t;
        t.clear();
        while (members) {
            const int k = __ffs(members) - 1;
            members &= members - 1;
            if (!PSMEM && !(k & 1) && !LEAN_SPAN(((int64_t)blockIdx.x * W + k / 2) * PF, PF, p.warp_extent, p.err)) continue;
            const float *row = reinterpret_cast<const float *>(k & 1 ? tail_part + (k / 2 - warp) * (S * STAGE)
                                                                     : head_part + (int64_t)(k / 2 - warp) * (PF * 4)) + h * PO;
            t.add(*reinterpret_cast<const float2 *>(row), *reinterpret_cast<const float4 *>(row + 4 + d));
        }
        if (head.first >= 0 && head.first + head.n <= b_n) {
            store_result(p, f, h, d, t.o, t.top, t.sum);
        } else {  // the block's part of the item that began before it, or of the one that goes on after it
            const int64_t at = ((int64_t)blockIdx.x * 2 + (head.first < 0 ? 0 : 1)) * PF + h * PO;
            float *row = p.cta_parts + at;
            if (!LEAN_SPAN(at, 8 + d, p.part_extent, p.err)) continue;
            *reinterpret_cast<float4 *>(row + 4 + d) = t.o;
            if (d == 0) *reinterpret_cast<float2 *>(row) = make_float2(t.top, t.sum);
        }
    }
    // The item that begins in this block and goes on in the next ones, for the kernel that adds its parts up.
    if (threadIdx.x == 0) {
        Shared x = {-1, 0};
        if (leaders) {
            const Record q = rec[31 - __clz(leaders)];
            if (q.first >= 0 && q.first + q.n > b_n) {
                const unsigned last = q.first + b_lo + q.n - 1;  // the last of its units, and the block that has it
                const unsigned n = units / blocks, rest = units - n * blocks;
                const unsigned b = last < rest * (n + 1) ? last / (n + 1) : rest + (last - rest * (n + 1)) / n;
                x = Shared{q.item, (int)(b - blockIdx.x) + 1};
            }
        }
        if (LEAN_IN(blockIdx.x, kAttMaxCtas, p.err)) p.shared[blockIdx.x] = x;
    }
}

// Parts of items shared by blocks, added up: 32 x 4 outputs of an item at a time, up to kAtOnce parts' loads under
// way in a warp.  Items of few parts are taken by single warps, those of many by whole blocks, whose warps take the
// parts in turn.
constexpr int kSumWarps = 8, kAtOnce = 10;
template <int H, int DP>
__global__ void __launch_bounds__(kSumWarps * 32) attend_sum_kernel(const AttArgs p, int blocks) {
    constexpr int JOBS = H * DP / 128, PF = part_floats(H, DP), PO = 4 + DP;
    __shared__ Shared item[kAttMaxCtas];
    __shared__ unsigned few_s[kSumWarps], many_s[kSumWarps];
    __shared__ float4 out_s[kSumWarps][32];
    __shared__ float2 ml_s[kSumWarps][32];
    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Shared mine = {-1, 0};
    if (threadIdx.x < blocks && LEAN_IN(threadIdx.x, kAttMaxCtas, p.err)) item[threadIdx.x] = mine = p.shared[threadIdx.x];
    const unsigned few = __ballot_sync(0xffffffffu, mine.item >= 0 && mine.parts <= kAtOnce);
    const unsigned many = __ballot_sync(0xffffffffu, mine.parts > kAtOnce);
    if (lane == 0) {
        few_s[warp] = few;
        many_s[warp] = many;
    }
    __syncthreads();
    auto nth_block = [&](const unsigned *m, int n) {  // block whose bit is the n-th that is set, -1: there are fewer
        for (int i = 0; i < kSumWarps; ++i) {
            const int c = __popc(m[i]);
            if (n < c) return 32 * i + nth_bit(m[i], n);
            n -= c;
        }
        return -1;
    };
    Sums t;
    auto take = [&](int b, int job, int from, int step) {  // parts from, from + step .. of the item that begins in block b
        const int parts = item[b].parts, e = (job * 32 + lane) * 4;
        const int64_t first = (int64_t)b * 2 * PF + e / DP * PO;
        const float *at = p.cta_parts + first;
        t.clear();
        for (int k0 = from; k0 < parts; k0 += kAtOnce * step) {
            float2 ml[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int k = k0 + i * step;
                if (k < parts) {
                    const int64_t skip = (int64_t)(k * 2 + (k == 0)) * PF;
                    const float *row = at + skip;
                    ml[i] = make_float2(-CUDART_INF_F, 0.f);
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (LEAN_SPAN(first + skip, 8 + e % DP, p.part_extent, p.err)) {
                        ml[i] = *reinterpret_cast<const float2 *>(row);
                        v[i] = *reinterpret_cast<const float4 *>(row + 4 + e % DP);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (k0 + i * step < parts) t.add(ml[i], v[i]);
        }
    };
    auto store = [&](int b, int job) {
        const int e = (job * 32 + lane) * 4;
        store_result(p, open_item(p, item[b].item, H), e / DP, e % DP, t.o, t.top, t.sum);
    };
    for (int job = blockIdx.x;; job += gridDim.x) {
        const int b = nth_block(many_s, job / JOBS);
        if (b < 0) break;
        take(b, job % JOBS, warp, kSumWarps);
        __syncthreads();
        ml_s[warp][lane] = make_float2(t.top, t.sum);
        out_s[warp][lane] = t.o;
        __syncthreads();
        if (warp == 0) {
            t.clear();
#pragma unroll
            for (int i = 0; i < kSumWarps; ++i) t.add(ml_s[i][lane], out_s[i][lane]);
            store(b, job % JOBS);
        }
    }
    for (int job = blockIdx.x + warp * gridDim.x;; job += gridDim.x * kSumWarps) {
        const int b = nth_block(few_s, job / JOBS);
        if (b < 0) break;
        take(b, job % JOBS, 0, 1);
        store(b, job % JOBS);
    }
}

template <typename C, int DP, int PARTS, bool WIDE>
lean_status launch_attend(const AttArgs &p, int64_t flags, void *stream) {
    static std::atomic<uint64_t> done{0};
    auto kern = attend_kernel<C, DP, PARTS, WIDE>;
    if (!step_ensure_smem(kern, att_smem<DP>(WIDE ? 16 : 8), done)) return LEAN_ERR_CUDA;
    // no more blocks than there can be units for
    constexpr int W = AttShape<DP>::kWarps;
    const int64_t units = ((int64_t)p.width * p.page + 2 * kUnit) / kUnit * p.n_seqs * p.hkv * p.tiles;
    const int64_t grid = std::min<int64_t>(std::min(step_sm_count(), kAttMaxCtas), std::max<int64_t>(1, units / W));
    const lean_status st = step_launch(kern, grid, W * 32, att_smem<DP>(WIDE ? 16 : 8), flags, stream, p);
    // (no item can be shared by blocks where each gets its own whatever the lengths are)
    const int64_t most = ((int64_t)p.width * p.page + 2 * kUnit - 1) / kUnit;
    const bool by_item = (int64_t)p.n_seqs * p.hkv * p.tiles <= grid && (most + W - 1) / W <= kJoinUnits;
    if (st != LEAN_OK || grid == 1 || by_item) return st;
    constexpr int H = WIDE ? 16 : 8;
    return step_launch(attend_sum_kernel<H, DP>, grid, kSumWarps * 32, 0, LEAN_FLAG_EARLY_WEIGHTS, stream, p, (int)grid);
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

int att_heads(int64_t hq, int64_t hkv) { return hq / hkv > 8 ? 16 : 8; }
int att_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

bool att_sizes_ok(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim) {
    return n_seqs > 0 && hkv > 0 && hq > 0 && hq <= 65536 && hq % hkv == 0 && dim > 0 && dim % 8 == 0 &&
           dim <= kAttMaxDim && n_seqs <= INT32_MAX / hq;
}

}  // namespace

extern "C" int64_t lean_paged_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                                        int64_t head_dim) {
    if (!att_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim)) return -1;
    // what blocks share, a part per warp and two per block, and what a warp folds, of the largest grid
    const int h = att_heads(n_q_heads, n_kv_heads), d = att_dim(head_dim);
    return kSharedBytes + (int64_t)kAttMaxCtas * 4 * ((8 + 2) * part_floats(h, d) + 8 * fold_floats(h, d));
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
    const int64_t group = a->n_q_heads / a->n_kv_heads, tiles = group > 8 ? (group + 15) / 16 : 1;
    if ((a->table_width * a->page_size / kUnit + 2 + kItemUnits) * a->n_seqs * a->n_kv_heads * tiles > UINT32_MAX)
        return LEAN_ERR_SHAPE;  // units are counted in 32 bits
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
    p.shared = reinterpret_cast<Shared *>(ws);
    p.warp_parts = reinterpret_cast<float *>(ws + kSharedBytes);
    const int part = part_floats(att_heads(a->n_q_heads, a->n_kv_heads), att_dim(a->head_dim));
    p.cta_parts = p.warp_parts + kAttMaxCtas * 8 * part;
    p.folds = reinterpret_cast<f32x2 *>(p.cta_parts + kAttMaxCtas * 2 * part);
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
    p.group = (int)group;
    p.tiles = (int)tiles;
    p.dim = (int)a->head_dim;
    p.page = (int)a->page_size;
    p.paged = a->page_size >= kUnit;
    p.whole = a->page_size % kUnit == 0;
    p.width = (int)a->table_width;
    p.window = (int)std::min<int64_t>(a->window, INT32_MAX);
    p.act = (int)a->act_dtype;
    p.scale_log2 = (float)(a->scale * 1.4426950408889634);
    p.cache_extent = (a->n_pages - 1) * a->page_stride + (a->page_size - 1) * a->place_stride +
                     (a->n_kv_heads - 1) * a->cache_head_stride + a->head_dim;
    p.warp_extent = (int64_t)kAttMaxCtas * 8 * part;
    p.part_extent = (int64_t)kAttMaxCtas * 2 * part;
    p.fold_extent = (int64_t)kAttMaxCtas * 8 * fold_floats(att_heads(a->n_q_heads, a->n_kv_heads), att_dim(a->head_dim));
    p.q_extent = (a->n_seqs - 1) * a->q_stride + (a->n_q_heads - 1) * a->q_head_stride + a->head_dim;
    p.out_extent = (a->n_seqs - 1) * a->out_stride + (a->n_q_heads - 1) * a->out_head_stride + a->head_dim;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    return a->cache_dtype == LEAN_BF16 ? pick_dim<__nv_bfloat16>(p, a->flags, stream)
                                       : pick_dim<__half>(p, a->flags, stream);
}
