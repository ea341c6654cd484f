// attend.cuh -- lean_paged_attention's kernels: attention of one new token per
// sequence over the paged cache (attend.cu: caches of 16 bits and the call;
// attend8.cu: caches in 8 bits; beside.cu and beside8.cu: sequences' own tokens in
// lean_prefix_attention).
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
// Caches in 8 bits, codes c with a scale s for each token and kv head: codes become
// f16 operands by byte permutes and a subtraction, exactly; scores are multiplied by
// the keys' scales, p by the values', relative to a power of two that follows the
// largest.  Half the bytes, but the same products and more instructions: 384
// sequences as above 61.5 us, one of 131072 32.3, 613 tokens 11.1; issue slots are
// 59% busy in the first, and a warp's time for a unit bounds all of them.
// Pages of 16 tokens or more hold a unit in one page or two, and two pages cost
// little (384 sequences as above: 69 us with pages of 24, 72 of 20).  In smaller
// pages every token is looked up: 90 us with pages of 8, 99 of one.
#pragma once
#include "step_common.cuh"

using namespace lean;

namespace lean {

constexpr int kAttMaxDim = 256;
constexpr int kAttMaxCtas = 160;  // of a launch: at most one per SM
constexpr int kAttMaxWarps = 16;  // of a block
constexpr int kAttRoomWarps = 8;  // of a block, that the workspace has parts for
constexpr int kUnit = 16;         // tokens
constexpr int kAttItemUnits = 4;  // empty units counted to an item (below)
constexpr int64_t kSharedBytes = 2048;  // a Shared for each block

struct Shared {  // an item that begins in a block and goes on in others (-1: none), and how many blocks it has
    int item, parts;
};

// Prefixes that sequences share (prefix.cuh): prefix i's tokens, its sequences starts[i]..starts[i + 1] - 1, whose query
// heads that share a kv head are rows, and its part of the list of items, `rows` rows by tiles of 128 keys.
constexpr int kTileRows = 128, kTileKeys = 128;
// Tiles of a block's time that an item costs beside its own (q, the first scores, the last outputs): 5 to 8 us, which are
// about four of 16-bit caches (96 sequences on 32768 tokens: 44.6 us, counted as two 47.8) and two in 8 bits.
__host__ __device__ constexpr int item_tiles(bool in8) { return in8 ? 2 : 4; }
struct PrefixList {
    const int32_t *starts, *lens;
    int n, n_seqs, group, hkv, rows, most, item_tiles;  // most: tokens that a prefix's pages can hold
    unsigned sms, own_most;                 // SMs, and the most blocks that sequences' own tokens can take
    float unit_ns, tile_ns;                 // what a unit of those and a tile of a prefix take of an SM's time
};
struct Prefix {
    int first, count, len, keys, tiles;  // keys: tiles of keys; tiles: of rows, for a kv head
    __device__ __forceinline__ unsigned cost(const PrefixList &p) const {  // (the call refuses lists that 32 bits do not count)
        return (unsigned)p.hkv * tiles * (keys + (keys > 0 ? p.item_tiles : 0));
    }
};
__device__ __forceinline__ Prefix open_prefix(const PrefixList &p, int i, unsigned *err) {
    Prefix x;
    const bool in = LEAN_IN(i, p.n, err);
    x.first = in ? min(max(p.starts[i], 0), p.n_seqs) : 0;
    const int end = in ? min(max(p.starts[i + 1], 0), p.n_seqs) : 0;
    x.count = max(0, end - x.first);
    x.len = min(in ? max(p.lens[i], 0) : 0, p.most);
    x.keys = x.len / kTileKeys + (x.len % kTileKeys != 0);
    x.tiles = (x.count * p.group - 1 + p.rows) / p.rows;  // (rows + 255 is below 2^31: the call's limits)
    if (x.tiles == 0) x.keys = 0;
    return x;
}
// The two kernels of one call run beside one another: of the SMs, as many as this for `units` units of sequences' own
// tokens where the prefixes have `tiles` tiles, so that both end together; the SMs that no tile needs at least.  With a and
// b for all of their units and tiles on one of s SMs, and d that an item's beginning costs every block of the second:
// a / n = b / (s - n) + d.  (In proportion to a and b, one rate for every type: 48 us where this takes 44, 96 sequences on
// 32768 tokens, 16/2 heads of 128.)  Where they came to different numbers blocks would only wait for SMs.
__device__ __forceinline__ unsigned own_blocks(const PrefixList &p, unsigned units, unsigned tiles) {
    if (tiles == 0) return p.own_most;
    const float s = p.sms, a = (float)units * p.unit_ns, d = p.item_tiles * p.tile_ns;
    const float c = d * s + a + (float)tiles * p.tile_ns;
    const unsigned n = (unsigned)__float2int_rn(2.f * a * s / (c + sqrtf(fmaxf(0.f, c * c - 4.f * d * a * s))));
    return min(p.own_most, min(p.sms - 1, max(max(1u, n), p.sms > tiles ? p.sms - tiles : 1)));
}

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
    int act, out_act;
    PrefixList list;  // (beside a kernel for prefixes)
    float scale_log2;
    const float *k_scales, *v_scales;  // of caches in 8 bits
    int64_t scale_page, scale_place, scale_hs;
    int64_t cache_extent, q_extent, out_extent;  // elements, for the checked build
    int64_t warp_extent, part_extent, fold_extent, scale_extent;
    int most_ctas;  // blocks that the workspace has room for
    unsigned *err;
};

// The kernels for a cache type; flags and stream as the calls have them (attend.cu, attend8.cu).
lean_status attend_cache16(const AttArgs &p, bool bf16, int64_t flags, void *stream);
lean_status attend_cache8(const AttArgs &p, int64_t flags, void *stream);
// The same beside a kernel for prefixes, heads of 128 at most (beside.cu, beside8.cu).
lean_status attend_beside16(const AttArgs &p, bool bf16, int64_t flags, void *stream);
lean_status attend_beside8(const AttArgs &p, int64_t flags, void *stream);
// What lean_paged_attention refuses, and its workspace, by sizes alone.
bool att_sizes_ok(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim);
// The workspace's parts, of att_workspace_bytes() bytes, as the kernel for caches in 8 bits or in 16 has them.
int64_t att_workspace_bytes(int64_t hq, int64_t hkv, int64_t dim);
void att_workspace(AttArgs &p, void *workspace, bool in8);

}  // namespace lean

namespace {

// Warps of a block (in 8 bits a unit is half the bytes and more instructions: at heads of 64, where 128 registers do, 16
// warps take 61 us where 8 take 78, 384 sequences as above), stages of a warp's queue: 128-192 KB of loads an SM can have
// under way.
__host__ __device__ constexpr int att_warps(bool in8, int dp, bool wide) {
    return dp == 256 ? 4 : in8 && !wide && dp == 64 ? 16 : 8;
}
template <typename C, int DP, bool WIDE>
struct AttShape {
    static constexpr bool kIn8 = sizeof(C) == 1;
    static constexpr int kWarps = att_warps(kIn8, DP, WIDE);
    static constexpr int kStages = kIn8 ? (DP == 64 ? (WIDE ? 8 : 4) : DP == 128 ? 5 : 3) : DP == 64 ? 5 : DP == 128 ? 3 : 2;
    static constexpr int kStageBytes = kUnit * DP * 2 * (int)sizeof(C);  // K and V
    static constexpr int kScaleBytes = kIn8 ? 2 * kUnit * 4 : 0;         // their scales
    static constexpr int kQueues = kWarps * kStages * (kStageBytes + kScaleBytes);
    // at 256 the warps' q as well (up to 12 registers per 16 elements)
    static constexpr int kSmem = 512 + kQueues + kWarps * (DP == 256 ? DP / 16 * 12 * 128 : 0);
};
// The matrix instructions' type: of a cache in 8 bits, whose codes are exact in it, f16.
template <typename C>
struct Operand {
    using type = C;
};
template <>
struct Operand<int8_t> {
    using type = __half;
};
// A part: maxima, sums and outputs of a group of H heads.
__host__ __device__ constexpr int part_floats(int heads, int dp) { return heads * (dp + 4); }
// What a warp folds: each lane's outputs, references and sums.
__host__ __device__ constexpr int fold_floats(int heads, int dp) { return heads * (dp + 8); }
// Shared memory of a block: queues; q at 256 (above); and, where it fits, a part per warp.
constexpr int kMaxSmem = 232448 - 1536;  // of 227 KB, less static variables
template <typename C, int DP, bool WIDE>
__host__ __device__ constexpr bool parts_in_smem() {
    using S = AttShape<C, DP, WIDE>;
    return S::kSmem + S::kWarps * part_floats(WIDE ? 16 : 8, DP) * 4 <= kMaxSmem;
}
template <typename C, int DP, bool WIDE>
__host__ __device__ constexpr int att_smem() {
    using S = AttShape<C, DP, WIDE>;
    return S::kSmem + (parts_in_smem<C, DP, WIDE>() ? S::kWarps * part_floats(WIDE ? 16 : 8, DP) * 4 : 0);
}

// 16 bytes of which `real` (16 or 0) are copied and the rest zero
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
// 4 bytes, or as many zeros
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
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

// Four bytes c as f16: 1024 + (c + 128) has c + 128 in its low bits, and the difference to 1152 is exact.  SEL: the
// places of two bytes, 4 (0x64) between and after them.
template <int SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t biased) {
    uint32_t h;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(h) : "r"(biased), "r"(0x64646464), "n"(SEL));
    const uint32_t bias = 0x64806480;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&d);
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
constexpr int kItemUnits = kAttItemUnits;

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
    if (LEAN_SPAN(at, 4, p.out_extent, p.err)) store_out<4>(p.out, at, p.out_act, v);
    const int64_t at_lse = (int64_t)f.s * p.hq + f.h0 + h;
    if (d == 0 && p.lse && LEAN_IN(at_lse, (int64_t)p.n_seqs * p.hq, p.err)) p.lse[at_lse] = natural_lse(top, sum);
}

// WIDE: 9 to 16 query heads in a group, one per row; else up to 8, two rows each.
// BESIDE: beside a kernel for prefixes, whose blocks may begin only when what came before this one is done (they do not wait
// for it themselves); blocks as own_blocks() says, parts of shared items left to the kernel after both.  (Asked for in
// p.list instead, at run time, it cost lean_paged_attention in 8 bits 7%.)
template <typename C, int DP, int PARTS, bool WIDE, bool BESIDE>
__global__ void __launch_bounds__(AttShape<C, DP, WIDE>::kWarps * 32, 1) attend_kernel(const AttArgs p) {
    using P = typename Operand<C>::type;
    constexpr bool IN8 = AttShape<C, DP, WIDE>::kIn8;
    constexpr int W = AttShape<C, DP, WIDE>::kWarps, S = AttShape<C, DP, WIDE>::kStages, T = W * 32;
    constexpr int STAGE = AttShape<C, DP, WIDE>::kStageBytes, EPP = 16 / (int)sizeof(C);  // elements of a 16-byte piece
    constexpr int H = WIDE ? 16 : 8, NH = WIDE ? 2 : 1;  // heads of a group, of a thread
    // a row's bytes and lanes, rows of a copy instruction
    constexpr int RB = DP * (int)sizeof(C), LPR = RB / 16, RPI = 32 / LPR;
    constexpr int KS = DP / 16;                                // steps of the contraction, and pairs of output tiles
    constexpr int AREGS = WIDE ? 4 * PARTS : 4 + (PARTS > 2 ? 2 : 0);  // of q per step
    constexpr bool QSMEM = DP == 256;                                  // no registers left for q
    constexpr int PF = part_floats(H, DP), PO = 4 + DP;                // a head's row of a part: m, l, -, out
    constexpr bool PSMEM = parts_in_smem<C, DP, WIDE>();
    // registers for q as it was read: beside the accumulators, and all through the item before
    constexpr bool EARLY_Q = !WIDE && DP <= 128, AHEAD_Q = !WIDE && DP == 64;
    static_assert(PF * 4 <= S * STAGE, "a part fits a queue");
    static_assert(W <= kAttMaxWarps, "a lane for each record");
    static_assert(PSMEM || W <= kAttRoomWarps, "the workspace has parts for as many");
    static_assert(AttShape<C, DP, WIDE>::kSmem <= kMaxSmem, "shared memory");
    constexpr int AT = 2;  // steps of the values whose products are under way at once (more spill)
    extern __shared__ uint8_t queue_raw[];
    uint8_t *queue = queue_raw + (512 - smem_addr(queue_raw) % 512) % 512;
    __shared__ unsigned scan[W], tile_scan[W];
    __shared__ int longest[W];
    __shared__ unsigned units_before[T];
    __shared__ Record rec[2 * W];

    if (BESIDE) {
        pdl_wait();
        pdl_launch_dependents();
    } else {
        step_begin();
    }
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r = lane / 4, c4 = lane % 4;
    // The dimension of the first of a thread's pair j, of q's rows and of the outputs: in 16 bits as the matrix
    // instructions have them; in 8 bits a thread has four neighbours, the bytes of one register: of the contraction in
    // an order of its own (q's is the same), of the outputs even ones in one tile and odd ones in the other.
    auto dim_of = [&](int j) { return IN8 ? 16 * (j >> 1) + 4 * c4 + 2 * (j & 1) : 8 * j + 2 * c4; };
    // what a row's pieces are moved by in shared memory (rows of 64 bytes: two of them have all banks)
    auto turned = [](int row) { return RB == 64 ? (row >> 1) & 3 : row & 7; };
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
    if (BESIDE) {
        unsigned tiles = 0;
        for (int i = threadIdx.x; i < p.list.n; i += T) tiles += open_prefix(p.list, i, p.err).cost(p.list);
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        if (lane == 0) tile_scan[warp] = tiles;
    }
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
    unsigned grid = gridDim.x;
    if (BESIDE) {
        unsigned tiles = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) tiles += tile_scan[i];
        grid = own_blocks(p.list, units, tiles);
    }
    const int64_t items = (int64_t)p.n_seqs * groups;
    const bool by_item = items <= grid && (unsigned)((most + W - 1) / W) <= units / (grid * W) + kJoinUnits;
    const int blocks = by_item ? (int)items : (int)min(grid, units / W + (units % W != 0));
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
    uint8_t *const head_part = PSMEM ? queue + AttShape<C, DP, WIDE>::kSmem - 512 + warp * (PF * 4)
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
        const C *k_lane = static_cast<const C *>(p.k) + EPP * col, *v_lane = static_cast<const C *>(p.v) + EPP * col;
        const uint32_t to_lane = my_queue + lr * RB + ((col ^ turned(lr)) * 16);
        const int real = EPP * col < p.dim ? 16 : 0;
        // scales: of a unit's keys, lanes 0-15, and values
        const uint32_t my_scales = smem_addr(queue) + W * S * STAGE + warp * (S * AttShape<C, DP, WIDE>::kScaleBytes);
        const float *scale_lane = lane < kUnit ? p.k_scales : p.v_scales;

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
                    if (IN8) {
                        const int64_t at = (int64_t)page_id * p.scale_page + (int64_t)(next.in_page + lane % kUnit) * p.scale_place +
                                           (int64_t)next.kvh * p.scale_hs;
                        const bool in = LEAN_IN(at, p.scale_extent, p.err);
                        cp_async4(my_scales + stage * AttShape<C, DP, WIDE>::kScaleBytes + 4 * lane, scale_lane + (in ? at : 0), in ? 4 : 0);
                    }
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
                    int64_t at_scale = -1;
                    if (in_unit >= next.x.start - t0 && in_unit < next.x.len - t0) {
                        const bool first = !p.paged || in_unit < in_first;
                        const int id = first ? page_id : last_id;
                        const int64_t place = !p.paged ? (t0 + in_unit) % p.page
                                                       : (int64_t)next.in_page + in_unit - (first ? 0 : p.page);
                        off = (int64_t)id * p.page_stride + place * p.place_stride + (int64_t)next.kvh * p.cache_hs;
                        if (id < 0 || id >= p.n_pages) off = -2;
                        else if (!LEAN_SPAN(off, p.dim, p.cache_extent, p.err)) off = -1;
                        if (IN8 && off >= 0) {
                            at_scale = (int64_t)id * p.scale_page + place * p.scale_place + (int64_t)next.kvh * p.scale_hs;
                            if (!LEAN_IN(at_scale, p.scale_extent, p.err)) at_scale = -1;
                        }
                    }
                    if (IN8) {  // what is not attended has scale 0, keys that are not there NaN, which reaches out and lse
                        const uint32_t to = my_scales + stage * AttShape<C, DP, WIDE>::kScaleBytes + 4 * lane;
                        if (off == -2 && lane < kUnit) asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(0x7fffffff) : "memory");
                        else cp_async4(to, scale_lane + (at_scale >= 0 ? at_scale : 0), at_scale >= 0 ? 4 : 0);
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
                            if (IN8 || o != -2)
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
                    const int d = dim_of(i);
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
        // (in 8 bits, where a piece is a step: tokens 0-7, 8-15 of the even and of the odd step, K like V)
        const uint32_t v_row = my_queue + kUnit * RB + (((lane >> 3) & 1) * 8 + (lane & 7)) * RB +
                               (((lane >> 4) ^ turned(lane & 7)) * 16);
        const uint32_t k_row = IN8 ? v_row - kUnit * RB
                                   : my_queue + ((lane >> 4) * 8 + (lane & 7)) * RB + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
        // q as rows of the matrix instruction, part by part
        uint32_t qa[QSMEM ? 1 : KS][AREGS];
        uint32_t *q_shared = reinterpret_cast<uint32_t *>(queue + AttShape<C, DP, WIDE>::kQueues) + warp * (KS * AREGS * 32);
        // outputs and sums of the item since its last fold, with reference m
        f32x2 acc[2 * KS][NH];
        float m[NH], l[NH], zs[NH];
        // (8 bits) the values' scales are taken into p, relative to 2^(v_ref - 126), which is above the largest so far
        int v_ref = 1;
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
                    const int fe = e == 0 || e == 255 ? 127 : min(253, max(1, 254 + PartRange<P>::kLiftQ - e));
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
                        const uint32_t lo = take_part<P>(f[0][2 * st].x, f[0][2 * st].y);
                        const uint32_t hi = take_part<P>(f[0][2 * st + 1].x, f[0][2 * st + 1].y);
                        if (WIDE) {
                            a[4 * part] = lo;
                            a[4 * part + 2] = hi;
                            a[4 * part + 1] = take_part<P>(f[NH - 1][2 * st].x, f[NH - 1][2 * st].y);
                            a[4 * part + 3] = take_part<P>(f[NH - 1][2 * st + 1].x, f[NH - 1][2 * st + 1].y);
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
                v_ref = 1;
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
            uint32_t codes[4];
            float2 ks[2], vs[2];  // scales of tokens 2 c4 and 2 c4 + 1, and of those 8 further on
            if constexpr (IN8) {
                const float2 *at = reinterpret_cast<const float2 *>(queue + (my_scales - smem_addr(queue)) +
                                                                    stage * AttShape<C, DP, WIDE>::kScaleBytes) + c4;
                ks[0] = at[0];
                ks[1] = at[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // an infinite one is NaN, as the scores of such a key are
                    ks[j].x += ks[j].x - ks[j].x;
                    ks[j].y += ks[j].y - ks[j].y;
                }
                vs[0] = at[8];
                vs[1] = at[12];
            }
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                uint32_t b[4], a[AREGS];
                if constexpr (IN8) {
                    if (!(st & 1)) {
                        ldmatrix4(codes, (k_row + stage * STAGE) ^ (16 * st));
#pragma unroll
                        for (int i = 0; i < 4; ++i) codes[i] ^= 0x80808080u;
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        b[2 * j] = codes_f16<0x4140>(codes[2 * (st & 1) + j]);
                        b[2 * j + 1] = codes_f16<0x4342>(codes[2 * (st & 1) + j]);
                    }
                } else {
                    ldmatrix4(b, (k_row + stage * STAGE) ^ (32 * st));
                }
#pragma unroll
                for (int i = 0; i < AREGS; ++i)
                    a[i] = QSMEM ? q_shared[(st * AREGS + i) * 32 + lane] : qa[QSMEM ? 0 : st][i];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (WIDE) {
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            mma<P>(st & 1 ? sd[j] : sc[j], a[4 * part], a[4 * part + 1], a[4 * part + 2], a[4 * part + 3],
                                   b[2 * j], b[2 * j + 1]);
                    } else {
                        mma<P>(sc[j], a[0], a[1], a[2], a[3], b[2 * j], b[2 * j + 1]);
                        if (PARTS > 2) mma<P>(sd[j], a[AREGS - 2], 0u, a[AREGS - 1], 0u, b[2 * j], b[2 * j + 1]);
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
                    if constexpr (IN8) e[h][i] *= i & 1 ? ks[j].y : ks[j].x;
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
                const float mn = top - m[h] <= PartRange<P>::kSlack ? m[h] : top;
                const float ms = mn == -CUDART_INF_F ? 0.f : mn;
                const float fall = ex2(m[h] - ms);
                fall2[h] = pack2(fall, fall);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[h][i] = ex2(e[h][i] - ms) * PartRange<P>::kLift;
                    sum += e[h][i];
                }
                l[h] = fmaf(l[h], fall, sum);
            }
            float v_fall = 1.f;  // of what is there, to the values' new reference
            if constexpr (IN8) {
                float top = fmaxf(fmaxf(vs[0].x, vs[0].y), fmaxf(vs[1].x, vs[1].y));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int now = max(v_ref, min(252, (int)(__float_as_uint(top) >> 23 & 0xff)));
                v_fall = __uint_as_float((uint32_t)max(0, 127 + v_ref - now) << 23);
                v_ref = now;
                const float down = __uint_as_float((uint32_t)(253 - now) << 23);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    fall2[h] = mul2(fall2[h], pack2(v_fall, v_fall));
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[h][i] *= (i & 1 ? vs[i >> 1].y : vs[i >> 1].x) * down;
                }
            }
            uint32_t pa[PARTS][4];
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    pa[part][h] = take_part<P>(e[h][0], e[h][1]);
                    pa[part][2 + h] = take_part<P>(e[h][2], e[h][3]);
                }
            // ---- values: a unit's products summed from 0, then one addition in fp32 (the instruction cuts off what is
            // small next to its accumulator: 8192 keys 17 nats below one left nothing there, 2.3e-4 of the output)
#pragma unroll
            for (int st = 0; st < KS; st += AT) {
                uint32_t b[AT][4];
                float d[2 * AT][4] = {};
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    if constexpr (IN8) {
                        if (i == 0) {
                            ldmatrix4_trans(codes, (v_row + stage * STAGE) ^ (16 * st));
#pragma unroll
                            for (int k = 0; k < 4; ++k) codes[k] ^= 0x80808080u;
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // tokens 0-7, 8-15; even dimensions, odd ones
                            b[i][k] = codes_f16<0x4240>(codes[2 * i + k]);
                            b[i][2 + k] = codes_f16<0x4341>(codes[2 * i + k]);
                        }
                    } else {
                        ldmatrix4_trans(b[i], (v_row + stage * STAGE) ^ (32 * (st + i)));
                    }
                }
#pragma unroll
                for (int part = 0; part < (WIDE ? PARTS : PARTS - 1); ++part)
#pragma unroll
                    for (int i = 0; i < 2 * AT; ++i) {
                        const uint32_t b0 = b[i / 2][2 * (i & 1)], b1 = b[i / 2][2 * (i & 1) + 1];
                        if (WIDE) mma<P>(d[i], pa[part][0], pa[part][1], pa[part][2], pa[part][3], b0, b1);
                        else if (part == 0) mma<P>(d[i], pa[0][0], pa[1][0], pa[0][2], pa[1][2], b0, b1);
                        else mma<P>(d[i], pa[PARTS - 1][0], 0u, pa[PARTS - 1][2], 0u, b0, b1);
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
                    const float g = IN8 ? f * PartRange<P>::kLift : f;
                    f2[h] = pack2(g, g);
                }
                const float v_up = __uint_as_float((uint32_t)(253 - v_ref) << 23);
#pragma unroll
                for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const f32x2 then = folded[(j * NH + h) * 32];
                        acc[j][h] = fma2(IN8 ? mul2(then, pack2(v_up, v_up)) : then, f2[h], acc[j][h]);
                    }
            };
            // (8 bits: what is folded is in the values' own size, without the lift, by which scales of 1e30 would not fit)
            const float v_size = IN8 ? __uint_as_float((uint32_t)(v_ref + 1) << 23) : 1.f;
            const float v_fold = v_size * (1.f / PartRange<P>::kLift);
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
                        folded[(j * NH + h) * 32] = IN8 ? mul2(acc[j][h], pack2(v_fold, v_fold)) : acc[j][h];
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
                    float inv = !whole ? 1.f / PartRange<P>::kLift : sum == 0.f ? 0.f : 1.f / sum;
                    if (IN8) inv *= v_size;
                    sum *= 1.f / PartRange<P>::kLift;
                    const int64_t at = (int64_t)cur.s * p.os + (int64_t)(h0 + row) * p.ohs;
                    if (c4 == 0) {
                        if (leaves) *reinterpret_cast<float2 *>(part + row * PO) = make_float2(m[h], sum);
                        else if (whole && p.lse && LEAN_IN((int64_t)cur.s * p.hq + h0 + row, (int64_t)p.n_seqs * p.hq, p.err))
                            p.lse[(int64_t)cur.s * p.hq + h0 + row] = natural_lse(m[h], sum);
                    }
#pragma unroll
                    for (int j = 0; j < 2 * KS; ++j) {
                        float2 a = unpack2(acc[j][h]);
                        if constexpr (IN8) {  // an even dimension and the odd one after it
                            const float2 even = unpack2(acc[j & ~1][h]), odd = unpack2(acc[j | 1][h]);
                            a = j & 1 ? make_float2(even.y, odd.y) : make_float2(even.x, odd.x);
                        }
                        const float o[2] = {a.x * inv, a.y * inv};
                        if (leaves) *reinterpret_cast<float2 *>(part + row * PO + 4 + dim_of(j)) = make_float2(o[0], o[1]);
                        else if (whole && dim_of(j) < p.dim && LEAN_SPAN(at + dim_of(j), 2, p.out_extent, p.err))
                            store_out<2>(p.out, at + dim_of(j), p.out_act, o);
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

// No more blocks of eight warps than there can be units for.  (Blocks of 16 as well: with a kv head of each sequence to a
// block there is nothing to join.  A decode step of 32 layers, 15/5 heads, one sequence of 200 tokens in 8 bits, 1.36 ms
// counted by 16, 1.25 by eight.)
inline int64_t att_grid(const AttArgs &p, int W) {
    const int64_t units = ((int64_t)p.width * p.page + 2 * kUnit) / kUnit * p.n_seqs * p.hkv * p.tiles;
    return std::min<int64_t>(std::min(step_sm_count(), p.most_ctas), std::max<int64_t>(1, units / std::min(W, 8)));
}

template <typename C, int DP, int PARTS, bool WIDE, bool BESIDE>
lean_status launch_attend(const AttArgs &p, int64_t flags, void *stream) {
    static std::atomic<uint64_t> done{0};
    auto kern = attend_kernel<C, DP, PARTS, WIDE, BESIDE>;
    if (!step_ensure_smem(kern, att_smem<C, DP, WIDE>(), done)) return LEAN_ERR_CUDA;
    constexpr int W = AttShape<C, DP, WIDE>::kWarps;
    const int64_t grid = att_grid(p, W);
    const lean_status st = step_launch(kern, grid, W * 32, att_smem<C, DP, WIDE>(), flags, stream, p);
    // (no item can be shared by blocks where each gets its own whatever the lengths are)
    const int64_t most = ((int64_t)p.width * p.page + 2 * kUnit - 1) / kUnit;
    const bool by_item = (int64_t)p.n_seqs * p.hkv * p.tiles <= grid && (most + W - 1) / W <= kJoinUnits;
    if (st != LEAN_OK || grid == 1 || by_item) return st;
    if constexpr (!BESIDE)
        return step_launch(attend_sum_kernel<WIDE ? 16 : 8, DP>, grid, kSumWarps * 32, 0, LEAN_FLAG_EARLY_WEIGHTS, stream, p, (int)grid);
    else return st;
}
template <typename C, int DP, bool BESIDE>
lean_status pick_attend(const AttArgs &p, int64_t flags, void *stream) {
    const bool wide = p.group > 8;
    if (p.act == LEAN_F32)
        return wide ? launch_attend<C, DP, 3, true, BESIDE>(p, flags, stream) : launch_attend<C, DP, 3, false, BESIDE>(p, flags, stream);
    return wide ? launch_attend<C, DP, 2, true, BESIDE>(p, flags, stream) : launch_attend<C, DP, 2, false, BESIDE>(p, flags, stream);
}
template <typename C>
lean_status pick_dim(const AttArgs &p, int64_t flags, void *stream) {
    if (p.dim <= 64) return pick_attend<C, 64, false>(p, flags, stream);
    if (p.dim <= 128) return pick_attend<C, 128, false>(p, flags, stream);
    return pick_attend<C, 256, false>(p, flags, stream);
}

}  // namespace
