// prefix.cuh -- lean_prefix_attention's kernels: the attention of many sequences'
// new tokens to prefixes that they share (prefix.cu: caches of 16 bits and the
// call; prefix8.cu: caches in 8 bits).
//
//   z_j = scale q . k_j,  p_j = e^(z_j - m),  out = sum p_j v_j / sum p_j
//
// over a prefix's tokens, then over a sequence's own (the kernels of attend.cuh),
// joined by their maxima and sums.
//
// The query heads that share a kv head, of all sequences that share a prefix, are
// rows of one matrix: S = Q K^T and O = P V are products that the fifth-generation
// tensor cores take, 128 rows by 128 keys at a time, and a prefix's keys and
// values are read once for 256 rows.  Below about 290 rows HBM bounds the call,
// above it the tensor cores do.
//
//   - Work is a list of items: 256 (or 128) rows of a prefix and kv head, over tiles
//     of 128 keys.  Every block takes an equal run of tiles, whatever the prefixes'
//     lengths and numbers of sequences are, and leaves maxima, sums and outputs of
//     its part of an item in the workspace; a last kernel adds up the parts and the
//     sequence's own tokens.
//   - A block has four loader warps (keys and values into swizzled tiles, two of each
//     under way), one warp that issues matrix instructions, and two groups of 128
//     threads, a thread to a row, that turn S into P.  The groups take turns: while one
//     works on its scores the tensor cores have the other's products.  With two tiles
//     of rows (NQ = 2) each group has its own 128 rows and all keys; with one, both
//     have the same rows and every other tile of keys.
//   - S and O lie in tensor memory; P replaces S there and is read as an operand
//     from it.  O is summed over one tile only and then added in fp32 registers: the
//     tensor cores cut off what is small next to their accumulator, and a new maximum
//     needs no pass over O.
//   - q is scaled by a power of two as in attend.cuh and split in QP parts of the
//     operands' type, p in PP: one each for 16-bit activations (q is exact in one; p
//     errs by half a step, 2^-8 of itself in bf16, as out itself is rounded), three
//     and two for fp32.
//   - Caches in 8 bits become f16 on the way into shared memory (exact); scores are
//     multiplied by the keys' scales, p by the values', relative to the tile's
//     largest.
#pragma once
#include <cuda.h>

#include <type_traits>

#include "../../include/lean_cache.h"
#include "attend.cuh"
#include "tensor.cuh"

namespace lean {

constexpr int kTileRows = 128, kTileKeys = 128, kHalfKeys = 64;
constexpr int kPrefixMaxCtas = 160;
constexpr int kPrefixThreads = 512;
// Tiles of a block's time that an item costs beside its own (q, the first scores, the last outputs).
constexpr int kItemTiles = 2;
// Halves of tiles whose products are summed in tensor memory before they are added in fp32 (one part of p): what is below
// 2^-24 of a sum is cut off when it is added, 16 keys at a time, so that a row errs by 2^-16 of its largest sum at most.
constexpr int kFoldHalves = 32;

struct PrefixArgs {
    const void *q, *k, *v;
    const float *k_scales, *v_scales;
    const int32_t *table, *lens, *starts;
    int64_t qs, qhs, page_stride, place_stride, cache_hs, scale_page, scale_place, scale_hs, table_stride, n_pages;
    int n_prefixes, n_seqs, hq, hkv, group, dim, page, width, act;
    float scale_log2;
    // workspace: where each prefix's items begin in the list (and, last, how long it is); maxima and sums, outputs, of
    // the parts that begin an item, by row (and half, with one tile of rows), then those that go on with one, by block
    unsigned long long *plan;
    float2 *ml;
    float *o;
    int64_t parts;  // how many there are
    // a sequence's own tokens, and what comes out
    const float *own_out, *own_lse;
    void *out;
    float *lse;
    int64_t os, ohs;
    int64_t cache_extent, scale_extent, q_extent, out_extent;  // elements, for the checked build
    unsigned *err;
};

// Keys and values of caches of 16 bits as tensors [page][head][place][dim] for the copy engine, in boxes of `box` places by
// 64 dimensions (box 0: pages whose size no multiple of 8 divides, or strides that it does not take).
struct PrefixMaps {
    CUtensorMap k, v;
    int box;
};

lean_status prefix_cache16(const PrefixArgs &p, bool bf16, bool two, int64_t flags, void *stream);
lean_status prefix_cache8(const PrefixArgs &p, bool two, int64_t flags, void *stream);

}  // namespace lean

namespace {

constexpr unsigned kErrPrefixWait = 4u;  // as the tensor-core products: a bounded wait ran out
constexpr uint64_t kPrefixWaitNs = 2000000000ull;

// A prefix: its sequences, keys, and its items in the list.
struct Prefix {
    int first, count, len, keys, tiles;  // keys: tiles of keys; tiles: of rows, for a kv head
    __device__ __forceinline__ unsigned long long cost(int hkv) const {
        return (unsigned long long)hkv * tiles * (keys + (keys > 0 ? kItemTiles : 0));
    }
};
__device__ __forceinline__ Prefix open_prefix(const PrefixArgs &p, int i, int rows) {
    Prefix x;
    const bool in = LEAN_IN(i, p.n_prefixes, p.err);
    x.first = in ? min(max(p.starts[i], 0), p.n_seqs) : 0;
    const int end = in ? min(max(p.starts[i + 1], 0), p.n_seqs) : 0;
    x.count = max(0, end - x.first);
    const int64_t most = (int64_t)p.width * p.page;
    const int len = in ? max(p.lens[i], 0) : 0;
    x.len = len > most ? (int)most : len;
    x.keys = x.len / kTileKeys + (x.len % kTileKeys != 0);
    x.tiles = (int)(((int64_t)x.count * p.group + rows - 1) / rows);
    if (x.tiles == 0) x.keys = 0;
    return x;
}
// A list of units cut into equal runs, none of them empty (blocks past the units have none): where a block's run begins,
// and the block that has a unit.
struct Runs {
    unsigned long long each;
    unsigned rest, blocks;
    __device__ __forceinline__ Runs(unsigned long long total, unsigned n) {
        blocks = total < n ? max(1u, (unsigned)total) : n;
        each = total / blocks;
        rest = (unsigned)(total % blocks);
    }
    __device__ __forceinline__ unsigned long long begin(unsigned b) const { return each * b + rest * b / blocks; }
    __device__ __forceinline__ unsigned of(unsigned long long u) const {
        unsigned lo = 0, hi = blocks - 1;  // the last block that begins at u or before it
        while (lo < hi) {
            const unsigned mid = (lo + hi + 1) / 2;
            if (begin(mid) <= u) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// A block's run of the list, item by item; every role walks it by itself.
struct Walk {
    int i;                       // prefix
    Prefix x;
    unsigned long long off;      // place in the prefix's part of the list
    unsigned long long left;     // of the run
    // the part of an item that comes next: keys' tiles from..to-1
    int kvh, tile, from, to;
    // false: no more
    __device__ __forceinline__ bool next(const PrefixArgs &p, int rows) {
        while (left > 0) {
            while (off >= x.cost(p.hkv)) {
                off -= x.cost(p.hkv);
                if (++i >= p.n_prefixes) return false;
                x = open_prefix(p, i, rows);
            }
            const int each = x.keys + kItemTiles;
            const int item = (int)(off / each);
            from = (int)(off - (unsigned long long)item * each);
            const int take = (int)min(left, (unsigned long long)(each - from));
            to = min(from + take, x.keys);
            off += take;
            left -= take;
            if (from < to) {
                kvh = item / x.tiles;
                tile = item - kvh * x.tiles;
                return true;
            }
        }
        return false;
    }
};

template <typename C, int DP, int QP, int PP, int NQ>
struct PrefixShape {
    static constexpr bool kIn8 = sizeof(C) == 1;
    static constexpr int kChunks = DP / 64, kChunkBytes = kTileRows * 128, kTileBytes = kChunks * kChunkBytes;
    static constexpr int kQ = NQ * QP * kTileBytes;
    // two tiles of keys and two of values; with three parts of q only one of the values fits
    static constexpr int kKStages = 2, kVStages = QP == 3 && DP == 128 ? 1 : 2;
    static constexpr int kOff = kQ + (kKStages + kVStages) * kTileBytes;  // rows' places, two tiles
    static constexpr int kScaleAt = kOff + 2 * kTileKeys * 8;             // scales of four tiles, keys and values
    static constexpr int kBars = kScaleAt + (kIn8 ? 4 * 2 * kTileKeys * 4 : 0);
    static constexpr int kSmem = kBars + 512;
    static constexpr int kSmemAsked = kSmem + 1008;  // (the tiles begin on 1024 bytes)
    // Tensor memory, 512 columns: for each group of rows its outputs, in what is left buffers for the scores of 64 keys,
    // which become p: part 0 (and 1) of 32 keys in the first 16 (and next 16) of their own 32 columns, a third beyond them.
    static constexpr int kWidth = PP == 3 ? 96 : 64, kBuffers = (256 - DP) / kWidth;
    static_assert(kBuffers >= 1 && kBuffers <= 3, "tensor memory");
    __device__ static __forceinline__ uint32_t scores(int g, unsigned b) { return (g * kBuffers + b) * kWidth; }
    __device__ static __forceinline__ uint32_t outputs(int g) { return 512 - 2 * DP + g * DP; }
    __device__ static __forceinline__ uint32_t part(int chunk, int k) { return k < 2 ? 32 * chunk + 16 * k : 64 + 16 * chunk; }
};

struct PrefixBars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // a stage's tile is there, was used
    uint64_t s_full[2][3], p_full[2][3], o_full[2][3];      // of a group's buffers: scores, p, products are done
    uint64_t q_full, q_free;                                // q is there; both groups are done with it
    uint64_t rows_full[2], tops_full[2];                    // a tile's rows' places, the warps' largest scales are there
    uint64_t scales_full[4];
    uint64_t last;                                          // every matrix instruction is done
    uint32_t tmem;
    int dead;            // a wait ran out: everyone leaves
    int tile_exp[4];     // exponents of the tiles' largest value scales
    float warp_top[2][4];
    int start_i;         // the run's first prefix and place in it
    unsigned long long start_off;
};
static_assert(sizeof(PrefixBars) <= 512, "room for the barriers");

// A box of a tensor map into shared memory; its bytes are counted on `bar`.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int place, int head, int page, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4,%5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(place), "r"(head), "r"(page), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void store8(float *to, const float *f) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]),
                 "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Wait for a phase; false: it, or another wait of the block, ran out.
__device__ __forceinline__ bool phase_wait(PrefixBars &b, uint64_t *bar, uint32_t parity, unsigned *err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(&b.dead)) return false;
        if (globaltimer_ns() - t0 > kPrefixWaitNs) {
            *reinterpret_cast<volatile int *>(&b.dead) = 1;
            atomicOr(err, kErrPrefixWait);
            return false;
        }
    }
    return true;
}

// The same for a warp, whose lanes stay together: false if it is for one of them.
__device__ __forceinline__ bool warp_wait(PrefixBars &b, uint64_t *bar, uint32_t parity, unsigned *err) {
    return __all_sync(0xffffffffu, phase_wait(b, bar, parity, err));
}

// Row r of a tile's item: its sequence and query head; false: the item has fewer.
__device__ __forceinline__ bool row_of(const PrefixArgs &p, const Walk &w, int64_t r, int &seq, int &head) {
    if (r >= (int64_t)w.x.count * p.group) return false;
    seq = w.x.first + (int)(r / p.group);
    head = w.kvh * p.group + (int)(r % p.group);
    return true;
}

template <typename C, int DP, int QP, int PP, int NQ>
__global__ void __launch_bounds__(kPrefixThreads, 1) prefix_kernel(const __grid_constant__ PrefixMaps maps, const PrefixArgs p) {
    using S = PrefixShape<C, DP, QP, PP, NQ>;
    using T = typename Operand<C>::type;
    constexpr bool IN8 = S::kIn8, BF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int KS = S::kKStages, VS = S::kVStages, NB = S::kBuffers, ROWS = NQ * kTileRows;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *smem = raw_smem + (1024 - smem_addr(raw_smem) % 1024) % 1024;
    uint8_t *const q_tiles = smem, *const k_tiles = smem + S::kQ, *const v_tiles = k_tiles + KS * S::kTileBytes;
    int64_t *const row_off = reinterpret_cast<int64_t *>(smem + S::kOff);
    float *const scales = reinterpret_cast<float *>(smem + S::kScaleAt);  // [tile % 4][key's, value's][128]
    PrefixBars &bars = *reinterpret_cast<PrefixBars *>(smem + S::kBars);
    step_begin();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;

    // ---- this block's run of the list
    unsigned long long *const before = reinterpret_cast<unsigned long long *>(smem);  // (the tiles' room, unused yet)
    const int per = (p.n_prefixes + kPrefixThreads - 1) / kPrefixThreads;
    const int lo = min(p.n_prefixes, (int)threadIdx.x * per), hi = min(p.n_prefixes, lo + per);
    unsigned long long mine = 0;
    for (int i = lo; i < hi; ++i) mine += open_prefix(p, i, ROWS).cost(p.hkv);
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) before[warp] = incl;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_full[i], 4);
            mbar_init(&bars.v_full[i], 4);
            mbar_init(&bars.k_empty[i], NQ);  // (with one tile of rows each tile of keys is one group's)
            mbar_init(&bars.v_empty[i], NQ);
            for (int b = 0; b < 3; ++b) {
                mbar_init(&bars.s_full[i][b], 1);
                mbar_init(&bars.p_full[i][b], 4);
                mbar_init(&bars.o_full[i][b], 1);
            }
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars.scales_full[i], 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.rows_full[i], 4);
            mbar_init(&bars.tops_full[i], 4);
        }
        mbar_init(&bars.q_full, 8);
        mbar_init(&bars.q_free, 10);
        mbar_init(&bars.last, 4);
        bars.dead = 0;
        bars.start_i = -1;
        fence_mbar_init();
    }
    __syncthreads();
    unsigned long long begins = incl - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kPrefixThreads / 32; ++i) {
        if (i < warp) begins += before[i];
        total += before[i];
    }
    const Runs runs(total, gridDim.x);
    const bool has_run = blockIdx.x < runs.blocks;
    const unsigned long long run_lo = has_run ? runs.begin(blockIdx.x) : 0, run_hi = has_run ? runs.begin(blockIdx.x + 1) : 0;
    if (blockIdx.x == 0) {  // for the kernel that adds the parts up
        unsigned long long at = begins;
        for (int i = lo; i < hi; ++i) {
            if (LEAN_IN(i, p.n_prefixes + 1, p.err)) p.plan[i] = at;
            at += open_prefix(p, i, ROWS).cost(p.hkv);
        }
        if (threadIdx.x == 0 && LEAN_IN(p.n_prefixes, p.n_prefixes + 1, p.err)) p.plan[p.n_prefixes] = total;
    }
    if (run_lo < run_hi && begins <= run_lo && run_lo < begins + mine) {  // one thread's
        unsigned long long off = run_lo - begins;
        int i = lo;
        for (;; ++i) {
            const unsigned long long c = open_prefix(p, i, ROWS).cost(p.hkv);
            if (off < c) break;
            off -= c;
        }
        bars.start_i = i;
        bars.start_off = off;
    }
    if (warp == 12) tm_alloc(&bars.tmem, 512);
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = bars.tmem;
    Walk w;
    w.i = max(bars.start_i, 0);
    w.off = bars.start_off;
    w.left = bars.start_i < 0 ? 0 : run_hi - run_lo;
    if (w.left > 0) w.x = open_prefix(p, w.i, ROWS);

    if (warp < 8) {
        // ---- scores to probabilities, products to outputs: a thread has a row
        regs_up<PP == 1 ? 168 : 192>();
        const int g = warp / 4, r = threadIdx.x % kTileRows;
        const uint32_t lanes = (uint32_t)(warp % 4) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t s_group = tmem + lanes + S::scores(g, 0), o_at = tmem + lanes + S::outputs(g);
        unsigned done = 0;          // half tiles of this group so far: buffer done % NB, whose phase is done / NB
        unsigned tiles_before = 0;  // of the run, by loader's count (scales)
        bool ok = true;
        uint32_t q_phase = 1;  // (the phase before the first counts as done)
        while (ok && w.next(p, ROWS)) {
            // where this row's part goes (-1: the item has no such row)
            int seq, head;
            const bool real = row_of(p, w, (int64_t)w.tile * ROWS + (NQ == 2 ? g * kTileRows : 0) + r, seq, head);
            int64_t part_at = -1;
            if (real) {
                const int64_t first = (int64_t)seq * p.hq + head;
                part_at = w.from == 0 ? (NQ == 2 ? first : 2 * first + g)
                                      : (NQ == 2 ? 1 : 2) * (int64_t)p.n_seqs * p.hq + (int64_t)blockIdx.x * 256 + g * kTileRows + r;
                if (!LEAN_IN(part_at, p.parts, p.err)) part_at = -1;
            }
            // q of this row, scaled by a power of two, in parts
            float zs;
            {
                float f[DP];
                const int64_t at = real ? (int64_t)seq * p.qs + (int64_t)head * p.qhs : 0;
                float top = 0.f;
#pragma unroll
                for (int d = 0; d < DP; d += 8) {
                    const bool in = real && d < p.dim && LEAN_SPAN(at + d, 8, p.q_extent, p.err);
                    if (QP == 3 && p.act == LEAN_F32) {
                        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                        if (in) {
                            a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at + d);
                            b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at + d + 4);
                        }
                        f[d] = a.x; f[d + 1] = a.y; f[d + 2] = a.z; f[d + 3] = a.w;
                        f[d + 4] = b.x; f[d + 5] = b.y; f[d + 6] = b.z; f[d + 7] = b.w;
                    } else {
                        uint4 a = make_uint4(0, 0, 0, 0);
                        if (in) a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at + d);
                        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            RawPair<false> pair;
                            pair.v = u[i];
                            const float2 v = pair.get(p.act);
                            f[d + 2 * i] = v.x;
                            f[d + 2 * i + 1] = v.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[d + i]));
                }
                const int e = (int)(__float_as_uint(top) >> 23);
                const int fe = e == 0 || e == 255 ? 127 : min(253, max(1, 254 + PartRange<T>::kLiftQ - e));
                float up = __uint_as_float((uint32_t)fe << 23);
                zs = p.scale_log2 * __uint_as_float((uint32_t)(254 - fe) << 23);
                if (zs < 0.f) {  // so that the largest product is the largest score
                    zs = -zs;
                    up = -up;
                }
                if (zs == 0.f) zs = 1.17549435e-38f;  // (masked scores are -inf times this)
                ok = warp_wait(bars, &bars.q_free, q_phase, p.err);
                if (!ok) break;
                q_phase ^= 1;
#pragma unroll
                for (int d = 0; d < DP; d += 8) {
                    // (with one tile of rows each group writes half of it)
                    if (NQ == 1 && (DP == 128 ? d / 64 : d / 32) != g) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[d + i] *= up;
#pragma unroll
                    for (int part = 0; part < QP; ++part) {
                        uint4 a;
                        a.x = take_part<T>(f[d], f[d + 1]);
                        a.y = take_part<T>(f[d + 2], f[d + 3]);
                        a.z = take_part<T>(f[d + 4], f[d + 5]);
                        a.w = take_part<T>(f[d + 6], f[d + 7]);
                        *reinterpret_cast<uint4 *>(q_tiles + ((NQ == 2 ? g : 0) * QP + part) * S::kTileBytes +
                                                   d / 64 * S::kChunkBytes + r * 128 + ((d / 8 % 8) ^ (r & 7)) * 16) = a;
                    }
                }
                smem_to_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full);
            }
            constexpr float kLog2Lift = PartRange<T>::kLift == 1.f ? 0.f : 13.f, kDown = 1.f / PartRange<T>::kLift;
            float m = -CUDART_INF_F, l = 0.f;
            int v_ref = 1;
            // What a tile's largest score and scales make of the references: m, v_ref; what is multiplied with the sums
            // and the outputs so far, added to the exponents, and multiplied with the sum of p.
            float fall, o_fall, shift, back;
            auto refer = [&](float top, unsigned slot) {
                // (m as in attend.cuh: within kSlack of the largest score so far)
                const float mn = top - m <= PartRange<T>::kSlack ? m : top;
                const float ms = mn == -CUDART_INF_F ? 0.f : mn;
                fall = o_fall = ex2(m - ms);
                bool moved = !(mn == m);
                m = mn;
                shift = kLog2Lift - ms;
                back = 1.f;
                if (IN8) {
                    // values' scales lie in 0.5..1 times 2^(exponent of the tile's largest - 126); sums are relative to
                    // 2^(v_ref - 126); what is below 2^-60 of the largest may count as 2^-60 of it
                    const int e = bars.tile_exp[slot], now = max(v_ref, e), below = min(now - e, 60);
                    o_fall *= __uint_as_float((uint32_t)max(0, 127 + v_ref - now) << 23);
                    shift -= (float)below;
                    back = __uint_as_float((uint32_t)(127 + below) << 23);
                    moved = moved || now != v_ref;
                    v_ref = now;
                }
                return moved;
            };
            auto size = [&]() { return IN8 ? kDown * __uint_as_float((uint32_t)(v_ref + 1) << 23) : kDown; };
            // Halves of tiles in turn (of the last one the second may have no keys; keys that are not there score -inf).
            int t = w.from + (NQ == 2 ? 0 : g), half = 0, limit = 0;  // limit: keys of the half that are there, or more
            unsigned n = 0, slot = 0;
            uint32_t s_at = 0;
            const float *ks = nullptr, *vs = nullptr;
            auto scores_wait = [&]() {
                limit = w.x.len - t * kTileKeys - half * kHalfKeys;
                n = tiles_before + (t - w.from);
                slot = n % 4;
                ks = scales + slot * 2 * kTileKeys + half * kHalfKeys;
                vs = ks + kTileKeys;
                s_at = s_group + done % NB * S::kWidth;
                bool got = true;
                if (IN8 && half == 0) got = warp_wait(bars, &bars.scales_full[slot], n / 4 & 1, p.err);
                got = got && warp_wait(bars, &bars.s_full[g][done % NB], done / NB & 1, p.err);
                tm_after();
                return got;
            };
            auto publish = [&]() {
                tm_wait_st();
                tm_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[g][done % NB]);
                ++done;
            };
            auto products_wait = [&]() {  // of all that were published
                const bool got = warp_wait(bars, &bars.o_full[g][(done - 1) % NB], (done - 1) / NB & 1, p.err);
                tm_after();
                return got;
            };
            auto advance_half = [&]() {
                if (half == 0 && limit > kHalfKeys) {
                    half = 1;
                } else {
                    half = 0;
                    t += NQ == 2 ? 1 : 2;
                }
            };
            if constexpr (PP == 1) {
                // outputs stay in tensor memory for kFoldHalves halves, then go to the row's part in the workspace
                int in_sum = 0;       // halves whose products lie there
                bool folded = false;  // the part has some already, with reference m_part
                float m_part = -CUDART_INF_F;
                while (t < w.to) {
                    ok = scores_wait();
                    if (!ok) break;
                    uint32_t x[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tm_ld32(s_at + 32 * c, x[c]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) tm_wait_ld(x[c]);
                    if (IN8) {
#pragma unroll
                        for (int i = 0; i < kHalfKeys; i += 2) {
                            const float2 z = unpack2(mul2(pack2(__uint_as_float(x[i / 32][i % 32]), __uint_as_float(x[i / 32][i % 32 + 1])),
                                                          *reinterpret_cast<const f32x2 *>(ks + i)));
                            x[i / 32][i % 32] = __float_as_uint(z.x);
                            x[i / 32][i % 32 + 1] = __float_as_uint(z.y);
                        }
                    }
                    if (limit < kHalfKeys) {
#pragma unroll
                        for (int i = 0; i < kHalfKeys; ++i)
                            if (i >= limit) x[i / 32][i % 32] = 0xff800000u;
                    }
                    float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int i = 0; i < kHalfKeys; ++i) tops[i % 4] = fmaxf(tops[i % 4], __uint_as_float(x[i / 32][i % 32]));
                    const bool moved = refer(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * zs, slot);
                    const f32x2 zs2 = pack2(zs, zs), shift2 = pack2(shift, shift);
                    f32x2 sum2[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t part[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 a = unpack2(fma2(pack2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])), zs2, shift2));
                            float2 e = make_float2(ex2(a.x), ex2(a.y));
                            sum2[i / 2 % 2] = add2(sum2[i / 2 % 2], pack2(e.x, e.y));
                            if (IN8) e = unpack2(mul2(pack2(e.x, e.y), *reinterpret_cast<const f32x2 *>(vs + 32 * c + i)));
                            part[i / 2] = take_part<T>(e.x, e.y);
                        }
                        tm_st16(s_at + S::part(c, 0), part);  // (over the scores, which are in registers)
                    }
                    if (__any_sync(0xffffffffu, moved) && in_sum > 0) {  // new references: what is there is rescaled
                        ok = products_wait();
                        if (!ok) break;
#pragma unroll
                        for (int c = 0; c < DP; c += 32) {
                            uint32_t y[32];
                            tm_ld32(o_at + c, y);
                            tm_wait_ld(y);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t z[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) z[i] = __float_as_uint(__uint_as_float(y[16 * h + i]) * o_fall);
                                tm_st16(o_at + c + 16 * h, z);
                            }
                        }
                    }
                    publish();
                    const float2 sum = unpack2(add2(sum2[0], sum2[1]));
                    l = fmaf(l, fall, (sum.x + sum.y) * back);
                    advance_half();
                    if (++in_sum == kFoldHalves || t >= w.to) {
                        ok = products_wait();
                        if (!ok) break;
                        const float f = ex2(m_part - (m == -CUDART_INF_F ? 0.f : m)), up = size();
                        float *o = p.o + part_at * DP;
#pragma unroll
                        for (int c = 0; c < DP; c += 32) {
                            uint32_t y[32];
                            tm_ld32(o_at + c, y);
                            tm_wait_ld(y);
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                if (part_at < 0) break;
                                float z[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) z[k] = __uint_as_float(y[i + k]) * up;
                                if (folded) {
                                    const Vec<float, 4> a = load_vec<float, 4>(o + c + i), b = load_vec<float, 4>(o + c + i + 4);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        z[k] = fmaf(a.v[k], f, z[k]);
                                        z[4 + k] = fmaf(b.v[k], f, z[4 + k]);
                                    }
                                }
                                store8(o + c + i, z);
                            }
                            __syncwarp();
                        }
                        tm_before();
                        folded = true;
                        m_part = m;
                        in_sum = 0;
                    }
                }
                tiles_before += w.to - w.from;
                if (!ok) break;
            } else {
                f32x2 acc[DP / 2];
#pragma unroll
                for (int i = 0; i < DP / 2; ++i) acc[i] = 0;
                while (t < w.to) {
                    ok = scores_wait();
                    if (!ok) break;
                    if (limit < kHalfKeys) {
#pragma unroll 1
                        for (int c = limit / 32 * 32; c < kHalfKeys; c += 32) {
                            uint32_t x[32];
                            tm_ld32(s_at + c, x);
                            tm_wait_ld(x);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t y[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) y[i] = c + 16 * h + i < limit ? x[16 * h + i] : 0xff800000u;
                                tm_st16(s_at + c + 16 * h, y);
                            }
                        }
                        tm_wait_st();
                    }
                    float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int c = 0; c < kHalfKeys; c += 32) {
                        uint32_t x[32];
                        tm_ld32(s_at + c, x);
                        tm_wait_ld(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float z = __uint_as_float(x[i]);
                            if (IN8) z *= ks[c + i];
                            tops[i % 4] = fmaxf(tops[i % 4], z);
                        }
                    }
                    refer(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * zs, slot);
                    const f32x2 zs2 = pack2(zs, zs), shift2 = pack2(shift, shift);
                    f32x2 sum2[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t x[32];
                        tm_ld32(s_at + 32 * c, x);
                        tm_wait_ld(x);
                        uint32_t part[PP][16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            f32x2 z = pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                            if (IN8) z = mul2(z, *reinterpret_cast<const f32x2 *>(ks + 32 * c + i));
                            const float2 a = unpack2(fma2(z, zs2, shift2));
                            float2 e = make_float2(ex2(a.x), ex2(a.y));
                            sum2[i / 2 % 2] = add2(sum2[i / 2 % 2], pack2(e.x, e.y));
                            if (IN8) e = unpack2(mul2(pack2(e.x, e.y), *reinterpret_cast<const f32x2 *>(vs + 32 * c + i)));
#pragma unroll
                            for (int k = 0; k < PP; ++k) part[k][i / 2] = take_part<T>(e.x, e.y);
                        }
#pragma unroll
                        for (int k = 0; k < PP; ++k) tm_st16(s_at + S::part(c, k), part[k]);  // over scores already used
                    }
                    publish();
                    const float2 sum = unpack2(add2(sum2[0], sum2[1]));
                    l = fmaf(l, fall, (sum.x + sum.y) * back);
                    ok = products_wait();
                    if (!ok) break;
                    const f32x2 fall2 = pack2(o_fall, o_fall);
#pragma unroll
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t x[32];
                        tm_ld32(o_at + c, x);
                        tm_wait_ld(x);
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            acc[(c + i) / 2] = fma2(acc[(c + i) / 2], fall2, pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                    }
                    tm_before();
                    advance_half();
                }
                tiles_before += w.to - w.from;
                if (!ok) break;
                if (part_at >= 0) {
                    const float up = size();
#pragma unroll
                    for (int d = 0; d < DP; d += 8) {
                        float z[8];
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            const float2 a = unpack2(acc[(d + k) / 2]);
                            z[k] = a.x * up;
                            z[k + 1] = a.y * up;
                        }
                        store8(p.o + part_at * DP + d, z);
                    }
                }
            }
            if (lane == 0) mbar_arrive(&bars.q_free);  // (its last products are done)
            if (part_at >= 0) p.ml[part_at] = make_float2(m, l * kDown);
        }
    } else if (warp < 12) {
        // ---- keys and values into shared memory
        regs_down<PP == 1 ? 112 : IN8 ? 88 : 72>();
        const int t = threadIdx.x - 256;
        unsigned n = 0;
        bool ok = true;
        auto page_of = [&](int tok) {
            const int64_t e = (int64_t)w.i * p.table_stride + tok / p.page;
            return tok < w.x.len && LEAN_IN(e, (int64_t)(p.n_prefixes - 1) * p.table_stride + p.width, p.err) ? p.table[e] : 0;
        };
        // place of token `tok`, in page `id`, in the caches; -1: past the prefix, -2: no page of the cache
        auto place_of = [&](int tok, int id) -> int64_t {
            if (tok >= w.x.len) return -1;
            if (id < 0 || id >= p.n_pages) {
                atomicOr(p.err, kErrSlot);
                return -2;
            }
            const int64_t off = (int64_t)id * p.page_stride + (int64_t)(tok % p.page) * p.place_stride + (int64_t)w.kvh * p.cache_hs;
            return LEAN_SPAN(off, p.dim, p.cache_extent, p.err) ? off : -1;
        };
        auto arrive = [&](uint64_t *bar) {  // of four warps, what each of whose lanes has written
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        if constexpr (IN8) {
            // A thread looks up a key's row and scales, then takes 16-byte pieces of all rows through registers, where
            // they become f16: the pieces of the next tile are under way while this one's are converted.
            constexpr int PR = DP / 16;  // pieces of a row
            uint4 xk[PR], xv[PR];
            float sk = 1.f, sv = 0.f;
            auto load = [&](const void *cache, unsigned tile, uint4 (&x)[PR]) {
                const int64_t *off = row_off + (tile & 1) * kTileKeys;
#pragma unroll
                for (int i = 0; i < PR; ++i) {
                    const int c = t % PR;
                    const int64_t o = off[(i * kTileKeys + t) / PR];
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (o >= 0 && 16 * c < p.dim) x[i] = *reinterpret_cast<const uint4 *>(static_cast<const int8_t *>(cache) + o + 16 * c);
                }
            };
            auto convert = [&](uint8_t *tile, const uint4 (&x)[PR]) {
#pragma unroll
                for (int i = 0; i < PR; ++i) {
                    const int row = (i * kTileKeys + t) / PR, c = t % PR;
                    const uint32_t u[4] = {x[i].x ^ 0x80808080u, x[i].y ^ 0x80808080u, x[i].z ^ 0x80808080u, x[i].w ^ 0x80808080u};
                    uint8_t *to = tile + c / 4 * S::kChunkBytes + row * 128;
                    *reinterpret_cast<uint4 *>(to + ((2 * c % 8) ^ (row & 7)) * 16) =
                        make_uint4(codes_f16<0x4140>(u[0]), codes_f16<0x4342>(u[0]), codes_f16<0x4140>(u[1]), codes_f16<0x4342>(u[1]));
                    *reinterpret_cast<uint4 *>(to + ((2 * c % 8 + 1) ^ (row & 7)) * 16) =
                        make_uint4(codes_f16<0x4140>(u[2]), codes_f16<0x4342>(u[2]), codes_f16<0x4140>(u[3]), codes_f16<0x4342>(u[3]));
                }
                smem_to_async();
            };
            // the rows of tile number m of the run, at kt of its prefix, whose pages are known; scales under way
            auto rows = [&](unsigned m, int kt, int id) {
                const int tok = kt * kTileKeys + t;
                const int64_t off = place_of(tok, id);
                row_off[(m & 1) * kTileKeys + t] = off;
                sk = off == -2 ? CUDART_NAN_F : 1.f;
                sv = 0.f;
                if (off >= 0) {
                    const int64_t at = (int64_t)id * p.scale_page + (int64_t)(tok % p.page) * p.scale_place + (int64_t)w.kvh * p.scale_hs;
                    if (LEAN_IN(at, p.scale_extent, p.err)) {
                        sk = p.k_scales[at];
                        sv = p.v_scales[at];
                    }
                }
                arrive(&bars.rows_full[m & 1]);
            };
            auto wait_rows = [&](unsigned m) { return warp_wait(bars, &bars.rows_full[m & 1], m / 2 & 1, p.err); };
            auto finish_scales = [&](unsigned m) {  // relative to the tile's largest
                float top = fmaxf(sv, 0.f);
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (lane == 0) bars.warp_top[m & 1][warp - 8] = top;
                arrive(&bars.tops_full[m & 1]);
                if (!warp_wait(bars, &bars.tops_full[m & 1], m / 2 & 1, p.err)) return false;
                const float *tops = bars.warp_top[m & 1];
                top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                const int e = min(252, max(1, (int)(__float_as_uint(top) >> 23)));
                float *to = scales + m % 4 * 2 * kTileKeys + t;
                to[0] = sk + (sk - sk);  // (an infinite one is NaN, as the scores of such a key are)
                to[kTileKeys] = sv * __uint_as_float((uint32_t)(253 - e) << 23);
                if (t == 0) bars.tile_exp[m % 4] = e;
                arrive(&bars.scales_full[m % 4]);
                return true;
            };
            while (ok && w.next(p, ROWS)) {
                rows(n, w.from, page_of(w.from * kTileKeys + t));
                int next_id = w.from + 1 < w.to ? page_of((w.from + 1) * kTileKeys + t) : 0;
                ok = wait_rows(n);
                if (!ok) break;
                load(p.k, n, xk);
                load(p.v, n, xv);
                ok = finish_scales(n);
                for (int kt = w.from; ok && kt < w.to; ++kt, ++n) {
                    const bool more = kt + 1 < w.to;
                    if (more) {
                        rows(n + 1, kt + 1, next_id);
                        if (kt + 2 < w.to) next_id = page_of((kt + 2) * kTileKeys + t);
                    }
                    if (n >= KS) ok = warp_wait(bars, &bars.k_empty[n % KS], (n / KS - 1) & 1, p.err);
                    if (!ok) break;
                    convert(k_tiles + n % KS * S::kTileBytes, xk);
                    arrive(&bars.k_full[n % KS]);
                    if (more) {
                        ok = wait_rows(n + 1);
                        if (!ok) break;
                        load(p.k, n + 1, xk);
                    }
                    if (n >= VS) ok = warp_wait(bars, &bars.v_empty[n % VS], (n / VS - 1) & 1, p.err);
                    if (!ok) break;
                    convert(v_tiles + n % VS * S::kTileBytes, xv);
                    arrive(&bars.v_full[n % VS]);
                    if (more) {
                        load(p.v, n + 1, xv);
                        ok = finish_scales(n + 1);
                    }
                }
            }
        } else {
            // Whole tiles in pages that the cache has: boxes of a page each, by the copy engine; a lane issues its own
            // page's.  (By cp.async, 32 for each of 128 threads: XX us.)  Others, whose last rows have to be zeros: row by
            // row.
            constexpr int PR = DP / 8;  // 16-byte pieces of a row
            const int boxes = maps.box > 0 ? kTileKeys / maps.box : 0;
            auto copy_rows = [&](const void *from, const int64_t *off, uint8_t *tile, bool is_k) {
                const C *cache = static_cast<const C *>(from);
#pragma unroll
                for (int i = 0; i < PR; ++i) {
                    const int row = (i * kTileKeys + t) / PR, c = t % PR;
                    const int64_t o = off[row];
                    const uint32_t to = smem_addr(tile + c / 8 * S::kChunkBytes + row * 128 + ((c % 8) ^ (row & 7)) * 16);
                    const bool in = o >= 0 && 8 * c < p.dim;
                    if (is_k && o == -2)  // keys that are not there: NaN, which reaches out and lse by itself
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to), "r"(0x7fff7fff) : "memory");
                    else
                        cp_async16(to, in ? cache + o + 8 * c : cache, in ? 16 : 0);
                }
                cp_async_commit();
            };
            auto copy_boxes = [&](const CUtensorMap *map, uint8_t *tile, uint64_t *full, int tok, int id) {
                if (warp == 8) {
                    if (lane == 0) mbar_arrive_expect_tx(full, S::kTileBytes);
                    __syncwarp();
                    if (lane < boxes) {
#pragma unroll
                        for (int c = 0; c < S::kChunks; ++c)
                            copy_box(smem_addr(tile + c * S::kChunkBytes + lane * maps.box * 128), map, 64 * c, tok % p.page, w.kvh, id, full);
                    }
                } else if (lane == 0) {
                    mbar_arrive(full);
                }
            };
            // the token whose page a thread looks up ahead: its box's first, or its row's
            auto mine = [&](int kt) { return kt * kTileKeys + (boxes > 0 ? lane * maps.box : t); };
            auto ahead = [&](int kt) { return boxes > 0 && lane >= boxes ? 0 : page_of(mine(kt)); };
            unsigned rows_n = 0;  // tiles taken row by row so far
            while (ok && w.next(p, ROWS)) {
                int next_id = ahead(w.from);
                for (int kt = w.from; ok && kt < w.to; ++kt, ++n) {
                    const int tok = mine(kt);
                    int id = next_id;
                    if (kt + 1 < w.to) next_id = ahead(kt + 1);
                    bool whole = boxes > 0 && kt * kTileKeys + kTileKeys <= w.x.len;
                    if (whole) {
                        bool fits = lane >= boxes || (id >= 0 && id < p.n_pages);
                        if (lane < boxes && fits)
                            fits = LEAN_SPAN((int64_t)id * p.page_stride + (int64_t)(tok % p.page) * p.place_stride + (int64_t)w.kvh * p.cache_hs,
                                             (maps.box - 1) * p.place_stride + p.dim, p.cache_extent, p.err);
                        whole = __all_sync(0xffffffffu, fits);
                    }
                    uint8_t *const kt_at = k_tiles + n % KS * S::kTileBytes, *const vt_at = v_tiles + n % VS * S::kTileBytes;
                    int64_t *offs = nullptr;
                    if (!whole) {
                        if (boxes > 0) id = page_of(kt * kTileKeys + t);
                        offs = row_off + (rows_n & 1) * kTileKeys;
                        offs[t] = place_of(kt * kTileKeys + t, id);
                        arrive(&bars.rows_full[rows_n & 1]);
                        ok = warp_wait(bars, &bars.rows_full[rows_n & 1], rows_n / 2 & 1, p.err);
                        if (!ok) break;
                        ++rows_n;
                    }
                    if (n >= KS) ok = warp_wait(bars, &bars.k_empty[n % KS], (n / KS - 1) & 1, p.err);
                    if (!ok) break;
                    if (whole) copy_boxes(&maps.k, kt_at, &bars.k_full[n % KS], tok, id);
                    else copy_rows(p.k, offs, kt_at, true);
                    if (n >= VS) ok = warp_wait(bars, &bars.v_empty[n % VS], (n / VS - 1) & 1, p.err);
                    if (!ok) break;
                    if (whole) {
                        copy_boxes(&maps.v, vt_at, &bars.v_full[n % VS], tok, id);
                    } else {
                        copy_rows(p.v, offs, vt_at, false);
                        cp_async_wait<1>();
                        smem_to_async();
                        arrive(&bars.k_full[n % KS]);
                        cp_async_wait<0>();
                        smem_to_async();
                        arrive(&bars.v_full[n % VS]);
                    }
                }
            }
            cp_async_wait<0>();
        }
        for (unsigned j = n > KS ? n - KS : 0; ok && j < n; ++j) ok = warp_wait(bars, &bars.k_empty[j % KS], j / KS & 1, p.err);
        for (unsigned j = n > VS ? n - VS : 0; ok && j < n; ++j) ok = warp_wait(bars, &bars.v_empty[j % VS], j / VS & 1, p.err);
    } else {
        regs_down<PP == 1 ? 64 : IN8 ? 40 : 56>();
        if (lane == 0) {
            // ---- matrix instructions: warps 12 and 13 issue the groups' scores, 14 and 15 their products.  (One thread
            // needs about 110 cycles for an instruction that runs for 64: one warp for all of them 58 us where four
            // take XX, 96 sequences on 32768 tokens.)
            const int g = warp % 2;
            unsigned n = 0;
            bool ok = true;
            auto halves_of = [&](unsigned t) { return w.x.len - (w.from + (int)t) * kTileKeys > kHalfKeys ? 2 : 1; };
            if (warp < 14) {
                const uint32_t idesc = tile_idesc(BF16, kHalfKeys, false);
                const uint32_t q_lower = tile_lower(smem_addr(q_tiles + (NQ == 2 ? g * QP * S::kTileBytes : 0)), 16);
                const uint32_t k_lower = tile_lower(smem_addr(k_tiles), 16);
                const int steps = (p.dim + 15) / 16;
                uint32_t q_phase = 0;
                unsigned u = 0;  // half tiles of this group
                while (ok && w.next(p, ROWS)) {
                    ok = phase_wait(bars, &bars.q_full, q_phase, p.err);
                    q_phase ^= 1;
                    const unsigned tiles = w.to - w.from;
                    for (unsigned t = NQ == 2 ? 0 : g; ok && t < tiles; t += NQ == 2 ? 1 : 2) {
                        const unsigned j = n + t;
                        ok = phase_wait(bars, &bars.k_full[j % KS], j / KS & 1, p.err);
                        const int halves = halves_of(t);
                        for (int half = 0; ok && half < halves; ++half, ++u) {
                            // p lies where the scores go: its products first
                            if (u >= NB) ok = phase_wait(bars, &bars.o_full[g][u % NB], (u / NB - 1) & 1, p.err);
                            if (!ok) break;
                            smem_to_async();
                            tm_after();
                            const uint32_t d = tmem + S::scores(g, u % NB);
                            const uint32_t b = k_lower + (j % KS * S::kTileBytes + half * kHalfKeys * 128 >> 4);
#pragma unroll
                            for (int part = 0; part < QP; ++part)
#pragma unroll
                                for (int s = 0; s < DP / 16; ++s) {
                                    const uint32_t in = (s / 4 * S::kChunkBytes + s % 4 * 32) >> 4;
                                    if (s < steps)
                                        tm_mma_ss(d, q_lower + (part * S::kTileBytes >> 4) + in, b + in, kTileUpper, idesc, part + s > 0);
                                }
                            tm_commit(&bars.s_full[g][u % NB]);
                        }
                        tm_commit(&bars.k_empty[j % KS]);
                    }
                    if (ok) mbar_arrive(&bars.q_free);  // (this phase of q_full has been seen)
                    n += tiles;
                }
            } else {
                // (with one stage for values, one thread takes both groups' tiles: each sees every phase of the stage)
                constexpr bool ALL = VS == 1;
                static_assert(!ALL || NQ == 1, "tiles in turn");
                const uint32_t idesc = tile_idesc(BF16, DP, true);
                const uint32_t v_lower = tile_lower(smem_addr(v_tiles), S::kChunkBytes);
                unsigned u0 = 0, u1 = 0;  // half tiles of this group, or of both
                while (ok && w.next(p, ROWS) && !(ALL && g == 1)) {
                    const unsigned tiles = w.to - w.from;
                    unsigned in_sum = 0;
                    for (unsigned t = NQ == 2 || ALL ? 0 : g; ok && t < tiles; t += NQ == 2 || ALL ? 1 : 2) {
                        const unsigned j = n + t;
                        const int of = ALL ? t % 2 : g;  // group
                        const int halves = halves_of(t);
                        for (int half = 0; ok && half < halves; ++half) {
                            const unsigned u = ALL && of ? u1 : u0;
                            // (p first: then what came before in this stage is done, and a phase is not mistaken for the
                            // one two before it)
                            ok = phase_wait(bars, &bars.p_full[of][u % NB], u / NB & 1, p.err);
                            if (half == 0) ok = ok && phase_wait(bars, &bars.v_full[j % VS], j / VS & 1, p.err);
                            if (!ok) break;
                            smem_to_async();
                            tm_after();
                            const uint32_t a = tmem + S::scores(of, u % NB), d = tmem + S::outputs(of);
                            const uint32_t b = v_lower + (j % VS * S::kTileBytes + half * kHalfKeys * 128 >> 4);
                            const bool add = PP == 1 && in_sum % kFoldHalves > 0;
#pragma unroll
                            for (int s = 0; s < kHalfKeys / 16; ++s)
#pragma unroll
                                for (int part = 0; part < PP; ++part)
                                    tm_mma_ts(d, a + S::part(s / 2, part) + s % 2 * 8, b + s * (2048 >> 4), kTileUpper, idesc,
                                              part + s > 0 || add);
                            tm_commit(&bars.o_full[of][u % NB]);
                            if (ALL && of) ++u1;
                            else ++u0;
                            ++in_sum;
                        }
                        tm_commit(&bars.v_empty[j % VS]);
                    }
                    n += tiles;
                }
            }
            tm_commit(&bars.last);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&bars.last, 0) && globaltimer_ns() - t0 < kPrefixWaitNs) {}
        }
    }
    tm_before();
    __syncthreads();
    if (warp == 12) tm_free(tmem, 512);
}

// Parts of a row, and the sequence's own tokens, added up: a warp to a row.
template <int DP, int NQ>
__global__ void __launch_bounds__(256) prefix_sum_kernel(const PrefixArgs p, unsigned blocks) {
    constexpr int V = DP / 32, ROWS = NQ * kTileRows, HALVES = NQ == 2 ? 1 : 2, U = 8;
    step_begin();
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= (int64_t)p.n_seqs * p.hq) return;
    const int seq = (int)(row / p.hq), head = (int)(row % p.hq);
    // its prefix: the last that begins at it or before
    int lo = 0, hi = p.n_prefixes;  // how many begin so: lo..hi
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool so = at < hi && LEAN_IN(at, p.n_prefixes + 1, p.err) && p.starts[at] <= seq;
        const int n = __popc(__ballot_sync(0xffffffffu, so));
        if (n == 0) break;
        hi = min(hi, lo + n * step);
        lo += (n - 1) * step + 1;
    }
    int parts = 0;
    int64_t more = 0;  // the first part that goes on
    if (lo > 0) {
        const Prefix x = open_prefix(p, lo - 1, ROWS);
        if (seq >= x.first && seq < x.first + x.count && x.keys > 0) {
            const int64_t r = (int64_t)(seq - x.first) * p.group + head % p.group;
            const int tile = (int)(r / ROWS), in = (int)(r % ROWS);
            const Runs runs(p.plan[p.n_prefixes], blocks);
            const unsigned long long at = p.plan[lo - 1] + ((unsigned long long)(head / p.group) * x.tiles + tile) * (x.keys + kItemTiles);
            const unsigned first = runs.of(at), last = runs.of(at + x.keys - 1);
            parts = (int)(last - first + 1) * HALVES;
            more = (int64_t)HALVES * p.n_seqs * p.hq + (int64_t)(first + 1) * 256 + in;
        }
    }
    float top = -CUDART_INF_F, sum = 0.f, o[V] = {};
    for (int k0 = 0; k0 < parts; k0 += 32) {
        const int k = k0 + lane, n = min(32, parts - k0);
        const int64_t at = k < HALVES ? HALVES * row + k : more + (int64_t)(k / HALVES - 1) * 256 + k % HALVES * kTileRows;
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        if (k < parts && LEAN_IN(at, p.parts, p.err)) ml = p.ml[at];
        float now = ml.x;
#pragma unroll
        for (int i = 16; i; i >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, i));
        now = fmaxf(now, top);
        const float ref = now == -CUDART_INF_F ? 0.f : now, old = ex2(top - ref), mine = ex2(ml.x - ref);
        top = now;
        sum = fmaf(sum, old, warp_sum(mine * ml.y));
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= old;
        for (int j0 = 0; j0 < n; j0 += U) {
            Vec<float, V> x[U];
            float f[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                f[j] = __shfl_sync(0xffffffffu, mine, min(j0 + j, 31));
                const int64_t from = __shfl_sync(0xffffffffu, at, min(j0 + j, 31));
                x[j] = Vec<float, V>{};
                if (j0 + j >= n) f[j] = 0.f;
                // (a part without keys has no outputs: they are not looked at)
                if (f[j] != 0.f && LEAN_IN(from, p.parts, p.err)) x[j] = load_vec<float, V>(p.o + from * DP + lane * V);
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf(f[j], x[j].v[i], o[i]);
        }
    }
    const float own = p.own_lse[row] * 1.4426950408889634f;
    if (own != -CUDART_INF_F) {  // (its sum is 1)
        const float now = fmaxf(own, top), ref = now == -CUDART_INF_F ? 0.f : now, old = ex2(top - ref), mine = ex2(own - ref);
        top = now;
        sum = fmaf(sum, old, mine);
        Vec<float, V> x = {};
        if (lane * V < p.dim) x = load_vec<float, V>(p.own_out + row * p.dim + lane * V);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(mine, x.v[i], o[i] * old);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= inv;
    const int64_t to = (int64_t)seq * p.os + (int64_t)head * p.ohs + lane * V;
    if (lane * V < p.dim && LEAN_SPAN(to, V, p.out_extent, p.err)) store_out<V>(p.out, to, p.act, o);
    if (lane == 0 && p.lse) p.lse[row] = natural_lse(top, sum);
}

template <typename C, int DP, int QP, int PP, int NQ>
lean_status launch_prefix(const PrefixMaps &maps, const PrefixArgs &p, int64_t flags, void *stream) {
    static std::atomic<uint64_t> done{0};
    using S = PrefixShape<C, DP, QP, PP, NQ>;
    static_assert(S::kSmemAsked <= 232448, "shared memory");
    auto kern = prefix_kernel<C, DP, QP, PP, NQ>;
    if (!step_ensure_smem(kern, S::kSmemAsked, done)) return LEAN_ERR_CUDA;
    return step_launch(kern, std::min(step_sm_count(), kPrefixMaxCtas), kPrefixThreads, S::kSmemAsked, flags, stream, maps, p);
}
// 16-bit activations whose q is exact in one part (f16 on bf16 caches is not): one part each, two tiles of rows where
// prefixes have more than one; else three parts of q and two of p.
template <typename C, int DP>
lean_status pick_prefix(const PrefixMaps &maps, const PrefixArgs &p, bool two, int64_t flags, void *stream) {
    const bool split = p.act == LEAN_F32 || (p.act == LEAN_F16 && std::is_same<C, __nv_bfloat16>::value);
    if (split) return launch_prefix<C, DP, 3, 3, 1>(maps, p, flags, stream);
    return two ? launch_prefix<C, DP, 1, 1, 2>(maps, p, flags, stream) : launch_prefix<C, DP, 1, 1, 1>(maps, p, flags, stream);
}

}  // namespace
