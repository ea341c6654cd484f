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
// tensor cores take, 128 rows at a time, and a prefix's keys and values are read
// once for 256 rows (128 where q and p are in three parts or prefixes have no more
// than 128 rows on average).  HBM would bound calls below about 290 rows a prefix, the
// tensor cores those above it; what does is the softmax between the two products
// (below).
//
//   - Work is a list of items: 256 (or 128) rows of a prefix and kv head, over tiles
//     of 128 keys.  Every block takes an equal run of tiles, whatever the prefixes'
//     lengths and numbers of sequences are, and leaves maxima, sums and outputs of
//     its part of an item in the workspace.  Sequences' own tokens are attended at
//     the same time on SMs of their own, as many as their share of the work asks for
//     (own_blocks(); one kernel after the other: 61 us in place of 47.8, 96 sequences
//     on 32768 tokens, 16/2 heads of 128); a last kernel adds up the parts of both.
//   - A block has two groups of 128 threads, a thread to a row, that turn S into P;
//     four warps that issue matrix instructions; and four that bring keys and values
//     into swizzled tiles, two of each under way.  With two tiles of rows (NQ = 2) each
//     group has its own 128 rows and all keys; with one, both have the same rows and
//     every other tile of keys.
//   - S and O lie in tensor memory, S in buffers of 64 keys, as many as fit (three for
//     heads of 64, two for heads of 128), so that products for the next keys run while a
//     group works on these.  P replaces S and is read as an operand from there.
//   - The reference of the exponentials only moves where p would become too large (for
//     f16, or on average above the 2^8 of attend.cuh): p is computed with the last one,
//     the sums say whether it held, and no maximum is looked for (77.6 -> 72.3 us, 256
//     sequences on 16384 tokens, 32/4 heads of 64).
//   - O is summed over 2048 keys in tensor memory, then added to the part in the
//     workspace in fp32: the tensor cores cut off what is small next to their
//     accumulator.  With p in three parts it is summed over 64 keys only and added in
//     registers (heads of 128 spill 180 bytes a thread in f16, 344 in bf16, 668 in 8
//     bits, of 64 84 to 124; with one part of p all spill 32 to 92).
//   - q is copied where the operands' type holds it; else it is scaled by a power of
//     two as in attend.cuh and split in three parts of that type, and p in three: fp32
//     out, and f16 out of bf16 caches.  16-bit out has p in one part, which errs by
//     half a step (2^-8 of itself in bf16, as out itself is rounded).
//   - Caches in 8 bits become f16 on the way into shared memory (exact); scores are
//     multiplied by the keys' scales, p by the values', relative to the largest of 32.
//
// Measured (GB300, in a graph, floors by bytes or tensor operations in brackets): 96
// sequences on 32768 tokens, 16/2 heads of 128, bf16, 44 us (13.5); 256 on 16384,
// 32/4 heads of 64, f16, 67 (18.0); 240 on 12 prompts in 8 bits, 91 (8.5); four on
// 2000, fp32 q, 19.3 (0.4).  What bounds heads of 64 is a group's time for 64 keys: 1300
// cycles (8 bits: 2200) in which two warps a scheduler wait for tensor memory, 64
// exponentials and their sum, one after the other; issue slots are 45% busy (8 bits
// 51%), the tensor pipe 28% (15%).  Heads of 128 (1700 cycles, 35%) wait for that pipe's
// operands from shared memory as well.  About 6 us pass before the first scores, 5 to 7
// in the last kernel.
#pragma once
#include <cuda.h>

#include <type_traits>

#include "../../include/lean_cache.h"
#include "attend.cuh"
#include "tensor.cuh"

namespace lean {

constexpr int kHalfKeys = 64;  // of a tile
constexpr int kPrefixMaxCtas = 160;
// Threads of a block (in 8 bits a fifth group of four warps issues copies), and the registers that each of
// its groups of 128 has after the start: together no more than the block is launched with, as many for each thread as the
// compiler gave the kernel (128, in 8 bits 96).  setmaxnreg waits forever for more than that, so that a launch asks first.
constexpr int prefix_threads(bool in8) { return in8 ? 640 : 512; }
struct PrefixRegs {
    int rows, loaders, mma, issuer;
};
constexpr PrefixRegs prefix_regs(bool in8, int pp) {
    return in8 ? (pp == 1 ? PrefixRegs{136, 72, 80, 56} : PrefixRegs{160, 56, 56, 48})
               : (pp == 1 ? PrefixRegs{152, 120, 88, 0} : PrefixRegs{192, 72, 56, 0});
}
constexpr bool prefix_regs_fit(int of_thread, bool in8, int pp) {
    const PrefixRegs r = prefix_regs(in8, pp);
    return (2 * r.rows + r.loaders + r.mma + r.issuer) * 128 <= of_thread * prefix_threads(in8);
}
static_assert(prefix_regs_fit(128, false, 1) && prefix_regs_fit(128, false, 3) && prefix_regs_fit(96, true, 1) &&
                  prefix_regs_fit(96, true, 3),
              "registers of a block");
// The kernel as it was built, asked once per device.
template <typename Kern>
inline bool prefix_regs_there(Kern kern, bool in8, int pp, std::atomic<uint64_t> &done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    cudaFuncAttributes built;
    if (cudaFuncGetAttributes(&built, kern) != cudaSuccess || !prefix_regs_fit(built.numRegs, in8, pp)) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}
// Halves of tiles whose products are summed in tensor memory before they are added in fp32 (one part of p): what is below
// 2^-24 of a sum is cut off when it is added, 16 keys at a time, so that a row errs by 2^-16 of its largest sum at most.
constexpr int kFoldHalves = 32;

struct PrefixArgs {
    const void *q, *k, *v;
    const float *k_scales, *v_scales;
    const int32_t *table;
    PrefixList list;
    int64_t qs, qhs, page_stride, place_stride, cache_hs, scale_page, scale_place, scale_hs, table_stride, n_pages;
    int n_prefixes, n_seqs, hq, hkv, group, dim, page, width, act;
    // sequences' own tokens: lengths, the most that their pages can hold, groups of query heads of a sequence
    const int32_t *own_lens;
    int own_most, own_groups;
    float scale_log2;
    // workspace: maxima and sums, outputs, of the parts that begin an item, by row (and half, with one tile of rows), then
    // those that go on with one, by block
    int2 *first;  // of a row with a prefix: the block that begins its item, and how many parts it has
    float2 *ml;
    float *o;
    int64_t parts;  // how many there are
    // a sequence's own tokens, and what comes out
    const float *own_out, *own_lse;
    const Shared *shared;     // items that blocks share, and their parts (attend.cuh)
    const float *cta_parts;
    int64_t part_extent;
    int own_heads, own_tiles, own_grid;
    void *out;
    float *lse;
    int64_t os, ohs;
    int64_t cache_extent, scale_extent, q_extent, out_extent;  // elements, for the checked build
    unsigned *err;
};

// Keys and values as tensors [page][head][place][dim] for the copy engine, in boxes of `box` places by 64 dimensions (in 8
// bits all of them; box 0: pages whose size no multiple of 8 divides, or strides that it does not take).
struct PrefixMaps {
    CUtensorMap k, v;
    int box;
};

// As many places, up to `most`, as a tile and every page are whole numbers of; 0 if fewer than 8.
inline int prefix_box(int page, int most) {
    int box = most;
    while (page % box) box /= 2;
    return box < 8 ? 0 : box;
}

enum class PrefixCache { kBf16, kF16, kI8 };
PrefixMaps prefix_maps(const PrefixArgs &p, PrefixCache type);

lean_status prefix_cache16(const PrefixArgs &p, bool bf16, bool two, int64_t flags, void *stream);
lean_status prefix_cache8(const PrefixArgs &p, bool two, int64_t flags, void *stream);

}  // namespace lean

namespace {

constexpr unsigned kErrPrefixWait = 4u;  // as the tensor-core products: a bounded wait ran out
constexpr uint64_t kPrefixWaitNs = 2000000000ull;

// A list of units cut into equal runs, none of them empty (blocks past the units have none): where a block's run begins,
// and the block that has a unit.
struct Runs {
    unsigned each, rest, blocks;  // the first `rest` blocks have one more
    __device__ __forceinline__ Runs(unsigned total, unsigned n) {
        blocks = min(max(1u, total), n);
        each = total / blocks;
        rest = total - each * blocks;
    }
    __device__ __forceinline__ unsigned begin(unsigned b) const { return each * b + min(b, rest); }
    __device__ __forceinline__ unsigned of(unsigned u) const {
        const unsigned longer = rest * (each + 1);
        return u < longer ? u / (each + 1) : rest + (u - longer) / each;
    }
};

// A block's run of the list, item by item; every role walks it by itself.
struct Walk {
    int i;                       // prefix
    Prefix x;
    unsigned off;                // place in the prefix's part of the list
    unsigned left;               // of the run
    unsigned unit, begin;        // the run's next unit, the first one of the part below
    // the part of an item that comes next: keys' tiles from..to-1
    int kvh, tile, from, to;
    // false: no more
    __device__ __forceinline__ bool next(const PrefixArgs &p) {
        while (left > 0) {
            while (off >= x.cost(p.list)) {
                off -= x.cost(p.list);
                if (++i >= p.n_prefixes) return false;
                x = open_prefix(p.list, i, p.err);
            }
            const int each = x.keys + p.list.item_tiles;
            const int item = (int)(off / each);
            from = (int)(off - (unsigned)item * each);
            const int take = (int)min(left, (unsigned)(each - from));
            to = min(from + take, x.keys);
            begin = unit;
            off += take;
            left -= take;
            unit += take;
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
    // caches in 8 bits: runs of rows as they lie in the cache, keys' then values' of a tile, kRawDepth for each of the four
    // warps that issue them in turn
    static constexpr int kRawRows = DP == 64 ? 64 : 32, kRawBytes = kRawRows * DP, kRuns = 2 * kTileKeys / kRawRows;
    static constexpr int kRawDepth = DP == 64 ? 2 : 1, kRaw = kIn8 ? 4 * kRawDepth : 0;
    static constexpr int kRawAt = kScaleAt + (kIn8 ? 4 * 2 * kTileKeys * 4 : 0);  // (a multiple of 128)
    static constexpr int kBars = kRawAt + kRaw * kRawBytes;
    static constexpr int kSmem = kBars + 640;
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
    uint64_t rows_full[2];                                  // a tile's rows' places are there
    uint64_t scales_full[4];
    uint64_t raw_full[8], raw_empty[8];                     // runs of rows in 8 bits are there, were used
    uint64_t tile_ready[4], tile_done[4];                   // what is known of a tile in 8 bits, and that it was taken
    uint64_t last;                                          // every matrix instruction is done
    uint32_t tmem;
    int dead;            // a wait ran out: everyone leaves
    int value_exp[4][4]; // exponents of the largest value scales of 32 keys, of four tiles
    int tile_whole[4];   // tiles in 8 bits: whether their rows come through the ring
    int start_i;         // the run's first prefix and place in it
    unsigned start_off;
};
static_assert(sizeof(PrefixBars) <= 640, "room for the barriers");

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

// The compiler lays what is behind such a condition away from the code around it.
__device__ __forceinline__ bool seldom(bool b) { return __builtin_expect(b, 0); }

// Wait for a phase; false: it, or another wait of the block, ran out.
__device__ __forceinline__ bool phase_wait(PrefixBars &b, uint64_t *bar, uint32_t parity, unsigned *err) {
    if (!seldom(!mbar_try_wait(bar, parity))) return true;
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

// q of a warp's 32 rows, lane l's at q_at (-1: none), as it is into a tile of q, with the signs turned by `flip`; read as
// below.
template <typename S, int DP, typename Mine, typename Ready>
__device__ __forceinline__ bool copy_q(const PrefixArgs &p, int64_t q_at, uint8_t *tile, int row0, int lane, uint32_t flip, Mine mine, Ready ready) {
    constexpr int LPR = DP / 8, RPI = 32 / LPR;
    const int c = lane % LPR;
    uint4 x[LPR];
#pragma unroll
    for (int i = 0; i < LPR; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, q_at, i * RPI + lane / LPR);
        x[i] = make_uint4(0, 0, 0, 0);
        if (mine(i) && at >= 0 && 8 * c < p.dim && LEAN_SPAN(at + 8 * c, 8, p.q_extent, p.err))
            x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at + 8 * c);
    }
    if (!ready()) return false;
#pragma unroll
    for (int i = 0; i < LPR; ++i) {
        const int row = row0 + i * RPI + lane / LPR;
        if (mine(i))
            *reinterpret_cast<uint4 *>(tile + c / 8 * S::kChunkBytes + row * 128 + ((c % 8) ^ (row & 7)) * 16) =
                make_uint4(x[i].x ^ flip, x[i].y ^ flip, x[i].z ^ flip, x[i].w ^ flip);
    }
    return true;
}

// q of a warp's 32 rows, lane l's at q_at (-1: none): scaled by a power of two and split in parts into tiles of q, E
// elements to a lane (16 bytes of them), so that a row is read by neighbouring lanes.  Rows whose turn is not `mine` are
// looked at but not written.  Returns the largest element of the lane's own row, as bits.
template <typename S, typename T, int DP, int QP, int E, typename Mine, typename Ready>
__device__ __forceinline__ uint32_t load_q(const PrefixArgs &p, int64_t q_at, uint8_t *tiles, int row0, int lane, float sign, Mine mine, Ready ready) {
    constexpr int LPR = DP / E, RPI = 32 / LPR, B = LPR < 8 ? LPR : 8;  // lanes of a row, rows at a time, times under way
    const int c = lane % LPR;
    uint32_t own = 0;
    bool ok = true;
#pragma unroll 1
    for (int it0 = 0; it0 < LPR; it0 += B) {
        uint4 x[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int64_t at = __shfl_sync(0xffffffffu, q_at, (it0 + i) * RPI + lane / LPR);
            x[i] = make_uint4(0, 0, 0, 0);
            if (at >= 0 && E * c < p.dim && LEAN_SPAN(at + E * c, E, p.q_extent, p.err))
                x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.q) + (at + E * c) * (16 / E));
        }
        if (it0 == 0) ok = ready();
        if (!ok) return 0xffffffffu;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int it = it0 + i;
            float f[E];
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (E == 4) {
                    f[k] = __uint_as_float(u[k]);
                } else {
                    RawPair<false> pair;
                    pair.v = u[k];
                    const float2 v = pair.get(p.act);
                    f[2 * k % E] = v.x;
                    f[(2 * k + 1) % E] = v.y;
                }
            }
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < E; ++k) top = fmaxf(top, fabsf(f[k]));
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t of_own = __float_as_uint(__shfl_sync(0xffffffffu, top, lane % RPI * LPR));
            if (lane / RPI == it) own = of_own;
            if (!mine(it)) continue;
            const int e = (int)(__float_as_uint(top) >> 23);
            const int fe = e == 0 || e == 255 ? 127 : min(253, max(1, 254 + PartRange<T>::kLiftQ - e));
            const float up = sign * __uint_as_float((uint32_t)fe << 23);
#pragma unroll
            for (int k = 0; k < E; ++k) f[k] *= up;
            const int row = row0 + it * RPI + lane / LPR, piece = E == 8 ? c : c / 2;
            uint8_t *to = tiles + piece / 8 * S::kChunkBytes + row * 128 + ((piece % 8) ^ (row & 7)) * 16 + (E == 8 ? 0 : c % 2 * 8);
#pragma unroll
            for (int part = 0; part < QP; ++part) {
                uint32_t a[E / 2];
#pragma unroll
                for (int k = 0; k < E / 2; ++k) a[k] = take_part<T>(f[2 * k], f[2 * k + 1]);
                if constexpr (E == 8) *reinterpret_cast<uint4 *>(to + part * S::kTileBytes) = make_uint4(a[0], a[1], a[2], a[3]);
                else *reinterpret_cast<uint2 *>(to + part * S::kTileBytes) = make_uint2(a[0], a[1]);
            }
        }
    }
    return own;
}

template <typename C, int DP, int QP, int PP, int NQ>
__global__ void __launch_bounds__(prefix_threads(sizeof(C) == 1), 1) prefix_kernel(const __grid_constant__ PrefixMaps maps, const PrefixArgs p) {
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
    // (No wait: the kernel before is attend.cuh's for this call, whose blocks let this one begin only when what came
    // before them is done, and nothing here is read or written there.  What they leave is waited for at the end, for the
    // kernel after this one.)
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;

    // ---- this block's run of the list
    unsigned *const before = reinterpret_cast<unsigned *>(smem);  // (the tiles' room, unused yet)
    constexpr int THREADS = prefix_threads(IN8);
    constexpr PrefixRegs REGS = prefix_regs(IN8, PP);
    auto own_len = [&](int i) { return i < p.n_seqs && LEAN_IN(i, p.n_seqs, p.err) ? p.own_lens[i] : 0; };
    const int len_ahead = own_len(threadIdx.x);
    const int per = (p.n_prefixes + THREADS - 1) / THREADS;
    const int lo = min(p.n_prefixes, (int)threadIdx.x * per), hi = min(p.n_prefixes, lo + per);
    unsigned mine = 0;
    for (int i = lo; i < hi; ++i) mine += open_prefix(p.list, i, p.err).cost(p.list);
    unsigned incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) before[warp] = incl;
    unsigned own = 0;  // units of sequences' own tokens, as attend.cuh counts them
    for (int i = threadIdx.x; i < p.n_seqs; i += THREADS) {
        const int len = min(max(i == (int)threadIdx.x ? len_ahead : own_len(i), 0), p.own_most);
        own += (unsigned)(max(1, len / kUnit + (len % kUnit != 0)) + kAttItemUnits) * p.own_groups;
    }
    own = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) before[32 + warp] = own;
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
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars.scales_full[i], 4);
            mbar_init(&bars.tile_ready[i], 4);
            mbar_init(&bars.tile_done[i], 4);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars.raw_full[i], 1);
            mbar_init(&bars.raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&bars.rows_full[i], 4);
        mbar_init(&bars.q_full, 8);
        mbar_init(&bars.q_free, 10);
        mbar_init(&bars.last, 4);
        bars.dead = 0;
        bars.start_i = -1;
        fence_mbar_init();
    }
    __syncthreads();
    unsigned begins = incl - mine, total = 0;
    own = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) begins += before[i];
        total += before[i];
        own += before[32 + i];
    }
    // (blocks past these find the SMs of attend.cuh's kernel free, when it is done, and have nothing to do)
    const Runs runs(total, max(1u, gridDim.x - min(gridDim.x, own_blocks(p.list, own, total))));
    const bool has_run = blockIdx.x < runs.blocks;
    const unsigned run_lo = has_run ? runs.begin(blockIdx.x) : 0, run_hi = has_run ? runs.begin(blockIdx.x + 1) : 0;
    if (run_lo < run_hi && begins <= run_lo && run_lo < begins + mine) {  // one thread's
        unsigned off = run_lo - begins;
        int i = lo;
        for (;; ++i) {
            const unsigned c = open_prefix(p.list, i, p.err).cost(p.list);
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
    w.unit = run_lo;
    if (w.left > 0) w.x = open_prefix(p.list, w.i, p.err);

    if (warp < 8) {
        // ---- scores to probabilities, products to outputs: a thread has a row
        regs_up<REGS.rows>();
        const int g = warp / 4, r = threadIdx.x % kTileRows;
        const uint32_t lanes = (uint32_t)(warp % 4) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t s_group = tmem + lanes + S::scores(g, 0), o_at = tmem + lanes + S::outputs(g);
        unsigned buf = 0, buf_phase = 0;  // the buffer of the next half tile, and its phase
        unsigned tiles_before = 0;  // of the run, by loader's count (scales)
        bool ok = true;
        uint32_t q_phase = 1;  // (the phase before the first counts as done)
        while (ok && w.next(p)) {
            // this row: where its q lies and its part goes (-1: the item has no such row)
            const int row = w.tile * ROWS + (NQ == 2 ? g * kTileRows : 0) + r;
            int64_t part_at = -1, q_at = -1;
            if (row < (int64_t)w.x.count * p.group) {
                const int seq = w.x.first + row / p.group, head = w.kvh * p.group + row % p.group;
                const int64_t first = (int64_t)seq * p.hq + head;
                q_at = (int64_t)seq * p.qs + (int64_t)head * p.qhs;
                part_at = w.from == 0 ? (NQ == 2 ? first : 2 * first + g)
                                      : (NQ == 2 ? 1 : 2) * (int64_t)p.n_seqs * p.hq + (int64_t)blockIdx.x * 256 + g * kTileRows + r;
                if (!LEAN_IN(part_at, p.parts, p.err)) part_at = -1;
                if (w.from == 0 && (NQ == 2 || g == 0) && LEAN_IN(first, (int64_t)p.n_seqs * p.hq, p.err)) {
                    p.first[first] = make_int2(blockIdx.x, (int)(runs.of(w.begin + w.x.keys - 1) - blockIdx.x) + 1);
                }
            }
            // q of this warp's rows; the scale of this one's scores
            float zs;
            {
                const float sign = p.scale_log2 < 0.f ? -1.f : 1.f;  // (so that the largest product is the largest score)
                auto ready = [&]() { return warp_wait(bars, &bars.q_free, q_phase, p.err); };
                uint8_t *const tiles = q_tiles + (NQ == 2 ? g * QP * S::kTileBytes : 0);
                auto turn = [&](int it) { return NQ == 2 || it % 2 == g; };  // (both groups have the same rows: half each)
                const int row0 = r - lane;
                zs = fabsf(p.scale_log2);
                if (QP == 1 && p.act == (BF16 ? LEAN_BF16 : LEAN_F16)) {  // the operands' own type: nothing to split or scale
                    ok = copy_q<S, DP>(p, q_at, tiles, row0, lane, sign < 0.f ? 0x80008000u : 0u, turn, ready);
                } else {
                    const uint32_t top = QP == 3 && p.act == LEAN_F32
                                             ? load_q<S, T, DP, QP, 4>(p, q_at, tiles, row0, lane, sign, turn, ready)
                                             : load_q<S, T, DP, QP, 8>(p, q_at, tiles, row0, lane, sign, turn, ready);
                    ok = top != 0xffffffffu;
                    const int e = (int)(top >> 23 & 0xff);
                    const int fe = e == 0 || e == 255 ? 127 : min(253, max(1, 254 + PartRange<T>::kLiftQ - e));
                    zs *= __uint_as_float((uint32_t)(254 - fe) << 23);
                }
                if (!ok) break;
                q_phase ^= 1;
                if (zs == 0.f) zs = 1.17549435e-38f;  // (masked scores are -inf times this)
                smem_to_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full);
            }
            // What p is multiplied with, as a power of two, and the sum of 32 of them up to which the references hold.  bf16
            // has fp32's range, but so do the sums of p v: as far as attend.cuh lets scores rise (up to a sum of 2^40 values
            // above 2^80 came out infinite where scores rose by 24 nats).  f16 ends at 2^-25 (half its smallest step) and
            // 65504: in one part p is lifted so that 32 equal ones stay below that and references seldom move (what is lost
            // of one is 2^-34 of the largest), in more as in attend.cuh.
            constexpr float kLog2Lift = BF16 ? 0.f : PP == 1 ? 9.f : 13.f;
            constexpr float kDown = BF16 ? 1.f : PP == 1 ? 1.f / 512 : 1.f / 8192;
            constexpr float kMostSum = BF16 ? 8192.f : 65504.f;
            static_assert(!BF16 || kMostSum == 32 << (int)PartRange<T>::kSlack, "as attend.cuh's");
            float m = -CUDART_INF_F, l = 0.f;
            int v_ref = 1;
            // The references m and v_ref: what they make of exponents and sums of 32 keys each.
            float shift[2], back[2];
            auto refer_scales = [&](const int *exps) {
                // values' scales lie in 0.5..1 times 2^(exponent of the largest of 32 - 126); sums are relative to
                // 2^(v_ref - 126); what is below 2^-60 of the largest may count as 2^-60 of it.  Larger ones than the
                // reference's make larger p, whose sums say whether they fit.
                const float up = kLog2Lift - (m == -CUDART_INF_F ? 0.f : m);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int below = min(v_ref - exps[c], 60);
                    shift[c] = up - (float)below;
                    back[c] = __uint_as_float((uint32_t)(127 + max(below, -60)) << 23);
                }
                return max(exps[0], exps[1]) <= v_ref + 60;
            };
            // New references for a half whose largest score is `top`, and what is multiplied with the sums and the outputs
            // so far.
            auto refer = [&](float top, const int *exps, float &fall, float &o_fall) {
                // (m as in attend.cuh: within kSlack of the largest score so far)
                const float mn = top - m <= PartRange<T>::kSlack ? m : top;
                fall = o_fall = ex2(m - (mn == -CUDART_INF_F ? 0.f : mn));
                m = mn;
                if (IN8) {
                    const int now = max(v_ref, max(exps[0], exps[1]));
                    o_fall *= __uint_as_float((uint32_t)max(0, 127 + v_ref - now) << 23);
                    v_ref = now;
                    refer_scales(exps);
                } else {
                    shift[0] = shift[1] = kLog2Lift - (m == -CUDART_INF_F ? 0.f : m);
                    back[0] = back[1] = 1.f;
                }
            };
            auto size = [&]() { return IN8 ? kDown * __uint_as_float((uint32_t)(v_ref + 1) << 23) : kDown; };
            // Halves of tiles in turn (of the last one the second may have no keys; keys that are not there score -inf).
            int t = w.from + (NQ == 2 ? 0 : g), half = 0, limit = 0;  // limit: keys of the half that are there, or more
            uint32_t s_at = 0;
            const float *ks = nullptr, *vs = nullptr;
            const int *exps = nullptr;
            auto scores_wait = [&]() {
                limit = w.x.len - t * kTileKeys - half * kHalfKeys;
                bool got = true;
                if (IN8) {
                    const unsigned n = tiles_before + (t - w.from), slot = n % 4;
                    exps = bars.value_exp[slot] + 2 * half;
                    ks = scales + slot * 2 * kTileKeys + half * kHalfKeys;
                    vs = ks + kTileKeys;
                    if (half == 0) got = warp_wait(bars, &bars.scales_full[slot], n / 4 & 1, p.err);
                }
                s_at = s_group + buf * S::kWidth;
                got = got && warp_wait(bars, &bars.s_full[g][buf], buf_phase, p.err);
                tm_after();
                return got;
            };
            auto publish = [&]() {
                tm_wait_st();
                tm_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[g][buf]);
                if (++buf == NB) {
                    buf = 0;
                    buf_phase ^= 1;
                }
            };
            auto products_wait = [&]() {  // of all that were published
                const bool first = buf == 0;
                const bool got = warp_wait(bars, &bars.o_full[g][first ? NB - 1 : buf - 1], first ? buf_phase ^ 1 : buf_phase, p.err);
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
                unsigned in_run = 0;  // halves of this part of the item so far
                bool folded = false;  // the part has some already, with reference m_part
                float m_part = -CUDART_INF_F;
                while (t < w.to) {
                    ok = scores_wait();
                    if (!ok) break;
                    uint32_t x[2][32];
                    tm_ld64(s_at, x);
                    if (IN8) {
#pragma unroll
                        for (int i = 0; i < kHalfKeys; i += 4) {
                            const float4 k = *reinterpret_cast<const float4 *>(ks + i);
                            uint32_t *z = &x[i / 32][i % 32];
                            const float2 a = unpack2(mul2(pack2(__uint_as_float(z[0]), __uint_as_float(z[1])), pack2(k.x, k.y)));
                            const float2 b = unpack2(mul2(pack2(__uint_as_float(z[2]), __uint_as_float(z[3])), pack2(k.z, k.w)));
                            z[0] = __float_as_uint(a.x);
                            z[1] = __float_as_uint(a.y);
                            z[2] = __float_as_uint(b.x);
                            z[3] = __float_as_uint(b.y);
                        }
                    }
                    if (seldom(limit < kHalfKeys)) {
#pragma unroll
                        for (int i = 0; i < kHalfKeys; ++i)
                            if (i >= limit) x[i / 32][i % 32] = 0xff800000u;
                    }
                    float sums[2];  // of the first 32 keys and of the others
                    auto exponentials = [&]() {
                        const f32x2 zs2 = pack2(zs, zs);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t part[16];
                            const f32x2 shift2 = pack2(shift[c], shift[c]);
                            f32x2 sum2 = 0;
                            float4 v;
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 a = unpack2(fma2(pack2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])), zs2, shift2));
                                float2 e = make_float2(ex2(a.x), ex2(a.y));
                                sum2 = add2(sum2, pack2(e.x, e.y));
                                if (IN8) {
                                    if (i % 4 == 0) v = *reinterpret_cast<const float4 *>(vs + 32 * c + i);
                                    e = unpack2(mul2(pack2(e.x, e.y), i % 4 == 0 ? pack2(v.x, v.y) : pack2(v.z, v.w)));
                                }
                                part[i / 2] = take_part<T>(e.x, e.y);
                            }
                            const float2 sum = unpack2(sum2);
                            sums[c] = sum.x + sum.y;
                            tm_st16(s_at + S::part(c, 0), part);  // (over the scores, which are in registers)
                        }
                    };
                    // With the references of the half before, as long as no p is too large; in the first half, and where
                    // they have to move, the largest score is looked for and p is computed again.
                    bool moves = in_run == 0;
                    if (!seldom(moves)) {
                        if (IN8) moves = !refer_scales(exps);
                        exponentials();
                        moves = moves || !(fmaxf(sums[0], sums[1]) <= kMostSum);
                    }
                    float fall = 1.f;
                    if (seldom(__any_sync(0xffffffffu, moves))) {
                        float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                        for (int i = 0; i < kHalfKeys; ++i) tops[i % 4] = fmaxf(tops[i % 4], __uint_as_float(x[i / 32][i % 32]));
                        float o_fall;
                        refer(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * zs, exps, fall, o_fall);
                        exponentials();
                        if (in_sum > 0) {  // what is there is rescaled
                            ok = products_wait();
                            if (!ok) break;
#pragma unroll
                            for (int c = 0; c < DP; c += 32) {
                                uint32_t y[32];
                                tm_ld32(o_at + c, y);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t z[16];
#pragma unroll
                                    for (int i = 0; i < 16; ++i) z[i] = __float_as_uint(__uint_as_float(y[16 * h + i]) * o_fall);
                                    tm_st16(o_at + c + 16 * h, z);
                                }
                            }
                        }
                    }
                    publish();
                    l = fmaf(l, fall, IN8 ? sums[0] * back[0] + sums[1] * back[1] : sums[0] + sums[1]);
                    ++in_run;
                    advance_half();
                    if (seldom(++in_sum == kFoldHalves || t >= w.to)) {
                        ok = products_wait();
                        if (!ok) break;
                        const float f = ex2(m_part - (m == -CUDART_INF_F ? 0.f : m)), up = size();
                        float *o = p.o + part_at * DP;
#pragma unroll
                        for (int c = 0; c < DP; c += 32) {
                            uint32_t y[32];
                            tm_ld32(o_at + c, y);
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
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float z = __uint_as_float(x[i]);
                            if (IN8) z *= ks[c + i];
                            tops[i % 4] = fmaxf(tops[i % 4], z);
                        }
                    }
                    float fall, o_fall;
                    refer(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * zs, exps, fall, o_fall);
                    const f32x2 zs2 = pack2(zs, zs);
                    f32x2 sum2[2] = {0, 0};  // of the first 32 keys and of the others
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t x[32];
                        tm_ld32(s_at + 32 * c, x);
                        uint32_t part[PP][16];
                        const f32x2 shift2 = pack2(shift[c], shift[c]);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            f32x2 z = pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                            if (IN8) z = mul2(z, *reinterpret_cast<const f32x2 *>(ks + 32 * c + i));
                            const float2 a = unpack2(fma2(z, zs2, shift2));
                            float2 e = make_float2(ex2(a.x), ex2(a.y));
                            sum2[c] = add2(sum2[c], pack2(e.x, e.y));
                            if (IN8) e = unpack2(mul2(pack2(e.x, e.y), *reinterpret_cast<const f32x2 *>(vs + 32 * c + i)));
#pragma unroll
                            for (int k = 0; k < PP; ++k) part[k][i / 2] = take_part<T>(e.x, e.y);
                        }
#pragma unroll
                        for (int k = 0; k < PP; ++k) tm_st16(s_at + S::part(c, k), part[k]);  // over scores already used
                    }
                    publish();
                    const float2 sum0 = unpack2(sum2[0]), sum1 = unpack2(sum2[1]);
                    l = fmaf(l, fall, (sum0.x + sum0.y) * back[0] + (sum1.x + sum1.y) * back[1]);
                    ok = products_wait();
                    if (!ok) break;
                    const f32x2 fall2 = pack2(o_fall, o_fall);
#pragma unroll
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t x[32];
                        tm_ld32(o_at + c, x);
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
        regs_down<REGS.loaders>();
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
            // Runs of rows as they lie in the cache, in the ring that the last four warps fill, become f16 (codes are
            // exact in it) in the operands' tiles; tiles that are not whole come row by row through registers.  (240
            // sequences on 12 prompts 96 us, with the sum as it is now 91; rows looked up and loaded by these threads 103,
            // boxes issued between their conversions 126.)
            constexpr int PR = DP / 16, RUNS = S::kRuns, PIECES = S::kRawRows * PR / 128;  // 16-byte pieces: of a row, of a thread
            uint8_t *const raw = smem + S::kRawAt;
            auto convert = [&](uint8_t *tile, int row, int c, uint4 x) {  // piece c of a row
                const uint32_t u[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
                uint8_t *to = tile + c / 4 * S::kChunkBytes + row * 128;
                *reinterpret_cast<uint4 *>(to + ((2 * c % 8) ^ (row & 7)) * 16) =
                    make_uint4(codes_f16<0x4140>(u[0]), codes_f16<0x4342>(u[0]), codes_f16<0x4140>(u[1]), codes_f16<0x4342>(u[1]));
                *reinterpret_cast<uint4 *>(to + ((2 * c % 8 + 1) ^ (row & 7)) * 16) =
                    make_uint4(codes_f16<0x4140>(u[2]), codes_f16<0x4342>(u[2]), codes_f16<0x4140>(u[3]), codes_f16<0x4342>(u[3]));
            };
            unsigned used = 0;  // runs
            while (ok && w.next(p)) {
                for (int kt = w.from; ok && kt < w.to; ++kt, ++n) {
                    ok = warp_wait(bars, &bars.tile_ready[n % 4], n / 4 & 1, p.err);
                    if (!ok) break;
                    uint8_t *const tiles[2] = {k_tiles + n % KS * S::kTileBytes, v_tiles + n % VS * S::kTileBytes};
                    if (bars.tile_whole[n % 4]) {
#pragma unroll 1
                        for (int run = 0; run < RUNS; ++run) {
                            const unsigned times = used / 4, slot = used % 4 + 4 * (times % S::kRawDepth);
                            if (run == 0 && n >= KS) ok = warp_wait(bars, &bars.k_empty[n % KS], (n / KS - 1) & 1, p.err);
                            if (run == RUNS / 2 && n >= VS) ok = ok && warp_wait(bars, &bars.v_empty[n % VS], (n / VS - 1) & 1, p.err);
                            ok = ok && warp_wait(bars, &bars.raw_full[slot], times / S::kRawDepth & 1, p.err);
                            if (!ok) break;
                            uint4 x[PIECES];
#pragma unroll
                            for (int i = 0; i < PIECES; ++i)
                                x[i] = *reinterpret_cast<const uint4 *>(raw + slot * S::kRawBytes + (i * 128 + t) * 16);
#pragma unroll
                            for (int i = 0; i < PIECES; ++i)
                                convert(tiles[run >= RUNS / 2], run % (RUNS / 2) * S::kRawRows + (i * 128 + t) / PR, t % PR, x[i]);
                            const bool last = run % (RUNS / 2) == RUNS / 2 - 1;
                            if (last) smem_to_async();
                            arrive(&bars.raw_empty[slot]);
                            if (last && lane == 0) mbar_arrive(run < RUNS / 2 ? &bars.k_full[n % KS] : &bars.v_full[n % VS]);
                            ++used;
                        }
                    } else {
                        const int64_t *const offs = row_off + (n & 1) * kTileKeys;
                        if (n >= KS) ok = warp_wait(bars, &bars.k_empty[n % KS], (n / KS - 1) & 1, p.err);
                        if (n >= VS) ok = ok && warp_wait(bars, &bars.v_empty[n % VS], (n / VS - 1) & 1, p.err);
                        if (!ok) break;
#pragma unroll 1
                        for (int kv = 0; kv < 2; ++kv) {
                            const int8_t *cache = static_cast<const int8_t *>(kv ? p.v : p.k);
#pragma unroll 1
                            for (int i = 0; i < PR; ++i) {
                                const int c = t % PR, row = (i * 128 + t) / PR;
                                const int64_t o = offs[row];
                                uint4 x = make_uint4(0, 0, 0, 0);
                                if (o >= 0 && 16 * c < p.dim) x = *reinterpret_cast<const uint4 *>(cache + o + 16 * c);
                                convert(tiles[kv], row, c, x);
                            }
                            smem_to_async();
                            arrive(kv ? &bars.v_full[n % VS] : &bars.k_full[n % KS]);
                        }
                    }
                    if (ok) arrive(&bars.tile_done[n % 4]);
                }
            }
        } else {
            // Whole tiles in pages that the cache has: boxes of a page each, by the copy engine; a lane issues its own
            // page's.  Others, whose last rows have to be zeros: row by row, with cp.async.
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
            while (ok && w.next(p)) {
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
        if (!ok) {  // a wait ran out: copies on their way land before the block's memory is another's
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000) {}
        }
        for (unsigned j = n > KS ? n - KS : 0; ok && j < n; ++j) ok = warp_wait(bars, &bars.k_empty[j % KS], j / KS & 1, p.err);
        for (unsigned j = n > VS ? n - VS : 0; ok && j < n; ++j) ok = warp_wait(bars, &bars.v_empty[j % VS], j / VS & 1, p.err);
    } else if (warp < 16) {
        regs_down<REGS.mma>();
        if (lane == 0) {
            // ---- matrix instructions: warps 12 and 13 issue the groups' scores, 14 and 15 their products.  (One thread
            // needs about 110 cycles for an instruction that runs for 64: with one warp for all of them 240 sequences on 12
            // prompts in 8 bits took 105 us, with four 91.)
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
                while (ok && w.next(p)) {
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
                            // (the smallest parts first: a sum is cut off relative to what it has come to)
#pragma unroll
                            for (int part = QP - 1; part >= 0; --part)
#pragma unroll
                                for (int s = 0; s < DP / 16; ++s) {
                                    const uint32_t in = (s / 4 * S::kChunkBytes + s % 4 * 32) >> 4;
                                    if (s < steps)
                                        tm_mma_ss(d, q_lower + (part * S::kTileBytes >> 4) + in, b + in, kTileUpper, idesc,
                                                  part < QP - 1 || s > 0);
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
                while (ok && w.next(p) && !(ALL && g == 1)) {
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
                            for (int part = PP - 1; part >= 0; --part)
#pragma unroll
                                for (int s = 0; s < kHalfKeys / 16; ++s)
                                    tm_mma_ts(d, a + S::part(s / 2, part) + s % 2 * 8, b + s * (2048 >> 4), kTileUpper, idesc,
                                              part < PP - 1 || s > 0 || add);
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
    if constexpr (IN8) {
        if (warp >= 16) {
            // ---- what is known of a tile, and its rows into the ring: each of four warps has 32 rows' scales and every
            // fourth run of the tile's rows, in stages of the ring of its own.  A lane looks up the page of a box of rows,
            // where pages do not fit boxes that of its row, a tile ahead.
            regs_down<REGS.issuer>();
            const int mine = warp - 16, box = maps.box, boxes = box > 0 ? kTileKeys / box : 0, lg = box > 0 ? 31 - __clz(box) : 0;
            uint8_t *const raw = smem + S::kRawAt;
            const int first_tok = boxes > 0 ? lane * box : 32 * mine + lane;  // of a tile: the lane's box's, or its row's
            const int page_step = kTileKeys / p.page, place_step = kTileKeys - page_step * p.page;
            unsigned n = 0, sent = 0;  // tiles, runs of this warp
            bool ok = true;
            while (ok && w.next(p)) {
                // the page (of the prefix) and place of the lane's token in the tile that is looked up, and those of the tile
                // at hand
                int page = (w.from * kTileKeys + first_tok) / p.page, place = w.from * kTileKeys + first_tok - page * p.page;
                auto look = [&](int kt) {
                    const int64_t e = (int64_t)w.i * p.table_stride + page;
                    const bool in = (boxes == 0 || lane < boxes) && kt * kTileKeys + first_tok < w.x.len &&
                                    LEAN_IN(e, (int64_t)(p.n_prefixes - 1) * p.table_stride + p.width, p.err);
                    return in ? p.table[e] : 0;
                };
                auto step = [&]() {
                    page += page_step;
                    place += place_step;
                    if (place >= p.page) {
                        place -= p.page;
                        ++page;
                    }
                };
                float sk, sv;
                int64_t off;
                bool whole;
                int id = look(w.from), at_place = place;
                step();
                int next_id = w.from + 1 < w.to ? look(w.from + 1) : 0;
                auto row = [&](int kt) {  // 32 mine + lane of tile kt; its scales under way
                    const int r = 32 * mine + lane, tok = kt * kTileKeys + r;
                    const bool real = id >= 0 && id < p.n_pages;
                    whole = boxes > 0 && kt * kTileKeys + kTileKeys <= w.x.len;
                    bool fits = (boxes > 0 && lane >= boxes) || real;
                    if (boxes > 0 && lane < boxes && real && whole)
                        fits = LEAN_SPAN((int64_t)id * p.page_stride + (int64_t)at_place * p.place_stride + (int64_t)w.kvh * p.cache_hs,
                                         (box - 1) * p.place_stride + p.dim, p.cache_extent, p.err);
                    whole = whole && __all_sync(0xffffffffu, fits);
                    const int of_id = boxes > 0 ? __shfl_sync(0xffffffffu, id, r >> lg) : id;
                    const int of_place = boxes > 0 ? __shfl_sync(0xffffffffu, at_place, r >> lg) + (r & (box - 1)) : at_place;
                    off = -1;
                    sk = 1.f;
                    sv = 0.f;
                    if (tok < w.x.len) {
                        if (of_id < 0 || of_id >= p.n_pages) {
                            off = -2;
                            sk = CUDART_NAN_F;
                            atomicOr(p.err, kErrSlot);
                        } else {
                            if (!whole) {
                                off = (int64_t)of_id * p.page_stride + (int64_t)of_place * p.place_stride + (int64_t)w.kvh * p.cache_hs;
                                if (!LEAN_SPAN(off, p.dim, p.cache_extent, p.err)) off = -1;
                            }
                            const int64_t at = (int64_t)of_id * p.scale_page + (int64_t)of_place * p.scale_place + (int64_t)w.kvh * p.scale_hs;
                            if (LEAN_IN(at, p.scale_extent, p.err)) {
                                sk = p.k_scales[at];
                                sv = p.v_scales[at];
                            }
                        }
                    }
                };
                row(w.from);
                for (int kt = w.from; kt < w.to; ++kt, ++n) {
                    // (with tile n - 2 taken, scores of n - 4 are done with their scales)
                    if (n >= 2) ok = warp_wait(bars, &bars.tile_done[(n - 2) % 4], (n - 2) / 4 & 1, p.err);
                    if (!ok) break;
                    auto send = [&](int run) {
                        const unsigned slot = mine + 4 * (sent % S::kRawDepth), times = sent / S::kRawDepth;
                        if (times > 0 && !warp_wait(bars, &bars.raw_empty[slot], (times - 1) & 1, p.err)) return false;
                        if (lane == 0) mbar_arrive_expect_tx(&bars.raw_full[slot], S::kRawBytes);
                        __syncwarp();
                        const int each = S::kRawRows >> lg, b = lane - run % (S::kRuns / 2) * each;
                        if (b >= 0 && b < each)
                            copy_box(smem_addr(raw + slot * S::kRawBytes + b * box * DP), run < S::kRuns / 2 ? &maps.k : &maps.v, 0,
                                     at_place, w.kvh, id, &bars.raw_full[slot]);
                        ++sent;
                        return true;
                    };
                    if (whole) ok = send(mine);  // (first: it takes longest)
                    if (!ok) break;
                    // the values' scales relative to the largest of 32
                    const uint32_t top = __reduce_max_sync(0xffffffffu, sv > 0.f ? __float_as_uint(sv) : 0u);
                    const int e = min(252, max(1, (int)(top >> 23)));
                    float *const to = scales + n % 4 * 2 * kTileKeys + 32 * mine + lane;
                    to[0] = sk + (sk - sk);  // (an infinite one is NaN, as the scores of such a key are)
                    to[kTileKeys] = sv * __uint_as_float((uint32_t)(253 - e) << 23);
                    if (!whole) row_off[(n & 1) * kTileKeys + 32 * mine + lane] = off;
                    if (lane == 0) {
                        bars.value_exp[n % 4][mine] = e;
                        if (mine == 0) bars.tile_whole[n % 4] = whole;
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars.tile_ready[n % 4]);
                        mbar_arrive(&bars.scales_full[n % 4]);
                    }
                    for (int run = mine + 4; ok && whole && run < S::kRuns; run += 4) ok = send(run);
                    if (!ok) break;
                    if (kt + 1 < w.to) {
                        id = next_id;
                        at_place = place;
                        row(kt + 1);
                        step();
                        if (kt + 2 < w.to) next_id = look(kt + 2);
                    }
                }
            }
            if (!ok) {  // as above
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000) {}
            }
        }
    }
    tm_before();
    __syncthreads();
    if (warp == 12) tm_free(tmem, 512);
    pdl_wait();
}

// Parts of a row, and the sequence's own tokens, added up: a warp to a row.
template <int DP, int NQ>
__global__ void __launch_bounds__(256) prefix_sum_kernel(const PrefixArgs p) {
    // U parts' loads under way in a warp: registers are what limits the warps of an SM (256 sequences on 16384 tokens, heads
    // of 64: six 66.9 us, eight 68.0, 16 71.3, 32 77; 96 on 32768, heads of 128: eight 46.1, 12 43.8, 16 44.3, 20 49)
    constexpr int V = DP / 32, ROWS = NQ * kTileRows, HALVES = NQ == 2 ? 1 : 2, U = DP == 64 ? 6 : 12;
    // (What the call is given is there: this kernel begins after blocks of the one before, and that after all that came
    // before the call.  Every thread waits before it ends, so that this kernel's end implies the end of the ones before.)
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= (int64_t)p.n_seqs * p.hq) {
        pdl_wait();
        return;
    }
    const int seq = (int)(row / p.hq), head = (int)(row % p.hq);
    // its prefix: the last that begins at it or before
    int lo = 0, hi = p.n_prefixes;  // how many begin so: lo..hi
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool so = at < hi && LEAN_IN(at, p.n_prefixes + 1, p.err) && p.list.starts[at] <= seq;
        const int n = __popc(__ballot_sync(0xffffffffu, so));
        if (n == 0) break;
        hi = min(hi, lo + n * step);
        lo += (n - 1) * step + 1;
    }
    Prefix x = {};
    if (lo > 0) x = open_prefix(p.list, lo - 1, p.err);
    pdl_wait();
    // asked for at once: the row's own result, and where its parts lie if it has a prefix
    const float own = p.own_lse[row] * 1.4426950408889634f;
    Vec<float, V> own_out = {};
    if (lane * V < p.dim) own_out = load_vec<float, V>(p.own_out + row * p.dim + lane * V);
    const int2 where = p.first[row];
    Shared shared[kAttMaxCtas / 32];
#pragma unroll
    for (int i = 0; i < kAttMaxCtas / 32; ++i) {
        const int b = 32 * i + lane;
        shared[i] = b < p.own_grid && LEAN_IN(b, kAttMaxCtas, p.err) ? p.shared[b] : Shared{-1, 0};
    }
    int parts = 0;
    int64_t more = 0;  // the first part that goes on
    if (lo > 0) {
        if (seq >= x.first && seq < x.first + x.count && x.keys > 0) {
            const int r = ((seq - x.first) * p.group + head % p.group) % ROWS;
            // (bounds: where seq_starts does not ascend, another prefix's block may have written it, or none)
            parts = min(max(where.y, 0), kPrefixMaxCtas) * HALVES;
            more = (int64_t)HALVES * p.n_seqs * p.hq + (int64_t)(min(max(where.x, 0), kPrefixMaxCtas) + 1) * 256 + r;
        }
    }
    // its own item's parts, if blocks share it (attend.cuh): of the block where it begins, and of the next ones
    const int item = (seq * p.hkv + head / p.group) * p.own_tiles + head % p.group / p.own_heads;
    int own_parts = 0, own_block = 0;
#pragma unroll
    for (int i = 0; i < kAttMaxCtas / 32; ++i) {
        const unsigned hit = __ballot_sync(0xffffffffu, shared[i].item == item);
        if (hit) {
            own_block = 32 * i + __ffs(hit) - 1;
            own_parts = __shfl_sync(0xffffffffu, shared[i].parts, __ffs(hit) - 1);
        }
    }
    float top = -CUDART_INF_F, sum = 0.f, o[V] = {};
    auto rescale = [&](float m) {  // to a reference not below m; what it is
        const float now = fmaxf(m, top), ref = now == -CUDART_INF_F ? 0.f : now, old = ex2(top - ref);
        top = now;
        sum *= old;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= old;
        return ref;
    };
    if (own_parts > 0) {
        const int pf = part_floats(p.own_heads, DP), po = DP + 4;
        for (int k0 = 0; k0 < own_parts; k0 += 8) {
            float2 ml[8];
            Vec<float, V> x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t at = ((int64_t)(own_block + k0 + k) * 2 + (k0 + k == 0)) * pf + (int64_t)(head % p.group % p.own_heads) * po;
                ml[k] = make_float2(-CUDART_INF_F, 0.f);
                x[k] = Vec<float, V>{};
                if (k0 + k < own_parts && LEAN_SPAN(at, po, p.part_extent, p.err)) {
                    ml[k] = *reinterpret_cast<const float2 *>(p.cta_parts + at);
                    x[k] = load_vec<float, V>(p.cta_parts + at + 4 + lane * V);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float w = ex2(ml[k].x - rescale(ml[k].x));
                sum = fmaf(w, ml[k].y, sum);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf(w, x[k].v[i], o[i]);
            }
        }
    } else if (own != -CUDART_INF_F) {  // (its sum is 1)
        const float w = ex2(own - rescale(own));
        sum = w;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = w * own_out.v[i];
    }
    for (int k0 = 0; k0 < parts; k0 += 32) {
        const int k = k0 + lane, n = min(32, parts - k0);
        const int64_t at = k < HALVES ? HALVES * row + k : more + (int64_t)(k / HALVES - 1) * 256 + k % HALVES * kTileRows;
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        if (k < parts && at < p.parts) ml = p.ml[at];
        float now = ml.x;
#pragma unroll
        for (int i = 16; i; i >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, i));
        const float mine = ex2(ml.x - rescale(now));
        sum += warp_sum(mine * ml.y);
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
                if (f[j] != 0.f && from < p.parts) x[j] = load_vec<float, V>(p.o + from * DP + lane * V);
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf(f[j], x[j].v[i], o[i]);
        }
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
    static std::atomic<uint64_t> smem_done{0}, regs_done{0};
    using S = PrefixShape<C, DP, QP, PP, NQ>;
    static_assert(S::kSmemAsked <= 232448, "shared memory");
    auto kern = prefix_kernel<C, DP, QP, PP, NQ>;
    if (!step_ensure_smem(kern, S::kSmemAsked, smem_done) || !prefix_regs_there(kern, S::kIn8, PP, regs_done)) return LEAN_ERR_CUDA;
    return step_launch(kern, std::min(step_sm_count(), kPrefixMaxCtas), prefix_threads(S::kIn8), S::kSmemAsked, flags, stream, maps, p);
}
// Whether q and p are split in parts.
inline bool splits(int act, bool bf16_cache) { return act == LEAN_F32 || (act == LEAN_F16 && bf16_cache); }
// 16-bit activations whose q is exact in one part (f16 on bf16 caches is not): one part each, two tiles of rows where
// prefixes have more than one; else three parts of each.
template <typename C, int DP>
lean_status pick_prefix(const PrefixMaps &maps, const PrefixArgs &p, bool two, int64_t flags, void *stream) {
    if (splits(p.act, std::is_same<C, __nv_bfloat16>::value)) return launch_prefix<C, DP, 3, 3, 1>(maps, p, flags, stream);
    return two ? launch_prefix<C, DP, 1, 1, 2>(maps, p, flags, stream) : launch_prefix<C, DP, 1, 1, 1>(maps, p, flags, stream);
}

}  // namespace
