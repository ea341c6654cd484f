// prefix.cu -- lean_prefix_attention: the call, and the kernels of prefix.cuh for
// caches of 16 bits.
#include "prefix.cuh"

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

}  // namespace

namespace lean {

// The caches as tensors in boxes of prefix_box() places (8 or more: rows of a tile lie in groups of 8; in 8 bits what a
// stage of the ring holds at most); none where a stride is 0 between rows that are not one.  16-bit rows are copied to where the matrix
// instructions read them, rows in 8 bits as they lie.
PrefixMaps prefix_maps(const PrefixArgs &p, PrefixCache type) {
    PrefixMaps m = {};
    const bool in8 = type == PrefixCache::kI8;
    const int box = prefix_box(p.page, !in8 ? kTileKeys : p.dim <= 64 ? 64 : 32);
    const EncodeTiled encode = encode_tiled();
    if (box == 0 || !encode || (p.page > 1 && p.place_stride == 0) || (p.hkv > 1 && p.cache_hs == 0) ||
        (p.n_pages > 1 && p.page_stride == 0))
        return m;
    const int64_t strides[3] = {p.place_stride, p.cache_hs, p.page_stride};
    cuuint64_t bytes[3];
    for (int i = 0; i < 3; ++i) {
        if (strides[i] >= (int64_t)1 << 38) return m;
        bytes[i] = strides[i] ? (in8 ? 1 : 2) * strides[i] : 16;
    }
    const cuuint64_t dims[4] = {(cuuint64_t)p.dim, (cuuint64_t)p.page, (cuuint64_t)p.hkv, (cuuint64_t)p.n_pages};
    const cuuint32_t boxes[4] = {in8 && p.dim > 64 ? 128u : 64u, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    const CUtensorMapDataType types[] = {CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                         CU_TENSOR_MAP_DATA_TYPE_UINT8};
    const void *from[2] = {p.k, p.v};
    CUtensorMap *to[2] = {&m.k, &m.v};
    for (int i = 0; i < 2; ++i)
        if (encode(to[i], types[(int)type], 4, const_cast<void *>(from[i]), dims, bytes, boxes, steps,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, in8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return m;
    m.box = box;
    return m;
}

lean_status prefix_cache16(const PrefixArgs &p, bool bf16, bool two, int64_t flags, void *stream) {
    const PrefixMaps maps = prefix_maps(p, bf16 ? PrefixCache::kBf16 : PrefixCache::kF16);
    if (bf16)
        return p.dim <= 64 ? pick_prefix<__nv_bfloat16, 64>(maps, p, two, flags, stream)
                           : pick_prefix<__nv_bfloat16, 128>(maps, p, two, flags, stream);
    return p.dim <= 64 ? pick_prefix<__half, 64>(maps, p, two, flags, stream)
                       : pick_prefix<__half, 128>(maps, p, two, flags, stream);
}

}  // namespace lean

namespace {

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
int prefix_dim(int64_t dim) { return dim <= 64 ? 64 : 128; }

bool prefix_sizes_ok(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim, int64_t n_prefixes) {
    return att_sizes_ok(n_seqs, hq, hkv, dim) && dim <= 128 && n_prefixes > 0 && n_prefixes <= n_seqs &&
           n_seqs <= (INT32_MAX - 512) / (hq / hkv);
}

// ns of an SM for 16 of a sequence's own tokens (16-bit and fp32 activations, caches of 16 and 8 bits, heads of up to 64
// and 128), and for a tile of keys (one tile of rows, two, one with q and p in parts), where an SM has many of them; GB300.
// Measured with up to eight query heads a kv head.
constexpr float kUnitNs[2][2][2] = {{{90, 165}, {80, 145}}, {{100, 190}, {103, 187}}};
constexpr float kTileNs[3][2][2] = {{{1050, 1250}, {1800, 3100}}, {{1250, 1700}, {2400, 3400}}, {{1950, 4100}, {2750, 5800}}};
// Of a unit of more than eight query heads a kv head, two for each thread (96 sequences with up to 500 tokens on prefixes of
// up to 16384, 12 heads a kv head, counted like the others and by this: 4 kv heads of 64 bf16 47.8 and 49.1 us, in 8 bits
// 87.0 and 71.3, fp32 q 103 and 88; 2 of 128 47.2 and 37.8, 65.4 and 66.0, 116 and 94; prefixes of up to 2000 12 to 25%
// less; by 2 about the same).
constexpr float kWideUnit = 1.5f;

// The workspace's parts: that of attend.cuh, rows' first parts, sequences' own results, maxima and sums, outputs.
struct PrefixRoom {
    int64_t first, own_out, own_lse, ml, o, bytes, parts;
};
PrefixRoom prefix_room(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim) {
    PrefixRoom r;
    const int64_t rows = n_seqs * hq;
    r.parts = 2 * rows + kPrefixMaxCtas * 256;
    r.first = up256(att_workspace_bytes(hq, hkv, dim));
    r.own_out = r.first + up256(rows * 8);
    r.own_lse = r.own_out + up256(rows * dim * 4);
    r.ml = r.own_lse + up256(rows * 4);
    r.o = r.ml + up256(r.parts * 8);
    r.bytes = r.o + r.parts * prefix_dim(dim) * 4;
    return r;
}

}  // namespace

extern "C" int64_t lean_prefix_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                                         int64_t head_dim, int64_t n_prefixes) {
    if (!prefix_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim, n_prefixes)) return -1;
    return prefix_room(n_seqs, n_q_heads, n_kv_heads, head_dim).bytes;
}

extern "C" lean_status lean_prefix_attention(const lean_prefix_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    const bool in8 = a->cache_dtype == LEAN_I8;
    if (!known_dtype(a->act_dtype) || (!in8 && a->cache_dtype != LEAN_BF16 && a->cache_dtype != LEAN_F16) ||
        !step_flags_ok(a->flags))
        return LEAN_ERR_FORMAT;
    if (!prefix_sizes_ok(a->n_seqs, a->n_q_heads, a->n_kv_heads, a->head_dim, a->n_prefixes) || a->n_pages <= 0 ||
        a->n_pages > INT32_MAX || a->page_size <= 0 || a->table_width <= 0 || a->table_width > INT32_MAX / a->page_size ||
        a->table_stride < a->table_width || a->prefix_width <= 0 ||
        a->prefix_width > (INT32_MAX - kTileKeys) / a->page_size ||  // (a tile's end is counted in 32 bits)
        a->prefix_stride < a->prefix_width)
        return LEAN_ERR_SHAPE;
    if (in8 && (a->head_dim % 16 || a->scale_page_stride < 0 || a->scale_place_stride < 0 || a->scale_head_stride < 0))
        return LEAN_ERR_SHAPE;
    if (!a->q || !a->k_cache || !a->v_cache || !a->prefix_table || !a->prefix_lens || !a->seq_starts || !a->block_table ||
        !a->seq_lens || !a->out || !a->workspace || (in8 && (!a->k_scales || !a->v_scales)))
        return LEAN_ERR_NULL;
    const int64_t act_strides[] = {a->q_stride, a->q_head_stride, a->out_stride, a->out_head_stride};
    const int64_t cache_strides[] = {a->page_stride, a->place_stride, a->cache_head_stride};
    for (int64_t s : act_strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        if (s % 8) return LEAN_ERR_ALIGN;
    }
    for (int64_t s : cache_strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        if (s % (in8 ? 16 : 8)) return LEAN_ERR_ALIGN;
    }
    const void *on16[] = {a->q, a->k_cache, a->v_cache, a->out}, *on4[] = {a->prefix_table, a->prefix_lens, a->seq_starts,
                                                                           a->block_table, a->seq_lens, a->lse};
    for (const void *x : on16)
        if (!step_aligned(x, 16)) return LEAN_ERR_ALIGN;
    for (const void *x : on4)
        if (!step_aligned(x, 4)) return LEAN_ERR_ALIGN;
    if (!step_aligned(a->workspace, 256) || (in8 && (!step_aligned(a->k_scales, 4) || !step_aligned(a->v_scales, 4))))
        return LEAN_ERR_ALIGN;
    const int64_t group = a->n_q_heads / a->n_kv_heads, tiles = group > 8 ? (group + 15) / 16 : 1;
    if ((a->table_width * a->page_size / kUnit + 2 + kAttItemUnits) * a->n_seqs * a->n_kv_heads * tiles > UINT32_MAX)
        return LEAN_ERR_SHAPE;  // attend.cuh counts units of sequences' own tokens in 32 bits
    // as prefix.cuh its items' tiles: a prefix's sequences fill at least all but one of its tiles of rows
    const int64_t columns = (a->prefix_width * a->page_size / kTileKeys + 1 + item_tiles(in8)) * a->n_kv_heads;
    if (columns > UINT32_MAX / (a->n_seqs * group / kTileRows + a->n_prefixes)) return LEAN_ERR_SHAPE;
    const PrefixRoom room = prefix_room(a->n_seqs, a->n_q_heads, a->n_kv_heads, a->head_dim);
    if (a->workspace_bytes < room.bytes) return LEAN_ERR_SHAPE;
    uint8_t *const ws = static_cast<uint8_t *>(a->workspace);
    unsigned *const err = error_word();
    if (!err) return LEAN_ERR_CUDA;

    AttArgs own = {};
    own.q = a->q;
    own.k = a->k_cache;
    own.v = a->v_cache;
    own.out = ws + room.own_out;
    own.lse = reinterpret_cast<float *>(ws + room.own_lse);
    own.table = a->block_table;
    own.lens = a->seq_lens;
    own.qs = a->q_stride;
    own.qhs = a->q_head_stride;
    own.os = a->n_q_heads * a->head_dim;
    own.ohs = a->head_dim;
    own.page_stride = a->page_stride;
    own.place_stride = a->place_stride;
    own.cache_hs = a->cache_head_stride;
    own.table_stride = a->table_stride;
    own.n_pages = a->n_pages;
    own.n_seqs = (int)a->n_seqs;
    own.hq = (int)a->n_q_heads;
    own.hkv = (int)a->n_kv_heads;
    own.group = (int)group;
    own.tiles = (int)tiles;
    own.dim = (int)a->head_dim;
    own.page = (int)a->page_size;
    own.paged = a->page_size >= kUnit;
    own.whole = a->page_size % kUnit == 0;
    own.width = (int)a->table_width;
    own.act = (int)a->act_dtype;
    own.out_act = LEAN_F32;
    own.scale_log2 = (float)(a->scale * 1.4426950408889634);
    own.cache_extent = (a->n_pages - 1) * a->page_stride + (a->page_size - 1) * a->place_stride +
                       (a->n_kv_heads - 1) * a->cache_head_stride + a->head_dim;
    own.q_extent = (a->n_seqs - 1) * a->q_stride + (a->n_q_heads - 1) * a->q_head_stride + a->head_dim;
    own.out_extent = a->n_seqs * a->n_q_heads * a->head_dim;
    own.err = err;
    att_workspace(own, ws, in8);
    if (in8) {
        own.k_scales = a->k_scales;
        own.v_scales = a->v_scales;
        own.scale_page = a->scale_page_stride;
        own.scale_place = a->scale_place_stride;
        own.scale_hs = a->scale_head_stride;
        own.scale_extent = (a->n_pages - 1) * a->scale_page_stride + (a->page_size - 1) * a->scale_place_stride +
                           (a->n_kv_heads - 1) * a->scale_head_stride + 1;
    }

    PrefixArgs p = {};
    p.q = own.q;
    p.k = own.k;
    p.v = own.v;
    p.k_scales = own.k_scales;
    p.v_scales = own.v_scales;
    p.table = a->prefix_table;
    p.qs = own.qs;
    p.qhs = own.qhs;
    p.page_stride = own.page_stride;
    p.place_stride = own.place_stride;
    p.cache_hs = own.cache_hs;
    p.scale_page = own.scale_page;
    p.scale_place = own.scale_place;
    p.scale_hs = own.scale_hs;
    p.table_stride = a->prefix_stride;
    p.n_pages = own.n_pages;
    p.n_prefixes = (int)a->n_prefixes;
    p.n_seqs = own.n_seqs;
    p.hq = own.hq;
    p.hkv = own.hkv;
    p.group = own.group;
    p.dim = own.dim;
    p.page = own.page;
    p.width = (int)a->prefix_width;
    p.act = own.act;
    p.scale_log2 = own.scale_log2;
    p.first = reinterpret_cast<int2 *>(ws + room.first);
    p.ml = reinterpret_cast<float2 *>(ws + room.ml);
    p.o = reinterpret_cast<float *>(ws + room.o);
    p.parts = room.parts;
    p.own_out = static_cast<const float *>(own.out);
    p.own_lse = own.lse;
    p.out = a->out;
    p.lse = a->lse;
    p.os = a->out_stride;
    p.ohs = a->out_head_stride;
    p.cache_extent = own.cache_extent;
    p.scale_extent = own.scale_extent;
    p.q_extent = own.q_extent;
    p.out_extent = (a->n_seqs - 1) * a->out_stride + (a->n_q_heads - 1) * a->out_head_stride + a->head_dim;
    p.err = err;

    // Two tiles of rows where a prefix has more than one of them on average (below that the second would mostly be empty);
    // from what the host knows, so that a large prefix among many small ones has single tiles as well.
    const bool bf16 = a->cache_dtype == LEAN_BF16;
    const bool two = !splits(p.act, bf16) && a->n_seqs * group > a->n_prefixes * kTileRows;
    // Both kernels run beside one another: by the times of their parts (own_blocks()).
    PrefixList list = {};
    list.starts = a->seq_starts;
    list.lens = a->prefix_lens;
    list.n = p.n_prefixes;
    list.n_seqs = p.n_seqs;
    list.group = p.group;
    list.hkv = p.hkv;
    list.rows = two ? 2 * kTileRows : kTileRows;
    list.most = (int)(a->prefix_width * a->page_size);
    list.sms = (unsigned)std::min(step_sm_count(), kPrefixMaxCtas);
    list.own_most = (unsigned)att_grid(own, att_warps(in8, prefix_dim(a->head_dim), group > 8));
    list.item_tiles = item_tiles(in8);
    const int wide = prefix_dim(a->head_dim) == 128;
    list.unit_ns = kUnitNs[a->act_dtype == LEAN_F32][in8][wide] * (group > 8 ? kWideUnit : 1.f);
    list.tile_ns = kTileNs[splits(p.act, bf16) ? 2 : two][in8][wide];
    p.list = own.list = list;
    p.own_lens = a->seq_lens;
    p.own_most = (int)(a->table_width * a->page_size);
    p.own_groups = own.hkv * own.tiles;
    p.own_heads = group > 8 ? 16 : 8;
    p.own_tiles = own.tiles;
    p.own_grid = (int)list.own_most;
    p.shared = own.shared;
    p.cta_parts = own.cta_parts;
    p.part_extent = own.part_extent;
    // Sequences' own tokens first: blocks of the prefixes' kernel begin beside theirs.
    lean_status st = in8 ? attend_beside8(own, a->flags, stream) : attend_beside16(own, bf16, a->flags, stream);
    if (st != LEAN_OK) return st;
    constexpr int64_t early = LEAN_FLAG_EARLY_WEIGHTS;
    st = in8 ? prefix_cache8(p, two, early, stream) : prefix_cache16(p, bf16, two, early, stream);
    if (st != LEAN_OK) return st;
    const int64_t grid = (a->n_seqs * a->n_q_heads + 7) / 8;
    if (p.dim <= 64) return step_launch(two ? prefix_sum_kernel<64, 2> : prefix_sum_kernel<64, 1>, grid, 256, 0, early, stream, p);
    return step_launch(two ? prefix_sum_kernel<128, 2> : prefix_sum_kernel<128, 1>, grid, 256, 0, early, stream, p);
}
