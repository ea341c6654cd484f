// attend.cu -- lean_paged_attention: the call, and the kernels of attend.cuh for
// caches of 16 bits.
#include "attend.cuh"

namespace {

int att_heads(int64_t hq, int64_t hkv) { return hq / hkv > 8 ? 16 : 8; }
int att_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

}  // namespace

namespace lean {

bool att_sizes_ok(int64_t n_seqs, int64_t hq, int64_t hkv, int64_t dim) {
    return n_seqs > 0 && hkv > 0 && hq > 0 && hq <= 65536 && hq % hkv == 0 && dim > 0 && dim % 8 == 0 &&
           dim <= kAttMaxDim && n_seqs <= INT32_MAX / hq;
}

// What blocks share; in floats, parts of warps and of blocks and what warps fold, of the largest grid.
int64_t att_workspace_bytes(int64_t hq, int64_t hkv, int64_t dim) {
    const int h = att_heads(hq, hkv), d = att_dim(dim);
    return kSharedBytes + (int64_t)kAttMaxCtas * 4 * ((kAttRoomWarps + 2) * part_floats(h, d) + kAttRoomWarps * fold_floats(h, d));
}
void att_workspace(AttArgs &p, void *workspace, bool in8) {
    const int h = p.group > 8 ? 16 : 8, d = att_dim(p.dim), part = part_floats(h, d), warps = att_warps(in8, d, p.group > 8);
    const int64_t floats = (att_workspace_bytes(p.hq, p.hkv, p.dim) - kSharedBytes) / 4;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.shared = reinterpret_cast<Shared *>(ws);
    p.warp_parts = reinterpret_cast<float *>(ws + kSharedBytes);
    // (blocks of more warps have their parts in shared memory, and the folds of 16 warps, heads of 64, that room as well:
    // for 155 blocks, where GB300 has 152 SMs)
    p.warp_extent = warps > kAttRoomWarps ? 0 : (int64_t)kAttMaxCtas * kAttRoomWarps * part;
    p.cta_parts = p.warp_parts + p.warp_extent;
    p.part_extent = (int64_t)kAttMaxCtas * 2 * part;
    p.folds = reinterpret_cast<f32x2 *>(p.cta_parts + p.part_extent);
    p.fold_extent = floats - p.warp_extent - p.part_extent;
    p.most_ctas = (int)std::min<int64_t>(kAttMaxCtas, p.fold_extent / (warps * fold_floats(h, d)));
}

lean_status attend_cache16(const AttArgs &p, bool bf16, int64_t flags, void *stream) {
    return bf16 ? pick_dim<__nv_bfloat16>(p, flags, stream) : pick_dim<__half>(p, flags, stream);
}

}  // namespace lean

extern "C" int64_t lean_paged_attention_workspace_bytes(int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads,
                                                        int64_t head_dim) {
    if (!att_sizes_ok(n_seqs, n_q_heads, n_kv_heads, head_dim)) return -1;
    return att_workspace_bytes(n_q_heads, n_kv_heads, head_dim);
}

extern "C" lean_status lean_paged_attention(const lean_attention_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    const bool in8 = a->cache_dtype == LEAN_I8;  // (the scales' fields are read for such caches only)
    if (!known_dtype(a->act_dtype) || (!in8 && a->cache_dtype != LEAN_BF16 && a->cache_dtype != LEAN_F16) ||
        !step_flags_ok(a->flags))
        return LEAN_ERR_FORMAT;
    if (!att_sizes_ok(a->n_seqs, a->n_q_heads, a->n_kv_heads, a->head_dim) || a->window < 0 || a->n_pages <= 0 ||
        a->n_pages > INT32_MAX || a->page_size <= 0 || a->table_width <= 0 ||
        a->table_width > INT32_MAX / a->page_size || a->table_stride < a->table_width)
        return LEAN_ERR_SHAPE;
    if (in8 && (a->head_dim % 16 || a->scale_page_stride < 0 || a->scale_place_stride < 0 || a->scale_head_stride < 0))
        return LEAN_ERR_SHAPE;
    if (!a->q || !a->k_cache || !a->v_cache || !a->block_table || !a->seq_lens || !a->out || !a->workspace ||
        (in8 && (!a->k_scales || !a->v_scales)))
        return LEAN_ERR_NULL;
    const int64_t strides[] = {a->q_stride, a->q_head_stride, a->out_stride, a->out_head_stride, a->page_stride,
                               a->place_stride, a->cache_head_stride};
    for (int64_t s : strides) {
        if (s < 0) return LEAN_ERR_SHAPE;
        if (s % 8) return LEAN_ERR_ALIGN;
    }
    if (in8 && ((a->page_stride | a->place_stride | a->cache_head_stride) % 16 || !step_aligned(a->k_scales, 4) ||
                !step_aligned(a->v_scales, 4)))
        return LEAN_ERR_ALIGN;
    if (!step_aligned(a->q, 16) || !step_aligned(a->k_cache, 16) || !step_aligned(a->v_cache, 16) ||
        !step_aligned(a->out, 16) || !step_aligned(a->block_table, 4) || !step_aligned(a->seq_lens, 4) ||
        !step_aligned(a->lse, 4) || !step_aligned(a->workspace, 256))
        return LEAN_ERR_ALIGN;
    const int64_t group = a->n_q_heads / a->n_kv_heads, tiles = group > 8 ? (group + 15) / 16 : 1;
    if ((a->table_width * a->page_size / kUnit + 2 + kAttItemUnits) * a->n_seqs * a->n_kv_heads * tiles > UINT32_MAX)
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
    p.act = p.out_act = (int)a->act_dtype;
    att_workspace(p, a->workspace, in8);
    if (in8) {
        p.k_scales = a->k_scales;
        p.v_scales = a->v_scales;
        p.scale_page = a->scale_page_stride;
        p.scale_place = a->scale_place_stride;
        p.scale_hs = a->scale_head_stride;
        p.scale_extent = (a->n_pages - 1) * a->scale_page_stride + (a->page_size - 1) * a->scale_place_stride +
                         (a->n_kv_heads - 1) * a->scale_head_stride + 1;
    }
    p.scale_log2 = (float)(a->scale * 1.4426950408889634);
    p.cache_extent = (a->n_pages - 1) * a->page_stride + (a->page_size - 1) * a->place_stride +
                     (a->n_kv_heads - 1) * a->cache_head_stride + a->head_dim;
    p.q_extent = (a->n_seqs - 1) * a->q_stride + (a->n_q_heads - 1) * a->q_head_stride + a->head_dim;
    p.out_extent = (a->n_seqs - 1) * a->out_stride + (a->n_q_heads - 1) * a->out_head_stride + a->head_dim;
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    return in8 ? attend_cache8(p, a->flags, stream) : attend_cache16(p, a->cache_dtype == LEAN_BF16, a->flags, stream);
}
