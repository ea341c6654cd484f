// kv_pages.cu -- lean_kv_pages: block tables, slot maps and the ring of free
// pages from the sequences' lengths.
//
// Three prefix sums over the sequences (new tokens, pages taken, pages given
// back) say where everything goes; after that every token and every page is
// independent.  The sums are cheap next to a launch (512 sequences: two trips
// through one block), so every block of the grid takes them for itself, over
// chunks of one sequence per thread, and then writes its share of the chunk's
// tokens and pages: one launch, no block waits for another.  Block 0 also
// writes what there is one of per sequence.  Inputs are never written (but for
// table and ring entries that no block reads), so the blocks need no order.
//
// Measured (GB300, calls in a graph): 64 sequences growing by a token 6.4 us, 509
// growing by 255000 tokens together 11.3 us.  Latency bounds both: a launch, the
// lengths, three sums with their barriers, the ring, the table.  The chain is longer
// than it has to be: pages taken and pages given back could share a sum, and the
// ring's new state could be left to block 0 after its tokens.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kPagesThreads = 512;
constexpr int kPagesWarps = kPagesThreads / 32;

struct PagesArgs {
    const int32_t *lens, *targets, *ring_state;
    int32_t *table, *ring, *lens_out, *ring_state_out, *status, *starts, *slots, *positions, *seqs;
    int64_t table_stride;
    int n_seqs, page, max_tokens, width, ring_size;
    unsigned *err;
};

// Exclusive prefix sum of v over the block; *total: the whole sum.  part: one
// int64 per warp, free for the next use after the caller's next barrier.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *part, int64_t *total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kPagesWarps; ++i) {
        if (i < warp) before += part[i];
        all += part[i];
    }
    *total = all;
    return before + s - v;
}

// A place in the ring, below two times its size, as one inside it.
__device__ __forceinline__ unsigned around(unsigned at, int size) {
    return at >= (unsigned)size ? at - (unsigned)size : at;
}

__global__ void __launch_bounds__(kPagesThreads) kv_pages_kernel(const PagesArgs p) {
    step_begin();
    __shared__ int64_t part[3][kPagesWarps];
    __shared__ int tok[kPagesThreads + 1];            // first token of the chunk's sequences
    __shared__ int len_s[kPagesThreads];              // length, or -1 - length where the sequence failed
    __shared__ int take_s[kPagesThreads], give_s[kPagesThreads], gives[kPagesThreads];
    // entries of the ring
    auto from_ring = [&](unsigned at) { return LEAN_IN(at, p.ring_size, p.err) ? p.ring[at] : -1; };
    const int head = p.ring_state[0], count = p.ring_state[1];
    const bool ring_ok = head >= 0 && head < p.ring_size && count >= 0 && count <= p.ring_size;
    // running sums over the chunks; int64: lengths of failed sequences count among the tokens
    int64_t tokens = 0, taken = 0, given = 0;
    // pages that really moved: up to the last sequence that got or gave any
    int64_t took = 0, gave = 0;
    const int G = gridDim.x;

    for (int first = 0; first < p.n_seqs; first += kPagesThreads) {
        const int s = first + threadIdx.x;
        const bool have_seq = s < p.n_seqs && LEAN_IN(s, p.n_seqs, p.err);
        const int len = have_seq ? p.lens[s] : 0, target = have_seq ? p.targets[s] : 0;
        int st = !ring_ok || len < 0 || target < 0 ? 4 : 0;
        const int64_t had = len > 0 ? ((int64_t)len + p.page - 1) / p.page : 0;
        const int64_t have = target > 0 ? ((int64_t)target + p.page - 1) / p.page : 0;
        if (st == 0 && (have > p.width || had > p.width)) st = 2;
        // new tokens, whatever becomes of the sequence (its place in the batch is its place)
        const int64_t fresh = len >= 0 && target > len ? (int64_t)target - len : 0;
        int64_t total;
        const int64_t t0 = tokens + block_scan(fresh, part[0], &total);
        tokens += total;
        if (st == 0 && fresh > 0 && t0 + fresh > p.max_tokens) st = 3;
        const int64_t need = st == 0 && have > had ? have - had : 0;
        const int64_t back = st == 0 && had > have ? had - have : 0;
        const int64_t f0 = taken + block_scan(need, part[1], &total);
        taken += total;
        if (need > 0 && f0 + need > count) st = 1;
        const int64_t b0 = given + block_scan(back, part[2], &total);
        given += total;
        if (back > 0 && (int64_t)count + b0 + back > p.ring_size) st = 4;  // more pages than there can be
        const int64_t cap = p.max_tokens;
        tok[threadIdx.x] = (int)(t0 < cap ? t0 : cap);
        if (threadIdx.x == kPagesThreads - 1 || s == p.n_seqs - 1)
            tok[threadIdx.x + 1] = (int)(t0 + fresh < cap ? t0 + fresh : cap);
        len_s[threadIdx.x] = st == 0 ? len : -1 - (len > 0 ? len : 0);
        take_s[threadIdx.x] = (int)(st == 0 && need > 0 ? f0 : 0);
        give_s[threadIdx.x] = (int)(st == 0 && back > 0 ? b0 : 0);
        gives[threadIdx.x] = (int)(st == 0 ? back : 0);
        if (blockIdx.x == 0 && have_seq && LEAN_IN(s, p.n_seqs, p.err)) {
            p.lens_out[s] = st == 0 ? target : len;
            p.status[s] = st;
            p.starts[s] = (int)(t0 < INT32_MAX ? t0 : INT32_MAX);
            if (s == p.n_seqs - 1) p.starts[s + 1] = (int)(t0 + fresh < INT32_MAX ? t0 + fresh : INT32_MAX);
        }
        int64_t m = st == 0 && need > 0 ? f0 + need : 0, r = st == 0 && back > 0 ? b0 + back : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const int64_t um = __shfl_xor_sync(0xffffffffu, m, o), ur = __shfl_xor_sync(0xffffffffu, r, o);
            m = um > m ? um : m;
            r = ur > r ? ur : r;
        }
        __syncthreads();  // the sums' last reads of part are over, and tok.. are written
        if (threadIdx.x % 32 == 0) {
            part[0][threadIdx.x / 32] = m;
            part[1][threadIdx.x / 32] = r;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPagesWarps; ++i) {
            took = part[0][i] > took ? part[0][i] : took;
            gave = part[1][i] > gave ? part[1][i] : gave;
        }

        // tokens of the chunk, over the threads of the grid
        const int n = p.n_seqs - first < kPagesThreads ? p.n_seqs - first : kPagesThreads;
        const int from = tok[0], to = tok[n];
        // (Four neighbours a thread where there are more than threads: one search, mostly one page and one 16-byte store
        // for them, 12.1 -> 11.1 us at 255000 tokens; else one, since a decode step's neighbours are of different
        // sequences, whose pages would be looked up one after the other.)
        const int K = to - from > G * kPagesThreads ? 4 : 1;
        for (int64_t i4 = (int64_t)from / K * K + K * ((int64_t)blockIdx.x * kPagesThreads + threadIdx.x); i4 < to;
             i4 += (int64_t)K * G * kPagesThreads) {
            int lo = 0, hi = n;  // the last sequence that begins at or before the first of them
            const int64_t at = i4 > from ? i4 : from;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tok[mid] <= at) lo = mid;
                else hi = mid;
            }
            int slot[4], position[4], seq[4], page_known = -1, seq_known = -1, id = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t i = i4 + k;
                slot[k] = -1;
                position[k] = 0;
                seq[k] = -1;
                if (i < from || i >= to || k >= K) continue;
                while (lo + 1 < n && tok[lo + 1] <= i) ++lo;
                const bool ok = len_s[lo] >= 0;
                const int had_len = ok ? len_s[lo] : -1 - len_s[lo];
                const int pos = had_len + (int)(i - tok[lo]);
                if (ok) {
                    const int page_at = pos / p.page, in = pos - page_at * p.page;
                    if (page_at != page_known || lo != seq_known) {
                        page_known = page_at;
                        seq_known = lo;
                        const int had_pages = (int)(((int64_t)had_len + p.page - 1) / p.page);
                        const int64_t entry = (int64_t)(first + lo) * p.table_stride + page_at;
                        if (!LEAN_IN(entry, (int64_t)(p.n_seqs - 1) * p.table_stride + p.width, p.err)) continue;
                        if (page_at < had_pages) {
                            id = p.table[entry];
                        } else {
                            id = from_ring(around((unsigned)head + take_s[lo] + page_at - had_pages, p.ring_size));
                            // a new page begins with a new token: that one enters it in the table
                            if (in == 0) p.table[entry] = id;
                        }
                    }
                    // (a page that is none, or whose slots pass 31 bits, is no place in any cache)
                    const int64_t at_slot = (int64_t)id * p.page + in;
                    if (id >= 0 && at_slot < INT32_MAX) slot[k] = (int)at_slot;
                    else atomicOr(p.err, kErrSlot);
                }
                position[k] = pos;
                seq[k] = first + lo;
            }
            auto put = [&](int32_t *to_, const int(&v)[4]) {
                if (!to_ || !LEAN_SPAN(at, (i4 + K < to ? i4 + K : to) - at, p.max_tokens, p.err)) return;
                if (K == 4 && i4 >= from && i4 + 4 <= to && ((uintptr_t)to_ & 15) == 0) {
                    *reinterpret_cast<int4 *>(to_ + i4) = make_int4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < K && i4 + k >= from && i4 + k < to) to_[i4 + k] = v[k];
                }
            };
            put(p.slots, slot);
            put(p.positions, position);
            put(p.seqs, seq);
        }
        // pages given back, a warp per sequence over the whole grid
        const int lane = threadIdx.x % 32;
        for (int k = blockIdx.x * kPagesWarps + threadIdx.x / 32; k < n; k += G * kPagesWarps) {
            const int g = gives[k];
            if (g == 0) continue;
            const int had_len = len_s[k];
            const int had_pages = (int)(((int64_t)had_len + p.page - 1) / p.page);
            const int64_t entry = (int64_t)(first + k) * p.table_stride + had_pages - g;
            const unsigned tail = around((unsigned)head + count, p.ring_size) + give_s[k];
#pragma unroll 4
            for (int j = lane; j < g; j += 32)
                if (LEAN_IN(entry + j, (p.n_seqs - 1) * p.table_stride + p.width, p.err) &&
                    LEAN_IN(around(tail + j, p.ring_size), p.ring_size, p.err))
                    p.ring[around(tail + j, p.ring_size)] = p.table[entry + j];
        }
        __syncthreads();
    }
    // the unused end of the batch (a limit without maps may be far past any batch)
    const int64_t used = p.slots || p.positions || p.seqs ? min(tokens, (int64_t)p.max_tokens) : p.max_tokens;
    for (int64_t i = used + (int64_t)blockIdx.x * kPagesThreads + threadIdx.x; i < p.max_tokens;
         i += (int64_t)G * kPagesThreads) {
        if (!LEAN_IN(i, p.max_tokens, p.err)) break;
        if (p.slots) p.slots[i] = -1;
        if (p.positions) p.positions[i] = 0;
        if (p.seqs) p.seqs[i] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.ring_state_out[0] = ring_ok ? (int)around((unsigned)(head + took), p.ring_size) : head;
        p.ring_state_out[1] = ring_ok ? (int)(count - took + gave) : count;
    }
}

}  // namespace

extern "C" lean_status lean_kv_pages(const lean_kv_pages_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!step_flags_ok(a->flags)) return LEAN_ERR_FORMAT;
    const int64_t big = INT32_MAX;  // (of sequences half: a chunk past the last one still has to be counted in 32 bits)
    if (a->n_seqs <= 0 || a->page_size <= 0 || a->max_tokens < 0 || a->table_width <= 0 ||
        a->table_stride < a->table_width || a->ring_size <= 0 || a->n_seqs > big / 2 || a->page_size > big ||
        a->max_tokens > big || a->table_stride > big || a->ring_size > big)
        return LEAN_ERR_SHAPE;
    // (blocks read the inputs while others write the outputs)
    if (a->lens_out && (a->lens_out == a->lens || a->lens_out == a->targets)) return LEAN_ERR_SHAPE;
    if (a->ring_state_out && a->ring_state_out == a->ring_state) return LEAN_ERR_SHAPE;
    if (!a->lens || !a->targets || !a->block_table || !a->free_ring || !a->ring_state || !a->lens_out ||
        !a->ring_state_out || !a->status || !a->token_starts)
        return LEAN_ERR_NULL;
    const void *all[] = {a->lens, a->targets, a->block_table, a->free_ring, a->ring_state, a->lens_out,
                         a->ring_state_out, a->status, a->token_starts, a->slots, a->positions, a->token_seqs};
    for (const void *q : all)
        if (!step_aligned(q, 4)) return LEAN_ERR_ALIGN;
    PagesArgs p = {a->lens, a->targets, a->ring_state, a->block_table, a->free_ring, a->lens_out,
                   a->ring_state_out, a->status, a->token_starts, a->slots, a->positions, a->token_seqs,
                   a->table_stride, (int)a->n_seqs, (int)a->page_size, (int)a->max_tokens, (int)a->table_width,
                   (int)a->ring_size, nullptr};
    p.err = error_word();
    if (!p.err) return LEAN_ERR_CUDA;
    // a block for every 512 tokens or 16 sequences, and one block per SM at most
    const int64_t grid = std::min<int64_t>(step_sm_count(),
                                           std::max<int64_t>((a->max_tokens + kPagesThreads - 1) / kPagesThreads,
                                                             (a->n_seqs + kPagesWarps - 1) / kPagesWarps));
    return step_launch(kv_pages_kernel, std::max<int64_t>(grid, 1), kPagesThreads, 0, a->flags, stream, p);
}
