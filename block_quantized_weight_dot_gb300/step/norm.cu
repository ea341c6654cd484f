// norm.cu -- lean_residual_norm: residual sum, gate and the RMS norms before
// and after a block, one pass over the row.
//
//   u = post_w x / rms(x),  h' = h + alpha gate u,  y = w h' / rms(h')
//   rms(v) = sqrt(mean(v^2) + eps)
//
// Every element of x, h and gate is read once and every element of h' and y
// written once: both sums of squares are taken from registers, so the work is
// bound by HBM (one token: by the launch and two trips through the SM).  A row
// belongs to `tpr` consecutive threads, each with NV vectors of VEC elements,
// loaded before anything is computed with them.
//
// Measured (GB300, calls in a graph): 8192 x 2048 bf16 with gate, norm after and
// fp32 residual 38.1 us, 6.16 TB/s of the 6.78 that a copy reaches; fp32 6.27
// TB/s; one row of 960 fp32 2.1 us.  On odd widths weights and a shared gate are read
// one element at a time: 8192 x 2049 63 us (35 at that rate of a copy), 16000 x 1001 59
// (33); rows past 16384 go by single elements, up to three times: 1024 x 20480 162 (43).
#include "step_common.cuh"

using namespace lean;

namespace {

struct NormArgs {
    const void *x, *h, *gate;
    const float *post_w, *w;
    void *h_out, *y;
    int64_t rows, xs, hs, gs, hos, ys, stride;  // stride: of all buffers, where it is one (SHIFT)
    int width;
    float eps, alpha;
    unsigned *err;
};

constexpr int kNormThreads = 512;  // of a row, at most

// Sum over the tpr threads of a row (whole warps); part: one float per warp of the block, not used for anything else.
__device__ __forceinline__ float row_sum(float v, int tpr, int row_in_block, float *part) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < tpr / 32; ++i) s += part[row_in_block * (tpr / 32) + i];
    return s;
}

// VEC elements as they lie in memory, in whole registers.
template <typename A, int VEC>
struct Raw {
    uint32_t w[(sizeof(A) * VEC + 3) / 4];
    __device__ __forceinline__ void load(const A *p) {
        if (sizeof(A) * VEC >= 16) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(A) * VEC / 16); ++i) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = q.x;
                w[(4 * i + 1) % kWords] = q.y;
                w[(4 * i + 2) % kWords] = q.z;
                w[(4 * i + 3) % kWords] = q.w;
            }
        } else if (sizeof(A) == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    __device__ __forceinline__ float get(int i) const;
    static constexpr int kWords = (sizeof(A) * VEC + 3) / 4;
};
template <typename A>
__device__ __forceinline__ float raw_element(uint32_t w, int half);
template <>
__device__ __forceinline__ float raw_element<float>(uint32_t w, int) { return __uint_as_float(w); }
template <>
__device__ __forceinline__ float raw_element<__nv_bfloat16>(uint32_t w, int half) {
    return __uint_as_float(half ? w & 0xffff0000u : w << 16);
}
template <>
__device__ __forceinline__ float raw_element<__half>(uint32_t w, int half) {
    const __half2 v = *reinterpret_cast<const __half2 *>(&w);
    return half ? __high2float(v) : __low2float(v);
}
template <typename A, int VEC>
__device__ __forceinline__ float Raw<A, VEC>::get(int i) const {
    return raw_element<A>(w[i * sizeof(A) / 4], i & 1);
}

// A vector of a row that may begin before its first element or end past its last one: what is not the row's is 0 and
// not stored.  `there`: false if the buffer has no such vector (checked build).
template <typename A, int VEC>
__device__ __forceinline__ void load_part(Raw<A, VEC> &v, const A *row, int c, int width, bool vector, bool there) {
    if (vector && there) {
        v.load(row + c);
        return;
    }
#pragma unroll
    for (int i = 0; i < Raw<A, VEC>::kWords; ++i) v.w[i] = 0;
    if (!there) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (c + j < 0 || c + j >= width) continue;
        if (sizeof(A) == 4) v.w[j % Raw<A, VEC>::kWords] = reinterpret_cast<const uint32_t *>(row)[c + j];
        else v.w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[c + j] << (j & 1 ? 16 : 0);
    }
}
template <typename A, int VEC>
__device__ __forceinline__ void store_part(A *row, int c, int width, const float *f, bool vector) {
    if (vector) {
        store_vec<A, VEC>(row + c, f);
        return;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        if (c + j >= 0 && c + j < width) row[c + j] = from_f<A>(f[j]);
}

// SHIFT: rows that do not begin on 16 bytes, with one stride for all buffers, so that all of them have vectors at the
// same columns; the first and the last vector of a row are then partial.
template <typename A, typename R, int VEC, int NV, bool SHIFT>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs p, int tpr) {
    step_begin();
    __shared__ float part[2][kNormThreads / 32];
    const int mine = (int)threadIdx.x / tpr, t = threadIdx.x - mine * tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + mine;
    const bool live = row < p.rows;
    const float inv = 1.f / (float)p.width;
    // column of the thread's vector i
    const int shift = SHIFT ? -(int)(row * p.stride % VEC) : 0;
    auto column = [&](int i) { return (t + i * tpr) * VEC + shift; };
    auto whole = [&](int c) { return !SHIFT || (c >= 0 && c + VEC <= p.width); };

    auto inside = [&](int64_t at, bool v, int64_t stride) {  // (a partial vector looks at every element for itself)
        return !v || LEAN_SPAN(at, VEC, (p.rows - 1) * stride + p.width, p.err);
    };

    Raw<A, VEC> xr[NV], gr[NV];
    Raw<R, VEC> hr[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = column(i);
        const bool v = whole(c);
        in[i] = live && c < p.width;
        if (in[i] && p.x)
            load_part(xr[i], static_cast<const A *>(p.x) + row * p.xs, c, p.width, v, inside(row * p.xs + c, v, p.xs));
        if (in[i] && p.h)
            load_part(hr[i], static_cast<const R *>(p.h) + row * p.hs, c, p.width, v, inside(row * p.hs + c, v, p.hs));
        if (in[i] && p.gate)
            load_part(gr[i], static_cast<const A *>(p.gate) + row * p.gs, c, p.width, v && !(SHIFT && p.gs == 0),
                      inside(row * p.gs + c, v, p.gs));
    }
    float post = 1.f;
    if (p.post_w) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i])
#pragma unroll
                for (int j = 0; j < VEC; ++j) s = fmaf(xr[i].get(j), xr[i].get(j), s);
        post = rsqrtf(fmaf(row_sum(s, tpr, mine, part[0]), inv, p.eps));
    }
    float v[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
        const int c = column(i);
        Raw<float, VEC> pw;
        if (p.post_w) load_part(pw, p.post_w, c, p.width, !SHIFT, inside(c, !SHIFT, 0));
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float u = 0.f;
            if (p.x) {
                u = xr[i].get(j);
                if (p.post_w) u = u * post * pw.get(j);
                if (p.gate) u *= gr[i].get(j);
                u *= p.alpha;
            }
            v[i][j] = p.h ? hr[i].get(j) + u : u;
            s = fmaf(v[i][j], v[i][j], s);
        }
        if (p.h_out && inside(row * p.hos + c, whole(c), p.hos))
            store_part<R, VEC>(static_cast<R *>(p.h_out) + row * p.hos, c, p.width, v[i], whole(c));
    }
    if (!p.y) return;
    const float r = rsqrtf(fmaf(row_sum(s, tpr, mine, part[1]), inv, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
        const int c = column(i);
        Raw<float, VEC> wv;
        if (p.w) load_part(wv, p.w, c, p.width, !SHIFT, inside(c, !SHIFT, 0));
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] *= p.w ? r * wv.get(j) : r;
        if (inside(row * p.ys + c, whole(c), p.ys))
            store_part<A, VEC>(static_cast<A *>(p.y) + row * p.ys, c, p.width, v[i], whole(c));
    }
}

// Rows too long for the registers of one block: one block per row, up to three
// passes over it (the later ones from L2).  Nothing is written before the last
// pass, in which each thread reads what it then overwrites, so that h_out may
// be h and y may be x here too.
template <typename A, typename R>
__global__ void __launch_bounds__(kNormThreads) norm_long_kernel(const NormArgs p) {
    step_begin();
    __shared__ float part[2][kNormThreads / 32];
    const int64_t row = blockIdx.x;
    const A *x = p.x ? static_cast<const A *>(p.x) + row * p.xs : nullptr;
    const A *gate = p.gate ? static_cast<const A *>(p.gate) + row * p.gs : nullptr;
    const R *h = p.h ? static_cast<const R *>(p.h) + row * p.hs : nullptr;
    const float inv = 1.f / (float)p.width;
    auto at = [&](const auto *v, int c, int64_t stride) {  // element c of the row
        return LEAN_IN(row * stride + c, (p.rows - 1) * stride + p.width, p.err) ? to_f(v[c]) : 0.f;
    };
    float post = 1.f;
    if (p.post_w) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.width; c += kNormThreads) s = fmaf(at(x, c, p.xs), at(x, c, p.xs), s);
        post = rsqrtf(fmaf(row_sum(s, kNormThreads, 0, part[0]), inv, p.eps));
    }
    auto value = [&](int c) {
        float u = 0.f;
        if (x) {
            u = at(x, c, p.xs);
            if (p.post_w) u = u * post * at(p.post_w, c, 0);
            if (gate) u *= at(gate, c, p.gs);
            u *= p.alpha;
        }
        return h ? at(h, c, p.hs) + u : u;
    };
    float r = 0.f;
    if (p.y) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.width; c += kNormThreads) {
            const float v = value(c);
            s = fmaf(v, v, s);
        }
        r = rsqrtf(fmaf(row_sum(s, kNormThreads, 0, part[1]), inv, p.eps));
    }
    for (int c = threadIdx.x; c < p.width; c += kNormThreads) {
        const float v = value(c);
        if (p.h_out && LEAN_IN(row * p.hos + c, (p.rows - 1) * p.hos + p.width, p.err))
            static_cast<R *>(p.h_out)[row * p.hos + c] = from_f<R>(v);
        if (p.y && LEAN_IN(row * p.ys + c, (p.rows - 1) * p.ys + p.width, p.err))
            static_cast<A *>(p.y)[row * p.ys + c] = from_f<A>(v * (p.w ? r * at(p.w, c, 0) : r));
    }
}

// How a row is cut: nv vectors for each of tpr threads.  Few rows: as many threads as vectors (latency).  Many: the cut
// that leaves the fewest threads idle in the last vector, two or three vectors and 256 threads rather than more (a row
// of 1024 vectors on 512 threads leaves one block an SM, whose barriers nothing hides: 59.8 us at 2048 x 8192 bf16
// against 46.7 on 256).
struct Cut {
    int nv, tpr;
};
Cut cut_row(int64_t nvec, const int *nvs, int n, bool few) {
    Cut best = {0, 0};
    float least = 1e30f;
    for (int i = 0; i < n; ++i) {
        const int64_t tpr = ((nvec + nvs[i] - 1) / nvs[i] + 31) / 32 * 32;
        if (tpr > kNormThreads) continue;
        const float idle = (float)(tpr * nvs[i]) / (float)nvec;
        const float cost = few ? (float)nvs[i]
                               : idle + (tpr > 256 ? 0.5f : 0.f) + (i == 0 ? 0.15f : 0.f) + (i == n - 1 ? 0.05f : 0.f);
        if (cost < least) {
            least = cost;
            best = Cut{nvs[i], (int)tpr};
        }
    }
    return best;
}

template <typename A, typename R>
lean_status launch_norm(const NormArgs &p, bool vec8, bool shifted, int64_t flags, void *stream) {
    const bool few = p.rows <= 2 * step_sm_count();
    static const int vec_nvs[] = {1, 2, 3, 4}, one_nvs[] = {2, 4, 8};
    const Cut c = vec8      ? cut_row((p.width + 7) / 8, vec_nvs, 4, few)
                  : shifted ? cut_row((p.width + 14) / 8, vec_nvs, 4, few)
                            : cut_row(p.width, one_nvs, 3, few);
    if (c.nv == 0) return step_launch(norm_long_kernel<A, R>, p.rows, kNormThreads, 0, flags, stream, p);
    const int rows = std::max(1, 128 / c.tpr), block = rows * c.tpr;
    const int64_t grid = (p.rows + rows - 1) / rows;
    auto go = [&](auto kern) { return step_launch(kern, grid, block, 0, flags, stream, p, c.tpr); };
    if (vec8) {
        if (c.nv == 1) return go(norm_kernel<A, R, 8, 1, false>);
        if (c.nv == 2) return go(norm_kernel<A, R, 8, 2, false>);
        if (c.nv == 3) return go(norm_kernel<A, R, 8, 3, false>);
        return go(norm_kernel<A, R, 8, 4, false>);
    }
    if (shifted) {
        if (c.nv == 1) return go(norm_kernel<A, R, 8, 1, true>);
        if (c.nv == 2) return go(norm_kernel<A, R, 8, 2, true>);
        if (c.nv == 3) return go(norm_kernel<A, R, 8, 3, true>);
        return go(norm_kernel<A, R, 8, 4, true>);
    }
    if (c.nv == 2) return go(norm_kernel<A, R, 1, 2, false>);
    if (c.nv == 4) return go(norm_kernel<A, R, 1, 4, false>);
    return go(norm_kernel<A, R, 1, 8, false>);
}

}  // namespace

extern "C" lean_status lean_residual_norm(const lean_norm_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!known_dtype(a->act_dtype) || (a->res_dtype != LEAN_F32 && a->res_dtype != a->act_dtype) ||
        !step_flags_ok(a->flags))
        return LEAN_ERR_FORMAT;
    if (a->rows <= 0 || a->width <= 0 || a->rows > INT32_MAX / 2 || a->width > INT32_MAX / 2 || a->x_stride < 0 || a->h_stride < 0 ||
        a->gate_stride < 0 || a->h_out_stride < 0 || a->y_stride < 0)
        return LEAN_ERR_SHAPE;
    if (a->rows > 1 && ((a->h_out && a->h_out_stride < a->width) || (a->y && a->y_stride < a->width)))
        return LEAN_ERR_SHAPE;
    if ((!a->x && !a->h) || (!a->h_out && !a->y) || (!a->x && (a->gate || a->post_w))) return LEAN_ERR_NULL;
    const int64_t as = dtype_size(a->act_dtype), rs = dtype_size(a->res_dtype);
    if (!step_aligned(a->x, as) || !step_aligned(a->gate, as) || !step_aligned(a->y, as) ||
        !step_aligned(a->h, rs) || !step_aligned(a->h_out, rs) || !step_aligned(a->w, 4) ||
        !step_aligned(a->post_w, 4))
        return LEAN_ERR_ALIGN;
    // 16-byte vectors when every row of every buffer allows them
    const int64_t any = a->width | a->x_stride | a->h_stride | a->gate_stride | a->h_out_stride | a->y_stride;
    const bool on16 = step_aligned(a->x, 16) && step_aligned(a->h, 16) && step_aligned(a->gate, 16) &&
                      step_aligned(a->h_out, 16) && step_aligned(a->y, 16);
    const bool vec8 = on16 && any % 8 == 0 && step_aligned(a->w, 16) && step_aligned(a->post_w, 16);
    // or where they all begin at the same distance from one
    const int64_t stride = a->x ? a->x_stride : a->h_stride;
    const bool shifted = on16 && !vec8 && (!a->h || a->h_stride == stride) && (!a->h_out || a->h_out_stride == stride) &&
                         (!a->y || a->y_stride == stride) && (!a->gate || a->gate_stride == stride || a->gate_stride == 0);
    NormArgs p = {a->x, a->h, a->gate, a->post_w, a->w, a->h_out, a->y, a->rows, a->x_stride, a->h_stride,
                  a->gate_stride, a->h_out_stride, a->y_stride, stride, (int)a->width, (float)a->eps,
                  (float)a->res_scale, nullptr};
#ifdef LEAN_DEBUG
    p.err = error_word();
#endif
    typedef __nv_bfloat16 b16;
    const bool same = a->res_dtype == a->act_dtype;
    switch (a->act_dtype) {
    case LEAN_F32: return launch_norm<float, float>(p, vec8, shifted, a->flags, stream);
    case LEAN_BF16:
        return same ? launch_norm<b16, b16>(p, vec8, shifted, a->flags, stream)
                    : launch_norm<b16, float>(p, vec8, shifted, a->flags, stream);
    default:
        return same ? launch_norm<__half, __half>(p, vec8, shifted, a->flags, stream)
                    : launch_norm<__half, float>(p, vec8, shifted, a->flags, stream);
    }
}
