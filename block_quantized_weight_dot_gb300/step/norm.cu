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
#include "step_common.cuh"

using namespace lean;

namespace {

struct NormArgs {
    const void *x, *h, *gate;
    const float *post_w, *w;
    void *h_out, *y;
    int64_t rows, xs, hs, gs, hos, ys;
    int width;
    float eps, alpha;
    unsigned *err;
};

constexpr int kNormThreads = 512;  // of a row, at most

// Sum over the tpr threads of a row (a power of two, 32 at least); part: one
// float per warp of the block, not used for anything else.
__device__ __forceinline__ float row_sum(float v, int tpr, float *part) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    const int warp = threadIdx.x / 32, first = (threadIdx.x & ~(tpr - 1)) / 32;
    if (threadIdx.x % 32 == 0) part[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < tpr / 32; ++i) s += part[first + i];
    return s;
}

template <typename A, typename R, int VEC, int NV>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs p, int tpr) {
    step_begin();
    __shared__ float part[2][kNormThreads / 32];
    const int t = threadIdx.x & (tpr - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < p.rows;
    const float inv = 1.f / (float)p.width;

    Vec<A, VEC> xr[NV], gr[NV];
    Vec<R, VEC> hr[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        in[i] = live && c < p.width;
        if (in[i] && p.x && LEAN_SPAN(row * p.xs + c, VEC, (p.rows - 1) * p.xs + p.width, p.err))
            xr[i] = load_vec<A, VEC>(static_cast<const A *>(p.x) + row * p.xs + c);
        if (in[i] && p.h && LEAN_SPAN(row * p.hs + c, VEC, (p.rows - 1) * p.hs + p.width, p.err))
            hr[i] = load_vec<R, VEC>(static_cast<const R *>(p.h) + row * p.hs + c);
        if (in[i] && p.gate && LEAN_SPAN(row * p.gs + c, VEC, (p.rows - 1) * p.gs + p.width, p.err))
            gr[i] = load_vec<A, VEC>(static_cast<const A *>(p.gate) + row * p.gs + c);
    }
    float post = 1.f;
    if (p.post_w) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i])
#pragma unroll
                for (int j = 0; j < VEC; ++j) s = fmaf(to_f(xr[i].v[j]), to_f(xr[i].v[j]), s);
        post = rsqrtf(fmaf(row_sum(s, tpr, part[0]), inv, p.eps));
    }
    float v[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
        const int c = (t + i * tpr) * VEC;
        Vec<float, VEC> pw;
        if (p.post_w) pw = load_vec<float, VEC>(p.post_w + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float u = 0.f;
            if (p.x) {
                u = to_f(xr[i].v[j]);
                if (p.post_w) u = u * post * pw.v[j];
                if (p.gate) u *= to_f(gr[i].v[j]);
                u *= p.alpha;
            }
            v[i][j] = p.h ? to_f(hr[i].v[j]) + u : u;
            s = fmaf(v[i][j], v[i][j], s);
        }
        if (p.h_out && LEAN_SPAN(row * p.hos + c, VEC, (p.rows - 1) * p.hos + p.width, p.err))
            store_vec<R, VEC>(static_cast<R *>(p.h_out) + row * p.hos + c, v[i]);
    }
    if (!p.y) return;
    const float r = rsqrtf(fmaf(row_sum(s, tpr, part[1]), inv, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
        const int c = (t + i * tpr) * VEC;
        Vec<float, VEC> wv;
        if (p.w) wv = load_vec<float, VEC>(p.w + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] *= p.w ? r * wv.v[j] : r;
        if (LEAN_SPAN(row * p.ys + c, VEC, (p.rows - 1) * p.ys + p.width, p.err))
            store_vec<A, VEC>(static_cast<A *>(p.y) + row * p.ys + c, v[i]);
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
    float post = 1.f;
    if (p.post_w) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.width; c += kNormThreads) s = fmaf(to_f(x[c]), to_f(x[c]), s);
        post = rsqrtf(fmaf(row_sum(s, kNormThreads, part[0]), inv, p.eps));
    }
    auto value = [&](int c) {
        float u = 0.f;
        if (x) {
            u = to_f(x[c]);
            if (p.post_w) u = u * post * p.post_w[c];
            if (gate) u *= to_f(gate[c]);
            u *= p.alpha;
        }
        return h ? to_f(h[c]) + u : u;
    };
    float r = 0.f;
    if (p.y) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.width; c += kNormThreads) {
            const float v = value(c);
            s = fmaf(v, v, s);
        }
        r = rsqrtf(fmaf(row_sum(s, kNormThreads, part[1]), inv, p.eps));
    }
    for (int c = threadIdx.x; c < p.width; c += kNormThreads) {
        const float v = value(c);
        if (p.h_out && LEAN_IN(row * p.hos + c, (p.rows - 1) * p.hos + p.width, p.err))
            static_cast<R *>(p.h_out)[row * p.hos + c] = from_f<R>(v);
        if (p.y && LEAN_IN(row * p.ys + c, (p.rows - 1) * p.ys + p.width, p.err))
            static_cast<A *>(p.y)[row * p.ys + c] = from_f<A>(v * (p.w ? r * p.w[c] : r));
    }
}

int pow2_at_least(int64_t v) {
    int p = 1;
    while (p < v) p *= 2;
    return p;
}

template <typename A, typename R>
lean_status launch_norm(const NormArgs &p, bool vec8, int64_t flags, void *stream) {
    const int vec = vec8 ? 8 : 1, most = vec8 ? 4 : 8;  // vectors of a thread, at most
    const int64_t nvec = (p.width + vec - 1) / vec;
    if (nvec > (int64_t)kNormThreads * most)
        return step_launch(norm_long_kernel<A, R>, p.rows, kNormThreads, 0, flags, stream, p);
    // few rows: as many threads as there are vectors (latency); many: two vectors a thread
    const int want = p.rows <= 2 * step_sm_count() ? 1 : 2;
    const int tpr = std::min(kNormThreads, std::max(32, pow2_at_least((nvec + want - 1) / want)));
    const int block = std::max(tpr, 128), nv = pow2_at_least((nvec + tpr - 1) / tpr);
    const int64_t grid = (p.rows + block / tpr - 1) / (block / tpr);
    if (vec8) {
        if (nv == 1) return step_launch(norm_kernel<A, R, 8, 1>, grid, block, 0, flags, stream, p, tpr);
        if (nv == 2) return step_launch(norm_kernel<A, R, 8, 2>, grid, block, 0, flags, stream, p, tpr);
        return step_launch(norm_kernel<A, R, 8, 4>, grid, block, 0, flags, stream, p, tpr);
    }
    if (nv <= 2) return step_launch(norm_kernel<A, R, 1, 2>, grid, block, 0, flags, stream, p, tpr);
    if (nv == 4) return step_launch(norm_kernel<A, R, 1, 4>, grid, block, 0, flags, stream, p, tpr);
    return step_launch(norm_kernel<A, R, 1, 8>, grid, block, 0, flags, stream, p, tpr);
}

}  // namespace

extern "C" lean_status lean_residual_norm(const lean_norm_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!known_dtype(a->act_dtype) || (a->res_dtype != LEAN_F32 && a->res_dtype != a->act_dtype) ||
        !step_flags_ok(a->flags))
        return LEAN_ERR_FORMAT;
    if (a->rows <= 0 || a->width <= 0 || a->width > INT32_MAX / 2 || a->x_stride < 0 || a->h_stride < 0 ||
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
    const bool vec8 = any % 8 == 0 && step_aligned(a->x, 16) && step_aligned(a->h, 16) &&
                      step_aligned(a->gate, 16) && step_aligned(a->h_out, 16) && step_aligned(a->y, 16) &&
                      step_aligned(a->w, 16) && step_aligned(a->post_w, 16);
    NormArgs p = {a->x, a->h, a->gate, a->post_w, a->w, a->h_out, a->y, a->rows, a->x_stride, a->h_stride,
                  a->gate_stride, a->h_out_stride, a->y_stride, (int)a->width, (float)a->eps,
                  (float)a->res_scale, nullptr};
#ifdef LEAN_DEBUG
    p.err = error_word();
#endif
    typedef __nv_bfloat16 b16;
    const bool same = a->res_dtype == a->act_dtype;
    switch (a->act_dtype) {
    case LEAN_F32: return launch_norm<float, float>(p, vec8, a->flags, stream);
    case LEAN_BF16:
        return same ? launch_norm<b16, b16>(p, vec8, a->flags, stream)
                    : launch_norm<b16, float>(p, vec8, a->flags, stream);
    default:
        return same ? launch_norm<__half, __half>(p, vec8, a->flags, stream)
                    : launch_norm<__half, float>(p, vec8, a->flags, stream);
    }
}
