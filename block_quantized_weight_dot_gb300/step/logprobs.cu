// logprobs.cu -- lean_token_logprobs: log probabilities of given tokens, with
// ranks, entropy and the top alternatives.
//
// One block per row: a pass for the largest logit, a pass for the sums and the
// rank, and one more for every alternative.
#include "step_common.cuh"

using namespace lean;

namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;

struct LpArgs {
    const void *x;
    const int32_t *ids;
    float *logprobs, *entropy, *top_lp;
    int32_t *ranks, *top_ids;
    int64_t stride;
    int64_t rows;
    int vocab, top_k;
    float scale;
    unsigned *err;
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LpArgs p) {
    step_begin();
    __shared__ float f[3][kLpWarps];
    __shared__ int n[kLpWarps];
    __shared__ float best_v;
    __shared__ int best_i;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.stride;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float m = -3.402823466e38f;
    for (int i = threadIdx.x; i < p.vocab; i += kLpThreads) m = fmaxf(m, to_f(x[i]));
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) f[0][warp] = m;
    __syncthreads();
    for (int w = 0; w < kLpWarps; ++w) m = fmaxf(m, f[0][w]);
    const int id = p.ids ? p.ids[row] : 0;
    const bool id_ok = id >= 0 && id < p.vocab;
    const float mine = id_ok ? to_f(x[id]) : 0.f;
    float s = 0.f, t = 0.f;
    int c = 0;
    for (int i = threadIdx.x; i < p.vocab; i += kLpThreads) {
        const float v = to_f(x[i]), d = (v - m) * p.scale, e = __expf(d);
        s += e;
        t = d < -200.f ? t : fmaf(e, d, t);
        c += v > mine;
    }
    __syncthreads();
    s = warp_sum(s);
    t = warp_sum(t);
    for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (lane == 0) {
        f[1][warp] = s;
        f[2][warp] = t;
        n[warp] = c;
    }
    __syncthreads();
    s = t = 0.f;
    c = 0;
    for (int w = 0; w < kLpWarps; ++w) {
        s += f[1][w];
        t += f[2][w];
        c += n[w];
    }
    const float log_s = logf(s);
    if (threadIdx.x == 0) {
        if (p.logprobs)
            p.logprobs[row] = !id_ok ? CUDART_NAN_F : s == 0.f ? -CUDART_INF_F : (mine - m) * p.scale - log_s;
        if (p.ranks) p.ranks[row] = id_ok ? c : -1;
        if (p.ids && !id_ok) atomicOr(p.err, kErrTokenId);
        if (p.entropy) p.entropy[row] = s == 0.f ? 0.f : log_s - t / s;
    }
    float last = CUDART_INF_F;
    int last_i = -1;
    for (int k = 0; k < p.top_k; ++k) {  // the largest after (last, last_i)
        float bv = -CUDART_INF_F;
        int bi = INT32_MAX;
        for (int i = threadIdx.x; i < p.vocab; i += kLpThreads) {
            const float v = to_f(x[i]);
            if ((v < last || (v == last && i > last_i)) && (v > bv || (v == bv && i < bi)) && v > -CUDART_INF_F) {
                bv = v;
                bi = i;
            }
        }
        for (int o = 16; o; o >>= 1) {
            const float v = __shfl_xor_sync(0xffffffffu, bv, o);
            const int i = __shfl_xor_sync(0xffffffffu, bi, o);
            if (v > bv || (v == bv && i < bi)) {
                bv = v;
                bi = i;
            }
        }
        __syncthreads();
        if (lane == 0) {
            f[0][warp] = bv;
            n[warp] = bi;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kLpWarps; ++w)
                if (f[0][w] > bv || (f[0][w] == bv && n[w] < bi)) {
                    bv = f[0][w];
                    bi = n[w];
                }
            best_v = bv;
            best_i = bi;
            p.top_ids[row * p.top_k + k] = bi == INT32_MAX ? -1 : bi;
            p.top_lp[row * p.top_k + k] = bi == INT32_MAX ? -CUDART_INF_F : (bv - m) * p.scale - log_s;
        }
        __syncthreads();
        last = best_v;
        last_i = best_i;
    }
}

}  // namespace

extern "C" int64_t lean_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top_k) {
    if (rows <= 0 || rows > INT32_MAX || vocab < 1 || vocab > (1 << 20) || top_k < 0 || top_k > LEAN_MAX_TOP) return -1;
    return 256;
}

extern "C" lean_status lean_token_logprobs(const lean_logprobs_args *a, void *stream) {
    if (!a) return LEAN_ERR_NULL;
    if (!known_dtype(a->dtype) || !step_flags_ok(a->flags)) return LEAN_ERR_FORMAT;
    const int64_t need = lean_token_logprobs_workspace_bytes(a->rows, a->vocab, a->top_k);
    if (need < 0 || a->stride < 0 || (a->rows > 1 && a->stride < a->vocab) || !(a->scale > 0) || a->scale > 3e38)
        return LEAN_ERR_SHAPE;
    if (!a->logits || !a->workspace || (!a->ids && (a->logprobs || a->ranks)) ||
        (a->top_k > 0 && (!a->top_ids || !a->top_logprobs)))
        return LEAN_ERR_NULL;
    if (!step_aligned(a->logits, dtype_size(a->dtype)) || !step_aligned(a->ids, 4) || !step_aligned(a->logprobs, 4) ||
        !step_aligned(a->ranks, 4) || !step_aligned(a->entropy, 4) || !step_aligned(a->top_ids, 4) ||
        !step_aligned(a->top_logprobs, 4) || !step_aligned(a->workspace, 256))
        return LEAN_ERR_ALIGN;
    if (a->workspace_bytes < need) return LEAN_ERR_SHAPE;
    LpArgs p = {a->logits, a->ids, a->logprobs, a->entropy, a->top_logprobs, a->ranks, a->top_ids, a->stride,
                a->rows, (int)a->vocab, (int)a->top_k, (float)a->scale, error_word()};
    if (!p.err) return LEAN_ERR_CUDA;
    switch (a->dtype) {
    case LEAN_F32: return step_launch(logprobs_kernel<float>, a->rows, kLpThreads, 0, a->flags, stream, p);
    case LEAN_BF16: return step_launch(logprobs_kernel<__nv_bfloat16>, a->rows, kLpThreads, 0, a->flags, stream, p);
    default: return step_launch(logprobs_kernel<__half>, a->rows, kLpThreads, 0, a->flags, stream, p);
    }
}
