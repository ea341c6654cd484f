// step_common.cuh -- what the step operators (norm, rope, kv_pages, attend,
// logprobs) share: element types, 16-byte vectors of elements, block-wide
// sums and the launch with its flag.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/lean_step.h"
#include "../csrc/debug.cuh"
#include "../csrc/dispatch.h"
#include "../csrc/ptx.cuh"

namespace lean {

// bits of the device error word set by the step operators
constexpr unsigned kErrSlot = 64u;      // a page or slot outside the cache
constexpr unsigned kErrTokenId = 256u;  // a token id outside the vocabulary

inline bool known_dtype(int64_t t) { return t == LEAN_F32 || t == LEAN_BF16 || t == LEAN_F16; }
inline int64_t dtype_size(int64_t t) { return t == LEAN_F32 ? 4 : 2; }
inline bool step_aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool step_flags_ok(int64_t flags) { return (flags & ~(int64_t)LEAN_FLAG_EARLY_WEIGHTS) == 0; }

// SMs of the current device, read once per device.
inline int step_sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
            return 152;
        cache[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

// Raise a kernel's dynamic shared memory limit, once per device.
template <typename Kern>
inline bool step_ensure_smem(Kern kern, size_t bytes, std::atomic<uint64_t> &done) {
    if (bytes <= 48 * 1024) return true;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// shared: how much of an SM's L1 should be shared memory, in percent (-1: as the driver likes).  Two kernels that are
// to overlap ask for the same: an SM has to be idle to change it.
template <typename... KArgs, typename... Args>
inline lean_status step_launch_with(int shared, void (*kern)(KArgs...), int64_t grid, int block, size_t smem,
                                    int64_t flags, void *stream, Args... args) {
    if (grid < 1 || grid > INT32_MAX) return LEAN_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    if (flags & LEAN_FLAG_EARLY_WEIGHTS) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (shared >= 0) {
        attr[cfg.numAttrs].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
        attr[cfg.numAttrs++].val.sharedMemCarveout = shared;
    }
    cfg.attrs = attr;
    cudaGetLastError();
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? LEAN_OK : LEAN_ERR_CUDA;
}
template <typename... KArgs, typename... Args>
inline lean_status step_launch(void (*kern)(KArgs...), int64_t grid, int block, size_t smem, int64_t flags,
                               void *stream, Args... args) {
    return step_launch_with(-1, kern, grid, block, smem, flags, stream, args...);
}

// First thing in every kernel here: let the next kernel's launch begin, and
// wait for the kernel before (both do nothing without LEAN_FLAG_EARLY_WEIGHTS
// on the launches concerned).  Every thread waits, so that this kernel's end
// implies the end of the one before it.
__device__ __forceinline__ void step_begin() {
    pdl_launch_dependents();
    pdl_wait();
}

// ---- elements -------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// N elements of type T that lie N * sizeof(T) apart from alignment: one or more
// 16-byte (or the one smaller) accesses.
template <typename T, int N>
struct alignas((sizeof(T) * N) >= 16 ? 16 : sizeof(T) * N) Vec {
    T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, N> *>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const float *f) {
    Vec<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f<T>(f[i]);
    *reinterpret_cast<Vec<T, N> *>(p) = o;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace lean
