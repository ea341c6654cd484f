// beside.cu -- the kernels of attend.cuh for caches of 16 bits, beside a kernel for prefixes.
#include "attend.cuh"

namespace lean {

lean_status attend_beside16(const AttArgs &p, bool bf16, int64_t flags, void *stream) {
    if (bf16)
        return p.dim <= 64 ? pick_attend<__nv_bfloat16, 64, true>(p, flags, stream)
                           : pick_attend<__nv_bfloat16, 128, true>(p, flags, stream);
    return p.dim <= 64 ? pick_attend<__half, 64, true>(p, flags, stream) : pick_attend<__half, 128, true>(p, flags, stream);
}

}  // namespace lean
