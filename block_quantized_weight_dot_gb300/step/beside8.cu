// beside8.cu -- the kernels of attend.cuh for caches in 8 bits, beside a kernel for prefixes.
#include "attend.cuh"

namespace lean {

lean_status attend_beside8(const AttArgs &p, int64_t flags, void *stream) {
    return p.dim <= 64 ? pick_attend<int8_t, 64, true>(p, flags, stream) : pick_attend<int8_t, 128, true>(p, flags, stream);
}

}  // namespace lean
