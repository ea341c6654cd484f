// attend8.cu -- the kernels of attend.cuh for caches in 8 bits.
#include "attend.cuh"

namespace lean {

lean_status attend_cache8(const AttArgs &p, int64_t flags, void *stream) { return pick_dim<int8_t>(p, flags, stream); }

}  // namespace lean
