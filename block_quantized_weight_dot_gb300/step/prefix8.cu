// prefix8.cu -- the kernels of prefix.cuh for caches in 8 bits.
#include "prefix.cuh"

namespace lean {

lean_status prefix_cache8(const PrefixArgs &p, bool two, int64_t flags, void *stream) {
    const PrefixMaps maps = prefix_maps(p, PrefixCache::kI8);
    return p.dim <= 64 ? pick_prefix<int8_t, 64>(maps, p, two, flags, stream)
                       : pick_prefix<int8_t, 128>(maps, p, two, flags, stream);
}

}  // namespace lean
