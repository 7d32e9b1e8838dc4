// cache8.cu -- the cache-reading kernel's instances over e4m3 rows.
#include "cache.cuh"

namespace mog {

cudaError_t launch_split8(const CacheArgs &a, const DiffArgs &d, void *out, bool diff, bool bf_out, bool wide, int splits,
                          cudaStream_t s) {
    if (diff) return bf_out ? pick_split<true, true, true>(a, d, out, wide, splits, s) : pick_split<true, true, false>(a, d, out, wide, splits, s);
    return bf_out ? pick_split<true, false, true>(a, d, out, wide, splits, s) : pick_split<true, false, false>(a, d, out, wide, splits, s);
}

}  // namespace mog
