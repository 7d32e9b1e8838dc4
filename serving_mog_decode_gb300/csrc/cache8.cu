// cache8.cu -- the cache-reading kernel's instances over e4m3 rows.
#include "cache.cuh"

namespace mog {

cudaError_t launch_split8(const CacheArgs &a, const DiffArgs &d, void *out, bool diff, bool bf_out, bool wide, int splits,
                          cudaStream_t s) {
    if (diff) return bf_out ? pick_split<true, true, 1>(a, d, out, wide, splits, s) : pick_split<true, true, 2>(a, d, out, wide, splits, s);
    return bf_out ? pick_split<true, false, 1>(a, d, out, wide, splits, s) : pick_split<true, false, 2>(a, d, out, wide, splits, s);
}

}  // namespace mog
