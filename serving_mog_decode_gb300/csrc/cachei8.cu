// cachei8.cu -- the cache-reading kernel's instances over int8 rows with a scale per block.
#include "cache.cuh"

namespace mog {

cudaError_t launch_spliti8(const CacheArgs &a, const DiffArgs &d, void *out, bool diff, bool bf_out, bool wide, int splits,
                           cudaStream_t s) {
    if (diff) return bf_out ? pick_split<true, true, true, true>(a, d, out, wide, splits, s) : pick_split<true, true, false, true>(a, d, out, wide, splits, s);
    return bf_out ? pick_split<true, false, true, true>(a, d, out, wide, splits, s) : pick_split<true, false, false, true>(a, d, out, wide, splits, s);
}

}  // namespace mog
