// cache16.cu -- the cache-reading kernel's instances over bf16 rows with one map and a bf16 output: cross attention
// of one token.
#include "cache.cuh"

namespace mog {

cudaError_t launch_split16(const CacheArgs &a, const DiffArgs &d, void *out, bool wide, int splits, cudaStream_t s) {
    return pick_split<false, false, true>(a, d, out, wide, splits, s);
}

}  // namespace mog
