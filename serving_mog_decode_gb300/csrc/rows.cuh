// rows.cuh -- rows of new tokens on their way into a mog_cache: packed bf16 arithmetic and the
// scale of an e4m3 row, shared by the store (cache.cu) and the stores with rotary positions (rows.cu).
#pragma once

#include "common.cuh"

namespace mog {

__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {  // (a NaN half gives way)
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {  // bf16 pair -> two codes
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(bf_hi(w)), "f"(bf_lo(w)));
    return c;
}

// Exponent e of a row's e4m3 scale 2^e: the least one (>= -126) with amax <= 448*2^e, amax the
// row's largest finite magnitude (0 if that is 0), so that dividing by it is exact and the only
// rounding is the one to e4m3.  The row's elements are in N words of each of LANES neighbouring
// lanes, all of which are in `group`.
template <int LANES, int N>
__device__ __forceinline__ int e4m3_row_exp(const uint32_t (&w)[N], unsigned group) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) m = bf2_max(m, w[k] & 0x7fff7fffu);
    float amax = fmaxf(bf_lo(m), bf_hi(m));
    if (amax == INFINITY) {  // the largest finite magnitude instead
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float p = fabsf(bf_lo(w[k])), q = fabsf(bf_hi(w[k]));
            amax = fmaxf(amax, fmaxf(p < INFINITY ? p : 0.f, q < INFINITY ? q : 0.f));
        }
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
    // amax = m * 2^E, 1 <= m < 2: 448 = 1.75 * 2^8
    const int bits = __float_as_int(amax), E = (bits >> 23) - 127;
    const int e = E - 8 + ((bits & 0x7fffff) > 0x600000);
    return amax > 0.f ? max(e, -126) : 0;
}
// 2^-e in both halves of a word, -126 <= -e <= 126
__device__ __forceinline__ uint32_t bf2_pow2_neg(int e) {
    const uint32_t inv = (uint32_t)(127 - e) << 7;
    return inv | inv << 16;
}

}  // namespace mog
