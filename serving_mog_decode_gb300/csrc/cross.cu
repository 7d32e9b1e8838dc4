// cross.cu -- cross attention (mog_cross_attend): several query tokens of each sequence, or one, to the
// rows of a bf16 cache, all of which every query sees (an encoder's states, a document).
//
//   out = softmax(tau q.K^T) V     per query token and head, over the keys [0, N_b)
//
// The T x G query rows that share a KV head are packed (token, then head), 128 to a tile.  A CTA
// has two streams over tiles of 128 keys: two query tiles that share every key tile, or, where only one
// is left, one query tile whose streams take alternate key tiles and are joined at the end.  While the
// softmax of one stream runs, the tensor cores work for the other:
//
//   warps 0-3, 4-7  softmax of stream 0, 1: a thread has one query row; it reads its 128 logits from
//                   tensor memory, takes the running maximum, and writes the weights back as bf16 where the logits were
//   warp 8          issues the MMAs: S = Q K^T (128 x 128 x 128) and O += P V, P from tensor memory
//   warp 9          TMA copies of K and V tiles through a ring of 32 KB slots, in the order of their use
//
// Tensor memory holds S (then P) and O of both streams, 512 columns.  O is rescaled only when a row's
// maximum has risen by more than 2^8 since the last time: weights are then at most 2^8, and O and
// their sum (fp32) lose nothing.  Weights are rounded to bf16 (2^-9 of each; the product's other operand is bf16),
// an error of the size of the output's own rounding; their sum is of the unrounded ones.
#include <cuda.h>

#include <algorithm>

#include "tc.cuh"
#include "internal.h"

namespace mog {

constexpr int CX_M = 128, CX_KEYS = 128;         // query rows and keys of a tile
constexpr int CX_TILE = CX_KEYS * MOG_D * 2;     // bytes of a tile (K, V or Q): two halves of 64 dimensions
constexpr int CX_HALF = CX_TILE / 2;
// Slots of 32 KB.  Two query tiles: one ring of five.  One query tile: the second one's place is a sixth, and each
// stream has a ring of three of its own.
constexpr int CX_SLOTS = 6, CX_RING = 5, CX_OWN = 3;
constexpr int CX_THREADS = 384, CX_MMA = 8, CX_LOAD = 9;  // (warps 10, 11 fill the third warpgroup)
// Registers: 168 a thread at launch; the softmax warps take 208, the others leave theirs at 80
// (256 * 208 + 128 * 80 = 63488 of 384 * 168 = 64512).
constexpr int CX_REGS_MORE = 208, CX_REGS_LESS = 80;
constexpr int CX_SMEM = (2 + CX_RING) * CX_TILE + 1024;
constexpr int CX_PART = MOG_D + 4;               // floats of a partial: maximum, sum, 2 unused, accumulators
constexpr float CX_RISE = 8.f;                   // log2 of the rise of a maximum that O is rescaled for

struct CrossArgs {
    const uint16_t *q;
    uint16_t *out;
    int64_t qb, qt, qh, ob, ot, oh;
    const int *lengths, *count;
    int n_max, t_max, h_kv, G;
    const int *bt;
    int pshift, pps, n_pages;
    int bmul, hmul;  // contiguous: 0 where all sequences (heads) are one in memory
    float scale2;    // tau * log2(e)
    float *part;     // splits > 1: [split][unit][row][CX_PART]
    int splits, rows_pad;
};

// Query rows of sequence b that share a KV head.
__device__ __forceinline__ int cross_rows(const CrossArgs &a, int b) {
    const int t = a.count ? min(max(a.count[b], 0), a.t_max) : a.t_max;
    return t * a.G;
}

// Key tiles [first, first + n) of split s of a sequence of `len` keys.
__device__ __forceinline__ void split_tiles(int len, int splits, int s, int &first, int &n) {
    const int nt = (int)(((unsigned)len + CX_KEYS - 1) / CX_KEYS);
    const int per = (nt + splits - 1) / splits;
    first = min(s * per, nt);
    n = min(per, nt - first);
}

// V tile, [128 keys][64 dims] twice, as the MN-major operand B (N = dimensions, K = keys): 64
// dimensions by 8 keys per swizzle atom, key atoms 1024 bytes apart, halves of the dimensions CX_HALF.
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
    uint64_t d = smem_desc_sw128(addr);
    d &= ~((uint64_t)0x3FFF << 16);
    return d | (uint64_t)(CX_HALF >> 4) << 16;
}
// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, int accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// After tmem_wait_ld: loaded values are not used before this point.
__device__ __forceinline__ void settle(uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t f32x2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// the two softmax groups' barrier
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct CrossBars {
    uint64_t full[CX_SLOTS];  // a copy is there
    // The logits of a stream's even and odd tiles.  That tile j + 1's are there says also that all earlier MMAs are
    // through, and so that V of tile j and K of tile j + 1 are free: the only signal that the copying warp needs.  It may
    // be a tile late with its wait, which is why even and odd ones have a barrier each.
    uint64_t s_full[2][2];
    uint64_t p_full[2][2];    // a stream's weights, of each half of the keys
    uint64_t o_full[2], v_tail;
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// Zeros in rows [row, row + n) of a tile, by a warp.
__device__ __forceinline__ void zero_rows(uint32_t tile, int row, int n) {
    for (int i = row * 8 + (threadIdx.x & 31); i < (row + n) * 8; i += 32) {
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(tile + 16 * i), "r"(0) : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(tile + CX_HALF + 16 * i), "r"(0) : "memory");
    }
}

// 32 dimensions from 32 c on of row `r` of a warp's 32 output rows, as bf16 in shared memory: 16-byte chunk ch
// of a row at chunk ch ^ (r & 7), without bank conflicts for a row a lane and for 16 lanes a row.
__device__ __forceinline__ void put32(uint32_t out, int r, int c, const float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(out + r * 256 + (((4 * c + i) ^ (r & 7)) << 4)),
                     "r"(cvt_bf2(v[8 * i], v[8 * i + 1])), "r"(cvt_bf2(v[8 * i + 2], v[8 * i + 3])),
                     "r"(cvt_bf2(v[8 * i + 4], v[8 * i + 5])), "r"(cvt_bf2(v[8 * i + 6], v[8 * i + 7])) : "memory");
}

template <bool PAGED>
__global__ void __launch_bounds__(CX_THREADS, 1) k_cross(CrossArgs a, const __grid_constant__ CUtensorMap kmap,
                                                         const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t cx_raw[];
    __shared__ __align__(8) CrossBars bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    __shared__ float2 s_ml[CX_M];
    const int u = blockIdx.y, b = u / a.h_kv, h = u - b * a.h_kv, split = blockIdx.z;
    const int rows = cross_rows(a, b), row0 = blockIdx.x * 2 * CX_M;
    if (row0 >= rows) return;
    const bool pair = row0 + CX_M < rows;  // two query tiles
    const int len = min(max(a.lengths[b], 0), a.n_max);
    int first, nt;
    split_tiles(len, a.splits, split, first, nt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = smem_u32(cx_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u, sR = sQ + (pair ? 2 : 1) * CX_TILE;
    const int ways = pair ? 1 : 2, ring = pair ? CX_RING : CX_OWN;  // rings, and their slots
    auto bar = [&](const uint64_t &x) { return smem_u32(&x); };
    // tiles of stream s, and its j-th
    auto n_of = [&](int s) { return pair ? nt : (nt - s + 1) >> 1; };
    auto tile_of = [&](int s, int j) { return first + (pair ? j : 2 * j + s); };
    const int tail = nt > 0 ? max(0, (first + nt) * CX_KEYS - len) : 0;  // rows of the last tile behind the sequence's end

    if (tid == CX_LOAD * 32) {
        for (int i = 0; i < CX_SLOTS; ++i) mbar_init(bar(bars.full[i]), 1);
        for (int i = 0; i < 2; ++i) {
            for (int k = 0; k < 2; ++k) mbar_init(bar(bars.s_full[i][k]), 1), mbar_init(bar(bars.p_full[i][k]), CX_M);
            mbar_init(bar(bars.o_full[i]), 1);
        }
        mbar_init(bar(bars.v_tail), 1);
        fence_barrier_init();
        s_fail = 0;
    }
    if (warp == CX_MMA) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    // copies, by their warp
    const int gr = PAGED ? min(CX_KEYS, 1 << a.pshift) : CX_KEYS, ng = CX_KEYS / gr;  // rows of a copy, copies of a tile
    int issued[2] = {0, 0};  // copies of each ring
    bool copies_ok = true;
    auto load = [&](int s, const CUtensorMap *map, int tile, bool value) {
        const int i = issued[s], slot = s * CX_OWN + i % ring, round = i / ring;
        if (round > 0) {  // copy i - ring, V of tile f - 1 or K of tile f, has been used
            const int f = (i - ring + 1) >> 1;
            copies_ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.s_full[pair ? 1 : s][f & 1]), (f >> 1) & 1));
        }
        if (!copies_ok) return;
        const uint32_t dst = sR + slot * CX_TILE;
        const int key = tile * CX_KEYS + lane * gr;  // lane g: the tile's g-th copy
        int page = 0;
        const bool seen = lane < ng && key < len;
        bool there = seen;
        if (PAGED && seen) {
            page = __ldg(a.bt + (int64_t)b * a.pps + (key >> a.pshift));
            there = (unsigned)page < (unsigned)a.n_pages;
        }
        const unsigned have = __ballot_sync(0xffffffffu, there);
        if (PAGED && value) {  // a page that is none: its weights are zero, and so must its values be finite
            const unsigned none = __ballot_sync(0xffffffffu, seen && !there);
            for (int g = 0; none >> g; ++g)
                if (none >> g & 1) zero_rows(dst, g * gr, gr);
            if (none) fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(bar(bars.full[slot]), (uint32_t)__popc(have) * gr * 256);
        __syncwarp();
        if (there) {
            const int row = PAGED ? key & ((1 << a.pshift) - 1) : key;
            const int c2 = PAGED ? h : h * a.hmul, c3 = PAGED ? page : b * a.bmul;
            tma_load_4d(dst + lane * gr * 128, map, 0, row, c2, c3, bar(bars.full[slot]));
            tma_load_4d(dst + CX_HALF + lane * gr * 128, map, 64, row, c2, c3, bar(bars.full[slot]));
        }
        ++issued[s];
    };
    if (warp == CX_LOAD) {  // the first keys, before all else
        __syncwarp();  // (its first lane has made the barriers)
        for (int t = 0; t < min(nt, ways); ++t) load(t, &kmap, first + t, false);
    }
    // queries: rows of 256 bytes in the layout that the K tiles have
    if (warp != CX_LOAD && nt > 0) {
        for (int i = tid < CX_LOAD * 32 ? tid : tid - 32; i < (pair ? 2 : 1) * CX_M * 16; i += CX_THREADS - 32) {
            const int r = i >> 4, ch = i & 15, row = row0 + r;
            const int t = row / a.G, g = row - t * a.G;
            const uint32_t at = sQ + (r >> 7) * CX_TILE + (ch >> 3) * CX_HALF + (r & 127) * 128 + (((ch ^ r) & 7) << 4);
            const bool in = row < rows;
            cp_async16(at, a.q + (in ? b * a.qb + t * a.qt + (int64_t)(h * a.G + g) * a.qh + 8 * ch : 0), in ? 16 : 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto tS = [&](int s) { return tmem + (uint32_t)(s * 128); };
    auto tO = [&](int s) { return tmem + (uint32_t)(256 + s * 128); };

    if (warp >= CX_MMA) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CX_REGS_LESS));
        if (warp == CX_LOAD) {
            // -------------------------------------------------------------- copies
            // in the order of their use: of a ring K, V, K, V, ...
            for (int t = 0; t < nt && copies_ok; ++t) {
                const int s = pair ? 0 : t & 1;
                load(s, &vmap, first + t, true);
                if (t + ways < nt && copies_ok) load(s, &kmap, first + t + ways, false);
            }
            bool ok = copies_ok;
            if (tail > 0 && ok) {
                // rows behind the sequence's end: their weights are zero, and so must their values be finite
                const int s = pair ? 0 : (nt - 1) & 1, i = issued[s] - 1, slot = s * CX_OWN + i % ring;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.full[slot]), (i / ring) & 1));
                zero_rows(sR + slot * CX_TILE, CX_KEYS - tail, tail);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bars.v_tail));
            }
            if (!ok) atomicExch(&s_fail, 1);
            // no copy outlives the CTA
            for (int s = 0; s < ways; ++s)
                for (int i = max(0, issued[s] - ring); i < issued[s]; ++i) mbar_wait(bar(bars.full[s * CX_OWN + i % ring]), (i / ring) & 1);
        } else if (warp == CX_MMA) {
            // ---------------------------------------------------------------- MMAs
            // One thread, the streams in turn: while it waits for the weights of one, the MMAs of the other run.
            if (elect_one()) {
                constexpr uint32_t ID_S = idesc_bf16_f32(CX_M, CX_KEYS), ID_O = idesc_bf16_f32(CX_M, MOG_D) | 1u << 16;
                const uint64_t qd = smem_desc_sw128(sQ), kd = smem_desc_sw128(sR), vd = v_desc(sR);
                bool ok = true;
                int at0 = 0, at1 = CX_OWN;  // the next slot of each ring, and its phase
                uint32_t phase0 = 0, phase1 = 0;
                auto next_copy = [&](int &at, uint32_t &phase, int end) {  // its slot, once it is there
                    const int slot = at;
                    ok = ok && mbar_wait(bar(bars.full[slot]), phase);
                    if (++at == end) at -= ring, phase ^= 1;
                    return slot;
                };
                auto mma_s = [&](int s, int j, int slot) {
                    const uint64_t q = qd + (pair ? s : 0) * (CX_TILE >> 4), k = kd + slot * (CX_TILE >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const int off = ((ks >> 2) * CX_HALF + (ks & 3) * 32) >> 4;
                        tc_mma(tS(s), q + off, k + off, ID_S, ks != 0);
                    }
                    tc_commit(bar(bars.s_full[s][j & 1]));
                };
                // stream s's j-th tile; v, k: the slots of its values and of the next tile's keys
                auto step = [&](int s, int j, int v, int k, bool more) {
                    const uint64_t d = vd + v * (CX_TILE >> 4);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        ok = ok && mbar_wait(bar(bars.p_full[s][c]), j & 1);
                        if (!ok) return;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 4 * c; ks < 4 * c + 4; ++ks)
                            tc_mma_ts(tO(s), tS(s) + 8 * ks, d + ks * (2048 >> 4), ID_O, ks != 0 || j != 0);
                    }
                    if (more) mma_s(s, j + 1, k);
                    else tc_commit(bar(bars.o_full[s]));
                };
                if (pair) {
                    if (nt > 0) {
                        const int k = next_copy(at0, phase0, CX_RING);
                        if (ok) mma_s(0, 0, k), mma_s(1, 0, k);
                    }
                    for (int j = 0; j < nt && ok; ++j) {
                        const bool more = j + 1 < nt;
                        const int v = next_copy(at0, phase0, CX_RING), k = more ? next_copy(at0, phase0, CX_RING) : 0;
                        if (!more && tail > 0) ok = ok && mbar_wait(bar(bars.v_tail), 0);
                        step(0, j, v, k, more);
                        if (ok) step(1, j, v, k, more);
                    }
                } else {
                    if (nt > 0) {
                        const int k = next_copy(at0, phase0, CX_OWN);
                        if (ok) mma_s(0, 0, k);
                    }
                    if (nt > 1 && ok) {
                        const int k = next_copy(at1, phase1, 2 * CX_OWN);
                        if (ok) mma_s(1, 0, k);
                    }
                    for (int j = 0; 2 * j < nt && ok; ++j) {
                        bool more = 2 * j + 2 < nt;
                        int v = next_copy(at0, phase0, CX_OWN), k = more ? next_copy(at0, phase0, CX_OWN) : 0;
                        if (2 * j + 1 == nt && tail > 0) ok = ok && mbar_wait(bar(bars.v_tail), 0);
                        step(0, j, v, k, more);
                        if (2 * j + 1 >= nt || !ok) break;
                        more = 2 * j + 3 < nt;
                        v = next_copy(at1, phase1, 2 * CX_OWN), k = more ? next_copy(at1, phase1, 2 * CX_OWN) : 0;
                        if (2 * j + 2 == nt && tail > 0) ok = ok && mbar_wait(bar(bars.v_tail), 0);
                        step(1, j, v, k, more);
                    }
                }
                if (!ok) atomicExch(&s_fail, 1);
            }
            __syncwarp();
        }
    } else {
        // ----------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CX_REGS_MORE));
        const int s = warp >> 2, r = tid & 127, n = n_of(s);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        int page = 0, gshift = 0;  // paged: the page of the next tile's group `lane`
        auto page_of = [&](int j) {
            if (!PAGED || j >= n) return;
            const int key = tile_of(s, j) * CX_KEYS + (lane << gshift);
            page = -1;
            if (lane < CX_KEYS >> gshift && key < len) page = __ldg(a.bt + (int64_t)b * a.pps + (key >> a.pshift));
        };
        if (PAGED) gshift = min(a.pshift, 7);
        page_of(0);
        for (int j = 0; j < n; ++j) {
            const int left = len - tile_of(s, j) * CX_KEYS;
            unsigned groups = 0xffffffffu;
            if (PAGED) {
                groups = __ballot_sync(0xffffffffu, (unsigned)page < (unsigned)a.n_pages);
                page_of(j + 1);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.s_full[s][j & 1]), (j >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            uint32_t x[4][32];
            float(&v)[128] = reinterpret_cast<float(&)[128]>(x);
            const bool cut = left < CX_KEYS || (PAGED && groups != (1u << (CX_KEYS >> gshift)) - 1u);
            tmem_ld32_nowait(tS(s) + lanes, x[0]);
            tmem_ld32_nowait(tS(s) + lanes + 32, x[1]);
            tmem_wait_ld();
            settle(x[0]), settle(x[1]);
            tmem_ld32_nowait(tS(s) + lanes + 64, x[2]);  // (while the maximum of the first ones is taken)
            tmem_ld32_nowait(tS(s) + lanes + 96, x[3]);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c == 1) {
                    tmem_wait_ld();
                    settle(x[2]), settle(x[3]);
                }
                if (cut) {
#pragma unroll
                    for (int i = 64 * c; i < 64 * c + 64; ++i)
                        if (i >= left || (PAGED && !(groups >> (i >> gshift) & 1u))) v[i] = -INFINITY;
                }
#pragma unroll
                for (int i = 64 * c; i < 64 * c + 64; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mx[k] = fmax3(mx[k], v[i + k], v[i + 4 + k]);
            }
            float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2, f = a.scale2;
            const bool big = fabsf(top) > 16777216.f && fabsf(top) < INFINITY;
            const float mn = fmaxf(m, top);
            if (j == 0) m = mn;
            const bool need = mn > m + CX_RISE;
            if (__any_sync(0xffffffffu, big || need)) {
                // Logits so large that a rounded maximum could leave a weight over 2: rounded first, so that the
                // largest weight is 1.
                if (__any_sync(0xffffffffu, big)) {
#pragma unroll
                    for (int i = 0; i < CX_KEYS; ++i) v[i] = __fmul_rn(v[i], f);
                    f = 1.f;
                }
                if (__any_sync(0xffffffffu, need)) {  // (not of the first tile)
                    const float al = need ? ex2(m - mn) : 1.f;
                    if (need) m = mn;
                    l *= al;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32_nowait(tO(s) + lanes + 32 * c, o);
                        tmem_wait_ld();
                        settle(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                        tmem_st32(tO(s) + lanes + 32 * c, o);
                    }
                }
            }
            const float sh = m == -INFINITY ? 0.f : -m;
            const uint64_t f2 = f32x2(f, f), sh2 = f32x2(sh, sh);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float y0, y1;
                    unpack2(fma2(f32x2(v[64 * c + 2 * i], v[64 * c + 2 * i + 1]), f2, sh2), y0, y1);
                    y0 = ex2(y0), y1 = ex2(y1);
                    sum[i & 1] = add2(sum[i & 1], f32x2(y0, y1));
                    p[i] = cvt_bf2(y0, y1);
                }
                tmem_st32(tS(s) + lanes + 32 * c, p);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(bars.p_full[s][c]));  // (the product starts on the first half)
            }
            float s0, s1;
            unpack2(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
        }
        // ----------------------------------------------------------------- outputs
        const int row = row0 + (pair ? s * CX_M : 0) + r;
        if (n > 0) ok = ok && mbar_wait(bar(bars.o_full[s]), 0);
        if (!pair && n_of(1 - s) > 0) ok = ok && mbar_wait(bar(bars.o_full[1 - s]), 0);  // (the ring is idle then)
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) atomicExch(&s_fail, 1);
        tc_fence_after();
        float *xch = reinterpret_cast<float *>(cx_raw + (sR - raw));  // [dimension][row]
        float mine = 1.f, his = 0.f;
        if (!pair) {
            if (s == 1) {
                s_ml[r] = make_float2(m, l);
                if (ok && n > 0)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        tmem_ld32(tO(1) + lanes + 32 * c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) xch[(32 * c + i) * CX_M + r] = o[i];
                    }
            }
            softmax_sync();
            if (s == 0) {
                const float2 ml = s_ml[r];
                const float mn = fmaxf(m, ml.x), sh = mn == -INFINITY ? 0.f : mn;
                mine = ex2(m - sh), his = n_of(1) > 0 ? ex2(ml.x - sh) : 0.f;
                m = mn;
                l = l * mine + ml.y * his;
            }
        }
        const bool failed = *(volatile int *)&s_fail != 0;
        if (pair || s == 0) {
            const bool write = row < rows;
            const uint32_t stage = sQ + (pair ? s : 0) * CX_TILE + (warp & 3) * 32 * 256;  // (the queries have been read)
            float *part = a.part + (((int64_t)split * gridDim.y + u) * a.rows_pad + row) * CX_PART;
            const float inv = a.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;  // (nothing seen: zeros; a sum that is NaN stays)
            mine *= inv, his *= inv;
            if (a.splits > 1 && write) *reinterpret_cast<float2 *>(part) = make_float2(failed ? __int_as_float(0x7fffffff) : m, l);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(tO(s) + lanes + 32 * c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    o[i] *= mine;
                    if (!pair && n_of(1) > 0) o[i] += xch[(32 * c + i) * CX_M + r] * his;
                    if (failed) o[i] = __int_as_float(0x7fffffff);  // a wait gave up: NaN, not a wrong number
                }
                if (write && a.splits > 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4 *>(part + 4 + 32 * c + 4 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                } else {
                    put32(stage, lane, c, o);
                }
                __syncwarp();
            }
            if (a.splits == 1) {
                // two rows at a time, 16 lanes each
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int k = 2 * i + (lane >> 4), ch = lane & 15, to = row - lane + k;
                    uint4 x;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                 : "r"(stage + k * 256 + ((ch ^ (k & 7)) << 4)));
                    if (to >= rows) continue;
                    const int t = to / a.G, g = to - t * a.G;
                    *reinterpret_cast<uint4 *>(a.out + b * a.ob + t * a.ot + (int64_t)(h * a.G + g) * a.oh + 8 * ch) = x;
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == CX_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Folds the partials of the splits: a warp per query row, four dimensions a lane.
__global__ void __launch_bounds__(256) k_cross_merge(CrossArgs a, int units) {
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t per = (int64_t)a.t_max * a.G;
    if (i >= units * per) return;
    const int u = (int)(i / per), row = (int)(i - u * per), b = u / a.h_kv, h = u - b * a.h_kv;
    if (row >= cross_rows(a, b)) return;
    const float *p = a.part + ((int64_t)u * a.rows_pad + row) * CX_PART;
    const int64_t step = (int64_t)units * a.rows_pad * CX_PART;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool nan = false;
    for (int k = 0; k < a.splits; k += 4) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const bool ok = k + x < a.splits;
            const float *r = p + (k + x) * step;
            ml[x] = ok ? __ldcg(reinterpret_cast<const float2 *>(r)) : make_float2(-INFINITY, 0.f);
            v[x] = ok ? __ldcg(reinterpret_cast<const float4 *>(r + 4) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            nan |= ml[x].x != ml[x].x;
            const float mn = fmaxf(m, ml[x].x), sh = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(m - sh), g = ex2(ml[x].x - sh);
            m = mn;
            l = l * f + ml[x].y * g;
            acc.x = acc.x * f + v[x].x * g, acc.y = acc.y * f + v[x].y * g;
            acc.z = acc.z * f + v[x].z * g, acc.w = acc.w * f + v[x].w * g;
        }
    }
    const float inv = nan ? __int_as_float(0x7fffffff) : l == 0.f ? 0.f : 1.f / l;
    const int t = row / a.G, g = row - t * a.G;
    uint16_t *dst = a.out + b * a.ob + t * a.ot + (int64_t)(h * a.G + g) * a.oh + 4 * lane;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_bf2(acc.x * inv, acc.y * inv), cvt_bf2(acc.z * inv, acc.w * inv));
}

// Splits of the keys for `ctas` CTAs over up to `tiles` key tiles: the number whose waves end first,
// in tile times, a CTA's start and end costing about 6 and the fold of the partials about 12.
int cross_splits(int64_t ctas, int64_t tiles) {
    const int64_t sms = num_sms();
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int s = 1; s <= 64 && (s == 1 || tiles >= 4LL * s); ++s) {
        const int64_t c = ceil_div64(ctas * s, sms) * (ceil_div64(tiles, s) + 6) + (s > 1 ? 12 : 0);
        if (c < cost) cost = c, best = s;
    }
    return best;
}

static bool row_map(CUtensorMap *map, const void *base, int64_t rows, int64_t h, int64_t b, int64_t sn, int64_t sh,
                    int64_t sb, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)MOG_D, (cuuint64_t)rows, (cuuint64_t)h, (cuuint64_t)b};
    // (a dim of one entry: any stride)
    const cuuint64_t strides[3] = {(cuuint64_t)sn * 2, h > 1 ? (cuuint64_t)sh * 2 : 256, b > 1 ? (cuuint64_t)sb * 2 : 256};
    for (int i = 0; i < 3; ++i)
        if (strides[i] == 0 || (strides[i] & 15) || strides[i] >= (1ull << 40)) return false;
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t cross_scratch(int batch, int h_kv, int G, int t_max, int n_max) {
    const int64_t rows = (int64_t)t_max * G, qt = ceil_div64(rows, 2 * CX_M), units = (int64_t)batch * h_kv;
    const int splits = cross_splits(units * qt, ceil_div64(n_max, CX_KEYS));
    return splits > 1 ? (size_t)splits * units * rows * CX_PART * sizeof(float) : 0;
}

cudaError_t launch_cross(const mog_cache *c, const int32_t *lengths, int n_max, int batch, const RowsIn &r, float *scratch,
                         cudaStream_t s) {
    CrossArgs a{};
    a.q = static_cast<const uint16_t *>(r.q), a.out = static_cast<uint16_t *>(r.qo);
    a.qb = r.qs[0], a.qt = r.qs[1], a.qh = r.qs[2], a.ob = r.os[0], a.ot = r.os[1], a.oh = r.os[2];
    a.lengths = lengths, a.count = r.count, a.n_max = n_max, a.t_max = r.t_max, a.h_kv = r.h_kv, a.G = r.h_q / r.h_kv;
    a.bt = c->block_table, a.pshift = c->block_table ? log2_exact(c->page_rows) : 0, a.pps = c->pages_per_seq;
    a.n_pages = c->n_pages;
    a.scale2 = (float)(1.4426950408889634 / sqrt((double)MOG_D));
    const bool paged = c->block_table != nullptr;
    // a stride of 0 (one memory for all): a dim of one entry
    const int64_t h = !paged && c->stride_h == 0 ? 1 : r.h_kv, b = paged ? c->n_pages : c->stride_b == 0 ? 1 : batch;
    a.hmul = h > 1, a.bmul = b > 1;
    CUtensorMap km, vm;
    const int box = paged ? std::min(CX_KEYS, c->page_rows) : CX_KEYS;
    const int64_t n = paged ? c->page_rows : c->n_cap;
    if (!row_map(&km, c->k, n, h, b, c->stride_n, c->stride_h, c->stride_b, box) ||
        !row_map(&vm, c->v, n, h, b, c->stride_n, c->stride_h, c->stride_b, box))
        return cudaErrorInvalidValue;
    const int64_t rows = (int64_t)r.t_max * a.G, qt = ceil_div64(rows, 2 * CX_M), units = (int64_t)batch * r.h_kv;
    a.splits = cross_splits(units * qt, ceil_div64(n_max, CX_KEYS));
    a.rows_pad = (int)rows, a.part = scratch;
    const auto fn = paged ? k_cross<true> : k_cross<false>;
    const cudaError_t e = ensure_smem((const void *)fn, CX_SMEM);
    if (e != cudaSuccess) return e;
    fn<<<dim3((unsigned)qt, (unsigned)units, a.splits), CX_THREADS, CX_SMEM, s>>>(a, km, vm);
    if (a.splits > 1) k_cross_merge<<<(unsigned)ceil_div64(units * rows, 8), 256, 0, s>>>(a, (int)units);
    return cudaGetLastError();
}

}  // namespace mog
