// cache.cuh -- decode attentions over a mog_cache (bf16, e4m3 or int8 rows, contiguous or paged):
// the kernel that reads the cache.  Its instances are compiled in cache.cu (bf16 rows, differential), cache16.cu
// (bf16 rows, one map), cache8.cu (e4m3 rows) and cachei8.cu (int8 rows).
//
// dense_decode8: softmax(tau q.K^T) V of an 8-bit cache whose row i stands for
// k_scale[i]*code_i and v_scale[i]*code_i.  mog_diff_decode: the difference of two softmax
// maps over one set of values, normalised.  mog_cross_attend with one token: as dense_decode8, over bf16 rows.
// Each is a split kernel and a fold of its partials,
// or, for short caches, one kernel whose clusters take a unit each and fold it themselves.
//
// Split (k_cache_split): the tiles (128 8-bit rows, 64 of bf16) of all (sequence, KV head) units form one list;
// CTA c takes tiles [c*chunk, (c+1)*chunk) of it, so ragged batches load every SM alike
// (the lengths are read on the device: a captured graph replays with grown sequences).  Its
// copies run ahead across unit borders.  Each unit that a CTA touches leaves one partial
// (max, sum, acc per head) in slot c + unit, which no other pair (c, unit) shares, because
// along the list either c or the unit grows by one.
//
// One warp takes 16 rows (bf16) or 32 (8-bit) of each tile.  Up to 8 columns (query heads, or
// the two maps of up to 4 differential heads) sit in N of m16n8k16 with the rows in M
// ("narrow"); up to 16 columns sit in M with the rows in N ("wide").  Either way a value
// row is read once for all of them, and no column of the product is padding at its limit.
// The wide form needs no transposition between the two products (its weights leave the first
// one in the layout that the second takes) and a maximum over 4 lanes instead of 8.
//
// 8-bit rows are read by 16-byte loads in the order the fragments want (dimensions are
// permuted alike in K and q, and, for e4m3, back in the output), then widened in registers to fp16,
// which holds every e4m3 and int8 value exactly.  An int8 tile's V is read by the transposing ldmatrix for bytes, and the rows
// of a block of 16 are taken in the order in which that hands them out (block_row): no shuffle of bytes is left before
// widening, which for int8 takes five instructions for four codes instead of e4m3's two.  The scale of an int8 block is copied to each of its rows
// in the stage, so that all 8-bit rows are alike from there on.  q enters as fp16 scaled by a power of two of its
// own, so that its elements down to 2^-29 of the largest are exact.  Weights p * v_scale enter
// the P.V product as fp16, 2^14 times their share of a running unit: high + low parts (2^-22
// relative), or the high part alone (2^-11; weight_parts), and no better than 2^-39 of the unit.  The unit is at most 2^15 times the largest weight
// of a row that is not zero (new_unit).  bf16 rows go through ldmatrix; their weights are three bf16
// parts (2^-24), or two for a bf16 output (2^-16).  All sums are fp32.
//
// Bound by: HBM in the narrow form (whole steps: 1M e4m3 tokens, 8 KV heads, G = 4: 315 us,
// 7.0 TB/s; differential, 4 x 128K bf16 tokens in 64-row pages, G = 4: 310 us, 6.9 TB/s; over e4m3 rows
// 171 us, 6.5 TB/s); the wide form too over bf16 rows (G = 5: 315 us), but over e4m3 rows by the latencies of its
// chains (G = 5, 4 x 128K: 220 us, 5.0 TB/s; 43% of issue slots, 37% of the tensor pipe).  int8 rows: 1M tokens, 8 KV heads,
// G = 4: 380 us, 5.65 TB/s; not HBM (78%) but the waits between a warp's products and its widening, at 54% of the
// issue slots (three CTAs of four warps, which the registers allow).  Wide int8 (G = 12, 256K tokens, 8 heads: 126 us, 4.3 TB/s; e4m3
// 114) runs in the two CTAs and 32 rows a warp that were chosen by measurements of e4m3 rows (below); other splits were not measured for it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.cuh"
#include "internal.h"

namespace mog {

constexpr int CT_WARPS = 4;
constexpr int CL_PER_SM = 2, CL_STAGES = 3;  // CTAs per SM and stages of the cluster form: short caches, latency
constexpr int CT_THREADS = 32 * CT_WARPS;
constexpr int W_EXP = 14;           // fp16 weights: 2^14 times their share of the unit
// 16-bit parts that a weight of the second product is held in.  A bf16 output takes one less where that
// is worth something: bf16 weights stay within 2^-16 of theirs, a 256th of the output's half step,
// and the step is 1% to 4% faster (2 x 4K tokens, G = 4: 11.3 us against 11.6; 4 x 128K, G = 5: 313 against 316);
// one fp16 part, within 2^-11, an eighth of that half step, is for the wide form alone (16 heads, 512K: 174 us
// against 204; the narrow form: 1M tokens, G = 4: 308 against 311).
constexpr int weight_parts(bool e4m3, bool wide, bool bf16_out) {
    return (e4m3 ? 2 : 3) - (bf16_out && (wide || !e4m3) ? 1 : 0);
}
constexpr int V_RANGE = 10 << 23;   // value scales within 2^10 of the unit's are in order (a difference of float bits)
constexpr float M_RISE = 4.f;       // m may rise by 2^4 before rows of zeros are looked for again
constexpr int V_NONE = 0x7fffffff;  // no unit yet

// A tile is copied by the whole CTA, 2 KB of neighbouring rows per instruction, and each
// warp consumes BLK blocks of 16 of its rows.  Stages are aligned to 128 bytes: 16 bytes off,
// the copies of the same kernel were 5% slower (1M e4m3 tokens, 8 heads: 329 against 316 us).
template <bool ROW8_, bool WIDE_, bool CLUSTER = false, bool I8_ = false>
struct Tile {
    static constexpr bool ROW8 = ROW8_, WIDE = WIDE_, I8 = I8_;  // 8-bit rows (e4m3 or int8); up to 16 columns; int8
    // A unit's first tile is looked at before its products, where a warp has one tile or a few (1000 tokens: 5.6 us
    // against 5.8 after them); elsewhere that would cost registers (8 x 16-64K, 32 KV heads: 403 against 381).
    static constexpr bool EARLY = CLUSTER;
    static constexpr int BLK = ROW8 ? 2 : 1;              // blocks of 16 rows per warp
    static constexpr int WROWS = 16 * BLK;                // rows per warp
    static constexpr int ROWS = CT_WARPS * WROWS;
    // Three CTAs per SM, but two of the wide e4m3 form: it is bound by the latencies of its
    // longer chains, which 255 registers (32 rows a warp in flight, no spills) hide better than
    // a third CTA (16 heads, 512K: 204 us against 231 with three CTAs and 16 rows a warp).
    static constexpr int PER_SM = CLUSTER ? CL_PER_SM : ROW8 && WIDE ? 2 : 3;
    static constexpr int ROW = ROW8 ? MOG_D : 2 * MOG_D;  // bytes
    static constexpr int KV = ROWS * ROW;                 // bytes of the K or V tile: 16 KB
    static constexpr int AUX = 2 * KV;                    // K scales, V scales
    static constexpr int MASK = AUX + (ROW8 ? 2 * ROWS * 4 : 0);  // bit per row
    static constexpr int STAGE = MASK + 128;              // rows stay aligned to 128 bytes
    static constexpr int STAGES = CLUSTER ? CL_STAGES : ROW8 && WIDE ? 3 : 2;   // 32 KB each: 96 KB or more in flight per SM
    static constexpr int COLS = WIDE ? 16 : 8;
    static constexpr int XCH = 2 * COLS * MOG_D * 4;      // two warps' accumulators, in a consumed stage
    // a cluster's CTA leaves its partial behind that in stage 0, or behind the stages
    static constexpr int PART = STAGE >= XCH + COLS * PART_W * 4 ? XCH : STAGES * STAGE;
    static constexpr int SMEM = STAGES * STAGE + (PART == XCH ? 0 : COLS * PART_W * 4);
};

struct CacheArgs {
    const uint8_t *K, *V;
    const float *ks, *vs;
    int64_t sb, sh, sn;     // bytes between pages (or sequences), heads, rows
    int64_t ssb, ssh, ssn;  // the same of the scales, in floats
    int sshift;             // log2 of the rows of a scale (int8; else 0)
    const int *bt;
    int pshift, pps, n_pages;
    const int *lengths;
    int n_max, batch, h_kv, G;
    const uint16_t *q;
    int64_t qb, qh, ob, oh;  // own_rows: elements between sequences and heads of the queries, of the output
    const int *count;        // own_rows: null, or per sequence: at most 0: its output stays as it is
    float *part;
    float scale2;
    int small;  // the strides between rows, and between their scales, fit 32 bits
    int cs;  // CTAs of a cluster that works on one unit; 0: the tile list is split
};

// Queries and outputs with strides and counts of their own (qb .. count): cross attention, the reader of bf16 rows
// with one map.  The others' are contiguous, [batch][h_kv * G][128].
constexpr bool own_rows(bool row8, bool diff) { return !row8 && !diff; }

struct DiffArgs {
    const float *lam;  // [heads][4][64]
    int64_t lam_stride;
    const float *gamma;
    float lambda_init, eps;
};

template <int ROWS>
__device__ __forceinline__ int seq_tiles(const CacheArgs &a, int b) {
    const int n = min(max(a.lengths[b], 0), a.n_max);
    return (int)(((unsigned)n + ROWS - 1) / ROWS);
}

// Tiles of the whole batch, times h_kv: called by a full warp.
template <int ROWS>
__device__ __forceinline__ int total_tiles(const CacheArgs &a) {
    int s = 0;
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) s += seq_tiles<ROWS>(a, b);
    return warp_isum(s) * a.h_kv;
}

// Sequence holding tile `t` of the list and the list position of its first tile (called by
// a full warp; t < total).  Lengths of 128 sequences are loaded at a time.
template <int ROWS>
__device__ __forceinline__ void find_seq(const CacheArgs &a, int t, int &b, int &first) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 128) {
        int mine[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[i] = b0 + 32 * i + lane < a.batch ? seq_tiles<ROWS>(a, b0 + 32 * i + lane) * a.h_kv : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int end = mine[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += v;
            }
            const unsigned in = __ballot_sync(0xffffffffu, base + end > t);
            if (in) {
                const int l = __ffs(in) - 1;
                b = b0 + 32 * i + l;
                first = base + __shfl_sync(0xffffffffu, end - mine[i], l);
                return;
            }
            base += __shfl_sync(0xffffffffu, end, 31);
        }
    }
    b = a.batch;
    first = base;
}

// A place in the tile list.
template <int ROWS>
struct Cursor {
    int b, h, t, nt, n;  // sequence, head, tile, tiles of the sequence, its length
    __device__ __forceinline__ void seek(const CacheArgs &a, int tile) {
        int first;
        find_seq<ROWS>(a, tile, b, first);
        load(a);
        const int r = tile - first;
        h = nt > 0 ? r / nt : 0;
        t = r - h * nt;
    }
    __device__ __forceinline__ void load(const CacheArgs &a) {
        n = b < a.batch ? min(max(a.lengths[b], 0), a.n_max) : 0;
        nt = (int)(((unsigned)n + ROWS - 1) / ROWS);
    }
    __device__ __forceinline__ bool last() const { return t + 1 == nt; }
    __device__ __forceinline__ void next(const CacheArgs &a) {
        if (++t < nt) return;
        t = 0;
        if (++h < a.h_kv) return;
        h = 0;
        do {
            ++b;
            load(a);
        } while (nt == 0 && b < a.batch);
    }
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes));
}

// Shared-memory position of a 16-byte chunk of a row, conflict-free for the readers.  e4m3
// (128-byte rows): K is read at rows r, r+1 and chunks t (t < 4), V at rows 0, 2, 4, 6 (+1,
// +8) and two neighbouring chunks; int8's V by ldmatrix, 8 rows at a chunk.  bf16 (256-byte rows): ldmatrix.
template <bool ROW8>
__device__ __forceinline__ uint32_t swz_k(int row, int ch) {
    return ROW8 ? (uint32_t)(row * MOG_D + ((ch ^ ((row & 1) << 2)) << 4)) : swz(row, ch);
}
template <bool ROW8, bool I8>
__device__ __forceinline__ uint32_t swz_v(int row, int ch) {
    return ROW8 ? (uint32_t)(row * MOG_D + ((ch ^ (row & (I8 ? 7 : 6))) << 4)) : swz(row, ch);
}
// int8: the row of a block of 16 that the products take as their r-th.  ldmatrix hands out V with four
// neighbouring rows of a dimension in a word, rows 4t .. 4t+3 to lane t; the second product has them at 2t, 2t+1,
// 2t+8 and 2t+9.
template <bool I8>
__device__ __forceinline__ int block_row(int r) {
    const int r8 = r & 7;
    return I8 ? 2 * r8 - (r8 & 1) + 2 * (r >> 3) : r;
}

// Page of the tile's 16-row group `lane`, loaded one tile ahead of its use (unchecked: a
// check here would wait for the load).
template <class T, bool PAGED>
__device__ __forceinline__ void tile_page(const CacheArgs &a, const Cursor<T::ROWS> &c, int &pg) {
    if constexpr (PAGED) {
        const int lane = threadIdx.x & 31, row = c.t * T::ROWS + 16 * lane;
        pg = -1;
        if (lane < T::ROWS / 16 && row < c.n) pg = __ldg(a.bt + (int64_t)c.b * a.pps + (row >> a.pshift));
    }
}

// Start the copies of a tile.  Rows behind the sequence's end or in no page are zero and
// masked; they are never read.
template <class T, bool PAGED>
__device__ __forceinline__ void issue(const CacheArgs &a, const Cursor<T::ROWS> &c, int pg, uint32_t stage) {
    constexpr bool ROW8 = T::ROW8;
    constexpr int CH = T::ROW / 16;        // chunks per row
    constexpr int RP = CT_THREADS / CH;    // rows per instruction: 16 or 8
    const int tid = threadIdx.x, lane = tid & 31, ch = tid % CH, r0 = tid / CH;
    const int first = c.t * T::ROWS, left = c.n - first;  // rows of the sequence from here on
    const int pmask = (1 << a.pshift) - 1;
    const int64_t head = c.h * a.sh + r0 * a.sn + ch * 16 + (PAGED ? 0 : c.b * a.sb);
    // int8, contiguous: a tile all of whose rows are there, with strides of 32 bits between them, without the checks of its rows.
    // The kernel is bound by its instructions there (1M tokens, 8 KV heads, G = 4: 405 us against 429); in pages the
    // same made it slower (8 x 16-64K tokens, 32 KV heads: 502 us against 496).
    if (T::I8 && !PAGED && a.small && left >= T::ROWS) {
        const uint8_t *k = a.K + head + (int64_t)first * (int)a.sn;
        const int64_t v = a.V - a.K;
#pragma unroll
        for (int i = 0; i < T::ROWS / RP; ++i) {
            const uint8_t *src = k + (int64_t)(RP * i) * (int)a.sn;
            cp_async16(stage + swz_k<ROW8>(r0 + RP * i, ch), src);
            cp_async16(stage + T::KV + swz_v<ROW8, T::I8>(r0 + RP * i, ch), src + v);
        }
        if (tid >= T::ROWS) return;
        const int64_t so = c.b * a.ssb + c.h * a.ssh + (int64_t)((first + tid) >> a.sshift) * (int)a.ssn;
        cp_async4(stage + T::AUX + 4 * tid, a.ks + so, 4);
        cp_async4(stage + T::AUX + 4 * (T::ROWS + tid), a.vs + so, 4);
        if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + T::MASK + 4 * (tid >> 5)), "r"(0xffffffffu) : "memory");
        return;
    }
#pragma unroll
    for (int i = 0; i < T::ROWS / RP; ++i) {
        const int r = r0 + RP * i;
        const int page = PAGED ? __shfl_sync(0xffffffffu, pg, RP * i / 16) : 0;
        const bool ok = r < left && (!PAGED || (unsigned)page < (unsigned)a.n_pages);
        int64_t off = head + (int64_t)(PAGED ? (first + RP * i) & pmask : first + RP * i) * a.sn;
        if (PAGED) off += page * a.sb;
        off = ok ? off : 0;
        const int bytes = ok ? 16 : 0;
        cp_async16(stage + swz_k<ROW8>(r, ch), a.K + off, bytes);
        cp_async16(stage + T::KV + swz_v<ROW8, T::I8>(r, ch), a.V + off, bytes);
    }
    // thread r: row r's scales and whether it is there
    if (tid >= T::ROWS) return;
    const int page = PAGED ? __shfl_sync(0xffffffffu, pg, tid / 16) : c.b;
    const bool ok = tid < left && (!PAGED || (unsigned)page < (unsigned)a.n_pages);
    if (ROW8) {
        const int row = PAGED ? (first + tid) & pmask : first + tid;
        const int64_t so = ok ? page * a.ssb + c.h * a.ssh + (int64_t)(T::I8 ? row >> a.sshift : row) * a.ssn : 0;
        cp_async4(stage + T::AUX + 4 * tid, a.ks + so, ok ? 4 : 0);
        cp_async4(stage + T::AUX + 4 * (T::ROWS + tid), a.vs + so, ok ? 4 : 0);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + T::MASK + 4 * (tid >> 5)), "r"(mask) : "memory");
}

// Column -> (map, head).  Narrow: 4 + 4 columns of two maps; wide: 8 + 8.
template <bool DIFF, bool WIDE>
__device__ __forceinline__ void column(int c, int &map, int &head) {
    map = DIFF ? (WIDE ? c >> 3 : c >> 2) : 0;
    head = DIFF ? (WIDE ? c & 7 : c & 3) : c;
}

// Running state of a warp.  A lane holds two columns: 2t, 2t+1 (narrow) or g, g+8 (wide),
// with g = lane / 4, t = lane % 4; o[i][e] belongs to the lane's column e & 1 (narrow) or
// e >> 1 (wide).
template <bool WIDE>
struct State {
    static constexpr int NT = WIDE ? 16 : 8;
    float o[NT][4];
    float m[2], l[2];  // what logits are relative to (log2 domain): their maximum, but see new_unit; this lane's share of the sum
    // e4m3: bits of the least value scale in order; the largest is 2^ve, and o is in units of
    // 2^(m + ve - W_EXP) (the same in all lanes)
    int vlo;
    float rise;  // e4m3: how far m has risen since new_unit last looked
    __device__ __forceinline__ int ve() const { return (vlo >> 23) - 127 + (V_RANGE >> 23); }
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        vlo = V_NONE;
        rise = 0.f;
    }
    static __device__ __forceinline__ int col(int e) { return WIDE ? e >> 1 : e & 1; }
};

// q of a unit: B fragments in registers (narrow), or A fragments in shared memory (wide: 32
// registers otherwise).  f: the factor that turns an accumulator of the lane's column into a
// log2-domain logit.
struct QF {
    uint32_t b[8][2];
    float f[2];
};
typedef uint4 QShared[8][32];

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// One column's fragment pieces: this lane's dimensions of each of the 8 steps.
template <bool ROW8, bool DIFF, bool WIDE>
__device__ __forceinline__ float load_column(uint32_t (&w)[8][2], const CacheArgs &a, int unit, int c) {
    const int t = threadIdx.x & 3;
    int map, head;
    column<DIFF, WIDE>(c, map, head);
    const bool have = head < a.G;
    unit = min(unit, a.batch * a.h_kv - 1);  // (lengths that change under a call must not lead out of q)
    const uint16_t *row = a.q + ((int64_t)unit * a.G + (have ? head : 0)) * MOG_D;
    if (own_rows(ROW8, DIFF)) {
        const int b = unit / a.h_kv;
        row = a.q + b * a.qb + ((unit - b * a.h_kv) * a.G + (have ? head : 0)) * a.qh;
    }
    if (!ROW8) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const bool use = have && (!DIFF || (ks >> 2) == map);
            const uint32_t *p = reinterpret_cast<const uint32_t *>(row + ks * 16 + 2 * t);
            w[ks][0] = use ? p[0] : 0u;
            w[ks][1] = use ? p[4] : 0u;
        }
        return a.scale2;
    }
    // dimensions 16(t + 4j) .. +15, word k of chunk j in step 4j + k
    uint32_t raw[2][8];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const bool use = have && (!DIFF || j == map);
        const uint4 *p = reinterpret_cast<const uint4 *>(row + 16 * (t + 4 * j));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = use ? p[i] : make_uint4(0, 0, 0, 0);
            raw[j][4 * i] = v.x, raw[j][4 * i + 1] = v.y, raw[j][4 * i + 2] = v.z, raw[j][4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf_lo(raw[j][i])), fabsf(bf_hi(raw[j][i]))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // largest magnitude to [2^14, 2^15); below 2^-100 a head's logits are 0 to fp32
    const int e = max((__float_as_int(amax) >> 23) - 127, -100);
    const float up = pow2f(14 - e);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t r = raw[ks >> 2][2 * (ks & 3) + i];
            const __half2 h = __floats2half2_rn(bf_lo(r) * up, bf_hi(r) * up);
            w[ks][i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    return pow2f(e - 14) * a.scale2;
}

// (wide: the caller puts a CTA barrier between the last reads of qs, this, and the next reads)
template <bool ROW8, bool DIFF, bool WIDE>
__device__ __forceinline__ void load_q(QF &qf, QShared &qs, const CacheArgs &a, int unit) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const float f = load_column<ROW8, DIFF, WIDE>(qf.b, a, unit, g);
    if (!WIDE) {
        qf.f[0] = __shfl_sync(0xffffffffu, f, 8 * t);
        qf.f[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        return;
    }
    uint32_t w[8][2];
    qf.f[0] = f;
    qf.f[1] = load_column<ROW8, DIFF, WIDE>(w, a, unit, g + 8);
    if (threadIdx.x < 32) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) qs[ks][lane] = make_uint4(qf.b[ks][0], w[ks][0], qf.b[ks][1], w[ks][1]);
    }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool ROW8>
__device__ __forceinline__ void mma_t(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (ROW8) mma_f16(d, a, b0, b1);
    else mma_bf16(d, a, b0, b1);
}
// four 8-bit codes -> two fp16 pairs (exact).  int8: u = code + 128 is the low byte of the fp16 number
// 1024 + u, from which 1152 is taken.
template <bool I8>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (I8) {
        w ^= 0x80808080u;
        lo = __byte_perm(w, 0x64646464u, 0x4140);
        hi = __byte_perm(w, 0x64646464u, 0x4342);
        const uint32_t bias = 0x64806480u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(lo), "r"(bias));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(hi), "r"(bias));
        return;
    }
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}
// Two blocks of 16 rows by 16 bytes, transposed: r[2k], r[2k + 1]: of block k, bytes g and g + 8 of rows 4t .. 4t+3.
// Lane l: the address of row l % 16 of block l / 16.
__device__ __forceinline__ void ldsm_b8_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The largest part of (x, y) that 16 bits hold, and what is left.
template <bool ROW8>
__device__ __forceinline__ uint32_t part16(float &x, float &y) {
    if (ROW8) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        x -= f.x, y -= f.y;
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const uint32_t h = cvt_bf2(x, y);
    x -= bf_lo(h), y -= bf_hi(h);
    return h;
}

__device__ __forceinline__ float lds4(uint32_t addr) {
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ float2 lds8(uint32_t addr) {
    float2 r;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(addr));
    return r;
}

// Wide: the scales of a block's rows 2t, 2t+1, 2t+8, 2t+9 of the products.
template <bool I8>
__device__ __forceinline__ void row_scales(float (&k)[4], uint32_t at) {
    const int t = threadIdx.x & 3;
    const float2 x = lds8(at + (I8 ? 16 : 8) * t), y = lds8(at + (I8 ? 16 * t + 8 : 8 * t + 32));
    k[0] = x.x, k[1] = x.y, k[2] = y.x, k[3] = y.y;
}

// 16 rows by 16 dimensions of K: {rows g | rows g+8} x {dimension pairs 0 | 1} of step ks, as
// the operand with rows in M; its halves (0, 2) and (1, 3) are the two with 8 rows in N.
template <bool ROW8, bool I8>
__device__ __forceinline__ void k_frag(uint32_t (&a)[4], uint32_t sk, int ks, const uint4 &wa, const uint4 &wb) {
    if (ROW8) {
        widen<I8>(word(wa, ks & 3), a[0], a[2]);
        widen<I8>(word(wb, ks & 3), a[1], a[3]);
    } else {
        const int lane = threadIdx.x & 31, mat = lane >> 3, r8 = lane & 7;
        ldsm_x4(sk + swz_k<ROW8>((mat & 1) * 8 + r8, 2 * ks + (mat >> 1)), a[0], a[1], a[2], a[3]);
    }
}

// The largest of a column's values.
template <bool WIDE>
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
    for (int o = WIDE ? 1 : 4; o < (WIDE ? 4 : 32); o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
// Row (of a block of 16) and column (of the lane's two) of logit i.
template <bool WIDE, bool I8>
__device__ __forceinline__ int logit_row(int i) {
    const int lane = threadIdx.x & 31;
    return block_row<I8>(WIDE ? 2 * (lane & 3) + (i & 1) + 8 * (i >> 2) : (lane >> 2) + 8 * (i >> 1));
}
template <bool WIDE>
__device__ __forceinline__ constexpr int logit_col(int i) { return WIDE ? (i >> 1) & 1 : i & 1; }

__device__ __forceinline__ int exp_above(float x) { return (__float_as_int(x) >> 23) - 126; }  // |x| < 2^that, x >= 0

constexpr int F32_INF = 0x7f800000;
// vlo for a largest scale with the bits hi (ve >= -112).
__device__ __forceinline__ int scale_floor(int hi) { return (max((hi >> 23) + 1, 15) << 23) - V_RANGE; }

// e4m3, a tile's value rows: zero: is row `lane` all zeros (with a finite scale);  hi: the bits of the largest
// finite scale.  If the tile is a unit's first, without rows of zeros, and its scales are in order,
// they set the range (true).
template <bool WIDE, bool I8>
__device__ __forceinline__ bool first_tile(State<WIDE> &st, int mine, bool there, uint32_t sv, bool &zero, int &hi) {
    const int lane = threadIdx.x & 31;
    uint32_t any = 0;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {  // (the row's chunks in an order without bank conflicts)
        const uint4 x = lds16(sv + lane * MOG_D + (((ch + lane) & 7) << 4));
        any |= x.x | x.y | x.z | x.w;
    }
    zero = (any & (I8 ? 0xffffffffu : 0x7f7f7f7fu)) == 0 && mine < F32_INF;
    hi = __reduce_max_sync(0xffffffffu, mine < F32_INF ? mine : 0);
    if (st.vlo == V_NONE && hi - __reduce_min_sync(0xffffffffu, there ? mine : F32_INF) <= V_RANGE &&
        !__any_sync(0xffffffffu, there && zero)) {
        st.vlo = scale_floor(hi);
        return true;
    }
    return false;
}

// e4m3: a unit for a tile with value scales out of order.  Weights 2^s * v_scale are held in fp16
// as shares of the unit 2^(m + ve).  While the scales stay between 2^(ve - 10) and 2^ve, and m rises by
// less than 2^4 in all, the unit follows the largest logit alone.  A scale outside may belong to
// a row of zeros (kv_store gives it the scale 1) or to one without weight, and a row of zeros may have the largest
// logit; a unit made for it would leave the other rows' weights no bits.  So rows of zeros are
// left out (their scale in the stage becomes 0), and m becomes the largest s + log2 v_scale of the rest, less ve, or
// what o holds, if that is more.  It may end above or below the largest logit: bounds keep the sum, which counts
// rows of zeros too, inside fp32.
// A cache with such a tile everywhere (every 16th row zero, the rest's scales 2^-14) is read in 409 us in place
// of 316 (1M tokens, G = 4) and 277 in place of 204 (512K, G = 16).
// mine: the bits of the scale of row `lane`;  there: is that row in the cache.
template <class T, int NS>
__device__ __forceinline__ void new_unit(State<T::WIDE> &st, const float (&s)[T::BLK][NS], float (&mx)[2], int mine,
                                         bool there, uint32_t sv, uint32_t vsc) {
    constexpr bool WIDE = T::WIDE;
    static_assert(!T::ROW8 || T::WROWS == 32, "a lane per row");
    const int lane = threadIdx.x & 31;
    st.rise = 0.f;
    bool zero;
    int hi;
    if (first_tile<WIDE, T::I8>(st, mine, there, sv, zero, hi) && !T::EARLY) return;
    if (zero) asm volatile("st.shared.u32 [%0], %1;" ::"r"(vsc + 4 * lane), "r"(0) : "memory");
    hi = __reduce_max_sync(0xffffffffu, mine < F32_INF && !zero ? mine : 0);
    __syncwarp();
    const int ve_old = st.ve();
    if (st.vlo == V_NONE || (hi > 0 && (unsigned)(hi - st.vlo) > V_RANGE)) st.vlo = scale_floor(hi);
    int ve = st.ve();
    float far[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int blk = 0; blk < T::BLK; ++blk)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int v = __float_as_int(lds4(vsc + 4 * (16 * blk + logit_row<WIDE, T::I8>(i)))) & 0x7fffffff;
            // (rounded up: a weight must not pass the unit)
            const float x = v > 0 && v < F32_INF ? __fadd_ru(s[blk][i], (float)((v >> 23) - 126 - ve)) : -INFINITY;
            far[logit_col<WIDE>(i)] = fmaxf(far[logit_col<WIDE>(i)], x);
        }
    // a row of the largest logit would pass 2^80: a smaller ve (v_scale * 2^(W_EXP - ve) stays finite)
    float least = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        far[c] = column_max<WIDE>(far[c]);
        if (far[c] > -INFINITY) least = fminf(least, fmaxf(far[c] - mx[c], -512.f) + 80.f);
    }
    const int less = max((int)-warp_max(-least), max(-100, -112 - ve));
    ve += less;
    st.vlo += less * (1 << 23);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int d = ve_old - ve;
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < State<WIDE>::NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (State<WIDE>::col(e) == c) big = fmaxf(big, fabsf(st.o[i][e]));
        big = column_max<WIDE>(big);
        const float sum = column_max<WIDE>(st.l[c]);
        float m = fmaxf(__fadd_ru(far[c], (float)-less), mx[c] - 90.f);                   // this tile's terms of the sum: 2^90
        if (sum > 0.f) m = fmaxf(m, st.m[c] + (float)(max(exp_above(sum), -30) - 90));      // the sum: 2^90
        if (big > 0.f) m = fmaxf(m, __fadd_ru(st.m[c], (float)(d + max(exp_above(big), -30) - 30)));  // o: 2^30
        if (m == -INFINITY) continue;  // (nothing so far)
        m = ceilf(m);
        const float fl = ex2(st.m[c] - m), fo = ex2(fminf(st.m[c] - m + (float)d, 126.f));
        st.l[c] *= fl;
#pragma unroll
        for (int i = 0; i < State<WIDE>::NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (State<WIDE>::col(e) == c) st.o[i][e] *= fo;
        st.m[c] = mx[c] = m;
    }
}

// This warp's rows of a tile.
//
// The products of one tile start from zero on the tensor cores, which truncate their sums,
// and join the running sum rounded to nearest (the same fused multiply-add that rescales
// it): summing a 1M-token sequence on the tensor cores alone drifted by 1.1e-5.
template <class T, bool DIFF, int PARTS>
__device__ __forceinline__ void compute(State<T::WIDE> &st, const QF &qf, const QShared &qs, uint32_t stage) {
    constexpr bool ROW8 = T::ROW8, WIDE = T::WIDE;
    constexpr int BLK = T::BLK;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, mat = lane >> 3, r8 = lane & 7;
    const int wr = (threadIdx.x >> 5) * T::WROWS;  // this warp's first row (a multiple of 16)
    const uint32_t sk = stage + wr * T::ROW, sv = sk + T::KV, sc = stage + T::AUX + 4 * wr;
    constexpr uint32_t ALL = (uint32_t)((1ull << T::WROWS) - 1);
    const uint32_t rows = (__float_as_uint(lds4(stage + T::MASK + 4 * (wr / 32))) >> (wr % 32)) & ALL;
    if (rows == 0) return;

    int mine = 0;  // e4m3: the bits of the value scale of row `lane`
    bool fresh = false;
    if (ROW8 && T::EARLY) {
        mine = __float_as_int(lds4(sc + 4 * (T::ROWS + lane))) & 0x7fffffff;
        bool zero;
        int hi;
        if (st.vlo == V_NONE) fresh = first_tile<WIDE, T::I8>(st, mine, (rows >> lane) & 1u, sv, zero, hi);
    }

    // Logits s[blk][i]: narrow: rows g (i = 0, 1) and g+8 (2, 3) of columns 2t, 2t+1 (even and
    // odd i); wide: columns g (i = 0, 1, 4, 5) and g+8 of rows 2t, 2t+1 (0..3), 2t+8, 2t+9.
    // The two maps of a differential head accumulate apart (half j of the dimensions is map
    // j), so that a row's infinity in one does not meet the zeros of the other.
    constexpr int NS = WIDE ? 8 : 4;
    float s[BLK][NS];
    {
        float d[BLK][2][NS] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint4 wa[BLK], wb[BLK];
            if (ROW8) {
#pragma unroll
                for (int blk = 0; blk < BLK; ++blk) {
                    wa[blk] = lds16(sk + swz_k<ROW8>(16 * blk + block_row<T::I8>(g), t + 4 * j));
                    wb[blk] = lds16(sk + swz_k<ROW8>(16 * blk + block_row<T::I8>(g + 8), t + 4 * j));
                }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int ks = 4 * j + w, acc = DIFF ? j : 0;
                uint4 qw;
                if (WIDE) qw = qs[ks][lane];
                const uint32_t qa[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
                for (int blk = 0; blk < BLK; ++blk) {
                    uint32_t a[4];
                    k_frag<ROW8, T::I8>(a, sk, ks, wa[blk], wb[blk]);
                    float (&dd)[NS] = d[blk][acc];
                    if (WIDE) {
                        mma_t<ROW8>(reinterpret_cast<float (&)[4]>(dd[0]), qa, a[0], a[2]);
                        mma_t<ROW8>(reinterpret_cast<float (&)[4]>(dd[NS - 4]), qa, a[1], a[3]);
                    } else {
                        mma_t<ROW8>(reinterpret_cast<float (&)[4]>(dd[0]), a, qf.b[ks][0], qf.b[ks][1]);
                    }
                }
            }
        }
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int i = 0; i < NS; ++i)
                s[blk][i] = !DIFF ? d[blk][0][i] : WIDE ? d[blk][(i >> 1) & 1][i] : t >= 2 ? d[blk][1][i] : d[blk][0][i];
    }

    // log2-domain logits; row of s[blk][i]: rowof(i).  They are rounded before the maximum is taken
    // from them (no fused multiply-add in the exponent): the largest weight has to be 1 however
    // large the logits.
    auto rowof = [](int i) { return logit_row<WIDE, T::I8>(i); };
    auto colof = [](int i) { return logit_col<WIDE>(i); };
#pragma unroll
    for (int blk = 0; blk < BLK; ++blk) {
        float k[4];  // scales of this lane's rows of the block (narrow: two of them)
        if (ROW8 && WIDE) row_scales<T::I8>(k, sc + 64 * blk);
        else if (ROW8) k[0] = lds4(sc + 4 * (16 * blk + rowof(0))), k[1] = lds4(sc + 4 * (16 * blk + rowof(2)));
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const float kk = ROW8 ? k[WIDE ? (i & 1) + 2 * (i >> 2) : i >> 1] : 1.f;
            s[blk][i] *= kk * qf.f[colof(i)];
        }
    }
    if (rows != ALL) {  // the sequence's end, or a page that is none
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (!((rows >> (16 * blk + rowof(i))) & 1u)) s[blk][i] = -INFINITY;
    }

    // maxima, rescale factors, weights
    float al[2], sh[2], mx[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        mx[c] = -INFINITY;
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (colof(i) == c) mx[c] = fmaxf(mx[c], s[blk][i]);
        mx[c] = column_max<WIDE>(mx[c]);
    }
    float inv = 0.f;
    if (ROW8) {
        if (!T::EARLY) mine = __float_as_int(lds4(sc + 4 * (T::ROWS + lane))) & 0x7fffffff;
        const bool there = (rows >> lane) & 1u;
        // (infinite at first)
        st.rise = T::EARLY && fresh ? 0.f : st.rise + fmaxf(fmaxf(mx[0] - st.m[0], mx[1] - st.m[1]), 0.f);
        if (__any_sync(0xffffffffu, (there && (unsigned)(mine - st.vlo) > V_RANGE) || st.rise > M_RISE))
            new_unit<T>(st, s, mx, mine, there, sv, sc + 4 * T::ROWS);
        inv = pow2f(W_EXP - st.ve());
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        // the shift: 0 until a row has been seen, so that no infinities are subtracted
        const float mn = fmaxf(st.m[c], mx[c]);
        sh[c] = mn == -INFINITY ? 0.f : mn;
        al[c] = ex2(st.m[c] - sh[c]);
        st.m[c] = mn;
        st.l[c] *= al[c];
    }
    uint32_t pf[BLK][PARTS][NS / 2];  // weights as the second product's operand
#pragma unroll
    for (int blk = 0; blk < BLK; ++blk) {
        float v[4];
        const uint32_t vsc = sc + 4 * (T::ROWS + 16 * blk);
        if (ROW8 && WIDE) {
            row_scales<T::I8>(v, vsc);
            v[0] *= inv, v[1] *= inv, v[2] *= inv, v[3] *= inv;
        } else if (ROW8) {
            v[0] = lds4(vsc + 4 * rowof(0)) * inv, v[1] = lds4(vsc + 4 * rowof(2)) * inv;
        }
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
            float x = ex2(s[blk][i] - sh[colof(i)]), y = ex2(s[blk][i + 1] - sh[colof(i + 1)]);
            st.l[colof(i)] += x;
            st.l[colof(i + 1)] += y;
            if (ROW8) {
                x *= v[WIDE ? 2 * (i >> 2) : i >> 1];
                y *= v[WIDE ? 1 + 2 * (i >> 2) : i >> 1];
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const uint32_t h = part16<ROW8>(x, y);
                pf[blk][k][i / 2] = WIDE ? h : movmatrix_t(h);
            }
        }
    }

    // O = O diag(al) + P V, 16 dimensions at a time, lowest parts first.  a: V fragment with
    // {dimension set 0 | 1} x {rows 2t, 2t+1 | 2t+8, 2t+9}
    auto add = [&](int mt, const uint32_t (&a)[BLK][4]) {
        float d[WIDE ? 2 : 1][4] = {};
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int k = PARTS - 1; k >= 0; --k) {
                if (WIDE) {
                    const uint32_t p[4] = {pf[blk][k][0], pf[blk][k][1], pf[blk][k][NS / 2 - 2], pf[blk][k][NS / 2 - 1]};
                    mma_t<ROW8>(d[0], p, a[blk][0], a[blk][2]);
                    mma_t<ROW8>(d[WIDE ? 1 : 0], p, a[blk][1], a[blk][3]);
                } else {
                    mma_t<ROW8>(d[0], a[blk], pf[blk][k][0], pf[blk][k][1]);
                }
            }
#pragma unroll
        for (int k = 0; k < (WIDE ? 2 : 1); ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float &o = st.o[WIDE ? 2 * mt + k : mt][e];
                o = fmaf(o, al[State<WIDE>::col(e)], d[k][e]);
            }
    };
    if (T::I8) {
        // words of dimensions g and g + 8 of a block's 16, rows 4t .. 4t+3; all of them asked for at once (two
        // sets at a time: 395 us for 380 at 1M tokens; before the maxima: 391)
        uint32_t x[4][BLK][4];
#pragma unroll
        for (int mt = 0; mt < 8; mt += 2)
#pragma unroll
            for (int blk = 0; blk < BLK; ++blk)
                ldsm_b8_t(sv + swz_v<ROW8, T::I8>(16 * blk + (lane & 15), mt + (lane >> 4)), x[mt / 2][blk]);
#pragma unroll
        for (int mt = 0; mt < 8; mt += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t a[BLK][4];
#pragma unroll
                for (int blk = 0; blk < BLK; ++blk) {
                    widen<T::I8>(x[mt / 2][blk][2 * k], a[blk][0], a[blk][2]);
                    widen<T::I8>(x[mt / 2][blk][2 * k + 1], a[blk][1], a[blk][3]);
                }
                add(mt + k, a);
            }
        }
    } else if (ROW8) {
        // rows 2t, 2t+1, 2t+8, 2t+9 of a block, dimensions 16g .. 16g+15: word w holds
        // dimensions 16g + 4w .. +3, the sets 0 and 1 of mt = 2w, then of 2w + 1
        uint4 x[BLK][4];
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[blk][i] = lds16(sv + swz_v<ROW8, T::I8>(16 * blk + 2 * t + (i & 1) + 8 * (i >> 1), g));
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            const uint32_t sel = mt & 1 ? 0x7362u : 0x5140u;
            uint32_t a[BLK][4];
#pragma unroll
            for (int blk = 0; blk < BLK; ++blk) {
                widen<T::I8>(__byte_perm(word(x[blk][0], mt >> 1), word(x[blk][1], mt >> 1), sel), a[blk][0], a[blk][1]);
                widen<T::I8>(__byte_perm(word(x[blk][2], mt >> 1), word(x[blk][3], mt >> 1), sel), a[blk][2], a[blk][3]);
            }
            add(mt, a);
        }
    } else {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[BLK][4];
            ldsm_x4_t(sv + swz_v<ROW8, T::I8>((mat >> 1) * 8 + r8, 2 * mt + (mat & 1)), a[0][0], a[0][1], a[0][2], a[0][3]);
            add(mt, a);
        }
    }
}

// A unit's end: the four warps' states become one partial in `dst` ([columns][PART_W]).
// Accumulators pass through the stage that has just been consumed (word i of lane l at
// i*32 + l), maxima and sums through `ex`.  Called by the whole CTA.
struct Exchange {
    float m[CT_WARPS][16], l[CT_WARPS][16];
};
template <bool WIDE>
__device__ __forceinline__ int lane_column(int c) {  // the lane's column c (0, 1) among all
    const int lane = threadIdx.x & 31;
    return WIDE ? (lane >> 2) + 8 * c : 2 * (lane & 3) + c;
}
template <bool WIDE>
__device__ __forceinline__ void state_put(const State<WIDE> &st, float *x, Exchange &ex) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < State<WIDE>::NT * 4; ++i) x[i * 32 + lane] = st.o[i >> 2][i & 3];
    if (WIDE ? (lane & 3) == 0 : lane < 4) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            ex.m[w][lane_column<WIDE>(c)] = st.m[c];
            ex.l[w][lane_column<WIDE>(c)] = st.l[c];
        }
    }
}
template <bool WIDE>
__device__ __forceinline__ void state_fold(State<WIDE> &st, const float *x, const Exchange &ex, int from) {
    const int lane = threadIdx.x & 31;
    float mine[2], his[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float m2 = ex.m[from][lane_column<WIDE>(c)], mn = fmaxf(st.m[c], m2);
        const float sh = mn == -INFINITY ? 0.f : mn;
        mine[c] = ex2(st.m[c] - sh);
        his[c] = ex2(m2 - sh);
        st.m[c] = mn;
        st.l[c] = st.l[c] * mine[c] + ex.l[from][lane_column<WIDE>(c)] * his[c];
    }
#pragma unroll
    for (int i = 0; i < State<WIDE>::NT * 4; ++i) {
        const int c = State<WIDE>::col(i & 3);
        st.o[i >> 2][i & 3] = st.o[i >> 2][i & 3] * mine[c] + x[i * 32 + lane] * his[c];
    }
}

template <class T, bool DIFF>
__device__ __forceinline__ void flush(State<T::WIDE> &st, float *x, Exchange &ex, const CacheArgs &a, float *dst) {
    constexpr bool ROW8 = T::ROW8, WIDE = T::WIDE, E4M3 = T::ROW8 && !T::I8;  // (int8's dimensions are in the order of bf16's)
    using S = State<WIDE>;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int SW = S::NT * 4 * 32;  // words of a warp's accumulators
    static_assert(T::XCH == 2 * SW * 4 && T::AUX >= T::XCH, "two states fit in a stage");
    if (ROW8) {  // to the values' own unit
        const float u = pow2f(st.vlo == V_NONE ? 0 : st.ve() - W_EXP);
#pragma unroll
        for (int i = 0; i < S::NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[i][e] *= u;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = WIDE ? 1 : 4; o < (WIDE ? 4 : 32); o <<= 1) st.l[c] += __shfl_xor_sync(0xffffffffu, st.l[c], o);
    __syncthreads();  // every warp has read its rows of the stage
    if (w >= 2) state_put(st, x + (w - 2) * SW, ex);
    __syncthreads();
    if (w < 2) state_fold(st, x + w * SW, ex, w + 2);
    if (w == 1) {
        __syncwarp();
        state_put(st, x + SW, ex);
    }
    __syncthreads();
    if (w != 0) return;
    state_fold(st, x + SW, ex, 1);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        int map, head;
        column<DIFF, WIDE>(lane_column<WIDE>(c), map, head);
        if (head >= a.G) continue;
        float *r = dst + (int64_t)(map * a.G + head) * PART_W;
        if ((WIDE ? t : g) == 0) *reinterpret_cast<float2 *>(r) = make_float2(st.m[c], st.l[c]);
        r += PART_ACC;
        if (WIDE) {
            // o[2 mt + k][2c + e]: e4m3: dimension 16(2t + e) + 2 mt + k; bf16: 16 mt + 8 k + 2t + e
#pragma unroll
            for (int i = 0; i < S::NT; i += E4M3 ? 4 : 1) {
                if (E4M3) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4 *>(r + 16 * (2 * t + e) + i) =
                            make_float4(st.o[i][2 * c + e], st.o[(i + 1) % S::NT][2 * c + e],
                                        st.o[(i + 2) % S::NT][2 * c + e], st.o[(i + 3) % S::NT][2 * c + e]);
                } else {
                    *reinterpret_cast<float2 *>(r + 8 * i + 2 * t) = make_float2(st.o[i][2 * c], st.o[i][2 * c + 1]);
                }
            }
        } else {
            // o[mt][c + 2 k]: e4m3: dimension 16 g + 2 mt + k; bf16: 16 mt + 8 k + g
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (E4M3) {
                    *reinterpret_cast<float2 *>(r + 16 * g + 2 * i) = make_float2(st.o[i][c], st.o[i][c + 2]);
                } else {
                    r[16 * i + g] = st.o[i][c];
                    r[16 * i + g + 8] = st.o[i][c + 2];
                }
            }
        }
    }
}

// Weight of a differential head's second map (called by a full warp).
template <bool DIFF>
__device__ __forceinline__ float map_weight(const DiffArgs &d, int head) {
    if (!DIFF) return 0.f;
    const float *L = d.lam + d.lam_stride * head + 2 * (threadIdx.x & 31);
    const float2 x0 = *reinterpret_cast<const float2 *>(L), x1 = *reinterpret_cast<const float2 *>(L + 64);
    const float2 x2 = *reinterpret_cast<const float2 *>(L + 128), x3 = *reinterpret_cast<const float2 *>(L + 192);
    const float e1 = warp_sum(x0.x * x1.x + x0.y * x1.y), e2 = warp_sum(x2.x * x3.x + x2.y * x3.y);
    return expf(e1) - expf(e2) + d.lambda_init;
}

// Running fold of partials: maximum, sum, four dimensions of a lane.
struct Fold {
    float m, l;
    float4 acc;
    __device__ __forceinline__ void init() { m = -INFINITY, l = 0.f, acc = make_float4(0.f, 0.f, 0.f, 0.f); }
    template <int U>
    __device__ __forceinline__ void add(const float2 (&ml)[U], const float4 (&v)[U]) {
        float mn = m;
#pragma unroll
        for (int i = 0; i < U; ++i) mn = fmaxf(mn, ml[i].x);
        const float sh = mn == -INFINITY ? 0.f : mn, f = exp2f(m - sh);
        m = mn;
        l *= f;
        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float fi = exp2f(ml[i].x - sh);
            l += fi * ml[i].y;
            acc.x += fi * v[i].x, acc.y += fi * v[i].y, acc.z += fi * v[i].z, acc.w += fi * v[i].w;
        }
    }
};

// A head's output from the folds of its map (both maps: their difference, the root-mean-square
// norm and its weights), four dimensions a lane of a full warp, from element `at` of out on.
template <bool DIFF, bool BF16OUT>
__device__ __forceinline__ void finish(const Fold (&f)[DIFF ? 2 : 1], float weight, const DiffArgs &d, void *out,
                                       int64_t at) {
    const int lane = threadIdx.x & 31;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < (DIFF ? 2 : 1); ++k) {
        // nothing seen: zeros (a sum that is NaN stays NaN)
        const float x = (f[k].l == 0.f ? 0.f : 1.f / f[k].l) * (k ? -weight : 1.f);
        r.x += x * f[k].acc.x, r.y += x * f[k].acc.y, r.z += x * f[k].acc.z, r.w += x * f[k].acc.w;
    }
    if (DIFF) {
        const float ss = warp_sum(r.x * r.x + r.y * r.y + r.z * r.z + r.w * r.w);
        const float x = (1.f - d.lambda_init) / sqrtf(ss * (1.f / MOG_D) + d.eps);
        const float4 gm = d.gamma ? reinterpret_cast<const float4 *>(d.gamma)[lane] : make_float4(1.f, 1.f, 1.f, 1.f);
        r.x *= x * gm.x, r.y *= x * gm.y, r.z *= x * gm.z, r.w *= x * gm.w;
    }
    const int64_t o = at + 4 * lane;
    if (BF16OUT) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + o) = make_uint2(cvt_bf2(r.x, r.y), cvt_bf2(r.z, r.w));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + o) = r;
    }
}

// A cluster's end: every CTA has its partial at T::PART; CTA r of the cluster takes heads r,
// r + cs, ..., a warp each, and folds them over the cluster's shared memory.
template <class T, bool DIFF, bool BF16OUT>
__device__ __forceinline__ void cluster_end(const CacheArgs &a, const DiffArgs &d, void *out, uint32_t smem, int unit) {
    constexpr int M = DIFF ? 2 : 1, U = 8;
    const int rank = blockIdx.x % a.cs, w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = unit % a.h_kv;
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int head = rank + a.cs * w; head < a.G; head += a.cs * CT_WARPS) {
        Fold f[M];
#pragma unroll
        for (int k = 0; k < M; ++k) {
            f[k].init();
            const uint32_t at = smem + T::PART + (k * a.G + head) * PART_W * 4;
            for (int c0 = 0; c0 < a.cs; c0 += U) {
                float2 ml[U];
                float4 v[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    ml[i] = make_float2(-INFINITY, 0.f), v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c0 + i >= a.cs) continue;
                    uint32_t p;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(at), "r"(c0 + i));
                    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(ml[i].x), "=f"(ml[i].y) : "r"(p));
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(v[i].x), "=f"(v[i].y), "=f"(v[i].z), "=f"(v[i].w) : "r"(p + 4 * PART_ACC + 16 * lane));
                }
                f[k].add(ml, v);
            }
        }
        int64_t at = ((int64_t)unit * a.G + head) * MOG_D;
        if (own_rows(T::ROW8, DIFF)) {
            const int b = unit / a.h_kv;
            if (a.count && a.count[b] <= 0) continue;
            at = b * a.ob + (h * a.G + head) * a.oh;
        }
        finish<DIFF, BF16OUT>(f, map_weight<DIFF>(d, h * a.G + head), d, out, at);
    }
    // nobody leaves while its partial is read
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CLUSTER: the form with a cluster of a.cs CTAs per unit (a kernel of its own: the two in one cost
// the split form registers and 14% of its speed).
template <bool ROW8, bool WIDE, bool PAGED, bool DIFF, bool BF16OUT, bool CLUSTER, bool I8>
__global__ void __launch_bounds__(CT_THREADS, Tile<ROW8, WIDE, CLUSTER, I8>::PER_SM) k_cache_split(CacheArgs a, DiffArgs d, void *out) {
    extern __shared__ __align__(128) uint8_t csm[];
    __shared__ Exchange ex;
    __shared__ QShared qs;  // (wide)
    using T = Tile<ROW8, WIDE, CLUSTER, I8>;
    constexpr int PARTS = weight_parts(ROW8, WIDE, BF16OUT);
    const uint32_t stages = smem_u32(csm);
    const int G2 = DIFF ? 2 * a.G : a.G;
    Cursor<T::ROWS> ci, cc;  // the next tile to copy, the next to compute
    int cnt, pg = -1;  // tiles of this CTA; the page of the next tile's row group `lane`
    if (!CLUSTER) {
        pdl_trigger();
        const int total = total_tiles<T::ROWS>(a);
        const int chunk = (total + gridDim.x - 1) / gridDim.x;
        const int t0 = min((int64_t)blockIdx.x * chunk, (int64_t)total);
        cnt = min(chunk, total - t0);
        if (cnt <= 0) return;
        ci.seek(a, t0);
    } else {  // tiles rank, rank + cs, ... of one unit: the first one's pages are known before its length
        const int u = blockIdx.x / a.cs, rank = blockIdx.x - u * a.cs;
        ci.b = u / a.h_kv, ci.h = u - ci.b * a.h_kv, ci.t = rank;
        if constexpr (PAGED) {
            const int lane = threadIdx.x & 31, col = (rank * T::ROWS + 16 * lane) >> a.pshift;
            if (lane < T::ROWS / 16 && col < a.pps) pg = __ldg(a.bt + (int64_t)ci.b * a.pps + col);
        }
        ci.load(a);
        cnt = ci.nt > rank ? (ci.nt - rank - 1) / a.cs + 1 : 0;
        if (cnt == 0) {  // an empty partial
            for (int i = threadIdx.x; i < G2 * PART_W; i += CT_THREADS)
                reinterpret_cast<float *>(csm + T::PART)[i] = i % PART_W == 0 ? -INFINITY : 0.f;
            cluster_end<T, DIFF, BF16OUT>(a, d, out, stages, u);
            return;
        }
    }
    cc = ci;
    if (!CLUSTER) tile_page<T, PAGED>(a, ci, pg);
    int ahead = 0;  // tiles whose copies have started
    auto feed = [&](uint32_t stage) {
        if (ahead < cnt) {
            issue<T, PAGED>(a, ci, pg, stage);
            if (++ahead < cnt) {
                if (CLUSTER) ci.t += a.cs;
                else ci.next(a);
                tile_page<T, PAGED>(a, ci, pg);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < T::STAGES - 1; ++s) feed(stages + s * T::STAGE);
    int unit = cc.b * a.h_kv + cc.h;
    QF qf;
    load_q<ROW8, DIFF, WIDE>(qf, qs, a, unit);
    State<WIDE> st;
    st.init();
    int slot = 0;
    for (int i = 0; i < cnt; ++i) {
        cp_async_wait<T::STAGES - 2>();
        __syncthreads();  // the tile is there, and the stage before it has been consumed
        feed(stages + (slot == 0 ? T::STAGES - 1 : slot - 1) * T::STAGE);
        compute<T, DIFF, PARTS>(st, qf, qs, stages + slot * T::STAGE);
        const bool end = !CLUSTER && cc.last();
        if (end || i == cnt - 1) {
            float *dst = CLUSTER ? reinterpret_cast<float *>(csm + T::PART)
                              : a.part + ((int64_t)blockIdx.x + unit) * G2 * PART_W;
            flush<T, DIFF>(st, reinterpret_cast<float *>(csm + slot * T::STAGE), ex, a, dst);
            if (i == cnt - 1) break;
            st.init();
        }
        slot = slot + 1 == T::STAGES ? 0 : slot + 1;
        if (!CLUSTER) cc.next(a);
        if (end) {
            unit = cc.b * a.h_kv + cc.h;
            load_q<ROW8, DIFF, WIDE>(qf, qs, a, unit);
        }
    }
    cp_async_wait<0>();
    if (CLUSTER) cluster_end<T, DIFF, BF16OUT>(a, d, out, stages, unit);
}

template <bool ROW8, bool WIDE, bool PAGED, bool DIFF, bool BF16OUT, bool I8>
static cudaError_t launch_split(const CacheArgs &a, const DiffArgs &d, void *out, int splits, cudaStream_t s) {
    const int smem = a.cs ? Tile<ROW8, WIDE, true, I8>::SMEM : Tile<ROW8, WIDE, false, I8>::SMEM;
    const auto fn = a.cs ? k_cache_split<ROW8, WIDE, PAGED, DIFF, BF16OUT, true, I8>
                         : k_cache_split<ROW8, WIDE, PAGED, DIFF, BF16OUT, false, I8>;
    const cudaError_t e = ensure_smem((const void *)fn, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.cs ? a.cs * a.batch * a.h_kv : splits);
    cfg.blockDim = dim3(CT_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.cs;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.cs > 1;
    return cudaLaunchKernelEx(&cfg, fn, a, d, out);
}

// The instance for a call: launches it (a.cs > 0: as clusters, one launch; else the split of
// `splits` CTAs, whose partials k_cache_merge folds).
template <bool ROW8, bool DIFF, bool BF16OUT, bool I8 = false>
static cudaError_t pick_split(const CacheArgs &a, const DiffArgs &d, void *out, bool wide, int splits, cudaStream_t s) {
    if (a.bt) return wide ? launch_split<ROW8, true, true, DIFF, BF16OUT, I8>(a, d, out, splits, s)
                          : launch_split<ROW8, false, true, DIFF, BF16OUT, I8>(a, d, out, splits, s);
    return wide ? launch_split<ROW8, true, false, DIFF, BF16OUT, I8>(a, d, out, splits, s)
                : launch_split<ROW8, false, false, DIFF, BF16OUT, I8>(a, d, out, splits, s);
}

cudaError_t launch_split8(const CacheArgs &a, const DiffArgs &d, void *out, bool diff, bool bf_out, bool wide, int splits,
                          cudaStream_t s);
cudaError_t launch_split16(const CacheArgs &a, const DiffArgs &d, void *out, bool wide, int splits, cudaStream_t s);
cudaError_t launch_spliti8(const CacheArgs &a, const DiffArgs &d, void *out, bool diff, bool bf_out, bool wide, int splits,
                           cudaStream_t s);

}  // namespace mog
