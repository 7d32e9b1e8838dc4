// rows.cu -- rows of new tokens: rotary positions, alone or on the way into a cache
// (mog_rope_apply, mog_rope_store), int8 caches with a scale per block of tokens and head
// (mog_kv_store), and a cache's rows read back (mog_kv_load).
//
// Rotary positions.  Pair i of a row's first rot_dim dimensions is turned by the angle
// pos * f_i.  A frequency is held as turns per position in 64-bit fixed point, so that the angle is
// one integer product whose overflow drops the whole turns: off by less than 2^-31 of a turn at any
// position (in fp32, position 1M would leave a tenth of a radian).  A CTA computes the
// cosines and sines of its tokens once, into shared memory, for all their heads.  A prompt is bound by HBM: 24K tokens of
// 32 + 8 + 8 heads into bf16 pages, 590 MB, 90 us, 6.5 TB/s; a chunk's start and end show (4096 tokens of 40 + 8 + 8 heads,
// 117 MB: 22 us, 5.3 TB/s); a step's tokens are latency: 8 sequences, 4.7 us.  Four CTAs an SM (64 registers) against the
// three of 80: 94.2 us against 95.7, launch included.
//
// A row (256 bytes) is the work of eight lanes, two 16-byte chunks each.  Lane l's chunks hold whole
// pairs in either layout, of the frequencies 8l .. 8l+7: chunks 2l, 2l+1 of neighbouring pairs, chunks
// l, l + rot_dim/16 of pairs half a turned part apart, and so no lane needs another's elements.
#include <algorithm>

#include "rows.cuh"
#include "internal.h"

namespace mog {

// Four int8 codes -> floats: u = code + 128 is the low byte of the number 2^23 + u.
__device__ __forceinline__ float4 i8x4_to_float4(uint32_t w) {
    w ^= 0x80808080u;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 | i)) - 8388736.f;
    return make_float4(f[0], f[1], f[2], f[3]);
}

enum { TO_NONE, TO_BF16, TO_E4M3, TO_I8 };
constexpr int RW_THREADS = 256, RW_GROUPS = RW_THREADS / 8;
constexpr int RW_TOKENS = 16;  // tokens of a CTA's tile of whole rows
constexpr int RW_DEPTH = 4;    // rows in flight per group of lanes
constexpr float I8_MAX = 127.f, I8_LEAST = 1.17549435e-38f;  // 2^-126: the smallest scale of an int8 block

struct RowsArgs {
    const uint16_t *q, *k, *v;  // rows of new tokens; elements between sequences, tokens and heads:
    uint16_t *qo;
    int64_t qb, qt, qh, kb, kt, kh, ob, ot, oh;
    int h_q, h_kv, t_max;
    const int *pos, *count;
    int each;  // pos is [batch][t_max], not the first token's [batch]
    // rotary positions
    const int64_t *turns;
    int rot16, pairs, inverse;
    float factor;
    // cache (bytes between pages or sequences, heads, rows; the scales' in floats)
    uint8_t *K, *V;
    float *ks, *vs;
    int64_t sb, sh, sn, ssb, ssh, ssn;
    const int *bt;
    int pshift, pps, n_pages, n_cap, bshift;
    // the grid: tokens of a tile of whole rows, slices of the heads; int8: 16-row slabs of a tile,
    // slices of its heads, CTAs that store
    int tile, slices, slabs, kv_slices, kv_ctas;
};

// not ld.global.nc: q may be turned in place
__device__ __forceinline__ uint4 ldg_once16(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ int seq_count(const RowsArgs &a, int b) {
    return a.count ? min(max(a.count[b], 0), a.t_max) : a.t_max;
}

// Cosines and sines of tokens t0 .. t0+n-1 of sequence b, the frequencies 8l + 2j, 8l + 2j + 1 at
// cs[token][j][l].
__device__ __forceinline__ void fill_turns(const RowsArgs &a, float4 *cs, int b, int t0, int n) {
    const int nf = 4 * a.rot16;
    for (int i = threadIdx.x; i < n * nf; i += RW_THREADS) {
        const int tok = i / nf, e = i - tok * nf, j = e / a.rot16, l = e - j * a.rot16, t = t0 + tok;
        const int64_t p = a.each ? (int64_t)a.pos[(int64_t)b * a.t_max + t] : (int64_t)a.pos[b] + t;
        float c[2], s[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint64_t phase = (uint64_t)p * (uint64_t)a.turns[8 * l + 2 * j + x];
            // quarter turns and an eighth of a turn at most, so that rounding it to fp32 costs 2^-25.3 radians (2^-23.3 if half
            // a turn were rounded; more than the rest of the error together)
            const uint32_t turn = (uint32_t)(phase >> 32), quarter = (turn + (1u << 29)) >> 30;
            float co, si;
            sincospif((float)(int)(turn - (quarter << 30)) * 4.656612873077393e-10f, &si, &co);
            const float fc = quarter + 1 & 2 ? -a.factor : a.factor, fs = (quarter >> 1 & 1) != a.inverse ? -a.factor : a.factor;
            c[x] = (quarter & 1 ? si : co) * fc;
            s[x] = (quarter & 1 ? co : si) * fs;
        }
        cs[i] = make_float4(c[0], s[0], c[1], s[1]);
    }
}

// First elements of the lane's two chunks of a row.
__device__ __forceinline__ int2 lane_chunks(const RowsArgs &a, bool turn) {
    const int l = threadIdx.x & 7;
    return turn && !a.pairs && l < a.rot16 ? make_int2(8 * l, 8 * (l + a.rot16)) : make_int2(16 * l, 16 * l + 8);
}

__device__ __forceinline__ uint2 turned(float x, float y, float c, float s) {
    return make_uint2(__float_as_uint(fmaf(x, c, -y * s)), __float_as_uint(fmaf(y, c, x * s)));
}

// The lane's 16 elements, turned: rounded once, to bf16.
__device__ __forceinline__ void turn_row(uint32_t (&w)[8], const RowsArgs &a, const float4 *cs) {
    const int l = threadIdx.x & 7;
    if (l >= a.rot16) return;
    if (a.pairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 z = cs[j * a.rot16 + l];
            const uint2 p = turned(bf_lo(w[2 * j]), bf_hi(w[2 * j]), z.x, z.y);
            const uint2 r = turned(bf_lo(w[2 * j + 1]), bf_hi(w[2 * j + 1]), z.z, z.w);
            w[2 * j] = cvt_bf2(__uint_as_float(p.x), __uint_as_float(p.y));
            w[2 * j + 1] = cvt_bf2(__uint_as_float(r.x), __uint_as_float(r.y));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 z = cs[j * a.rot16 + l];
            const uint2 p = turned(bf_lo(w[j]), bf_lo(w[4 + j]), z.x, z.y);
            const uint2 r = turned(bf_hi(w[j]), bf_hi(w[4 + j]), z.z, z.w);
            w[j] = cvt_bf2(__uint_as_float(p.x), __uint_as_float(r.x));
            w[4 + j] = cvt_bf2(__uint_as_float(p.y), __uint_as_float(r.y));
        }
    }
}

__device__ __forceinline__ void load_chunks(uint32_t (&w)[8], const uint16_t *row, int2 at) {
    const uint4 x = ldg_once16(row + at.x), y = ldg_once16(row + at.y);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
}
__device__ __forceinline__ void store_chunks(uint16_t *row, int2 at, const uint32_t (&w)[8]) {
    *reinterpret_cast<uint4 *>(row + at.x) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(row + at.y) = make_uint4(w[4], w[5], w[6], w[7]);
}

// The slab and row of a position of sequence b; false if it is outside the cache or in no page.
__device__ __forceinline__ bool find_row(const RowsArgs &a, int b, int pos, int &slab, int &row) {
    if (pos < 0 || pos >= a.n_cap) return false;
    slab = b, row = pos;
    if (a.bt) {
        slab = __ldg(a.bt + (int64_t)b * a.pps + (pos >> a.pshift));
        row = pos & ((1 << a.pshift) - 1);
        if ((unsigned)slab >= (unsigned)a.n_pages) return false;
    }
    return true;
}

// Tokens t0 .. t0+n-1 of sequence b, heads h0 .. h0+nh-1 of the list queries, keys, values: a
// group of eight lanes takes every 32nd (token, head), heads fastest.
template <int TO>
__device__ __forceinline__ void whole_rows(const RowsArgs &a, const float4 *cs, int b, int t0, int n, int h0, int nh) {
    const int total = n * nh, dt = RW_GROUPS / nh, dh = RW_GROUPS - dt * nh;
    const unsigned group = 0xffu << (threadIdx.x & 24);
    int r = threadIdx.x / 8, t = r / nh, h = r - t * nh;
    for (; r < total; r += RW_GROUPS * RW_DEPTH) {
        uint32_t w[RW_DEPTH][8];
        int tt[RW_DEPTH], hh[RW_DEPTH];
#pragma unroll
        for (int u = 0; u < RW_DEPTH; ++u) {
            tt[u] = t, hh[u] = h0 + h;
            t += dt, h += dh;
            if (h >= nh) h -= nh, ++t;
            if (r + u * RW_GROUPS >= total) continue;
            const bool isq = hh[u] < a.h_q, isv = hh[u] >= a.h_q + a.h_kv;
            const int64_t tok = t0 + tt[u];
            const uint16_t *row = isq ? a.q + b * a.qb + tok * a.qt + hh[u] * a.qh
                                      : (isv ? a.v : a.k) + b * a.kb + tok * a.kt + (hh[u] - a.h_q - (isv ? a.h_kv : 0)) * a.kh;
            load_chunks(w[u], row, lane_chunks(a, !isv));
        }
#pragma unroll
        for (int u = 0; u < RW_DEPTH; ++u) {
            if (r + u * RW_GROUPS >= total) continue;
            const bool isq = hh[u] < a.h_q, isv = hh[u] >= a.h_q + a.h_kv;
            const int2 at = lane_chunks(a, !isv);
            const int tok = t0 + tt[u];
            if (!isv) turn_row(w[u], a, cs + tt[u] * 4 * a.rot16);
            if (isq) {
                store_chunks(a.qo + b * a.ob + (int64_t)tok * a.ot + hh[u] * a.oh, at, w[u]);
                continue;
            }
            if (TO == TO_NONE) continue;
            int slab, row;
            if (!find_row(a, b, (int)((unsigned)a.pos[b] + (unsigned)tok), slab, row)) continue;  // (past 2^31: negative)
            const int head = hh[u] - a.h_q - (isv ? a.h_kv : 0);
            uint8_t *dst = (isv ? a.V : a.K) + slab * a.sb + head * a.sh + row * a.sn;
            if (TO == TO_BF16) {
                store_chunks(reinterpret_cast<uint16_t *>(dst), at, w[u]);
                continue;
            }
            const int e = e4m3_row_exp<8>(w[u], group);
            const uint32_t inv2 = bf2_pow2_neg(e);
            uint32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = e4m3_pair(bf2_mul(w[u][i], inv2));
            *reinterpret_cast<uint2 *>(dst + at.x) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
            *reinterpret_cast<uint2 *>(dst + at.y) = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
            if ((threadIdx.x & 7) == 0)
                (isv ? a.vs : a.ks)[slab * a.ssb + head * a.ssh + row * a.ssn] = __int_as_float((e + 127) << 23);
        }
    }
}

template <int TO>
__global__ void __launch_bounds__(RW_THREADS, 4) k_rope_rows(RowsArgs a) {
    extern __shared__ float4 cs[];
    const int b = blockIdx.y, tile = blockIdx.x / a.slices, slice = blockIdx.x - tile * a.slices;
    const int t0 = tile * a.tile, n = min(a.tile, seq_count(a, b) - t0);
    const int heads = a.h_q + 2 * a.h_kv, per = (heads + a.slices - 1) / a.slices;
    const int h0 = slice * per, nh = min(per, heads - h0);
    if (n <= 0 || nh <= 0) return;
    fill_turns(a, cs, b, t0, n);
    __syncthreads();
    whole_rows<TO>(a, cs, b, t0, n, h0, nh);
}

// ------------------------------------------------------------------------------------
// int8 blocks.  A block of 2^bshift rows (16 .. 128) of one head has one scale s; its rows stand for
// s * code.  New rows behind those that the block holds raise its scale to amax / 127 if their
// largest magnitude needs it, and the codes it holds are then rounded anew (code * old/new); a
// block that holds none starts afresh.  s >= 2^-126, so that 1/s is finite.
//
// A warp takes 16 rows of one head's keys or values, in registers between the maximum and the
// rounding (one pass over the rows); a block is the work of one warp or of up to 8, which share their
// maxima in shared memory.  A CTA's tile is `slabs` times 16 positions, and 8 / slabs heads at a time.
//
// Bound by HBM together with the waits between a tile's loads and its maxima: 4 prompts, 24K tokens of 8 heads into 64-row
// pages, 100 MB read and 50 MB written: 27 us, 5.6 TB/s (issue 51%); with 32 query heads turned too, 22.5 KB a token: 85 us, 5.9 TB/s.
// With turns, registers for three CTAs an SM: 92 us for pairs in half the row and 102 for halves of all of it, launch included
// (100 and 106 as the compiler chooses them; 92 and 107 for four, where they spill); without turns, for four: as fast as three.
// ------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t u16x2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two elements' codes in bytes 0 and 1, as x * inv rounded to nearest even (|x * inv| < 2^22): the low byte of
// the number raised by 1.5 * 2^23.  CLAMP: infinities become +-127.
template <bool CLAMP>
__device__ __forceinline__ uint32_t i8_pair(uint32_t w, float inv) {
    float x = __fmul_rn(bf_lo(w), inv), y = __fmul_rn(bf_hi(w), inv);
    if (CLAMP) x = fminf(fmaxf(x, -I8_MAX), I8_MAX), y = fminf(fmaxf(y, -I8_MAX), I8_MAX);
    return __byte_perm(__float_as_uint(__fadd_rn(x, 12582912.f)), __float_as_uint(__fadd_rn(y, 12582912.f)), 0x0040);
}
template <bool CLAMP>
__device__ __forceinline__ void store_codes(uint8_t *row, int2 at, const uint32_t (&w)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __byte_perm(i8_pair<CLAMP>(w[2 * i], inv), i8_pair<CLAMP>(w[2 * i + 1], inv), 0x5410);
    *reinterpret_cast<uint2 *>(row + at.x) = make_uint2(c[0], c[1]);
    *reinterpret_cast<uint2 *>(row + at.y) = make_uint2(c[2], c[3]);
}
// four codes times `ratio`, rounded to nearest even
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __fmul_rn((float)((int)(w << (24 - 8 * i)) >> 24), ratio);
        r |= (__float_as_uint(__fadd_rn(x, 12582912.f)) & 0xffu) << (8 * i);
    }
    return r;
}

constexpr uint32_t I8_NAN = 0xffffu;  // a maximum: there is a NaN

template <bool TURN>
__global__ void __launch_bounds__(RW_THREADS, TURN ? 3 : 4) k_rows_i8(RowsArgs a) {
    extern __shared__ float4 cs[];
    __shared__ uint32_t s_amax[2][RW_THREADS / 32];
    const int b = blockIdx.y, count = seq_count(a, b);
    if (TURN && (int)blockIdx.x >= a.kv_ctas) {  // the queries
        const int x = blockIdx.x - a.kv_ctas, tile = x / a.slices, slice = x - tile * a.slices;
        const int t0 = tile * a.tile, n = min(a.tile, count - t0);
        const int per = (a.h_q + a.slices - 1) / a.slices, h0 = slice * per, nh = min(per, a.h_q - h0);
        if (n <= 0 || nh <= 0) return;
        fill_turns(a, cs, b, t0, n);
        __syncthreads();
        whole_rows<TO_NONE>(a, cs, b, t0, n, h0, nh);
        return;
    }
    const int64_t start = a.pos[b];
    const int lo = (int)max(start, (int64_t)0), hi = (int)max((int64_t)0, min(start + count, (int64_t)a.n_cap));  // the new rows' positions
    const int span = 16 * a.slabs, tile = blockIdx.x / a.kv_slices, slice = blockIdx.x - tile * a.kv_slices;
    const int64_t p0 = (int64_t)(lo / span + tile) * span;
    if (lo >= hi || p0 >= hi) return;
    const int base = (int)p0, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slab = w & (a.slabs - 1), s0 = base + 16 * slab, bw = 1 << (a.bshift - 4);
    const int b0 = s0 & -(1 << a.bshift);  // the block's first position
    const bool held = b0 < lo;  // it holds rows
    int page = 0, row0 = 0;     // where position s0 is
    const bool mine = b0 < hi && (int64_t)b0 + (1 << a.bshift) > lo && find_row(a, b, b0, page, row0);
    row0 += s0 - b0;
    int turn0 = 0;  // the position of the first token in cs
    if (TURN) {
        const int first = max(base, lo);  // (tokens before it are not turned here)
        fill_turns(a, cs, b, (int)(first - start), (int)min((int64_t)hi, p0 + span) - first);
        __syncthreads();
        turn0 = first;
    }
    const int heads = 2 * a.h_kv, per = (heads + a.kv_slices - 1) / a.kv_slices, step = RW_THREADS / 32 / a.slabs;
    const int j0 = slice * per, j1 = min(j0 + per, heads);
    for (int jb = j0, it = 0; jb < j1; jb += step, it ^= 1) {
        const int j = jb + w / a.slabs, head = j < a.h_kv ? j : j - a.h_kv;
        const bool isv = j >= a.h_kv, active = mine && j < j1;
        const int2 at = lane_chunks(a, TURN && !isv);
        const uint16_t *src = (isv ? a.v : a.k) + b * a.kb + head * a.kh;
        uint32_t x[4][8];
        unsigned here = 0;  // bit i: row 4i + lane/8 is new
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = s0 + 4 * i + (lane >> 3);
            if (active && p >= lo && p < hi) {
                here |= 1u << i;
                load_chunks(x[i], src + (p - start) * a.kt, at);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[i][k] = 0;
            }
        }
        float *scale = (isv ? a.vs : a.ks) + page * a.ssb + head * a.ssh + (row0 >> a.bshift) * a.ssn;
        const float old = active && held ? *scale : 0.f;
        if (TURN && !isv) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (here >> i & 1) turn_row(x[i], a, cs + (s0 + 4 * i + (lane >> 3) - turn0) * 4 * a.rot16);
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) m = u16x2_max(m, x[i][k] & 0x7fff7fffu);
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        const bool special = m >= 0x7f80u;
        if (special) {  // the largest finite magnitude, or a NaN
            uint32_t fin = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t p = x[i][k] & 0x7fffu, q = x[i][k] >> 16 & 0x7fffu;
                    fin = max(fin, max(p < 0x7f80u ? p : 0u, q < 0x7f80u ? q : 0u));
                }
            m = m > 0x7f80u ? I8_NAN : __reduce_max_sync(0xffffffffu, fin);
        }
        if (lane == 0) s_amax[it][w] = m;
        __syncthreads();  // (two buffers: the next round's maxima do not meet this one's readers)
        if (!active) continue;
        const int w0 = w & -bw;  // the block's warps
        for (int k = 0; k < bw; ++k) m = max(m, s_amax[it][w0 + k]);
        float s = fmaxf(fmaxf(old, __fmul_rn(__uint_as_float(m << 16), 1.f / I8_MAX)), I8_LEAST);
        if (m == I8_NAN || old != old) s = __int_as_float(0x7fffffff);  // a NaN: all of the block's rows are
        const float inv = __frcp_rn(s);
        if ((w & (bw - 1)) == 0 && lane == 0) *scale = s;
        if (s != s) continue;  // (codes stay)
        uint8_t *dst = (isv ? a.V : a.K) + page * a.sb + head * a.sh + row0 * a.sn;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!(here >> i & 1)) continue;
            uint8_t *row = dst + (4 * i + (lane >> 3)) * a.sn;
            if (special) store_codes<true>(row, at, x[i], inv);
            else store_codes<false>(row, at, x[i], inv);
        }
        if (held && s > old) {  // the codes that the slab holds, 16 a lane
            const float ratio = __fdiv_rn(old, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (s0 + 4 * i + (lane >> 3) >= lo) continue;
                uint4 *p = reinterpret_cast<uint4 *>(dst + (4 * i + (lane >> 3)) * a.sn + 16 * (lane & 7));
                const uint4 c = *p;
                *p = make_uint4(rescaled(c.x, ratio), rescaled(c.y, ratio), rescaled(c.z, ratio), rescaled(c.w, ratio));
            }
        }
    }
}

// ------------------------------------------------------------------------------------
// mog_kv_load: rows of a cache as bf16, eight lanes a row; bound by HBM, and close to it by the
// instructions of the addresses, so that a group of lanes keeps to one head's keys or values: of its
// addresses only the page and the row change (24K tokens of 8 heads from 64-row pages, 50 MB read, 100 MB
// written, 22 us of HBM time: 29 us, and 39 with heads fastest in one list).
// ------------------------------------------------------------------------------------
template <int FROM>
__global__ void __launch_bounds__(RW_THREADS) k_kv_load(RowsArgs a, uint16_t *ko, uint16_t *vo, int out32) {
    const int b = blockIdx.y, l = threadIdx.x & 7, per = 2 * a.h_kv, grp = threadIdx.x / 8;
    const int n = seq_count(a, b), start = a.pos[b];
    // groups side by side: per <= 32: whole tokens (the groups left over have nothing); else the heads in turns
    const int tokens = per <= RW_GROUPS ? RW_GROUPS / per : 1, wide = min(per, RW_GROUPS);
    const int tl = grp / wide;
    if (tl >= tokens) return;
    const int step = tokens * gridDim.x;
    for (int r = grp - tl * wide; r < per; r += wide) {
        const bool val = r >= a.h_kv;
        const int h = val ? r - a.h_kv : r;
        uint16_t *out = (val ? vo : ko) + b * a.kb + h * a.kh + 16 * l;
        const uint8_t *in = (val ? a.V : a.K) + h * a.sh + (FROM == TO_BF16 ? 32 : 16) * l;
        const float *scale = (val ? a.vs : a.ks) + h * a.ssh;
        for (int t = blockIdx.x * tokens + tl; t < n; t += step * RW_DEPTH) {
            uint4 x[RW_DEPTH], y[RW_DEPTH];
            float s[RW_DEPTH];
            bool have[RW_DEPTH];
#pragma unroll
            for (int u = 0; u < RW_DEPTH; ++u) {
                int slab, row;
                have[u] = t + u * step < n && find_row(a, b, (int)((unsigned)start + (unsigned)(t + u * step)), slab, row);
                if (!have[u]) continue;
                const uint8_t *src = in + slab * a.sb + row * a.sn;
                x[u] = ldg_nc16(src);
                if (FROM == TO_BF16) y[u] = ldg_nc16(src + 16);
                else s[u] = __ldg(scale + slab * a.ssb + (row >> a.bshift) * a.ssn);
            }
#pragma unroll
            for (int u = 0; u < RW_DEPTH; ++u) {
                if (!have[u]) continue;
                if (FROM != TO_BF16) {
                    const uint32_t c[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float4 f;
                        if (FROM == TO_E4M3) f = e4m3x4_to_float4(c[k]);
                        else f = i8x4_to_float4(c[k]);
                        o[2 * k] = cvt_bf2(f.x * s[u], f.y * s[u]), o[2 * k + 1] = cvt_bf2(f.z * s[u], f.w * s[u]);
                    }
                    x[u] = make_uint4(o[0], o[1], o[2], o[3]), y[u] = make_uint4(o[4], o[5], o[6], o[7]);
                }
                uint16_t *dst = out + (int64_t)(t + u * step) * a.kt;
                if (out32) {
                    stg32(dst, x[u], y[u]);
                } else {
                    *reinterpret_cast<uint4 *>(dst) = x[u];
                    *reinterpret_cast<uint4 *>(dst + 8) = y[u];
                }
            }
        }
    }
}

// --------------------------------------------------------------------------- launches

static void set_cache(RowsArgs &a, const mog_cache *c) {
    const int es = c->type == MOG_CACHE_BF16 ? 2 : 1;
    const int64_t cap = c->block_table ? (int64_t)c->pages_per_seq * c->page_rows : c->n_cap;
    a.K = static_cast<uint8_t *>(c->k), a.V = static_cast<uint8_t *>(c->v), a.ks = c->k_scale, a.vs = c->v_scale;
    a.sb = c->stride_b * es, a.sh = c->stride_h * es, a.sn = c->stride_n * es;
    a.ssb = c->scale_b, a.ssh = c->scale_h, a.ssn = c->scale_n;
    a.bt = c->block_table, a.pshift = c->block_table ? log2_exact(c->page_rows) : 0, a.pps = c->pages_per_seq;
    a.n_pages = c->n_pages, a.n_cap = (int)std::min<int64_t>(cap, INT32_MAX);
    a.bshift = c->type == MOG_CACHE_I8 ? log2_exact(c->block_rows) : 0;
}

static void set_rows(RowsArgs &a, const RowsIn &r) {
    a.q = static_cast<const uint16_t *>(r.q), a.qo = static_cast<uint16_t *>(r.qo);
    a.k = static_cast<const uint16_t *>(r.k), a.v = static_cast<const uint16_t *>(r.v);
    a.qb = r.qs[0], a.qt = r.qs[1], a.qh = r.qs[2], a.ob = r.os[0], a.ot = r.os[1], a.oh = r.os[2];
    a.kb = r.ks[0], a.kt = r.ks[1], a.kh = r.ks[2];
    a.h_q = r.h_q, a.h_kv = r.h_kv, a.t_max = r.t_max, a.pos = r.pos, a.count = r.count, a.each = r.each;
    if (!r.rope) return;
    a.turns = r.rope->turns, a.rot16 = r.rope->rot_dim / 16, a.pairs = r.rope->layout == MOG_ROPE_PAIRS;
    a.inverse = r.inverse, a.factor = r.rope->factor;
}

// CTAs for `tiles` tiles of each sequence: as many slices of the heads as give every SM four, but
// no slice with less than a round of work.
static int head_slices(int64_t tiles, int batch, int64_t most) {
    const int64_t want = ceil_div64(4LL * num_sms(), tiles * batch);
    return (int)std::max<int64_t>(1, std::min(want, most));
}

cudaError_t launch_rope(const mog_cache *c, int batch, const RowsIn &r, cudaStream_t s) {
    RowsArgs a{};
    if (c) set_cache(a, c);
    set_rows(a, r);
    a.tile = std::min(RW_TOKENS, r.t_max);
    const int heads = r.h_q + 2 * r.h_kv;
    const int64_t tiles = ceil_div64(r.t_max, a.tile);
    a.slices = head_slices(tiles, batch, ceil_div64((int64_t)heads * a.tile, RW_GROUPS));
    a.slices = std::min(a.slices, heads);
    const dim3 grid((unsigned)(tiles * a.slices), batch);
    const size_t smem = (size_t)a.tile * 4 * a.rot16 * sizeof(float4);
    if (!c) k_rope_rows<TO_NONE><<<grid, RW_THREADS, smem, s>>>(a);
    else if (c->type == MOG_CACHE_BF16) k_rope_rows<TO_BF16><<<grid, RW_THREADS, smem, s>>>(a);
    else k_rope_rows<TO_E4M3><<<grid, RW_THREADS, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_rows_i8(const mog_cache *c, int batch, const RowsIn &r, cudaStream_t s) {
    RowsArgs a{};
    set_cache(a, c);
    set_rows(a, r);
    // 64 positions a tile, or a block if that is more; a step's few tokens: a block
    const int bw = c->block_rows / 16;
    a.slabs = r.t_max >= 64 ? std::max(bw, 4) : bw;
    const int span = 16 * a.slabs, step = RW_THREADS / 32 / a.slabs;
    const int64_t tiles = ((int64_t)r.t_max + span - 2) / span + 1;
    a.kv_slices = head_slices(tiles, batch, ceil_div64(2 * r.h_kv, step));
    a.kv_ctas = (int)(tiles * a.kv_slices);
    int64_t ctas = a.kv_ctas;
    if (!r.rope) {
        k_rows_i8<false><<<dim3((unsigned)ctas, batch), RW_THREADS, 0, s>>>(a);
        return cudaGetLastError();
    }
    a.tile = std::min(RW_TOKENS, r.t_max);
    const int64_t qtiles = ceil_div64(r.t_max, a.tile);
    a.slices = std::min(r.h_q, head_slices(qtiles, batch, ceil_div64((int64_t)r.h_q * a.tile, RW_GROUPS)));
    ctas += qtiles * a.slices;
    const size_t smem = (size_t)std::max(span, a.tile) * 4 * a.rot16 * sizeof(float4);  // up to 64 KB
    const cudaError_t e = ensure_smem((const void *)k_rows_i8<true>, smem);
    if (e != cudaSuccess) return e;
    k_rows_i8<true><<<dim3((unsigned)ctas, batch), RW_THREADS, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_load(const mog_cache *c, int batch, const RowsIn &r, void *ko, void *vo, cudaStream_t s) {
    RowsArgs a{};
    set_cache(a, c);
    set_rows(a, r);
    const int64_t most = ceil_div64(16LL * num_sms(), batch);
    const int64_t want = ceil_div64(r.t_max, std::max(RW_GROUPS / (2 * r.h_kv), 1) * RW_DEPTH);
    const dim3 grid((unsigned)std::min(want, most), batch);
    uint16_t *k = static_cast<uint16_t *>(ko), *v = static_cast<uint16_t *>(vo);
    const int out32 = ((uintptr_t)ko | (uintptr_t)vo | (uintptr_t)(2 * a.kb) | (uintptr_t)(2 * a.kt) | (uintptr_t)(2 * a.kh)) % 32 == 0;
    if (c->type == MOG_CACHE_BF16) k_kv_load<TO_BF16><<<grid, RW_THREADS, 0, s>>>(a, k, v, out32);
    else if (c->type == MOG_CACHE_E4M3) k_kv_load<TO_E4M3><<<grid, RW_THREADS, 0, s>>>(a, k, v, out32);
    else k_kv_load<TO_I8><<<grid, RW_THREADS, 0, s>>>(a, k, v, out32);
    return cudaGetLastError();
}

}  // namespace mog
