// cache.cu -- decode attentions over a mog_cache (bf16 or e4m3 rows, contiguous or paged)
// and the store that writes it.
//
// dense_decode8: softmax(tau q.K^T) V of an e4m3 cache whose row i stands for
// k_scale[i]*code_i and v_scale[i]*code_i.  mog_diff_decode: the difference of two softmax
// maps over one set of values, normalised.  Both are one split kernel and one merge kernel.
//
// Split (k_cache_split): the 64-row tiles of all (sequence, KV head) units form one list;
// CTA c takes tiles [c*chunk, (c+1)*chunk) of it, so ragged batches load every SM alike
// (the lengths are read on the device: a captured graph replays with grown sequences).  Its
// copies run ahead across unit borders.  Each unit that a CTA touches leaves one partial
// (max, sum, acc per head) in slot c + unit, which no other pair (c, unit) shares, because
// along the list either c or the unit grows by one.
//
// Work of one warp: 16 rows of each tile; rows in the M dimension of m16n8k16, the heads of
// a KV head in N.  A differential head is two columns (its two maps): columns 0..3 and
// 4..7 of one block for up to 4 heads, blocks 0 and 1 for up to 8, so both maps share each
// value row that is read.
//
// e4m3 rows are read by 16-byte loads in the order the fragments want (dimensions are
// permuted alike in K and q, and back in the output), then widened in registers to fp16,
// which holds every e4m3 value exactly.  q enters as fp16 scaled by a power of two of its
// own, so that its elements down to 2^-29 of the largest are exact.  Weights enter the P.V
// product as fp16 (2^14 * p * v_scale / running power of two >= v_scale): high part alone
// (2^-12 relative) when the output is rounded to bf16, high + low parts (2^-22) when it
// stays fp32.  bf16 rows go through ldmatrix; their weights are bf16 high + low parts for
// a bf16 output (2^-17) and three parts (2^-24) for an fp32 one.  All sums are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.cuh"
#include "internal.h"

namespace mog {

constexpr int CT_WARPS = 4;
constexpr int CT_THREADS = 32 * CT_WARPS;
constexpr float W_SCALE = 16384.f;  // 2^14: scale of fp16 weights

// A tile is copied by the whole CTA, 2 KB of neighbouring rows per instruction, and each
// warp consumes BLK blocks of 16 of its rows.  Stages are aligned to 128 bytes: 16 bytes off,
// the copies of the same kernel were 5% slower (1M e4m3 tokens, 8 heads: 329 against 316 us).
template <bool E4M3>
struct Tile {
    static constexpr int BLK = E4M3 ? 2 : 1;              // blocks of 16 rows per warp
    static constexpr int WROWS = 16 * BLK;                // rows per warp
    static constexpr int ROWS = CT_WARPS * WROWS;
    static constexpr int ROW = E4M3 ? MOG_D : 2 * MOG_D;  // bytes
    static constexpr int KV = ROWS * ROW;                 // bytes of the K or V tile: 16 KB
    static constexpr int AUX = 2 * KV;                    // K scales, V scales
    static constexpr int MASK = AUX + (E4M3 ? 2 * ROWS * 4 : 0);  // bit per row
    static constexpr int STAGE = MASK + 128;              // rows stay aligned to 128 bytes
    static constexpr int STAGES = 2;  // 3 CTAs per SM: 96 KB in flight while 96 KB are consumed
    static constexpr int SMEM = STAGES * STAGE;
};

struct CacheArgs {
    const uint8_t *K, *V;
    const float *ks, *vs;
    int64_t sb, sh, sn;     // bytes between pages (or sequences), heads, rows
    int64_t ssb, ssh, ssn;  // the same of the scales, in floats
    const int *bt;
    int pshift, pps, n_pages;
    const int *lengths;
    int n_max, batch, h_kv, G;
    const uint16_t *q;
    float *part;
    float scale2;
};

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
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) s += seq_tiles<ROWS>(a, b);
    return warp_isum(s) * a.h_kv;
}

// Sequence holding tile `t` of the list and the list position of its first tile (called by
// a full warp; t < total).
template <int ROWS>
__device__ __forceinline__ void find_seq(const CacheArgs &a, int t, int &b, int &first) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int mine = b0 + lane < a.batch ? seq_tiles<ROWS>(a, b0 + lane) * a.h_kv : 0;
        int end = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += v;
        }
        const unsigned in = __ballot_sync(0xffffffffu, base + end > t);
        if (in) {
            const int l = __ffs(in) - 1;
            b = b0 + l;
            first = base + __shfl_sync(0xffffffffu, end - mine, l);
            return;
        }
        base += __shfl_sync(0xffffffffu, end, 31);
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
// +8) and two neighbouring chunks.  bf16 (256-byte rows): ldmatrix.
template <bool E4M3>
__device__ __forceinline__ uint32_t swz_k(int row, int ch) {
    return E4M3 ? (uint32_t)(row * MOG_D + ((ch ^ ((row & 1) << 2)) << 4)) : swz(row, ch);
}
template <bool E4M3>
__device__ __forceinline__ uint32_t swz_v(int row, int ch) {
    return E4M3 ? (uint32_t)(row * MOG_D + ((ch ^ (row & 6)) << 4)) : swz(row, ch);
}

// Page of the tile's 16-row group `lane`, loaded one tile ahead of its use (unchecked: a
// check here would wait for the load).
template <bool E4M3, bool PAGED>
__device__ __forceinline__ void tile_page(const CacheArgs &a, const Cursor<Tile<E4M3>::ROWS> &c, int &pg) {
    if constexpr (PAGED) {
        using T = Tile<E4M3>;
        const int lane = threadIdx.x & 31, row = c.t * T::ROWS + 16 * lane;
        pg = -1;
        if (lane < T::ROWS / 16 && row < c.n) pg = __ldg(a.bt + (int64_t)c.b * a.pps + (row >> a.pshift));
    }
}

// Start the copies of a tile.  Rows behind the sequence's end or in no page are zero and
// masked; they are never read.
template <bool E4M3, bool PAGED>
__device__ __forceinline__ void issue(const CacheArgs &a, const Cursor<Tile<E4M3>::ROWS> &c, int pg, uint32_t stage) {
    using T = Tile<E4M3>;
    constexpr int CH = T::ROW / 16;        // chunks per row
    constexpr int RP = CT_THREADS / CH;    // rows per instruction: 16 or 8
    const int tid = threadIdx.x, lane = tid & 31, ch = tid % CH, r0 = tid / CH;
    const int first = c.t * T::ROWS, left = c.n - first;  // rows of the sequence from here on
    const int pmask = (1 << a.pshift) - 1;
    const int64_t head = c.h * a.sh + r0 * a.sn + ch * 16 + (PAGED ? 0 : c.b * a.sb);
#pragma unroll
    for (int i = 0; i < T::ROWS / RP; ++i) {
        const int r = r0 + RP * i;
        const int page = PAGED ? __shfl_sync(0xffffffffu, pg, RP * i / 16) : 0;
        const bool ok = r < left && (!PAGED || (unsigned)page < (unsigned)a.n_pages);
        int64_t off = head + (int64_t)(PAGED ? (first + RP * i) & pmask : first + RP * i) * a.sn;
        if (PAGED) off += page * a.sb;
        off = ok ? off : 0;
        const int bytes = ok ? 16 : 0;
        cp_async16(stage + swz_k<E4M3>(r, ch), a.K + off, bytes);
        cp_async16(stage + T::KV + swz_v<E4M3>(r, ch), a.V + off, bytes);
    }
    // thread r: row r's scales and whether it is there
    if (tid >= T::ROWS) return;
    const int page = PAGED ? __shfl_sync(0xffffffffu, pg, tid / 16) : c.b;
    const bool ok = tid < left && (!PAGED || (unsigned)page < (unsigned)a.n_pages);
    if (E4M3) {
        const int64_t row = PAGED ? (first + tid) & pmask : first + tid;
        const int64_t so = ok ? page * a.ssb + c.h * a.ssh + row * a.ssn : 0;
        cp_async4(stage + T::AUX + 4 * tid, a.ks + so, ok ? 4 : 0);
        cp_async4(stage + T::AUX + 4 * (T::ROWS + tid), a.vs + so, ok ? 4 : 0);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + T::MASK + 4 * (tid >> 5)), "r"(mask) : "memory");
}

// Column -> (map, head) of a differential block layout, (0, column) otherwise.
template <bool DIFF, int NB>
__device__ __forceinline__ void column(int nb, int c, int &map, int &head) {
    map = DIFF ? (NB == 1 ? c >> 2 : nb) : 0;
    head = DIFF ? (NB == 1 ? c & 3 : c) : nb * 8 + c;
}

template <int NB>
struct State {
    float o[NB][8][4];  // [block][16 dimensions][...] of O^T
    float m[NB][2], l[NB][2];
    float vr;  // e4m3: power of two >= every v_scale seen (0: none yet); o is in units of vr / W_SCALE
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][t][e] = 0.f;
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.f;
        }
        vr = 0.f;
    }
};

// q of a unit as B fragments, and the factor that turns an accumulator of column (2t, 2t+1)
// into a log2-domain logit.
template <int NB>
struct QF {
    uint32_t b[NB][8][2];
    float f[NB][2];
};

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

template <bool E4M3, int NB, bool DIFF>
__device__ __forceinline__ void load_q(QF<NB> &qf, const CacheArgs &a, int unit) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        int map, head;
        column<DIFF, NB>(nb, g, map, head);
        const bool have = head < a.G;
        const uint16_t *row = a.q + ((int64_t)unit * a.G + (have ? head : 0)) * MOG_D;
        if (!E4M3) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const bool use = have && (!DIFF || (ks >> 2) == map);
                const uint32_t *p = reinterpret_cast<const uint32_t *>(row + ks * 16 + 2 * t);
                qf.b[nb][ks][0] = use ? p[0] : 0u;
                qf.b[nb][ks][1] = use ? p[4] : 0u;
            }
            qf.f[nb][0] = qf.f[nb][1] = a.scale2;
        } else {
            // this lane's dimensions: 16(t + 4j) .. +15, word w of chunk j in step 4j + w
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
            const float up = pow2f(14 - e), back = pow2f(max(e - 14, -126)) * a.scale2;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = raw[ks >> 2][2 * (ks & 3) + i];
                    const __half2 h = __floats2half2_rn(bf_lo(w) * up, bf_hi(w) * up);
                    qf.b[nb][ks][i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            qf.f[nb][0] = __shfl_sync(0xffffffffu, back, 8 * t);
            qf.f[nb][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
        }
    }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool E4M3>
__device__ __forceinline__ void mma_t(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (E4M3) mma_f16(d, a, b0, b1);
    else mma_bf16(d, a, b0, b1);
}
// four e4m3 bytes -> two fp16 pairs (exact)
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The largest part of (x, y) that 16 bits hold, and what is left.
template <bool E4M3>
__device__ __forceinline__ uint32_t part16(float &x, float &y) {
    if (E4M3) {
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

// This warp's rows of a tile.
//
// The products of one tile start from zero on the tensor cores, which truncate their sums,
// and join the running sum rounded to nearest (the same fused multiply-add that rescales
// it): summing a 1M-token sequence on the tensor cores alone drifted by 1.1e-5.
template <bool E4M3, int NB, bool DIFF, int PARTS>
__device__ __forceinline__ void compute(State<NB> &st, const QF<NB> &qf, uint32_t stage) {
    using T = Tile<E4M3>;
    constexpr int BLK = T::BLK;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, mat = lane >> 3, r8 = lane & 7;
    const int wr = (threadIdx.x >> 5) * T::WROWS;  // this warp's first row (a multiple of 16)
    const uint32_t sk = stage + wr * T::ROW, sv = sk + T::KV, sc = stage + T::AUX + 4 * wr;
    constexpr uint32_t ALL = (uint32_t)((1ull << T::WROWS) - 1);
    const uint32_t rows = (__float_as_uint(lds4(stage + T::MASK + 4 * (wr / 32))) >> (wr % 32)) & ALL;
    if (rows == 0) return;

    // logits: rows g (0, 1) and g+8 (2, 3) of columns 2t, 2t+1.  The two maps of a
    // differential block accumulate apart (half j of the dimensions is map j).
    float s[BLK][NB][4];
#pragma unroll
    for (int blk = 0; blk < BLK; ++blk) {
        float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[blk][nb][e] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint4 wa, wb;
            if (E4M3) {
                wa = lds16(sk + swz_k<E4M3>(16 * blk + g, t + 4 * j));
                wb = lds16(sk + swz_k<E4M3>(16 * blk + g + 8, t + 4 * j));
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int ks = 4 * j + w;
                uint32_t a[4];
                if (E4M3) {
                    widen(word(wa, w), a[0], a[2]);
                    widen(word(wb, w), a[1], a[3]);
                } else {
                    ldsm_x4(sk + swz_k<E4M3>((mat & 1) * 8 + r8, 2 * ks + (mat >> 1)), a[0], a[1], a[2], a[3]);
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (DIFF && NB == 2 && nb != j) continue;
                    if (DIFF && NB == 1 && j == 1) mma_t<E4M3>(s2, a, qf.b[nb][ks][0], qf.b[nb][ks][1]);
                    else mma_t<E4M3>(s[blk][nb], a, qf.b[nb][ks][0], qf.b[nb][ks][1]);
                }
            }
        }
        if (DIFF && NB == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[blk][0][e] = t >= 2 ? s2[e] : s[blk][0][e];
        }
    }

    // log2-domain logits
#pragma unroll
    for (int blk = 0; blk < BLK; ++blk) {
        float kA = 1.f, kB = 1.f;
        if (E4M3) kA = lds4(sc + 4 * (16 * blk + g)), kB = lds4(sc + 4 * (16 * blk + g + 8));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            s[blk][nb][0] *= kA * qf.f[nb][0];
            s[blk][nb][1] *= kA * qf.f[nb][1];
            s[blk][nb][2] *= kB * qf.f[nb][0];
            s[blk][nb][3] *= kB * qf.f[nb][1];
        }
    }
    if (rows != ALL) {  // the sequence's end, or a page that is none
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
            const bool okA = (rows >> (16 * blk + g)) & 1u, okB = (rows >> (16 * blk + g + 8)) & 1u;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (!okA) s[blk][nb][0] = s[blk][nb][1] = -INFINITY;
                if (!okB) s[blk][nb][2] = s[blk][nb][3] = -INFINITY;
            }
        }
    }
    float inv = 0.f;
    if (E4M3) {
        const float mine = fabsf(lds4(sc + 4 * (T::ROWS + lane)));
        if (__any_sync(0xffffffffu, mine > st.vr)) {  // a larger value scale: new unit
            const float vr = pow2f(min(max((__float_as_int(warp_max(mine)) >> 23) - 126, -100), 127));
            const float f = st.vr / vr;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st.o[nb][i][e] *= f;
            st.vr = vr;
        }
        inv = st.vr > 0.f ? W_SCALE / st.vr : 0.f;  // (rows whose scales are all 0 have no unit yet)
    }
    uint32_t pb[BLK][NB][PARTS][2];
    float al[NB][2];
    float vA[BLK], vB[BLK];
    if (E4M3) {
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
            vA[blk] = lds4(sc + 4 * (T::ROWS + 16 * blk + g)) * inv;
            vB[blk] = lds4(sc + 4 * (T::ROWS + 16 * blk + g + 8)) * inv;
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float sh[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[0][nb][e], s[0][nb][e + 2]);
            if (BLK == 2) mx = fmaxf(mx, fmaxf(s[BLK - 1][nb][e], s[BLK - 1][nb][e + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // the shift: 0 until a row has been seen, so that no infinities are subtracted
            const float mn = fmaxf(st.m[nb][e], mx);
            sh[e] = mn == -INFINITY ? 0.f : mn;
            al[nb][e] = ex2(st.m[nb][e] - sh[e]);
            st.m[nb][e] = mn;
            st.l[nb][e] *= al[nb][e];
        }
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
            float p0 = ex2(s[blk][nb][0] - sh[0]), p1 = ex2(s[blk][nb][1] - sh[1]);
            float p2 = ex2(s[blk][nb][2] - sh[0]), p3 = ex2(s[blk][nb][3] - sh[1]);
            st.l[nb][0] += p0 + p2;
            st.l[nb][1] += p1 + p3;
            if (E4M3) p0 *= vA[blk], p1 *= vA[blk], p2 *= vB[blk], p3 *= vB[blk];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                pb[blk][nb][i][0] = movmatrix_t(part16<E4M3>(p0, p1));
                pb[blk][nb][i][1] = movmatrix_t(part16<E4M3>(p2, p3));
            }
        }
    }

    // O^T = O^T diag(al) + V^T P^T, 16 dimensions at a time; lowest parts first
    if (E4M3) {
        // rows 2t, 2t+1, 2t+8, 2t+9 of a block, dimensions 16g .. 16g+15: word w holds
        // dimensions 16g + 4w .. +3, of tiles 2w (+0: row g of the fragment, +1: row g+8), 2w+1
        uint4 x[BLK][4];
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[blk][i] = lds16(sv + swz_v<E4M3>(16 * blk + 2 * t + (i & 1) + 8 * (i >> 1), g));
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t sel = hf ? 0x7362u : 0x5140u;
                float d[NB][4] = {};
#pragma unroll
                for (int blk = 0; blk < BLK; ++blk) {
                    uint32_t a[4];
                    widen(__byte_perm(word(x[blk][0], w), word(x[blk][1], w), sel), a[0], a[1]);
                    widen(__byte_perm(word(x[blk][2], w), word(x[blk][3], w), sel), a[2], a[3]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = PARTS - 1; i >= 0; --i) mma_f16(d[nb], a, pb[blk][nb][i][0], pb[blk][nb][i][1]);
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st.o[nb][2 * w + hf][e] = fmaf(st.o[nb][2 * w + hf][e], al[nb][e & 1], d[nb][e]);
            }
    } else {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[4];
            ldsm_x4_t(sv + swz_v<E4M3>((mat >> 1) * 8 + r8, 2 * mt + (mat & 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float d[4] = {};
#pragma unroll
                for (int i = PARTS - 1; i >= 0; --i) mma_bf16(d, a, pb[0][nb][i][0], pb[0][nb][i][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[nb][mt][e] = fmaf(st.o[nb][mt][e], al[nb][e & 1], d[e]);
            }
        }
    }
}

// A unit's end: the four warps' states become one partial in `dst` ([columns][PART_W]).
// Accumulators pass through the stage that has just been consumed (word i of lane l at
// i*32 + l), maxima and sums through `ex`.  Called by the whole CTA.
template <int NB>
struct Exchange {
    float m[CT_WARPS][NB * 8], l[CT_WARPS][NB * 8];
};
template <int NB>
__device__ __forceinline__ void state_put(const State<NB> &st, float *x, Exchange<NB> &ex) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[(nb * 32 + i) * 32 + lane] = st.o[nb][i >> 2][i & 3];
        if (lane < 4) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ex.m[w][nb * 8 + 2 * lane + e] = st.m[nb][e];
                ex.l[w][nb * 8 + 2 * lane + e] = st.l[nb][e];
            }
        }
    }
}
template <int NB>
__device__ __forceinline__ void state_fold(State<NB> &st, const float *x, const Exchange<NB> &ex, int from) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float mine[2], his[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float m2 = ex.m[from][nb * 8 + 2 * t + e], mn = fmaxf(st.m[nb][e], m2);
            const float sh = mn == -INFINITY ? 0.f : mn;
            mine[e] = ex2(st.m[nb][e] - sh);
            his[e] = ex2(m2 - sh);
            st.m[nb][e] = mn;
            st.l[nb][e] = st.l[nb][e] * mine[e] + ex.l[from][nb * 8 + 2 * t + e] * his[e];
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
            st.o[nb][i >> 2][i & 3] = st.o[nb][i >> 2][i & 3] * mine[i & 1] + x[(nb * 32 + i) * 32 + lane] * his[i & 1];
    }
}

template <bool E4M3, int NB, bool DIFF>
__device__ __forceinline__ void flush(State<NB> &st, float *x, Exchange<NB> &ex, const CacheArgs &a, float *dst) {
    using T = Tile<E4M3>;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int SW = 32 * 32 * NB;  // words of a warp's accumulators
    static_assert(T::AUX >= 2 * SW * 4, "two states fit in a stage");
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        if (E4M3) {  // to the values' own unit
            const float u = st.vr / W_SCALE;
#pragma unroll
            for (int i = 0; i < 32; ++i) st.o[nb][i >> 2][i & 3] *= u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) st.l[nb][e] += __shfl_xor_sync(0xffffffffu, st.l[nb][e], o);
    }
    __syncthreads();  // every warp has read its rows of the stage
    if (w >= 2) state_put(st, x + (w - 2) * SW, ex);
    __syncthreads();
    if (w < 2) state_fold(st, x + w * SW, ex, w + 2);
    if (w == 1) {
        __syncwarp();
        state_put(st, x + SW, ex);
    }
    __syncthreads();
    if (w == 0) {
        state_fold(st, x + SW, ex, 1);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int map, head;
                column<DIFF, NB>(nb, 2 * t + e, map, head);
                if (head >= a.G) continue;
                float *r = dst + (int64_t)(map * a.G + head) * PART_W;
                if (g == 0) *reinterpret_cast<float2 *>(r) = make_float2(st.m[nb][e], st.l[nb][e]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float lo = st.o[nb][i][e], hi = st.o[nb][i][e + 2];
                    if (E4M3) {
                        *reinterpret_cast<float2 *>(r + PART_ACC + 16 * g + 2 * i) = make_float2(lo, hi);
                    } else {
                        r[PART_ACC + 16 * i + g] = lo;
                        r[PART_ACC + 16 * i + g + 8] = hi;
                    }
                }
            }
    }
}

template <bool E4M3, int NB, bool PAGED, bool DIFF, int PARTS>
__global__ void __launch_bounds__(CT_THREADS, 3) k_cache_split(CacheArgs a) {
    extern __shared__ __align__(128) uint8_t csm[];
    __shared__ Exchange<NB> ex;
    using T = Tile<E4M3>;
    pdl_trigger();
    const int total = total_tiles<T::ROWS>(a);
    const int chunk = (total + gridDim.x - 1) / gridDim.x;
    const int t0 = min((int64_t)blockIdx.x * chunk, (int64_t)total), cnt = min(chunk, total - t0);
    if (cnt <= 0) return;
    const uint32_t stages = smem_u32(csm);
    Cursor<T::ROWS> ci, cc;  // the next tile to copy, the next to compute
    ci.seek(a, t0);
    cc = ci;
    int pg = 0;
    tile_page<E4M3, PAGED>(a, ci, pg);
    int ahead = 0;  // tiles whose copies have started
    auto feed = [&](uint32_t stage) {
        if (ahead < cnt) {
            issue<E4M3, PAGED>(a, ci, pg, stage);
            if (++ahead < cnt) {
                ci.next(a);
                tile_page<E4M3, PAGED>(a, ci, pg);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < T::STAGES - 1; ++s) feed(stages + s * T::STAGE);
    const int G2 = DIFF ? 2 * a.G : a.G;
    int unit = cc.b * a.h_kv + cc.h;
    QF<NB> qf;
    load_q<E4M3, NB, DIFF>(qf, a, unit);
    State<NB> st;
    st.init();
    int slot = 0;
    for (int i = 0; i < cnt; ++i) {
        cp_async_wait<T::STAGES - 2>();
        __syncthreads();  // the tile is there, and the stage before it has been consumed
        feed(stages + (slot == 0 ? T::STAGES - 1 : slot - 1) * T::STAGE);
        compute<E4M3, NB, DIFF, PARTS>(st, qf, stages + slot * T::STAGE);
        const bool end = cc.last();
        if (end || i == cnt - 1) {
            flush<E4M3, NB, DIFF>(st, reinterpret_cast<float *>(csm + slot * T::STAGE), ex, a,
                                  a.part + ((int64_t)blockIdx.x + unit) * G2 * PART_W);
            if (i == cnt - 1) break;
            st.init();
        }
        slot = slot + 1 == T::STAGES ? 0 : slot + 1;
        cc.next(a);
        if (end) {
            unit = cc.b * a.h_kv + cc.h;
            load_q<E4M3, NB, DIFF>(qf, a, unit);
        }
    }
    cp_async_wait<0>();
}

// One CTA per (unit, head): warp w folds partials w, w + 8, ... (each lane four dimensions),
// then the warps are folded and normalised; for a differential head both maps, their
// difference, the root-mean-square norm and its weights.
constexpr int CM_WARPS = 8;
template <int ROWS, bool DIFF, bool BF16OUT>
__global__ void __launch_bounds__(CM_WARPS * 32) k_cache_merge(CacheArgs a, DiffArgs d, void *out, int splits) {
    constexpr int M = DIFF ? 2 : 1;
    __shared__ float4 s_acc[M][CM_WARPS][32];
    __shared__ float s_m[M][CM_WARPS], s_l[M][CM_WARPS];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / a.G, head = blockIdx.x % a.G;
    const int b = unit / a.h_kv, h = unit % a.h_kv;
    // the unit's tiles in the list, and with them the CTAs that hold its partials
    int before = 0, all = 0;
    for (int i = lane; i < a.batch; i += 32) {
        const int nt = seq_tiles<ROWS>(a, i);
        all += nt;
        if (i < b) before += nt;
    }
    before = warp_isum(before), all = warp_isum(all);
    const int nt = seq_tiles<ROWS>(a, b), chunk = (all * a.h_kv + splits - 1) / splits;
    const int first = before * a.h_kv + h * nt;
    const int c0 = nt ? first / chunk : 0, c1 = nt ? (first + nt - 1) / chunk + 1 : 0;
    float weight = 0.f;
    if (DIFF) {
        const float *L = d.lam + d.lam_stride * (h * a.G + head) + 2 * lane;
        const float2 x0 = *reinterpret_cast<const float2 *>(L), x1 = *reinterpret_cast<const float2 *>(L + 64);
        const float2 x2 = *reinterpret_cast<const float2 *>(L + 128), x3 = *reinterpret_cast<const float2 *>(L + 192);
        const float e1 = warp_sum(x0.x * x1.x + x0.y * x1.y), e2 = warp_sum(x2.x * x3.x + x2.y * x3.y);
        weight = expf(e1) - expf(e2) + d.lambda_init;
    }
    pdl_wait();
    const int64_t step = (int64_t)M * a.G * PART_W;  // floats of a slot
#pragma unroll
    for (int k = 0; k < M; ++k) {
        const float *p = a.part + (int64_t)unit * step + (int64_t)(k * a.G + head) * PART_W;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int U = 4;
        for (int c = c0 + w; c < c1; c += CM_WARPS * U) {
            float2 ml[U];
            float4 v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool ok = c + CM_WARPS * i < c1;
                const float *r = p + (c + CM_WARPS * i) * step;
                ml[i] = ok ? __ldcg(reinterpret_cast<const float2 *>(r)) : make_float2(-INFINITY, 0.f);
                v[i] = ok ? __ldcg(reinterpret_cast<const float4 *>(r + PART_ACC) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
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
        s_acc[k][w][lane] = acc;
        if (lane == 0) s_m[k][w] = m, s_l[k][w] = l;
    }
    __syncthreads();
    if (w != 0) return;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < M; ++k) {
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < CM_WARPS; ++i) m = fmaxf(m, s_m[k][i]);
        const float sh = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < CM_WARPS; ++i) {
            const float fi = exp2f(s_m[k][i] - sh);
            const float4 v = s_acc[k][i][lane];
            l += fi * s_l[k][i];
            acc.x += fi * v.x, acc.y += fi * v.y, acc.z += fi * v.z, acc.w += fi * v.w;
        }
        // nothing seen: zeros (a sum that is NaN stays NaN)
        const float f = (l == 0.f ? 0.f : 1.f / l) * (k ? -weight : 1.f);
        r.x += f * acc.x, r.y += f * acc.y, r.z += f * acc.z, r.w += f * acc.w;
    }
    if (DIFF) {
        const float ss = warp_sum(r.x * r.x + r.y * r.y + r.z * r.z + r.w * r.w);
        const float f = (1.f - d.lambda_init) / sqrtf(ss * (1.f / MOG_D) + d.eps);
        const float4 gm = d.gamma ? reinterpret_cast<const float4 *>(d.gamma)[lane] : make_float4(1.f, 1.f, 1.f, 1.f);
        r.x *= f * gm.x, r.y *= f * gm.y, r.z *= f * gm.z, r.w *= f * gm.w;
    }
    const int64_t o = (int64_t)blockIdx.x * MOG_D + 4 * lane;
    if (BF16OUT) {
        const uint2 v = make_uint2(cvt_bf2(r.x, r.y), cvt_bf2(r.z, r.w));
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + o) = v;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + o) = r;
    }
}

int cache_splits(int units, int n_max) {
    // one wave of three CTAs per SM, and no more CTAs than tiles
    // (tiles of 64 rows: the smaller kind)
    const int64_t tiles = units * ceil_div64(n_max, Tile<false>::ROWS), slots = 3LL * num_sms();
    return (int)(tiles < slots ? tiles : slots);
}

template <bool E4M3, int NB, bool PAGED, bool DIFF, int PARTS>
static cudaError_t launch_split(const CacheArgs &a, int splits, cudaStream_t s) {
    const auto fn = k_cache_split<E4M3, NB, PAGED, DIFF, PARTS>;
    cudaError_t e = ensure_smem((const void *)fn, Tile<E4M3>::SMEM);
    if (e != cudaSuccess) return e;
    fn<<<splits, CT_THREADS, Tile<E4M3>::SMEM, s>>>(a);
    return cudaGetLastError();
}
template <bool E4M3, bool DIFF, int PARTS>
static cudaError_t pick_split(const CacheArgs &a, int splits, cudaStream_t s) {
    const bool one = (DIFF ? 2 : 1) * a.G <= 8;
    if (a.bt) return one ? launch_split<E4M3, 1, true, DIFF, PARTS>(a, splits, s) : launch_split<E4M3, 2, true, DIFF, PARTS>(a, splits, s);
    return one ? launch_split<E4M3, 1, false, DIFF, PARTS>(a, splits, s) : launch_split<E4M3, 2, false, DIFF, PARTS>(a, splits, s);
}

template <int ROWS>
static cudaError_t launch_merge(const cudaLaunchConfig_t &cfg, bool diff, bool bf_out, const CacheArgs &a,
                                const DiffArgs &d, void *out, int splits) {
    if (diff) return bf_out ? cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, true, true>, a, d, out, splits)
                            : cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, true, false>, a, d, out, splits);
    return bf_out ? cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, false, true>, a, d, out, splits)
                  : cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, false, false>, a, d, out, splits);
}

cudaError_t launch_cache_decode(const mog_cache *c, const int32_t *lengths, int n_max, int batch, int h_kv, int G,
                                const void *q, const mog_diff_params *diff, int out_type, void *out, float *scratch,
                                cudaStream_t s) {
    const bool e4 = c->type == MOG_CACHE_E4M3, bf_out = out_type == MOG_OUT_BF16;
    const int es = e4 ? 1 : 2;
    CacheArgs a{static_cast<const uint8_t *>(c->k), static_cast<const uint8_t *>(c->v), c->k_scale, c->v_scale,
                c->stride_b * es, c->stride_h * es, c->stride_n * es, c->scale_b, c->scale_h, c->scale_n,
                c->block_table, c->block_table ? log2_exact(c->page_rows) : 0, c->pages_per_seq, c->n_pages,
                lengths, n_max, batch, h_kv, G, static_cast<const uint16_t *>(q), scratch,
                (float)(LOG2E / sqrt(diff ? MOG_D / 2.0 : (double)MOG_D))};
    DiffArgs d{};
    if (diff) d = DiffArgs{diff->lam, diff->lam_heads > 1 ? 4 * (MOG_D / 2) : 0, diff->gamma, diff->lambda_init, diff->eps};
    const int splits = cache_splits(batch * h_kv, n_max);
    cudaError_t e;
    if (diff) {
        if (e4) e = bf_out ? pick_split<true, true, 1>(a, splits, s) : pick_split<true, true, 2>(a, splits, s);
        else e = bf_out ? pick_split<false, true, 2>(a, splits, s) : pick_split<false, true, 3>(a, splits, s);
    } else {
        e = bf_out ? pick_split<true, false, 1>(a, splits, s) : pick_split<true, false, 2>(a, splits, s);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(batch * h_kv * G);
    cfg.blockDim = dim3(CM_WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (e4) return launch_merge<Tile<true>::ROWS>(cfg, diff, bf_out, a, d, out, splits);
    return launch_merge<Tile<false>::ROWS>(cfg, diff, bf_out, a, d, out, splits);
}

// ------------------------------------------------------------------------------------
// mog_kv_store: rows of new keys and values to their positions.  One half-warp per row:
// its 128 elements are one 16-byte load a lane, the largest finite magnitude four shuffles.
// A row's e4m3 scale is the least power of two 2^e (e >= -126) with amax <= 448*2^e, so
// that dividing by it is exact and the only rounding is the one to e4m3.
// ------------------------------------------------------------------------------------
struct StoreArgs {
    uint8_t *K, *V;
    float *ks, *vs;
    int64_t sb, sh, sn, ssb, ssh, ssn;
    const int *bt;
    int pshift, pps, n_pages, n_cap;
    const int *pos, *count;
    const uint16_t *kn, *vn;
    int64_t nb, nt, nh;  // elements between sequences, tokens and heads of the new rows
    int t_max, h_kv;
};

constexpr int SR_THREADS = 256;

template <bool E4M3>
__global__ void __launch_bounds__(SR_THREADS) k_kv_store(StoreArgs a) {
    const int b = blockIdx.y;
    const int count = a.count ? min(max(a.count[b], 0), a.t_max) : a.t_max;
    const int64_t start = a.pos[b];
    const int64_t rows = (int64_t)count * 2 * a.h_kv;  // head fastest, then key or value, then token
    const int lane = threadIdx.x & 15;
    const int64_t step = (int64_t)gridDim.x * (SR_THREADS / 16);
    // (whole half-warps enter or leave: the shuffles below stay inside one)
    const unsigned half = 0xffffu << (threadIdx.x & 16);
    for (int64_t i = blockIdx.x * (int64_t)(SR_THREADS / 16) + threadIdx.x / 16; i < rows; i += step) {
        const int t = (int)(i / (2 * a.h_kv)), r = (int)(i - (int64_t)t * 2 * a.h_kv);
        const bool val = r >= a.h_kv;
        const int h = val ? r - a.h_kv : r;
        const int64_t pos = start + t;
        if (pos < 0 || pos >= a.n_cap) continue;
        int64_t slab = b, row = pos;
        if (a.bt) {
            slab = a.bt[(int64_t)b * a.pps + (pos >> a.pshift)];
            if (slab < 0 || slab >= a.n_pages) continue;
            row = pos & ((1 << a.pshift) - 1);
        }
        const uint4 x = ldg_nc16((val ? a.vn : a.kn) + b * a.nb + t * a.nt + h * a.nh + lane * 8);
        uint8_t *dst = (val ? a.V : a.K) + slab * a.sb + h * a.sh + row * a.sn;
        if (!E4M3) {
            *reinterpret_cast<uint4 *>(dst + lane * 16) = x;
            continue;
        }
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float u = fabsf(bf_lo(w[k])), v = fabsf(bf_hi(w[k]));
            amax = fmaxf(amax, u < INFINITY ? u : 0.f);
            amax = fmaxf(amax, v < INFINITY ? v : 0.f);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, o));
        // amax = m * 2^E, 1 <= m < 2: 448 = 1.75 * 2^8
        const int bits = __float_as_int(amax), E = (bits >> 23) - 127;
        int e = E - 8 + ((bits & 0x7fffff) > 0x600000);
        e = amax > 0.f ? max(e, -126) : 0;
        const float inv = pow2f(-e);
        uint32_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t u = 0;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint16_t p;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(bf_hi(w[2 * k + m]) * inv), "f"(bf_lo(w[2 * k + m]) * inv));
                u |= (uint32_t)p << (16 * m);
            }
            c[k] = u;
        }
        *reinterpret_cast<uint2 *>(dst + lane * 8) = make_uint2(c[0], c[1]);
        if (lane == 0) (val ? a.vs : a.ks)[slab * a.ssb + h * a.ssh + row * a.ssn] = pow2f(e);
    }
}

cudaError_t launch_kv_store(const mog_cache *c, int batch, int h_kv, int t_max, const int32_t *pos,
                            const int32_t *count, const void *kn, const void *vn, int64_t nb, int64_t nt,
                            int64_t nh, cudaStream_t s) {
    const bool e4 = c->type == MOG_CACHE_E4M3;
    const int es = e4 ? 1 : 2;
    const int64_t cap = c->block_table ? (int64_t)c->pages_per_seq * c->page_rows : c->n_cap;
    StoreArgs a{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale,
                c->stride_b * es, c->stride_h * es, c->stride_n * es, c->scale_b, c->scale_h, c->scale_n,
                c->block_table, c->block_table ? log2_exact(c->page_rows) : 0, c->pages_per_seq, c->n_pages,
                (int)(cap < INT32_MAX ? cap : INT32_MAX), pos, count, static_cast<const uint16_t *>(kn),
                static_cast<const uint16_t *>(vn), nb, nt, nh, t_max, h_kv};
    const int64_t rows = (int64_t)t_max * 2 * h_kv, per = SR_THREADS / 16;
    const int64_t most = ceil_div64(16LL * num_sms(), batch);
    const int64_t want = ceil_div64(rows, per);
    const dim3 grid((unsigned)(want < most ? want : most), batch);
    if (e4) k_kv_store<true><<<grid, SR_THREADS, 0, s>>>(a);
    else k_kv_store<false><<<grid, SR_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mog
