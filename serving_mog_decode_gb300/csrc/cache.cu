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

constexpr int CT_ROWS = 64;
constexpr int CT_THREADS = 128;
constexpr float W_SCALE = 16384.f;  // 2^14: scale of fp16 weights

template <bool E4M3, int NB>
struct Tile {
    static constexpr int ROW = E4M3 ? MOG_D : 2 * MOG_D;  // bytes
    static constexpr int KV = CT_ROWS * ROW;              // bytes of the K or V tile
    static constexpr int AUX = 2 * KV;                    // row masks, then K and V scales
    static constexpr int RAW = AUX + CT_ROWS * 4 * (E4M3 ? 3 : 1);
    static constexpr int XCH = 2 * 32 * 36 * 4 * NB;  // two warps' states (the exchange at a unit's end)
    static constexpr int STAGE = RAW > XCH ? RAW : XCH;
    // e4m3: 16.75 KB a stage, four of them and three CTAs per SM; bf16: 32.3 KB, two
    static constexpr int STAGES = E4M3 ? 4 : 2;
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

__device__ __forceinline__ int seq_tiles(const CacheArgs &a, int b) {
    const int n = min(max(a.lengths[b], 0), a.n_max);
    return (n + CT_ROWS - 1) / CT_ROWS;
}

// Tiles of the whole batch, times h_kv: called by a full warp.
__device__ __forceinline__ int total_tiles(const CacheArgs &a) {
    int s = 0;
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) s += seq_tiles(a, b);
    return warp_isum(s) * a.h_kv;
}

// Sequence holding tile `t` of the list and the list position of its first tile (called by
// a full warp; t < total).
__device__ __forceinline__ void find_seq(const CacheArgs &a, int t, int &b, int &first) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int mine = b0 + lane < a.batch ? seq_tiles(a, b0 + lane) * a.h_kv : 0;
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
struct Cursor {
    int b, h, t, nt, n;  // sequence, head, tile, tiles of the sequence, its length
    __device__ __forceinline__ void seek(const CacheArgs &a, int tile) {
        int first;
        find_seq(a, tile, b, first);
        load(a);
        const int r = tile - first;
        h = nt > 0 ? r / nt : 0;
        t = r - h * nt;
    }
    __device__ __forceinline__ void load(const CacheArgs &a) {
        n = b < a.batch ? min(max(a.lengths[b], 0), a.n_max) : 0;
        nt = (n + CT_ROWS - 1) / CT_ROWS;
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

// Shared-memory position of a 16-byte chunk of a 128-byte e4m3 row, conflict-free for the
// readers: K is read by rows r, r+1 and chunks t (t < 4), V by rows 0, 2, 4, 6 (+1, +8) and
// two neighbouring chunks.
__device__ __forceinline__ uint32_t swz8_k(int row, int ch) {
    return (uint32_t)(row * MOG_D + ((ch ^ ((row & 1) << 2)) << 4));
}
__device__ __forceinline__ uint32_t swz8_v(int row, int ch) {
    return (uint32_t)(row * MOG_D + ((ch ^ (row & 6)) << 4));
}

// Pages of the four 16-row groups of a tile, loaded one tile ahead of their use (unchecked:
// a check here would wait for the load).
template <bool PAGED>
__device__ __forceinline__ void tile_pages(const CacheArgs &a, const Cursor &c, int (&pg)[4]) {
    if constexpr (PAGED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = c.t * CT_ROWS + 16 * i;
            pg[i] = row < c.n ? __ldg(a.bt + (int64_t)c.b * a.pps + (row >> a.pshift)) : -1;
        }
    }
}

// Start the copies of one tile.  Rows behind the sequence's end or in no page are zero and
// masked; they are never read.
template <bool E4M3, int NB, bool PAGED>
__device__ __forceinline__ void issue(const CacheArgs &a, const Cursor &c, const int (&pg)[4], uint8_t *stage) {
    using T = Tile<E4M3, NB>;
    constexpr int CH = T::ROW / 16;             // chunks per row
    constexpr int STEP = CT_THREADS / CH;       // rows per pass
    const uint32_t sk = smem_u32(stage), sv = sk + T::KV;
    uint32_t *mask = reinterpret_cast<uint32_t *>(stage + T::AUX);
    const int ch = threadIdx.x % CH, r0 = threadIdx.x / CH;
    const int pmask = (1 << a.pshift) - 1;
#pragma unroll
    for (int i = 0; i < CT_ROWS / STEP; ++i) {
        const int r = r0 + STEP * i, pos = c.t * CT_ROWS + r;
        const int page = PAGED ? pg[(STEP * i) / 16] : c.b;
        const bool ok = pos < c.n && (!PAGED || (unsigned)page < (unsigned)a.n_pages);
        const int64_t slab = ok ? page : 0, row = ok ? (PAGED ? (pos & pmask) : pos) : 0;
        const int64_t off = slab * a.sb + c.h * a.sh + row * a.sn + ch * 16;
        const int bytes = ok ? 16 : 0;
        cp_async16(sk + (E4M3 ? swz8_k(r, ch) : swz(r, ch)), a.K + off, bytes);
        cp_async16(sv + (E4M3 ? swz8_v(r, ch) : swz(r, ch)), a.V + off, bytes);
        if (ch == 0) mask[r] = ok;
        if (E4M3 && ch < 2) {
            const int64_t so = slab * a.ssb + c.h * a.ssh + row * a.ssn;
            cp_async4(smem_u32(mask + (1 + ch) * CT_ROWS + r), (ch ? a.vs : a.ks) + so, ok ? 4 : 0);
        }
    }
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

// This warp's 16 rows of a tile.
template <bool E4M3, int NB, bool DIFF, int PARTS>
__device__ __forceinline__ void compute(State<NB> &st, const QF<NB> &qf, const uint8_t *stage) {
    using T = Tile<E4M3, NB>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, mat = lane >> 3, r8 = lane & 7;
    const int rb = (threadIdx.x >> 5) * 16;
    const uint32_t sk = smem_u32(stage), sv = sk + T::KV;
    const uint32_t *mask = reinterpret_cast<const uint32_t *>(stage + T::AUX);
    const float *sc = reinterpret_cast<const float *>(mask + CT_ROWS);
    const int rA = rb + g, rB = rA + 8;

    // logits: rows rA (0, 1) and rB (2, 3) of columns 2t, 2t+1.  The two maps of a
    // differential block accumulate apart (half j of the dimensions is map j).
    float s[NB][4], s2[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb][e] = 0.f;
        s2[e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint4 wa, wb;
        if (E4M3) {
            wa = lds16(sk + swz8_k(rA, t + 4 * j));
            wb = lds16(sk + swz8_k(rB, t + 4 * j));
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int ks = 4 * j + w;
            uint32_t a[4];
            if (E4M3) {
                widen(word(wa, w), a[0], a[2]);
                widen(word(wb, w), a[1], a[3]);
            } else {
                ldsm_x4(sk + swz(rb + (mat & 1) * 8 + r8, 2 * ks + (mat >> 1)), a[0], a[1], a[2], a[3]);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (DIFF && NB == 2 && nb != j) continue;
                if (DIFF && NB == 1 && j == 1) mma_t<E4M3>(s2, a, qf.b[nb][ks][0], qf.b[nb][ks][1]);
                else mma_t<E4M3>(s[nb], a, qf.b[nb][ks][0], qf.b[nb][ks][1]);
            }
        }
    }
    if (DIFF && NB == 1 && t >= 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][e] = s2[e];
    }

    const bool okA = mask[rA] != 0, okB = mask[rB] != 0;
    float kA = 1.f, kB = 1.f, vA = 1.f, vB = 1.f;
    if (E4M3) {
        kA = sc[rA], kB = sc[rB];
        vA = sc[CT_ROWS + rA], vB = sc[CT_ROWS + rB];
        const float vt = fmaxf(fabsf(vA), fabsf(vB));
        if (__any_sync(0xffffffffu, vt > st.vr)) {  // a larger value scale: new unit
            const float vr = pow2f(min(max((__float_as_int(warp_max(vt)) >> 23) - 126, -100), 127));
            const float f = st.vr / vr;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st.o[nb][i][e] *= f;
            st.vr = vr;
        }
        // a row's weight factor; a batch of rows whose scales are all 0 has no unit yet
        const float inv = st.vr > 0.f ? W_SCALE / st.vr : 0.f;
        vA *= inv, vB *= inv;
    }
    uint32_t pb[NB][PARTS][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float f0 = qf.f[nb][0], f1 = qf.f[nb][1];
        const float s0 = okA ? s[nb][0] * (kA * f0) : -INFINITY, s1 = okA ? s[nb][1] * (kA * f1) : -INFINITY;
        const float s2_ = okB ? s[nb][2] * (kB * f0) : -INFINITY, s3 = okB ? s[nb][3] * (kB * f1) : -INFINITY;
        float mx0 = fmaxf(s0, s2_), mx1 = fmaxf(s1, s3);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        // the shift: 0 until a row has been seen, so that no infinities are subtracted
        const float mn0 = fmaxf(st.m[nb][0], mx0), mn1 = fmaxf(st.m[nb][1], mx1);
        const float sh0 = mn0 == -INFINITY ? 0.f : mn0, sh1 = mn1 == -INFINITY ? 0.f : mn1;
        const float al0 = ex2(st.m[nb][0] - sh0), al1 = ex2(st.m[nb][1] - sh1);
        st.m[nb][0] = mn0;
        st.m[nb][1] = mn1;
        float p0 = ex2(s0 - sh0), p1 = ex2(s1 - sh1), p2 = ex2(s2_ - sh0), p3 = ex2(s3 - sh1);
        st.l[nb][0] = st.l[nb][0] * al0 + (p0 + p2);
        st.l[nb][1] = st.l[nb][1] * al1 + (p1 + p3);
        if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                st.o[nb][i][0] *= al0;
                st.o[nb][i][1] *= al1;
                st.o[nb][i][2] *= al0;
                st.o[nb][i][3] *= al1;
            }
        }
        if (E4M3) p0 *= vA, p1 *= vA, p2 *= vB, p3 *= vB;
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            pb[nb][i][0] = movmatrix_t(part16<E4M3>(p0, p1));
            pb[nb][i][1] = movmatrix_t(part16<E4M3>(p2, p3));
        }
    }

    // O^T += V^T P^T
    if (E4M3) {
        // rows 2t, 2t+1, 2t+8, 2t+9, dimensions 16g .. 16g+15: word w holds dimensions
        // 16g + 4w .. +3, of tiles 2w (+0: row g of the fragment, +1: row g+8) and 2w+1
        const uint4 x0 = lds16(sv + swz8_v(rb + 2 * t, g)), y0 = lds16(sv + swz8_v(rb + 2 * t + 1, g));
        const uint4 x1 = lds16(sv + swz8_v(rb + 2 * t + 8, g)), y1 = lds16(sv + swz8_v(rb + 2 * t + 9, g));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t sel = hf ? 0x7362u : 0x5140u;
                uint32_t a[4];
                widen(__byte_perm(word(x0, w), word(y0, w), sel), a[0], a[1]);
                widen(__byte_perm(word(x1, w), word(y1, w), sel), a[2], a[3]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) mma_f16(st.o[nb][2 * w + hf], a, pb[nb][i][0], pb[nb][i][1]);
            }
        }
    } else {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[4];
            ldsm_x4_t(sv + swz(rb + (mat >> 1) * 8 + r8, 2 * mt + (mat & 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < PARTS; ++i) mma_bf16(st.o[nb][mt], a, pb[nb][i][0], pb[nb][i][1]);
        }
    }
}

// Fold the state that another warp left in shared memory (word i of lane l at i*32 + l).
template <int NB>
__device__ __forceinline__ void state_put(const State<NB> &st, float *x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float *p = x + nb * 36 * 32 + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) p[i * 32] = st.o[nb][i >> 2][i & 3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            p[(32 + e) * 32] = st.m[nb][e];
            p[(34 + e) * 32] = st.l[nb][e];
        }
    }
}
template <int NB>
__device__ __forceinline__ void state_fold(State<NB> &st, const float *x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float *p = x + nb * 36 * 32 + lane;
        float mine[2], his[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float m2 = p[(32 + e) * 32], mn = fmaxf(st.m[nb][e], m2);
            const float sh = mn == -INFINITY ? 0.f : mn;
            mine[e] = ex2(st.m[nb][e] - sh);
            his[e] = ex2(m2 - sh);
            st.m[nb][e] = mn;
            st.l[nb][e] = st.l[nb][e] * mine[e] + p[(34 + e) * 32] * his[e];
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
            st.o[nb][i >> 2][i & 3] = st.o[nb][i >> 2][i & 3] * mine[i & 1] + p[i * 32] * his[i & 1];
    }
}

// A unit's end: the four warps' states become one partial in `dst` ([columns][PART_W]).
// `x` is a stage that nothing reads or fills any more.  Called by the whole CTA.
template <bool E4M3, int NB, bool DIFF>
__device__ __forceinline__ void flush(State<NB> &st, float *x, const CacheArgs &a, float *dst) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int SW = 36 * 32 * NB;
    if (E4M3) {  // to the values' own unit
        const float u = st.vr / W_SCALE;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 32; ++i) st.o[nb][i >> 2][i & 3] *= u;
    }
    __syncthreads();  // every warp has read its rows of the stage
    if (w >= 2) state_put(st, x + (w - 2) * SW);
    __syncthreads();
    if (w < 2) state_fold(st, x + w * SW);
    __syncthreads();
    if (w == 1) state_put(st, x);
    __syncthreads();
    if (w == 0) {
        state_fold(st, x);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = st.l[nb][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                int map, head;
                column<DIFF, NB>(nb, 2 * t + e, map, head);
                if (head >= a.G) continue;
                float *r = dst + (int64_t)(map * a.G + head) * PART_W;
                if (g == 0) *reinterpret_cast<float2 *>(r) = make_float2(st.m[nb][e], l);
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
    using T = Tile<E4M3, NB>;
    pdl_trigger();
    const int total = total_tiles(a);
    const int chunk = (total + gridDim.x - 1) / gridDim.x;
    const int t0 = min((int64_t)blockIdx.x * chunk, (int64_t)total), cnt = min(chunk, total - t0);
    if (cnt <= 0) return;
    Cursor ci, cc;
    ci.seek(a, t0);
    cc = ci;
    int pg[4];
    tile_pages<PAGED>(a, ci, pg);
    int ahead = 0;  // tiles whose copies have started
    auto feed = [&]() {
        if (ahead < cnt) {
            issue<E4M3, NB, PAGED>(a, ci, pg, csm + (ahead % T::STAGES) * T::STAGE);
            ++ahead;
            if (ahead < cnt) {
                ci.next(a);
                tile_pages<PAGED>(a, ci, pg);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < T::STAGES - 1; ++s) feed();
    const int G2 = DIFF ? 2 * a.G : a.G;
    int unit = cc.b * a.h_kv + cc.h;
    QF<NB> qf;
    load_q<E4M3, NB, DIFF>(qf, a, unit);
    State<NB> st;
    st.init();
    for (int i = 0; i < cnt; ++i) {
        cp_async_wait<T::STAGES - 2>();
        __syncthreads();
        feed();
        uint8_t *stage = csm + (i % T::STAGES) * T::STAGE;
        compute<E4M3, NB, DIFF, PARTS>(st, qf, stage);
        const bool end = cc.last();
        if (end || i == cnt - 1) {
            flush<E4M3, NB, DIFF>(st, reinterpret_cast<float *>(stage), a,
                                  a.part + ((int64_t)blockIdx.x + unit) * G2 * PART_W);
            if (i == cnt - 1) break;
            st.init();
        }
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
template <bool DIFF, bool BF16OUT>
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
        const int nt = seq_tiles(a, i);
        all += nt;
        if (i < b) before += nt;
    }
    before = warp_isum(before), all = warp_isum(all);
    const int nt = seq_tiles(a, b), chunk = (all * a.h_kv + splits - 1) / splits;
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
    const int64_t tiles = units * ceil_div64(n_max, CT_ROWS), slots = 3LL * num_sms();
    return (int)(tiles < slots ? tiles : slots);
}

template <bool E4M3, int NB, bool PAGED, bool DIFF, int PARTS>
static cudaError_t launch_split(const CacheArgs &a, int splits, cudaStream_t s) {
    const auto fn = k_cache_split<E4M3, NB, PAGED, DIFF, PARTS>;
    cudaError_t e = ensure_smem((const void *)fn, Tile<E4M3, NB>::SMEM);
    if (e != cudaSuccess) return e;
    fn<<<splits, CT_THREADS, Tile<E4M3, NB>::SMEM, s>>>(a);
    return cudaGetLastError();
}
template <bool E4M3, bool DIFF, int PARTS>
static cudaError_t pick_split(const CacheArgs &a, int splits, cudaStream_t s) {
    const bool one = (DIFF ? 2 : 1) * a.G <= 8;
    if (a.bt) return one ? launch_split<E4M3, 1, true, DIFF, PARTS>(a, splits, s) : launch_split<E4M3, 2, true, DIFF, PARTS>(a, splits, s);
    return one ? launch_split<E4M3, 1, false, DIFF, PARTS>(a, splits, s) : launch_split<E4M3, 2, false, DIFF, PARTS>(a, splits, s);
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
    if (diff) return bf_out ? cudaLaunchKernelEx(&cfg, k_cache_merge<true, true>, a, d, out, splits)
                            : cudaLaunchKernelEx(&cfg, k_cache_merge<true, false>, a, d, out, splits);
    return bf_out ? cudaLaunchKernelEx(&cfg, k_cache_merge<false, true>, a, d, out, splits)
                  : cudaLaunchKernelEx(&cfg, k_cache_merge<false, false>, a, d, out, splits);
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
