// cross.cu -- cross attention (mog_cross_attend): several query tokens of each sequence, or one, to the
// rows of a bf16 cache, all of which every query sees (an encoder's states, a document).
//
//   out = softmax(tau q.K^T) V     per query token and head, over the keys [0, N_b)
//
// The query rows that share a KV head are packed (token, then head), as many whole tokens as fit 128 rows to
// a tile.  A CTA has two streams over tiles of 128 keys: two query tiles that share every key tile ("pair"), or,
// where only one is left, one query tile whose streams take alternate key tiles and are joined at the end.  While
// the softmax of one stream runs, the tensor cores work for the other:
//
//   warps 0-3, 4-7  softmax of stream 0, 1: a thread has one query row; it reads its 128 logits from
//                   tensor memory, takes the running maximum, and writes the weights back as bf16 where the logits were
//   warp 8          issues the MMAs: S = Q K^T (128 x 128 x 128) and O += P V, P from tensor memory
//   warp 9          TMA copies of K and V tiles through a ring of 32 KB slots, in the order of their use
//   warp 10         TMA copies of the query tiles
//   warp 11         finds the items, a few ahead
//
// Work: an item is a pair of query tiles of a (sequence, KV head).  Lengths and counts are read on the device (a
// captured graph replays with others).  Either a CTA, one per SM, takes whole items, the longest sequences' first
// and in a snake (c, 2C - 1 - c, 2C + c, ...); or the key tiles of all items form one list, in units of two
// tile products, of which each CTA takes an equal share (sequences alike: of what whole rounds leave).  The parts of an item that several CTAs have are partials (at most
// two a CTA), which k_cross_merge folds.  cross_grid has the rule.  The copies of a CTA's next item run ahead.
//
// Bound by: the tensor cores, whose products the softmax does not hide completely.  4096 tokens of 32 heads over 32K rows
// of 8 KV heads: 1.33 to 1.46 ms, 1.50 to 1.65 PFLOP/s, the longer the GPU is at its power limit (1.40 ms in a graph of 20 calls: 1.57
// PFLOP/s, 0.83 of a library's matrix product in a burst, 0.93 of a sustained one); a unit (two tile products)
// takes about 2.9K cycles, 2048 of them the MMA pipe's, at 1.97 GHz.  The chain of a
// softmax tile is about 1300 cycles; an item's start and end (O read, normalised, stored) about 10K.  Few query rows (16
// tokens of 40 heads to 128K rows of 8 heads, 4 sequences, in pages): HBM, 335 us, 6.4 TB/s.
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
constexpr int CX_RING = 5;                       // slots of K and V tiles
constexpr int CX_THREADS = 384, CX_MMA = 8, CX_LOAD = 9, CX_Q = 10;
constexpr int CX_ITEMS = 4;                      // items found ahead
constexpr int CX_SORT = 64;                      // sequences that whole items are sorted over
constexpr int CX_ROUNDS = 64;                    // whole items of a CTA that are added up beforehand
// Registers: 168 a thread at launch; the softmax warps take 208, the others leave theirs at 80
// (256 * 208 + 128 * 80 = 63488 of 384 * 168 = 64512).
constexpr int CX_REGS_MORE = 208, CX_REGS_LESS = 80;
constexpr int CX_SMEM = (2 + CX_RING) * CX_TILE + 1024;
constexpr int CX_PART = MOG_D + 4;               // floats of a partial row: maximum, sum, 2 unused, accumulators
constexpr float CX_RISE = 8.f;                   // log2 of the rise of a maximum that O is rescaled for

struct CrossArgs {
    uint16_t *out;
    int64_t ob, ot, oh;
    const int *lengths, *count;
    int n_max, t_max, batch, h_kv, G;
    int tokens;      // of a query tile
    int qmul;        // 0 where the queries of all sequences are one in memory
    int out32;       // rows of the output begin at multiples of 32 bytes
    const int *bt;
    int pshift, pps, n_pages;
    int bmul, hmul;  // contiguous: 0 where all sequences (heads) are one in memory
    float scale2;    // tau * log2(e)
    // equal shares: [CTAs] what to fold at the beginning of a CTA's share and the partials
    // [2 * CTAs][part_rows][CX_PART]: of CTA c, slot 2c: the item that it does not begin, 2c + 1: that it does not end
    int4 *fold;
    float *part;
    int part_rows;
    int whole;       // whole items
    int polls;       // limit of the waits that last as long as an item: for the next one, for the queries' place
};

// A sequence as items of each of its KV heads: `pairs` of two query tiles, `units` units each, and one of a
// single query tile (`half` units) if half > 0.  An item without keys is a unit of its own (its rows are zeros).
struct CrossSeq {
    int count, len, nt, pairs, units, half;
    __device__ __forceinline__ void load(const CrossArgs &a, int b) {
        set(a, a.count ? min(max(a.count[b], 0), a.t_max) : a.t_max, min(max(a.lengths[b], 0), a.n_max));
    }
    __device__ __forceinline__ void set(const CrossArgs &a, int count_, int len_) {
        count = count_, len = len_;
        nt = (int)(((unsigned)len + CX_KEYS - 1) / CX_KEYS);
        const int tiles = (count + a.tokens - 1) / a.tokens;
        pairs = tiles >> 1;
        units = max(nt, 1);
        half = tiles & 1 ? max((nt + 1) >> 1, 1) : 0;
    }
    __device__ __forceinline__ int items() const { return pairs + (half > 0); }  // of a KV head
    __device__ __forceinline__ int cost() const { return pairs * units + half; }
};

// Whole items: sequences by their number of key tiles, the longest first, and where each one's items end in that
// order.  n = 0: not sorted; `items` of every (sequence, KV head), real or not.
struct CrossOrder {
    int n, items;
    int whole;                 // whole items: by cross_grid, or as `fits` finds
    int total, longest, most;  // units: of all items, of the longest one, of the CTA with the most
    int differ;                // sequences that are not like the first
    uint8_t seq[CX_SORT];
    int end[CX_SORT], count[CX_SORT], len[CX_SORT];  // (count, len: by sequence)
    // (by the whole CTA; followed by a barrier)
    __device__ __forceinline__ void make(const CrossArgs &a, int (&need)[CX_SORT], int (&key)[CX_SORT]) {
        const int tid = threadIdx.x, per = ((a.t_max + a.tokens - 1) / a.tokens + 1) / 2;
        const bool sort = a.batch <= CX_SORT && (a.whole ? a.batch * a.h_kv * per > (int)gridDim.x : a.batch > 1);
        if (tid == 0) {
            n = sort ? a.batch : 0, items = per, whole = a.whole;
            total = longest = most = differ = 0;
        }
        if (!sort) return;
        CrossSeq c;
        if (tid < a.batch) {
            c.load(a, tid);
            need[tid] = c.items() * a.h_kv, key[tid] = c.nt;
            count[tid] = c.count, len[tid] = c.len;
        }
        __syncthreads();
        if (tid < a.batch) {
            int rank = 0;
            int e = need[tid];
            for (int i = 0; i < a.batch; ++i)
                if (key[i] > key[tid] || (key[i] == key[tid] && i < tid)) ++rank, e += need[i];
            seq[rank] = (uint8_t)tid, end[rank] = e;
            if (!a.whole) {
                CrossSeq f;
                f.set(a, count[0], len[0]);
                atomicAdd(&total, c.cost() * a.h_kv);
                atomicMax(&longest, c.pairs ? c.units : c.half);
                atomicOr(&differ, c.nt != f.nt || c.pairs != f.pairs || c.half != f.half);
            }
        }
        if (!a.whole) fits(a);
    }
    // Sequences that differ, in a call whose largest lengths ask for equal shares: whole items if these leave the CTA with
    // the most to do little above the mean.  Equal shares of such sequences are more than their partials: CTAs are no longer in
    // step at the same key tiles, and L2 serves each on its own.  24 ragged batches, both ways: whole items are the faster
    // of the two up to 4/3 of the mean and 12 units (16 sequences, 16 heads, G = 8, 407 tokens to 1000 .. 4000 rows,
    // 515 units at most, 509 in the mean: 869 us against 1109; 4 sequences, 4 heads, 146 tokens, 30 and 12.5: 53.5
    // against 54.8; 4 sequences, 8 heads, G = 8, 69 tokens to 2000 .. 8000 rows, 59 and 17.9: 107 against 86).
    // (A function of its own: inlined, it moves the code of the main loops, which then take 2% longer.)
    __device__ __noinline__ void fits(const CrossArgs &a) {
        __syncthreads();
        const int ctas = gridDim.x, all = end[n - 1], limit = total / ctas + total / ctas / 3 + 12;
        if (!differ || longest > limit || all > CX_ROUNDS * ctas) return;
        const int c = threadIdx.x;
        if (c < ctas) {
            int sum = 0, k = 0;
            CrossSeq q;
            q.set(a, count[seq[0]], len[seq[0]]);
            for (int r = 0;; ++r) {
                const int i = r * ctas + (r & 1 ? ctas - 1 - c : c);
                if (i >= all) break;  // (those of later rounds are greater)
                while (end[k] <= i) ++k, q.set(a, count[seq[k]], len[seq[k]]);
                const int j = (i - (k ? end[k - 1] : 0)) % q.items();
                sum += j < q.pairs ? q.units : q.half;
            }
            atomicMax(&most, sum);
        }
        __syncthreads();
        if (threadIdx.x == 0) whole = most <= limit;
    }
};

// What a CTA works on next: `nt` key tiles from `first` on of an item.  The units of all items stay below 2^30.
struct Segment {
    CrossSeq q;
    int b, h, x;      // sequence, KV head, item
    int at;           // its unit in the item
    int left;         // units of the CTA from here on;  whole items: how many it has had
    bool pair, begins, ends;
    int first, nt;
    // Equal shares: the list's units, a share.  Sequences alike: CTAs first take `rounds` whole items each (`skipped`
    // in all), in step with one another, so that those of a KV head read its tiles from L2 at the same time; the
    // list is of the other items, pairs and then halves.
    int total, chunk, skipped, index;
    int rounds;
    bool even;

    __device__ __forceinline__ int units() const { return x < q.pairs ? q.units : q.half; }
    __device__ __forceinline__ void set(int most) {
        pair = x < q.pairs;
        const int n = min(units() - at, most);
        begins = at == 0, ends = at + n == units();
        first = pair ? at : 2 * at;
        nt = min(pair ? n : 2 * n, q.nt - first);
    }
    // The CTA's first segment; false if it has none (called by full warps).
    __device__ __forceinline__ bool start(const CrossArgs &a, const CrossOrder &o) {
        left = 0;
        if (o.whole) return take(a, o);
        plan(a, gridDim.x);
        if (rounds) return round(a);
        return share(a);
    }
    // Equal shares: how the work is laid out (called by full warps).
    __device__ __forceinline__ void plan(const CrossArgs &a, int ctas) {
        all_units(a);
        rounds = 0;
        if (even) {
            q.load(a, 0);
            const int units = a.batch * a.h_kv, p = units * q.pairs;
            rounds = p / ctas;
            skipped = rounds * ctas;
            total = (p - skipped) * q.units + units * q.half;
        }
        chunk = max((total + ctas - 1) / ctas, CX_LEAST);
    }
    static constexpr int CX_LEAST = 4;  // units of a share: fewer are not worth a CTA's start and its partials
    // sequences alike: the next whole item
    __device__ __forceinline__ bool round(const CrossArgs &a) {
        item(a, left++ * gridDim.x + blockIdx.x);
        q.load(a, b);
        set(INT32_MAX);
        return true;
    }
    // sequences alike: pair item i, or half item i - all pairs
    __device__ __forceinline__ void item(const CrossArgs &a, int i) {
        const int p = a.batch * a.h_kv * q.pairs, u = i < p ? i / q.pairs : i - p;
        x = i < p ? i - u * q.pairs : q.pairs;
        b = u / a.h_kv, h = u - b * a.h_kv;
        index = i, at = 0;
    }
    // the CTA's share of the list (called by full warps unless the sequences are alike)
    __device__ __forceinline__ bool share(const CrossArgs &a) {
        rounds = 0;
        const int p = blockIdx.x * chunk;  // (below total + 2^30)
        if (p >= total) return false;
        left = min(chunk, total - p);
        seek(a, p);
        set(left);
        return true;
    }
    // whole items: the next one of the snake
    __device__ __forceinline__ bool take(const CrossArgs &a, const CrossOrder &o) {
        while (true) {
            const int i = left * gridDim.x + (left & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            ++left;
            if (o.n == 0) {  // one item each, or too many sequences to sort: the sequences as they are
                const int unit = i / o.items;
                if (unit >= a.batch * a.h_kv) return false;
                b = unit / a.h_kv, h = unit - b * a.h_kv, x = i - unit * o.items;
                q.load(a, b);
                if (x < q.items()) break;
            } else {
                int k = 0;
                while (k < o.n && o.end[k] <= i) ++k;
                if (k == o.n) return false;
                b = o.seq[k];
                q.set(a, o.count[b], o.len[b]);
                const int r = i - (k ? o.end[k - 1] : 0), n = max(q.items(), 1);
                h = min(r / n, a.h_kv - 1), x = r - r / n * n;
                break;
            }
        }
        at = 0;
        set(INT32_MAX);
        return true;
    }
    // units of all sequences, and whether these are alike
    __device__ __forceinline__ void all_units(const CrossArgs &a) {
        const int lane = threadIdx.x & 31;
        CrossSeq f;
        f.load(a, 0);
        int s = 0;
        bool same = true;
        for (int i = lane; i < a.batch; i += 32) {
            CrossSeq c;
            c.load(a, i);
            s += c.cost() * a.h_kv;
            same = same && c.nt == f.nt && c.pairs == f.pairs && c.half == f.half;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        total = s;
        even = __all_sync(0xffffffffu, same) && s > 0;
    }
    // The item that holds unit p of the list (p < total; called by full warps unless the sequences are alike).
    __device__ __forceinline__ void seek(const CrossArgs &a, int p) {
        if (even) {
            const int pairs = a.batch * a.h_kv * q.pairs, first = (pairs - skipped) * q.units;
            const int i = p < first ? p / q.units : (p - first) / q.half, n = p < first ? i * q.units : first + i * q.half;
            item(a, (p < first ? skipped : pairs) + i);
            at = p - n;
            q.load(a, b);
            return;
        }
        const int lane = threadIdx.x & 31;
        int base = 0;
        b = a.batch - 1;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            CrossSeq c;
            int mine = 0;
            if (b0 + lane < a.batch) c.load(a, b0 + lane), mine = c.cost() * a.h_kv;
            int end = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += v;
            }
            const unsigned in = __ballot_sync(0xffffffffu, base + end > p);
            if (in) {
                const int l = __ffs(in) - 1;
                b = b0 + l;
                base += __shfl_sync(0xffffffffu, end - mine, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, end, 31);
        }
        q.load(a, b);
        const int c = max(q.cost(), 1), r = p - base;
        h = min(r / c, a.h_kv - 1);
        const int o = r - h * c;
        x = min(o / q.units, q.pairs);
        at = o - x * q.units;
    }
    __device__ __forceinline__ bool next(const CrossArgs &a, const CrossOrder &o) {
        if (o.whole) return take(a, o);
        if (rounds) return left < rounds ? round(a) : share(a);
        left -= min(units() - at, left);
        if (left <= 0) return false;
        if (even) {
            item(a, index + 1);
            q.load(a, b);
            set(left);
            return true;
        }
        at = 0;
        if (++x >= q.items()) {
            x = 0;
            if (++h == a.h_kv) {
                h = 0;
                do {
                    if (++b >= a.batch) return false;  // (lengths that changed under the call)
                    q.load(a, b);
                } while (q.count == 0);
            }
        }
        set(left);
        return true;
    }
    // What k_cross_merge has to do for the item in which the share of CTA c > 0 begins, if that is the first share to
    // begin inside it (by a full warp): (how many CTAs from c - 1 on have parts, 0 for none; sequence; KV head; item,
    // from 2^30 on: a pair).
    __device__ __forceinline__ int4 fold(const CrossArgs &a) {
        plan(a, gridDim.x);
        const int c = blockIdx.x, p = c * chunk;
        if (c == 0 || p >= total) return make_int4(0, 0, 0, 0);
        seek(a, p);
        const int begin = p - at, end = begin + units();
        if (at == 0 || begin < p - chunk) return make_int4(0, 0, 0, 0);
        return make_int4((end - 1) / chunk - c + 2, b, h, x + (x < q.pairs ? 1 << 30 : 0));
    }
    bool end;  // (no item any more)
    // tiles of stream s, its j-th; rows of the last tile behind the sequence's end
    __device__ __forceinline__ int n_of(int s) const { return pair ? nt : (nt - s + 1) >> 1; }
    __device__ __forceinline__ int tile_of(int s, int j) const { return first + (pair ? j : 2 * j + s); }
    __device__ __forceinline__ int tail() const { return max(0, (first + nt) * CX_KEYS - q.len); }
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
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
__device__ __forceinline__ void sts16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}
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

// Bit i: key k + i of a tile is behind the sequence's end (`left` keys of it are not), or in no page (bit j of
// groups: the page of keys j << gshift .. is one; gshift >= 4).
template <bool PAGED>
__device__ __forceinline__ uint32_t dead_keys(int k, int left, unsigned groups, int gshift) {
    uint32_t dead = left >= k + 32 ? 0u : left <= k ? 0xffffffffu : 0xffffffffu << (left - k);
    if (PAGED) {
        if (!(groups >> (k >> gshift) & 1u)) dead |= 0xffffu;
        if (!(groups >> ((k + 16) >> gshift) & 1u)) dead |= 0xffff0000u;
    }
    return dead;
}

// Barriers.  Every wait is for the phase after the last one that its waiter has seen.
struct CrossBars {
    uint64_t full[CX_RING];  // a copy is there
    // Copies that fall free together (V of a tile and K of the next one) are a group; the slot of its last one says so.
    uint64_t free[CX_RING];
    uint64_t q_full, q_free;  // the item's queries are there; their place, which the outputs pass through, is free
    uint64_t s_full[2];       // a stream's logits
    uint64_t p_full[2][2];    // its weights, of each half of the keys
    uint64_t o_full[2], o_free[2];  // its sums are through; have been read
    uint64_t j_full, j_free;  // one query tile: stream 1's maxima and sums are there; have been read
    uint64_t i_full[CX_ITEMS], i_free[CX_ITEMS];  // the items
    uint64_t v_tail[4];       // an item's last V: its rows behind the sequence's end are zero (the ring holds 2 such at most)
    uint64_t drained;         // no MMA runs any more
};

// The rows that the softmax thread r of stream s would have written of the CTA's items from the skip-th on are NaN, the
// partials' by their maxima: a wait has given up, and the items did not come.  (by full warps; a function of its own, as `fits`)
__device__ __noinline__ void lost_items(const CrossArgs &a, const CrossOrder &o, uint32_t skip, int s, int r) {
    Segment g;
    for (bool more = g.start(a, o); more; more = g.next(a, o)) {
        const int t0 = (2 * g.x + (g.pair ? s : 0)) * a.tokens;
        if (skip > 0) {
            --skip;
        } else if ((g.pair || s == 0) && r < min(a.tokens, g.q.count - t0) * a.G) {
            if (g.begins && g.ends) {
                const int t = r / a.G, hd = r - t * a.G;
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + g.b * a.ob + (t0 + t) * a.ot + (int64_t)(g.h * a.G + hd) * a.oh);
                for (int i = 0; i < MOG_D / 8; ++i) dst[i] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            } else {
                a.part[((2 * (int64_t)blockIdx.x + (g.begins ? 1 : 0)) * a.part_rows + (g.pair ? s * CX_M : 0) + r) * CX_PART] = __int_as_float(0x7fffffff);
            }
        }
        __syncwarp();
    }
}

template <bool PAGED>
__global__ void __launch_bounds__(CX_THREADS, 1) k_cross(CrossArgs a, const __grid_constant__ CUtensorMap qmap,
                                                         const __grid_constant__ CUtensorMap kmap,
                                                         const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t cx_raw[];
    __shared__ __align__(8) CrossBars bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    pdl_trigger();  // (k_cross_merge waits for the whole grid)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ Segment s_items[CX_ITEMS];  // what warp 11 has found for the others to do
    __shared__ CrossOrder s_order;
    s_order.make(a, *reinterpret_cast<int(*)[CX_SORT]>(cx_raw), *reinterpret_cast<int(*)[CX_SORT]>(cx_raw + 4 * CX_SORT));
    fence_proxy_async();  // (the queries may be copied to where that worked)
    __syncthreads();
    const uint32_t sQ = (smem_u32(cx_raw) + 1023u) & ~1023u, sR = sQ + 2 * CX_TILE;
    auto bar = [&](const uint64_t &x) { return smem_u32(&x); };
    float2 *s_ml = reinterpret_cast<float2 *>(cx_raw + (sQ + CX_TILE - smem_u32(cx_raw)));  // (one query tile: the other's place)
    if (tid == CX_LOAD * 32) {
        for (int i = 0; i < CX_RING; ++i) mbar_init(bar(bars.full[i]), 1), mbar_init(bar(bars.free[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bars.s_full[i]), 1);
            for (int k = 0; k < 2; ++k) mbar_init(bar(bars.p_full[i][k]), CX_M);
            mbar_init(bar(bars.o_full[i]), 1);
            mbar_init(bar(bars.o_free[i]), CX_M);
        }
        mbar_init(bar(bars.q_full), 1);
        mbar_init(bar(bars.q_free), 2 * CX_M);
        mbar_init(bar(bars.j_full), CX_M);
        mbar_init(bar(bars.j_free), CX_M);
        for (int i = 0; i < 4; ++i) mbar_init(bar(bars.v_tail[i]), 1);
        mbar_init(bar(bars.drained), 1);
        for (int i = 0; i < CX_ITEMS; ++i) mbar_init(bar(bars.i_full[i]), 1), mbar_init(bar(bars.i_free[i]), 11);  // (warps 0 .. 10)
        fence_barrier_init();
        s_fail = 0;
    }
    if (warp == CX_MMA) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // The CTA's it-th item (by a whole warp, or by one thread for its own); false behind the last one, and if it does not
    // come.  Every role goes through all that come, also after another wait that has given up.
    auto item_at = [&](uint32_t it) {
        if (!mbar_wait(bar(bars.i_full[it % CX_ITEMS]), (it / CX_ITEMS) & 1, a.polls)) {
            atomicExch(&s_fail, 1);
            return false;
        }
        return !s_items[it % CX_ITEMS].end;
    };
    auto warp_item_at = [&](uint32_t it) { return __all_sync(0xffffffffu, item_at(it)) != 0; };
    auto item_done = [&](uint32_t it) { mbar_arrive(bar(bars.i_free[it % CX_ITEMS])); };
    auto warp_item_done = [&](uint32_t it) {
        __syncwarp();
        if (lane == 0) item_done(it);
    };
    auto tS = [&](int s) { return tmem + (uint32_t)(s * 128); };
    auto tO = [&](int s) { return tmem + (uint32_t)(256 + s * 128); };

    if (warp >= CX_MMA) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CX_REGS_LESS));
        if (warp == CX_LOAD) {
            // -------------------------------------------------------------- copies of K and V
            const int gr = PAGED ? min(CX_KEYS, 1 << a.pshift) : CX_KEYS, ng = CX_KEYS / gr;  // rows of a copy, copies of a tile
            int slot = 0, issued = 0, tails = 0, b = 0, h = 0, len = 0;
            // bits by slot: the next phase of full; its occupant is the first of a group of two; the next phase of free
            uint32_t fullp = 0, two = 0, freep = 0;
            bool ok = true;
            // paged: the pages of a tile (lane g: of its g-th copy), asked for a tile ahead
            auto pages_of = [&](int tile) {
                const int key = tile * CX_KEYS + lane * gr;
                return PAGED && lane < ng && key < len ? __ldg(a.bt + (int64_t)b * a.pps + (key >> a.pshift)) : -1;
            };
            auto load = [&](const CUtensorMap *map, int tile, int page, bool value, bool first_of_two) {
                if (issued >= CX_RING) {  // the slot's last occupant has been used
                    const int w = two >> slot & 1 ? (slot + 1 == CX_RING ? 0 : slot + 1) : slot;
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.free[w]), (freep >> w & 1) ^ 1));
                }
                if (!ok) return;
                const uint32_t dst = sR + slot * CX_TILE;
                const int key = tile * CX_KEYS + lane * gr;  // lane g: the tile's g-th copy
                const bool seen = lane < ng && key < len, there = seen && (!PAGED || (unsigned)page < (unsigned)a.n_pages);
                const unsigned have = __ballot_sync(0xffffffffu, there);
                if (PAGED && value) {  // a page that is none: its weights are zero, and so must its values be finite
                    const unsigned none = __ballot_sync(0xffffffffu, seen && !there);
                    for (int i = 0; none >> i; ++i)
                        if (none >> i & 1) zero_rows(dst, i * gr, gr);
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
                const uint32_t bit = 1u << slot;
                fullp ^= bit;
                two = first_of_two ? two | bit : two & ~bit;
                if (!first_of_two) freep ^= bit;
                ++issued;
                slot = slot + 1 == CX_RING ? 0 : slot + 1;
            };
            for (uint32_t it = 0; warp_item_at(it); warp_item_done(it++)) {
                const Segment &g = s_items[it % CX_ITEMS];
                if (!ok) continue;
                // in the order of their use
                const int ways = g.pair ? 1 : 2, nt = g.nt, first = g.first;
                b = g.b, h = g.h, len = g.q.len;
                int ahead = pages_of(first), now[2] = {0, 0};  // of the next K; of the V to come
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= min(nt, ways) || !ok) continue;
                    now[t] = ahead;
                    ahead = t + 1 < nt ? pages_of(first + t + 1) : -1;
                    load(&kmap, first + t, now[t], false, t + 1 < min(nt, ways));
                }
                for (int t = 0; t < nt && ok; ++t) {
                    const bool more = t + ways < nt;
                    load(&vmap, first + t, now[0], true, more);
                    if (ways == 2) now[0] = now[1];
                    if (!more || !ok) continue;
                    (ways == 2 ? now[1] : now[0]) = ahead;
                    ahead = t + ways + 1 < nt ? pages_of(first + t + ways + 1) : -1;
                    load(&kmap, first + t + ways, ways == 2 ? now[1] : now[0], false, false);
                }
                if (nt > 0 && g.tail() > 0 && ok) {
                    // rows behind the sequence's end: their weights are zero, and so must their values be finite
                    const int last = slot == 0 ? CX_RING - 1 : slot - 1;
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.full[last]), (fullp >> last & 1) ^ 1));
                    zero_rows(sR + last * CX_TILE, CX_KEYS - g.tail(), g.tail());
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(bars.v_tail[tails++ & 3]));
                }
                if (!ok) atomicExch(&s_fail, 1);
            }
            // no copy outlives the CTA
            for (int i = 0; i < min(issued, CX_RING); ++i) mbar_wait(bar(bars.full[i]), (fullp >> i & 1) ^ 1);
        } else if (warp == CX_MMA) {
            // ---------------------------------------------------------------- MMAs
            // One thread, the streams in turn: while it waits for the weights of one, the MMAs of the other run.
            if (elect_one()) {
                constexpr uint32_t ID_S = idesc_bf16_f32(CX_M, CX_KEYS), ID_O = idesc_bf16_f32(CX_M, MOG_D) | 1u << 16;
                const uint64_t qd = smem_desc_sw128(sQ), kd = smem_desc_sw128(sR), vd = v_desc(sR);
                bool ok = true, pair = false;
                int at = 0;                         // the next slot of the ring
                uint32_t phase = 0, seg = 0, tails = 0;
                uint32_t pp0 = 0, pp1 = 0;          // the next phase of the streams' p_full
                auto next_copy = [&]() {            // its slot, once it is there
                    const int slot = at;
                    ok = ok && mbar_wait(bar(bars.full[slot]), phase);
                    if (++at == CX_RING) at = 0, phase ^= 1;
                    return slot;
                };
                auto mma_s = [&](int s, int slot) {
                    const uint64_t q = qd + (pair ? s : 0) * (CX_TILE >> 4), k = kd + slot * (CX_TILE >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const int off = ((ks >> 2) * CX_HALF + (ks & 3) * 32) >> 4;
                        tc_mma(tS(s), q + off, k + off, ID_S, ks != 0);
                    }
                    tc_commit(bar(bars.s_full[s]));
                };
                // a tile of stream s; v, k: the slots of its values and of the next tile's keys
                auto step = [&](int s, bool opens, int v, int k, bool more) {
                    const uint64_t d = vd + v * (CX_TILE >> 4);
                    uint32_t &pp = s ? pp1 : pp0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        ok = ok && mbar_wait(bar(bars.p_full[s][c]), pp);
                        if (!ok) return;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 4 * c; ks < 4 * c + 4; ++ks)
                            tc_mma_ts(tO(s), tS(s) + 8 * ks, d + ks * (2048 >> 4), ID_O, ks != 0 || !opens);
                    }
                    pp ^= 1;
                    if (more) mma_s(s, k);
                    else tc_commit(bar(bars.o_full[s]));
                };
                auto run = [&](const Segment &g) {
                    const int nt = g.nt, tail = g.tail();
                    pair = g.pair;
                    if (nt == 0) return;
                    ok = mbar_wait(bar(bars.q_full), seg & 1);
                    if (!ok) return;
                    tc_fence_after();
                    if (pair) {
                        const int k0 = next_copy();
                        if (!ok) return;
                        mma_s(0, k0), mma_s(1, k0);
                        tc_commit(bar(bars.free[k0]));
                        for (int s = 0; s < 2 && seg > 0; ++s) ok = ok && mbar_wait(bar(bars.o_free[s]), (seg - 1) & 1);
                        for (int j = 0; j < nt && ok; ++j) {
                            const bool more = j + 1 < nt;
                            const int v = next_copy(), k = more ? next_copy() : v;
                            if (!more && tail > 0) ok = ok && mbar_wait(bar(bars.v_tail[tails & 3]), (tails >> 2) & 1);
                            if (ok) step(0, j == 0, v, k, more);
                            if (ok) step(1, j == 0, v, k, more);
                            if (!ok) break;
                            tc_commit(bar(bars.free[k]));
                        }
                    } else {
                        int k0 = next_copy();
                        if (ok) mma_s(0, k0);
                        if (nt > 1 && ok) {
                            k0 = next_copy();
                            if (ok) mma_s(1, k0);
                        }
                        if (!ok) return;
                        tc_commit(bar(bars.free[k0]));
                        for (int s = 0; s < 2 && seg > 0; ++s) ok = ok && mbar_wait(bar(bars.o_free[s]), (seg - 1) & 1);
                        for (int t = 0; t < nt && ok; t += 2) {
                            bool more = t + 2 < nt;
                            int v = next_copy(), k = more ? next_copy() : v;
                            if (t + 1 == nt && tail > 0) ok = ok && mbar_wait(bar(bars.v_tail[tails & 3]), (tails >> 2) & 1);
                            if (ok) step(0, t == 0, v, k, more);
                            if (!ok) break;
                            tc_commit(bar(bars.free[k]));
                            if (t + 1 >= nt) break;
                            more = t + 3 < nt;
                            v = next_copy(), k = more ? next_copy() : v;
                            if (t + 2 == nt && tail > 0) ok = ok && mbar_wait(bar(bars.v_tail[tails & 3]), (tails >> 2) & 1);
                            if (ok) step(1, t == 0, v, k, more);
                            if (!ok) break;
                            tc_commit(bar(bars.free[k]));
                        }
                    }
                    ++seg;
                    tails += tail > 0;
                };
                for (uint32_t it = 0; item_at(it); item_done(it++)) {
                    if (ok) run(s_items[it % CX_ITEMS]);
                    if (!ok) atomicExch(&s_fail, 1);
                }
                tc_commit(bar(bars.drained));  // no MMA outlives the CTA
                mbar_wait(bar(bars.drained), 0);
            }
            __syncwarp();
        } else if (warp == CX_Q) {
            // ---------------------------------------------------------------- copies of the queries
            if (lane == 0) {
                const uint32_t bytes = (uint32_t)(a.tokens * a.G) * 256;  // of a tile; tokens from t_max on are zeros
                uint32_t seg = 0;
                bool ok = true;
                for (uint32_t it = 0; item_at(it); item_done(it++)) {
                    const Segment &g = s_items[it % CX_ITEMS];
                    if (!ok || g.nt == 0) continue;
                    if (seg > 0) ok = mbar_wait(bar(bars.q_free), (seg - 1) & 1, a.polls);
                    if (!ok) {
                        atomicExch(&s_fail, 1);
                        continue;
                    }
                    const int n = g.pair ? 2 : 1;
                    mbar_expect_tx(bar(bars.q_full), n * bytes);
                    for (int i = 0; i < n; ++i)
                        for (int d = 0; d < 2; ++d)
                            tma_load_5d(sQ + i * CX_TILE + d * CX_HALF, &qmap, 64 * d, 0, (2 * g.x + i) * a.tokens, g.h, g.b * a.qmul,
                                        bar(bars.q_full));
                    ++seg;
                }
                if (seg > 0) mbar_wait(bar(bars.q_full), (seg - 1) & 1);  // no copy outlives the CTA
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------------------- items
            Segment w;
            bool more = w.start(a, s_order), ok = true;
            for (uint32_t it = 0; ok; ++it) {
                if (it >= CX_ITEMS) ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.i_free[it % CX_ITEMS]), (it / CX_ITEMS - 1) & 1, a.polls));
                w.end = !more;
                if (lane == 0 && ok) {
                    s_items[it % CX_ITEMS] = w;
                    mbar_arrive(bar(bars.i_full[it % CX_ITEMS]));
                }
                if (!more) break;
                more = w.next(a, s_order);
            }
            if (!ok) atomicExch(&s_fail, 1);
            if (!a.whole) {
                const int4 f = s_order.whole ? make_int4(0, 0, 0, 0) : w.fold(a);
                if (lane == 0) a.fold[blockIdx.x] = f;
            }
        }
    } else {
        // ----------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CX_REGS_MORE));
        const int s = warp >> 2, r = tid & 127, gshift = PAGED ? min(a.pshift, 7) : 7;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        uint32_t sp = 0, op0 = 0, op1 = 0, joins = 0;       // the next phases of s_full and both o_full (op0: of q_full, too)
        const bool row = r < a.tokens * a.G;  // (the rows behind the tile's tokens hold anything)
        bool ok = true;
        uint32_t it = 0;
        for (; warp_item_at(it); warp_item_done(it++)) {
            const Segment &g = s_items[it % CX_ITEMS];
            const int n = g.n_of(s), n1 = g.n_of(1), len = g.q.len;
            const bool pair = g.pair, whole = g.begins && g.ends;
            auto q_done = [&]() {  // the thread's part in freeing the query tiles
                fence_proxy_async();
                mbar_arrive(bar(bars.q_free));
            };
            const int tile0 = g.tile_of(s, 0), tiles = pair ? 1 : 2;  // the stream's tiles: tile0, tile0 + tiles, ...
            const int *bt = PAGED ? a.bt + (int64_t)g.b * a.pps : nullptr;
            float m = -INFINITY, l = 0.f;
            int page = 0;  // paged: the page of the next tile's group `lane`
            auto page_of = [&](int j) {
                if (!PAGED || j >= n) return;
                const int key = (tile0 + j * tiles) * CX_KEYS + (lane << gshift);
                page = -1;
                if (lane < CX_KEYS >> gshift && key < len) page = __ldg(bt + (key >> a.pshift));
            };
            page_of(0);
            for (int j = 0; j < n && ok; ++j) {
                const int left = len - (tile0 + j * tiles) * CX_KEYS;
                unsigned groups = 0xffffffffu;
                if (PAGED) {
                    groups = __ballot_sync(0xffffffffu, (unsigned)page < (unsigned)a.n_pages);
                    page_of(j + 1);
                }
                ok = __all_sync(0xffffffffu, mbar_wait(bar(bars.s_full[s]), sp));
                sp ^= 1;
                if (!ok) break;
                if (j + 1 == n && pair && whole) q_done();  // (all of the stream's logits have been computed)
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
                        for (int w = 2 * c; w < 2 * c + 2; ++w) {
                            const uint32_t dead = dead_keys<PAGED>(32 * w, left, groups, gshift);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (dead >> i & 1) v[32 * w + i] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int i = 64 * c; i < 64 * c + 64; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = fmax3(mx[k], v[i + k], v[i + 4 + k]);
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2, f = a.scale2;
                const bool big = row && fabsf(top) > 16777216.f && fabsf(top) < INFINITY;
                const float mn = fmaxf(m, top);
                if (j == 0) m = mn;
                const bool need = row && mn > m + CX_RISE;
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
            // ------------------------------------------------------------- outputs
            const bool some = g.nt > 0, reads = some && (pair || s == 0), join = some && !pair;
            if (join) {  // stream 1's maxima and sums to stream 0, which reads both O
                if (s == 1) {
                    if (joins > 0) ok = ok && mbar_wait(bar(bars.j_free), (joins - 1) & 1);
                    // With one key tile the stream has waited for nothing of this item, and another warp's partial of the last one
                    // may still be passing through this place: it is free when the item's queries are there, which q_free has let in.
                    if (n == 0) ok = ok && mbar_wait(bar(bars.q_full), op0);
                    if (ok) s_ml[r] = make_float2(m, l);
                    else atomicExch(&s_fail, 1);  // (before stream 0 reads it)
                    mbar_arrive(bar(bars.j_full));
                } else {
                    ok = ok && mbar_wait(bar(bars.j_full), joins & 1);
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok && pair && whole && some) q_done();
            if (reads && ok) {
                if (join || s == 0) ok = mbar_wait(bar(bars.o_full[0]), op0);
                if (join ? n1 > 0 : s == 1) ok = ok && mbar_wait(bar(bars.o_full[1]), op1);
                ok = __all_sync(0xffffffffu, ok);
            }
            if (some) op0 ^= 1;
            if (n1 > 0) op1 ^= 1;
            if (!ok) atomicExch(&s_fail, 1);
            tc_fence_after();
            if (pair || s == 0) {
                float mine = 1.f, his = 0.f;
                if (join) {
                    const float2 ml = s_ml[r];
                    mbar_arrive(bar(bars.j_free));
                    if (whole) q_done(), q_done();  // (for stream 1 too, which may be an item ahead)
                    const float mn = fmaxf(m, ml.x), sh = mn == -INFINITY ? 0.f : mn;
                    mine = ex2(m - sh), his = n1 > 0 ? ex2(ml.x - sh) : 0.f;
                    m = mn;
                    l = l * mine + (n1 > 0 ? ml.y * his : 0.f);
                }
                const bool failed = !ok || *(volatile int *)&s_fail != 0;
                if (whole) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;  // (nothing seen: zeros; a sum that is NaN stays)
                    mine *= inv, his *= inv;
                }
                if (failed) mine = __int_as_float(0x7fffffff);  // a wait gave up: NaN, not a wrong number
                const int t0 = (2 * g.x + (pair ? s : 0)) * a.tokens;           // the tile's first token
                const int live = min(a.tokens, g.q.count - t0) * a.G;          // its rows
                const int w0 = (warp & 3) * 32, k0 = lane >> 4, ch = lane & 15;  // the warp's first row; what a lane copies
                const uint32_t stage = sQ + (pair ? s : 0) * CX_TILE + w0 * 256;
                float *part = a.part + ((2 * (int64_t)blockIdx.x + (g.begins ? 1 : 0)) * a.part_rows + (pair ? s * CX_M : 0)) * CX_PART;
                if (!whole && r < live) *reinterpret_cast<float2 *>(part + (int64_t)r * CX_PART) = make_float2(failed ? mine : m, l);
                auto get = [&](int c, float(&o)[32]) {  // 32 dimensions of the thread's row
                    if (some && ok) {
                        tmem_ld32(tO(s) + lanes + 32 * c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= mine;
                        if (join && n1 > 0) {
                            float o1[32];
                            tmem_ld32(tO(1) + lanes + 32 * c, o1);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] += o1[i] * his;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = mine;
                    }
                };
                auto o_read = [&]() {
                    tc_fence_before();
                    mbar_arrive(bar(bars.o_free[s]));
                    if (join) mbar_arrive(bar(bars.o_free[1]));
                };
                if (whole) {  // a row a thread
                    if (!some) mine = his = 0.f;  // no keys: zeros
                    const int t = r / a.G, hd = r - t * a.G;
                    uint16_t *dst = a.out + g.b * a.ob + (t0 + t) * a.ot + (int64_t)(g.h * a.G + hd) * a.oh;
                    // (loops that are not unrolled: code that runs once an item waits for its instructions more than for
                    // anything else)
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        get(c, o);
                        if (r < live) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t x[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) x[k] = cvt_bf2(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]);
                                uint16_t *to = dst + 32 * c + 16 * i;
                                const uint4 y = make_uint4(x[0], x[1], x[2], x[3]), z = make_uint4(x[4], x[5], x[6], x[7]);
                                if (a.out32) {
                                    stg32(to, y, z);
                                } else {
                                    *reinterpret_cast<uint4 *>(to) = y;
                                    *reinterpret_cast<uint4 *>(to + 8) = z;
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if (some) o_read();
                } else {
                    // A partial, fp32, 64 dimensions at a time: a warp's 32 rows pass through its part of the query tile, to
                    // leave in whole pieces of 256 bytes: 16-byte chunk ch of a row at chunk ch ^ (row & 7), without bank
                    // conflicts for a row a lane and for 16 lanes a row.
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        get(c, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sts16(stage + lane * 256 + (((8 * (c & 1) + i) ^ (lane & 7)) << 4), __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                                  __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
                        if (c & 1) {
                            __syncwarp();
#pragma unroll 4
                            for (int k = k0; k < 32; k += 2) {
                                const uint4 x = lds16(stage + k * 256 + ((ch ^ (k & 7)) << 4));
                                if (w0 + k < live) *reinterpret_cast<uint4 *>(part + (int64_t)(w0 + k) * CX_PART + 4 + 32 * (c - 1) + 4 * ch) = x;
                            }
                            __syncwarp();
                        }
                    }
                    o_read();
                    q_done();
                    if (join) q_done();
                }
                __syncwarp();
            }
            joins += join;
        }
        if (__any_sync(0xffffffffu, *(volatile int *)&s_fail != 0)) lost_items(a, s_order, it, s, r);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == CX_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Folds the partials of the items that several CTAs share: blocks (c - 1, *) that of a.fold[c], a warp per query row,
// four dimensions a lane.
__global__ void __launch_bounds__(256) k_cross_merge(CrossArgs a) {
    constexpr int U = 8;  // partials in flight
    const int lane = threadIdx.x & 31, c0 = blockIdx.x;
    pdl_wait();  // (by every block: nothing behind this kernel starts before k_cross has ended)
    const int4 f = __ldcg(a.fold + c0 + 1);
    if (f.x == 0) return;
    const int b = f.y, h = f.z, x = f.w & ((1 << 30) - 1), rows = f.w >> 30 ? 2 * CX_M : CX_M;
    const int count = a.count ? min(max(a.count[b], 0), a.t_max) : a.t_max;
    for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < rows; row += gridDim.y * 8) {
        const int r = row & (CX_M - 1), tile = 2 * x + (row >= CX_M);
        const int t = tile * a.tokens + r / a.G, hd = r % a.G;
        if (r >= a.tokens * a.G || t >= count) continue;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        bool nan = false;
        for (int k = 0; k < f.x; k += U) {
            float2 ml[U];
            float4 v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool ok = k + i < f.x;
                const int64_t slot = 2 * ((int64_t)c0 + k + i) + (k + i == 0 ? 1 : 0);
                const float *from = a.part + (slot * a.part_rows + row) * CX_PART;
                ml[i] = ok ? __ldcg(reinterpret_cast<const float2 *>(from)) : make_float2(-INFINITY, 0.f);
                v[i] = ok ? __ldcg(reinterpret_cast<const float4 *>(from + 4) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mn = m;
#pragma unroll
            for (int i = 0; i < U; ++i) mn = fmaxf(mn, ml[i].x), nan |= ml[i].x != ml[i].x;
            const float sh = mn == -INFINITY ? 0.f : mn, d = ex2(m - sh);
            m = mn;
            l *= d, acc.x *= d, acc.y *= d, acc.z *= d, acc.w *= d;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float e = ex2(ml[i].x - sh);
                l += ml[i].y * e;
                acc.x += v[i].x * e, acc.y += v[i].y * e, acc.z += v[i].z * e, acc.w += v[i].w * e;
            }
        }
        const float inv = nan ? __int_as_float(0x7fffffff) : l == 0.f ? 0.f : 1.f / l;
        uint16_t *dst = a.out + b * a.ob + t * a.ot + (int64_t)(h * a.G + hd) * a.oh + 4 * lane;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_bf2(acc.x * inv, acc.y * inv), cvt_bf2(acc.z * inv, acc.w * inv));
    }
}

// The grid and its work, by what the largest lengths and counts make of it.  Equal shares cost partials (up to 256 KB
// written and read by each CTA) and their fold, as much as about 8 units of work; whole items leave the SMs
// with unequal ones (8 sequences, 16 heads, 500 tokens to 375 .. 1500 rows: whole items 46 us, equal shares 84; 1 sequence,
// 8 heads, G = 4, 64 tokens to 4000 rows: 57 against 28).  A call laid out for equal shares whose sequences differ may still
// take whole items (CrossOrder::fits).
static void cross_grid(int batch, int h_kv, int G, int t_max, int n_max, int64_t &ctas, int &whole) {
    const int64_t tiles = ceil_div64(t_max, CX_M / G), nt = ceil_div64(n_max, CX_KEYS), per = ceil_div64(tiles, 2);
    const int64_t units = (int64_t)batch * h_kv, all = units * (tiles / 2 * nt + tiles % 2 * ceil_div64(nt, 2));
    const int64_t sms = num_sms(), longest = tiles > 1 ? nt : ceil_div64(nt, 2);
    whole = units * per <= (1 << 30) && ceil_div64(units * per, sms) * longest <= all / sms + 8;
    ctas = std::min(sms, whole ? units * per : ceil_div64(all, Segment::CX_LEAST));
}

// Tensor map of bf16 rows, `dims` of which the first is a row's 128 elements; strides in elements, of no account for a
// dim of one entry.  Boxes of 64 elements by `box`.  False if TMA cannot describe it.
static bool row_map(CUtensorMap *map, const void *base, int n, const int64_t *dims, const int64_t *strides, const int *box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[5], st[4];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < n; ++i) {
        d[i] = (cuuint64_t)dims[i], bx[i] = (cuuint32_t)box[i], es[i] = 1;
        if (i == 0) continue;
        st[i - 1] = dims[i] > 1 ? (cuuint64_t)strides[i] * 2 : 256;
        if (st[i - 1] == 0 || (st[i - 1] & 15) || st[i - 1] >= (1ull << 40)) return false;
    }
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n, const_cast<void *>(base), d, st, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int cross_part_rows(int G, int t_max) { return t_max > CX_M / G ? 2 * CX_M : CX_M; }

size_t cross_scratch(int batch, int h_kv, int G, int t_max, int n_max) {
    int64_t ctas;
    int whole;
    cross_grid(batch, h_kv, G, t_max, n_max, ctas, whole);
    return whole ? 0 : ctas * (sizeof(int4) + (size_t)2 * cross_part_rows(G, t_max) * CX_PART * sizeof(float));
}

cudaError_t launch_cross(const mog_cache *c, const int32_t *lengths, int n_max, int batch, const RowsIn &r, float *scratch,
                         cudaStream_t s, int polls) {
    CrossArgs a{};
    a.out = static_cast<uint16_t *>(r.qo), a.ob = r.os[0], a.ot = r.os[1], a.oh = r.os[2];
    a.lengths = lengths, a.count = r.count, a.n_max = n_max, a.t_max = r.t_max, a.batch = batch, a.h_kv = r.h_kv;
    a.G = r.h_q / r.h_kv, a.tokens = CX_M / a.G;
    a.bt = c->block_table, a.pshift = c->block_table ? log2_exact(c->page_rows) : 0, a.pps = c->pages_per_seq;
    a.n_pages = c->n_pages;
    a.scale2 = (float)(1.4426950408889634 / sqrt((double)MOG_D));
    // as many polls as the other waits (some seconds), and 16 for the 1.5 us of each key tile that an item may have
    a.polls = polls >= 0 ? polls : (1 << 20) + 16 * (int)ceil_div64(n_max, CX_KEYS);
    const bool paged = c->block_table != nullptr;
    // a stride of 0 (one memory for all): a dim of one entry
    const int64_t h = !paged && c->stride_h == 0 ? 1 : r.h_kv, b = paged ? c->n_pages : c->stride_b == 0 ? 1 : batch;
    const int64_t qb = r.qs[0] == 0 ? 1 : batch;
    a.hmul = h > 1, a.bmul = b > 1, a.qmul = qb > 1;
    CUtensorMap qm, km, vm;
    const int64_t dims[4] = {MOG_D, paged ? c->page_rows : c->n_cap, h, b}, st[4] = {1, c->stride_n, c->stride_h, c->stride_b};
    const int box[4] = {64, paged ? std::min(CX_KEYS, c->page_rows) : CX_KEYS, 1, 1};
    const int64_t qdims[5] = {MOG_D, a.G, r.t_max, r.h_kv, qb}, qst[5] = {1, r.qs[2], r.qs[1], a.G * r.qs[2], r.qs[0]};
    const int qbox[5] = {64, a.G, a.tokens, 1, 1};
    if (!row_map(&km, c->k, 4, dims, st, box) || !row_map(&vm, c->v, 4, dims, st, box) || !row_map(&qm, r.q, 5, qdims, qst, qbox))
        return cudaErrorInvalidValue;
    int64_t ctas;
    cross_grid(batch, r.h_kv, a.G, r.t_max, n_max, ctas, a.whole);
    a.out32 = ((uintptr_t)r.qo | (uintptr_t)(2 * a.ob) | (uintptr_t)(2 * a.ot) | (uintptr_t)(2 * a.oh)) % 32 == 0;
    a.fold = reinterpret_cast<int4 *>(scratch), a.part = scratch + 4 * ctas, a.part_rows = cross_part_rows(a.G, r.t_max);
    const auto fn = paged ? k_cross<true> : k_cross<false>;
    cudaError_t e = ensure_smem((const void *)fn, CX_SMEM);
    if (e != cudaSuccess) return e;
    fn<<<(unsigned)ctas, CX_THREADS, CX_SMEM, s>>>(a, qm, km, vm);
    if ((e = cudaGetLastError()) != cudaSuccess || a.whole || ctas == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas - 1, (unsigned)a.part_rows / 16);  // two rows a warp
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_cross_merge, a);
}

}  // namespace mog
