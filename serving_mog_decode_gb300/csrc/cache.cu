// cache.cu -- decode attentions over a mog_cache: the fold of the split form's partials and
// the launches; and the store that writes a cache.
#include <algorithm>

#include "cache.cuh"

namespace mog {

// Folds the partials of the split form.  HEADS = 1: a CTA's 16 warps share one (unit, head), warp
// w folding partials w, w + 16, ...; HEADS = 8: a warp per (unit, head), for batches of many
// short units, which have a partial or two each (whole step, 256 sequences of 1000 e4m3 tokens, 8 KV heads,
// G = 4: 103 us against 161; 4 sequences of 16000: 35.9 against 33.8).
template <int ROWS, bool DIFF, bool BF16OUT, int HEADS>
__global__ void __launch_bounds__(HEADS == 1 ? 512 : 256) k_cache_merge(CacheArgs a, DiffArgs d, void *out, int splits) {
    constexpr int M = DIFF ? 2 : 1, W = HEADS == 1 ? 16 : 1;  // warps of a head
    __shared__ float4 s_acc[M][W][32];
    __shared__ float2 s_ml[M][W];
    const int lane = threadIdx.x & 31, w = W == 1 ? 0 : threadIdx.x >> 5;
    const int row = HEADS == 1 ? blockIdx.x : blockIdx.x * HEADS + (threadIdx.x >> 5);
    if (row >= a.batch * a.h_kv * a.G) return;
    const int unit = row / a.G, head = row - unit * a.G;
    const int b = unit / a.h_kv, h = unit - b * a.h_kv;
    // the unit's tiles in the list, and with them the CTAs that hold its partials
    int before = 0, all = 0;
#pragma unroll 4
    for (int i = lane; i < a.batch; i += 32) {
        const int nt = seq_tiles<ROWS>(a, i);
        all += nt;
        if (i < b) before += nt;
    }
    before = warp_isum(before), all = warp_isum(all);
    const int nt = seq_tiles<ROWS>(a, b), chunk = (all * a.h_kv + splits - 1) / splits;
    const int first = before * a.h_kv + h * nt;
    const int c0 = nt ? first / chunk : 0, c1 = nt ? (first + nt - 1) / chunk + 1 : 0;
    const float weight = map_weight<DIFF>(d, h * a.G + head);
    pdl_wait();
    const int64_t step = (int64_t)M * a.G * PART_W;  // floats of a slot
    const float *p = a.part + (int64_t)unit * step + (int64_t)head * PART_W;
    Fold f[M];
#pragma unroll
    for (int k = 0; k < M; ++k) f[k].init();
    constexpr int U = (W == 1 ? 4 : 8) / M;  // partials in flight, of every map
    for (int c = c0 + w; c < c1; c += W * U) {
        float2 ml[M][U];
        float4 v[M][U];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int k = 0; k < M; ++k) {
                const bool ok = c + W * i < c1;
                const float *r = p + (c + W * i) * step + (int64_t)k * a.G * PART_W;
                ml[k][i] = ok ? __ldcg(reinterpret_cast<const float2 *>(r)) : make_float2(-INFINITY, 0.f);
                v[k][i] = ok ? __ldcg(reinterpret_cast<const float4 *>(r + PART_ACC) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int k = 0; k < M; ++k) f[k].add(ml[k], v[k]);
    }
    if (W > 1) {
#pragma unroll
        for (int k = 0; k < M; ++k) {
            s_acc[k][w][lane] = f[k].acc;
            if (lane == 0) s_ml[k][w] = make_float2(f[k].m, f[k].l);
        }
        __syncthreads();
        if (w != 0) return;
#pragma unroll
        for (int k = 0; k < M; ++k) {
            float2 ml[W];
            float4 v[W];
#pragma unroll
            for (int i = 0; i < W; ++i) ml[i] = s_ml[k][i], v[i] = s_acc[k][i][lane];
            f[k].init();
            f[k].add(ml, v);
        }
    }
    finish<DIFF, BF16OUT>(f, weight, d, out, row);
}

int cache_splits(int units, int n_max) {
    // one wave of three CTAs per SM, and no more CTAs than tiles (of 64 rows, the smaller kind)
    const int64_t tiles = units * ceil_div64(n_max, 64), slots = 3LL * num_sms();
    return (int)(tiles < slots ? tiles : slots);
}

// CTAs of a cluster per unit, or 0 for the split form with its second kernel.  One launch saves
// the partials' way through L2, a launch and the scratch, but has no more than 8 CTAs for a
// KV head.  It is taken while all clusters fit on the GPU together (two CTAs per SM, three
// stages each) and no CTA has more than 8 tiles of 64 rows, 4 if there is not a CTA for every SM.
// Kernel times, one launch against two: 8 KV heads and G = 4 of e4m3, 1000 tokens 5.1 us against
// 6.4 (12 against 18 with the host's part), 2000 6.2 against 7.0, 4096 8.4 against 8.2 (2 KV heads
// 8.2 against 6.8; differential over bf16 10.9 against 9.4); 32 KV heads, 4096 tokens 10.1
// against 13.3.  Clusters of 16 were slower throughout.
constexpr int CLUSTER_MAX = 8;

int cache_cluster(int units, int n_max) {
    const int64_t tiles = ceil_div64(n_max, 64), sms = num_sms(), slots = CL_PER_SM * sms;
    int cs = 1;
    while (cs < CLUSTER_MAX && cs < tiles && (int64_t)units * cs * 2 <= slots) cs *= 2;
    const int64_t ctas = (int64_t)units * cs, most = ctas >= sms ? 8 : 4;
    return ctas <= slots && tiles <= cs * most ? cs : 0;
}

template <int ROWS, int HEADS>
static cudaError_t launch_merge(cudaStream_t s, bool diff, bool bf_out, const CacheArgs &a, const DiffArgs &d, void *out,
                                int splits) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div64((int64_t)a.batch * a.h_kv * a.G, HEADS));
    cfg.blockDim = dim3(HEADS == 1 ? 512 : 256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (diff) return bf_out ? cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, true, true, HEADS>, a, d, out, splits)
                            : cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, true, false, HEADS>, a, d, out, splits);
    return bf_out ? cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, false, true, HEADS>, a, d, out, splits)
                  : cudaLaunchKernelEx(&cfg, k_cache_merge<ROWS, false, false, HEADS>, a, d, out, splits);
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
                (float)(LOG2E / sqrt(diff ? MOG_D / 2.0 : (double)MOG_D)), cache_cluster(batch * h_kv, n_max)};
    DiffArgs d{};
    if (diff) d = DiffArgs{diff->lam, diff->lam_heads > 1 ? 4 * (MOG_D / 2) : 0, diff->gamma, diff->lambda_init, diff->eps};
    const bool wide = (diff ? 2 : 1) * G > 8;
    const int per_sm = !e4 ? 3 : wide ? Tile<true, true>::PER_SM : Tile<true, false>::PER_SM;
    const int rows = !e4 ? 64 : wide ? Tile<true, true>::ROWS : Tile<true, false>::ROWS;
    const int splits = std::min(cache_splits(batch * h_kv, n_max), per_sm * num_sms());
    while (a.cs > 1 && a.cs / 2 >= ceil_div64(n_max, rows)) a.cs /= 2;  // as many CTAs as tiles do
    const cudaError_t e = e4 ? launch_split8(a, d, out, diff != nullptr, bf_out, wide, splits, s)
                          : bf_out ? pick_split<false, true, true>(a, d, out, wide, splits, s)
                                   : pick_split<false, true, false>(a, d, out, wide, splits, s);
    if (e != cudaSuccess || a.cs) return e;
    // a unit has splits / units partials and one more: a CTA per head from about five
    if (splits > 4 * batch * h_kv)
        return rows == 128 ? launch_merge<128, 1>(s, diff, bf_out, a, d, out, splits)
                           : launch_merge<64, 1>(s, diff, bf_out, a, d, out, splits);
    return rows == 128 ? launch_merge<128, 8>(s, diff, bf_out, a, d, out, splits)
                       : launch_merge<64, 8>(s, diff, bf_out, a, d, out, splits);
}

// ------------------------------------------------------------------------------------
// mog_kv_store: rows of new keys and values to their positions.  A row is the work of four
// lanes, 32 elements each, four 16-byte loads in flight: the kernel is bound by the instructions
// of a row's addresses as much as by HBM, and fewer lanes share them among more elements (24K
// tokens of 8 heads in 16-row pages, 100 MB read, 50 MB written, 22 us of HBM time: 16 lanes 45 us,
// 8 lanes 24, 4 lanes 21.6 with part of the rows in L2, 27.0 without; into bf16 rows, 201 MB: 33 us without, 0.90
// of the copy rate).  Elements stay packed in pairs:
// their magnitudes' maximum and their scaling are bf16x2 instructions, exact both.
// A row's e4m3 scale is the least power of two 2^e (e >= -126) with amax <= 448*2^e, so
// that dividing by it is exact and the only rounding is the one to e4m3.
// ------------------------------------------------------------------------------------
// S: type of the strides, 32 bits where they all fit (the products that make an address are then one
// instruction each: 24.4 us against 26.1 with eight lanes a row).
template <class S>
struct StoreArgs {
    uint8_t *K, *V;
    float *ks, *vs;
    S sb, sh, sn, ssb, ssh, ssn;
    const int *bt;
    int pshift, pps, n_pages, n_cap;
    const int *pos, *count;
    const uint16_t *kn, *vn;
    S nb, nt, nh;  // elements between sequences, tokens and heads of the new rows
    int t_max, h_kv;
};

constexpr int SR_THREADS = 256, SR_LANES = 4, SR_VECS = 16 / SR_LANES;  // 16-byte pieces of a row per lane

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

template <bool E4M3, class S>
__global__ void __launch_bounds__(SR_THREADS) k_kv_store(StoreArgs<S> a) {
    const int b = blockIdx.y, lane = threadIdx.x % SR_LANES;
    const int count = a.count ? min(max(a.count[b], 0), a.t_max) : a.t_max;
    const int per = 2 * a.h_kv, rows = count * per;  // head fastest, then key or value, then token
    const int start = a.pos[b];
    const int step = gridDim.x * (SR_THREADS / SR_LANES), dt = step / per, dr = step - dt * per;
    int i = blockIdx.x * (SR_THREADS / SR_LANES) + threadIdx.x / SR_LANES;
    int t = i / per, r = i - t * per;
    // (whole groups of lanes enter or leave: the shuffles below stay inside one)
    const unsigned group = ((1u << SR_LANES) - 1u) << (threadIdx.x & (32 - SR_LANES));
    for (; i < rows; i += step) {  // (rows and step stay below 2^30)
        const bool val = r >= a.h_kv;
        const int h = val ? r - a.h_kv : r;
        const int pos = (int)((unsigned)start + (unsigned)t);  // (past 2^31: negative, and so left out)
        const uint16_t *src = (val ? a.vn : a.kn) + (int64_t)b * a.nb + (int64_t)t * a.nt + (int64_t)h * a.nh + lane * 8;
        t += dt;
        r += dr;
        if (r >= per) r -= per, ++t;
        if (pos < 0 || pos >= a.n_cap) continue;
        int slab = b, row = pos;
        if (a.bt) {
            slab = a.bt[(int64_t)b * a.pps + (pos >> a.pshift)];
            row = pos & ((1 << a.pshift) - 1);
            if ((unsigned)slab >= (unsigned)a.n_pages) continue;
        }
        uint32_t w[4 * SR_VECS];  // piece k: elements 8*(lane + SR_LANES*k) ..
#pragma unroll
        for (int k = 0; k < SR_VECS; ++k) {
            const uint4 x = ldg_nc16(src + 8 * SR_LANES * k);
            w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
        }
        uint8_t *dst = (val ? a.V : a.K) + (int64_t)slab * a.sb + (int64_t)h * a.sh + (int64_t)row * a.sn;
        if (!E4M3) {
#pragma unroll
            for (int k = 0; k < SR_VECS; ++k)
                *reinterpret_cast<uint4 *>(dst + 16 * (lane + SR_LANES * k)) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            continue;
        }
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4 * SR_VECS; ++k) m = bf2_max(m, w[k] & 0x7fff7fffu);
        float amax = fmaxf(bf_lo(m), bf_hi(m));
        if (amax == INFINITY) {  // the largest finite magnitude instead
            amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4 * SR_VECS; ++k) {
                const float p = fabsf(bf_lo(w[k])), q = fabsf(bf_hi(w[k]));
                amax = fmaxf(amax, fmaxf(p < INFINITY ? p : 0.f, q < INFINITY ? q : 0.f));
            }
        }
#pragma unroll
        for (int o = 1; o < SR_LANES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
        // amax = m * 2^E, 1 <= m < 2: 448 = 1.75 * 2^8
        const int bits = __float_as_int(amax), E = (bits >> 23) - 127;
        int e = E - 8 + ((bits & 0x7fffff) > 0x600000);
        e = amax > 0.f ? max(e, -126) : 0;
        const uint32_t inv = (uint32_t)(127 - e) << 7, inv2 = inv | inv << 16;  // 2^-e twice, -126 <= -e <= 126
        // (a product below bf16's normal range rounds, but e4m3 has only 0 there)
#pragma unroll
        for (int k = 0; k < SR_VECS; ++k) {
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = e4m3_pair(bf2_mul(w[4 * k + j], inv2));
            *reinterpret_cast<uint2 *>(dst + 8 * (lane + SR_LANES * k)) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        }
        if (lane == 0)
            (val ? a.vs : a.ks)[(int64_t)slab * a.ssb + (int64_t)h * a.ssh + (int64_t)row * a.ssn] = pow2f(e);
    }
}

template <class S>
static cudaError_t launch_store(const mog_cache *c, int batch, int h_kv, int t_max, const int32_t *pos,
                                const int32_t *count, const void *kn, const void *vn, int64_t nb, int64_t nt,
                                int64_t nh, cudaStream_t s) {
    const bool e4 = c->type == MOG_CACHE_E4M3;
    const int es = e4 ? 1 : 2;
    const int64_t cap = c->block_table ? (int64_t)c->pages_per_seq * c->page_rows : c->n_cap;
    const StoreArgs<S> a{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale,
                         (S)(c->stride_b * es), (S)(c->stride_h * es), (S)(c->stride_n * es), (S)c->scale_b,
                         (S)c->scale_h, (S)c->scale_n, c->block_table,
                         c->block_table ? log2_exact(c->page_rows) : 0, c->pages_per_seq, c->n_pages,
                         (int)(cap < INT32_MAX ? cap : INT32_MAX), pos, count, static_cast<const uint16_t *>(kn),
                         static_cast<const uint16_t *>(vn), (S)nb, (S)nt, (S)nh, t_max, h_kv};
    const int64_t rows = (int64_t)t_max * 2 * h_kv, per = SR_THREADS / SR_LANES;
    // up to 16 CTAs per SM; fewer rows: one per group of lanes
    const int64_t most = ceil_div64(16LL * num_sms(), batch);
    const int64_t want = ceil_div64(rows, per);
    const dim3 grid((unsigned)(want < most ? want : most), batch);
    if (e4) k_kv_store<true><<<grid, SR_THREADS, 0, s>>>(a);
    else k_kv_store<false><<<grid, SR_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_store(const mog_cache *c, int batch, int h_kv, int t_max, const int32_t *pos,
                            const int32_t *count, const void *kn, const void *vn, int64_t nb, int64_t nt,
                            int64_t nh, cudaStream_t s) {
    bool small = true;
    for (int64_t x : {2 * c->stride_b, 2 * c->stride_h, 2 * c->stride_n, c->scale_b, c->scale_h, c->scale_n, nb, nt, nh})
        small = small && x >= INT32_MIN && x <= INT32_MAX;
    return small ? launch_store<int>(c, batch, h_kv, t_max, pos, count, kn, vn, nb, nt, nh, s)
                 : launch_store<int64_t>(c, batch, h_kv, t_max, pos, count, kn, vn, nb, nt, nh, s);
}

}  // namespace mog
