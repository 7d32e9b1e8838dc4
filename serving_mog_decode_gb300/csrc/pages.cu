// pages.cu -- the pages of a paged KV cache as a resource: sequences share pages, give them
// back, grow into free ones and move together.  All state is on the device (block table,
// lengths, holders per page); no call waits for the GPU, so a decode loop can be captured
// with its page handling.
//
// Invariants, kept by every call: row b of the block table holds ceil(length/page_rows)
// pages and -1 behind them; refs[p] is the number of table entries that are p; a page that
// is partly filled and shared is the last one of every sequence that holds it.
//
// These calls are bound by launch latency and dependent reads on the table's side, by HBM
// where they copy pages (read once, written once).  A growth by one token without copies takes 3.7 us for 8
// sequences of one layer and 5.9 for 64 of 32 layers, whose copy kernel finds nothing to do (8.8 with e4m3
// rows: 128 pools, two copy kernels).  Only the holders of one last page that all grow at
// once are walked quadratically: 1024 of them take 58 us, 4096 take 460.  Metadata of a call is planned by one
// CTA (a page pool has at most a few hundred thousand pages: their holder counts come from
// L2), page bytes are copied by the whole GPU in a second kernel, launched early and
// waiting for the plan (programmatic dependent launch); small growth is one launch.
#include "common.cuh"
#include "internal.h"

namespace mog {

// Work buffer (int32): header, the list of copies (sources, destinations), and n_pages entries:
// the free pages found (grow) or, of a page that moves or is moved to, the number of its copy (compact;
// other entries are what earlier calls left, so that a number counts only if its copy names the page).
constexpr int PW_HEAD = 64;
enum { PW_STATUS = 0, PW_COPIES = 1, PW_LIVE = 2 };

struct PagesArgs {
    int n_pages, page_shift, batch, pps;
    int *table, *lengths, *refs, *work;
    __host__ __device__ int *src() const { return work + PW_HEAD; }
    __host__ __device__ int *dst() const { return src() + (n_pages > batch ? n_pages : batch); }
    __host__ __device__ int *map() const { return dst() + (n_pages > batch ? n_pages : batch); }
};

size_t pages_work_ints(int n_pages, int batch) {
    return PW_HEAD + 2 * (size_t)(n_pages > batch ? n_pages : batch) + (size_t)n_pages;
}

struct PoolArgs {
    int n;
    int64_t chunks;  // copy units of a page in the widest pool
    uint8_t *base[MOG_MAX_POOLS];
    int64_t stride[MOG_MAX_POOLS], bytes[MOG_MAX_POOLS];
};

// ---------------------------------------------------------------------------- assign
// table_new[b] = table_old[src[b]].  Every CTA owns eight table columns (a 32-byte sector of
// each row): it loads them for all sequences into shared memory before it writes any of
// them, so that sequences may take each other's pages in any pattern, in one launch.
// 64 rows go at a time, four of them in flight per thread: 288 rows of 129 pages take 3 us (32
// columns and an integer division per entry: 13 us).
constexpr int AS_THREADS = 512, AS_COLS = 8, AS_STEP = AS_THREADS / AS_COLS;

__global__ void __launch_bounds__(AS_THREADS) k_pages_assign(PagesArgs a, const int *src) {
    extern __shared__ int old[];  // [batch][AS_COLS], then [batch] sources
    int *from = old + a.batch * AS_COLS;
    const int c = threadIdx.x % AS_COLS, r = threadIdx.x / AS_COLS, col = blockIdx.x * AS_COLS + c;
    const bool in = col < a.pps;
#pragma unroll 4
    for (int b = r; b < a.batch; b += AS_STEP)
        if (in) old[b * AS_COLS + c] = a.table[(int64_t)b * a.pps + col];
    for (int b = threadIdx.x; b < a.batch; b += AS_THREADS) {
        const int s = src[b];
        const bool bad = s < -1 || s >= a.batch;
        from[b] = bad ? b : s;  // (a bad source: the sequence stays as it is)
        if (bad && blockIdx.x == 0) atomicOr(a.work + PW_STATUS, PAGES_BAD_INDEX);
    }
    __syncthreads();
#pragma unroll 4
    for (int b = r; b < a.batch; b += AS_STEP) {
        const int s = from[b];
        if (s == b || !in) continue;
        const int was = old[b * AS_COLS + c], now = s < 0 ? -1 : old[s * AS_COLS + c];
        if (was == now) continue;
        a.table[(int64_t)b * a.pps + col] = now;
        if ((unsigned)was < (unsigned)a.n_pages) atomicAdd(a.refs + was, -1);
        if ((unsigned)now < (unsigned)a.n_pages) atomicAdd(a.refs + now, 1);
        if (was >= a.n_pages || was < -1 || now >= a.n_pages || now < -1) atomicOr(a.work + PW_STATUS, PAGES_BAD_INDEX);
    }
    if (blockIdx.x != 0) return;
    __syncthreads();
    for (int b = threadIdx.x; b < a.batch; b += AS_THREADS) old[b] = a.lengths[b];
    __syncthreads();
    for (int b = threadIdx.x; b < a.batch; b += AS_THREADS) {
        const int s = from[b];
        if (s != b) a.lengths[b] = s < 0 ? 0 : old[s];
    }
}

// ------------------------------------------------------------------------- block scans

constexpr int PL_THREADS = 1024;

// Exclusive prefix of v over the CTA's threads in order; `sum` is the total.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int &sum) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the last scan's sums have been read
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    const int y = warp_sums[lane];
    int z = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, z, o);
        if (lane >= o) z += u;
    }
    sum = __shfl_sync(0xffffffffu, z, 31);
    return __shfl_sync(0xffffffffu, z - y, w) + x - v;
}

// Bit i set: refs[p0 + i] is not 0 (bit stays clear behind the pool's end).
constexpr int PL_PER = 16;  // pages per thread and step
__device__ __forceinline__ uint32_t live_bits(const PagesArgs &a, int64_t p0) {
    uint32_t m = 0;
    if (p0 + PL_PER <= a.n_pages && ((uintptr_t)a.refs & 15) == 0) {
#pragma unroll
        for (int i = 0; i < PL_PER / 4; ++i) {
            const int4 v = *reinterpret_cast<const int4 *>(a.refs + p0 + 4 * i);
            m |= (uint32_t)((v.x != 0) | ((v.y != 0) << 1) | ((v.z != 0) << 2) | ((v.w != 0) << 3)) << (4 * i);
        }
    } else {
        for (int i = 0; i < PL_PER; ++i)
            if (p0 + i < a.n_pages && a.refs[p0 + i] != 0) m |= 1u << i;
    }
    return m;
}

// ------------------------------------------------------------------------------ grow
// One CTA plans.  A sequence needs the pages between its old and new length and, where its
// last page is partly filled and still shared when its turn comes, one to replace that page
// by a copy.  The needs are numbered by a prefix sum in the order of the sequences; free
// pages are numbered in ascending order; need i takes free page i.  If there are fewer free
// pages than needs, nothing changes.
__device__ __forceinline__ void grow_plan(const PagesArgs &a, const int *n_new, int *pos, int *granted) {
    extern __shared__ int gsm[];
    int *first = gsm;                 // [batch + 1] first need of a sequence
    int *tail = first + a.batch + 1;  // [batch] its partly filled last page if it grows, else -1
    __shared__ int sums[32], bad;
    const int tid = threadIdx.x, R = 1 << a.page_shift;
    const int64_t cap = (int64_t)a.pps << a.page_shift;
    if (tid == 0) bad = 0;
    __syncthreads();
    for (int b = tid; b < a.batch; b += PL_THREADS) {
        const int len = a.lengths[b], n = n_new[b];
        int t = -1;
        if (len < 0 || len > cap || n < 0) {
            atomicOr(&bad, PAGES_BAD_INDEX);
        } else if (n > 0) {
            if ((int64_t)len + n > cap) atomicOr(&bad, PAGES_FULL);
            if (len & (R - 1)) {
                t = a.table[(int64_t)b * a.pps + (len >> a.page_shift)];
                if ((unsigned)t >= (unsigned)a.n_pages) {
                    atomicOr(&bad, PAGES_BAD_INDEX);
                    t = -1;
                }
            }
        }
        tail[b] = t;
    }
    __syncthreads();
    int base = 0;
    if (bad == 0) {
        for (int b0 = 0; b0 < a.batch; b0 += PL_THREADS) {
            const int b = b0 + tid;
            int need = 0;
            if (b < a.batch) {
                const int len = a.lengths[b], n = n_new[b], t = tail[b];
                if (n > 0)
                    need = (int)((((int64_t)len + n + R - 1) >> a.page_shift) - (((int64_t)len + R - 1) >> a.page_shift));
                if (t >= 0) {
                    int holders = a.refs[t];
                    // earlier sequences that leave the page
                    for (int i = 0; holders > 1 && i < b; ++i) holders -= tail[i] == t;
                    need += holders > 1;
                }
            }
            int sum;
            const int at = block_scan(need, sums, sum);
            if (b < a.batch) first[b] = base + at;
            base += sum;
        }
        if (tid == 0) first[a.batch] = base;
        __syncthreads();
    }
    // the lowest `base` free pages, in order
    int found = 0;
    int *list = a.map();
    for (int64_t p0 = 0; found < base && p0 < a.n_pages; p0 += PL_THREADS * PL_PER) {
        const int64_t p = p0 + (int64_t)tid * PL_PER;
        const int in = (int)min((int64_t)PL_PER, max((int64_t)0, a.n_pages - p));
        uint32_t free = in > 0 ? ~live_bits(a, p) & ((1u << in) - 1u) : 0u;
        int sum;
        int at = found + block_scan(__popc(free), sums, sum);
        for (; free && at < base; free &= free - 1, ++at) list[at] = (int)p + __ffs(free) - 1;
        found += sum;
    }
    __syncthreads();
    const int why = bad ? bad : found < base ? PAGES_FULL : 0;
    if (why) {
        for (int b = tid; b < a.batch; b += PL_THREADS) {
            pos[b] = a.lengths[b];
            granted[b] = 0;
        }
        if (tid == 0) {
            a.work[PW_COPIES] = 0;
            atomicOr(a.work + PW_STATUS, why);
        }
        return;
    }
    if (tid == 0) a.work[PW_COPIES] = 0;
    __syncthreads();
    for (int i = tid; i < base; i += PL_THREADS) {
        int lo = 0, hi = a.batch;  // the last sequence with first[b] <= i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int b = lo, len = a.lengths[b];
        const int pages = (int)(((int64_t)len + R - 1) >> a.page_shift);
        const int fresh = (int)((((int64_t)len + n_new[b] + R - 1) >> a.page_shift) - pages);
        const bool copy = first[b + 1] - first[b] > fresh;  // its first need replaces the last page
        const int k = i - first[b], page = list[i];
        const int slot = pages - (copy ? 1 : 0) + k;
        if (copy && k == 0) {
            const int c = atomicAdd(a.work + PW_COPIES, 1);
            a.src()[c] = tail[b];
            a.dst()[c] = page;
            atomicAdd(a.refs + tail[b], -1);
        }
        a.table[(int64_t)b * a.pps + slot] = page;
        a.refs[page] = 1;
    }
    __syncthreads();
    for (int b = tid; b < a.batch; b += PL_THREADS) {
        const int len = a.lengths[b], n = n_new[b];  // (n_new may be pos or granted of the call before)
        pos[b] = len;
        granted[b] = n;
        a.lengths[b] = len + n;
    }
}

// --------------------------------------------------------------------------- compact
// One CTA plans: the live pages behind the first n_live take, in order, the free places
// among them; every other page stays.  Sources and destinations are disjoint, so the
// copies need no order.
__global__ void __launch_bounds__(PL_THREADS) k_pages_plan(PagesArgs a) {
    __shared__ int sums[32];
    pdl_trigger();
    const int tid = threadIdx.x;
    int live = 0;
    for (int64_t p0 = 0; p0 < a.n_pages; p0 += PL_THREADS * PL_PER) {
        const int64_t p = p0 + (int64_t)tid * PL_PER;
        if (p < a.n_pages) live += __popc(live_bits(a, p));
    }
    int n_live;
    block_scan(live, sums, n_live);
    int holes = 0, movers = 0;
    for (int64_t p0 = 0; p0 < a.n_pages; p0 += PL_THREADS * PL_PER) {
        const int64_t p = p0 + (int64_t)tid * PL_PER;
        uint32_t h = 0, m = 0;
        if (p < a.n_pages) {
            const uint32_t l = live_bits(a, p);
            const int in = (int)min((int64_t)PL_PER, max((int64_t)0, n_live - p));  // pages in front
            const uint32_t front = (1u << in) - 1u;
            h = ~l & front;
            m = l & ~front;
        }
        int sh, sm;
        int ah = holes + block_scan(__popc(h), sums, sh), am = movers + block_scan(__popc(m), sums, sm);
        for (; h; h &= h - 1) a.dst()[ah++] = (int)p + __ffs(h) - 1;
        for (; m; m &= m - 1) a.src()[am++] = (int)p + __ffs(m) - 1;
        holes += sh;
        movers += sm;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += PL_THREADS) {  // holes == movers
        const int from = a.src()[i], to = a.dst()[i];
        a.map()[from] = a.map()[to] = i;
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
    }
    if (tid == 0) {
        a.work[PW_COPIES] = movers;
        a.work[PW_LIVE] = n_live;
    }
}

// ------------------------------------------------------------------------------ copies
// The page copies of a plan, over all pools.  A step of a CTA is CP_THREADS x 8 x 16 bytes, 32 KB:
// 16 sequences' 740 MB of pages moved in 140 us with 16 CTAs per SM; 16 KB steps took 149,
// 8 KB steps 153.
constexpr int CP_THREADS = 256, CP_DEPTH = 8, CP_UNIT = CP_THREADS * CP_DEPTH * 16;

// Steps first, first + stride, ... by CP_THREADS threads, of which this is `tid`.
__device__ __forceinline__ void copy_pages(const PagesArgs &a, const PoolArgs &pl, int n, int64_t first, int64_t stride,
                                           int tid) {
    const int64_t units = (int64_t)n * pl.n * pl.chunks;
    for (int64_t u = first; u < units; u += stride) {
        const int64_t c = u / (pl.n * pl.chunks), r = u - c * (pl.n * pl.chunks);
        const int k = (int)(r / pl.chunks);
        const int64_t off = (r - k * pl.chunks) * CP_UNIT, left = pl.bytes[k] - off;
        const uint8_t *from = pl.base[k] + __ldcg(a.src() + c) * pl.stride[k] + off;
        uint8_t *to = pl.base[k] + __ldcg(a.dst() + c) * pl.stride[k] + off;
        uint4 v[CP_DEPTH];
#pragma unroll
        for (int i = 0; i < CP_DEPTH; ++i) {
            const int o = (i * CP_THREADS + tid) * 16;
            if (o < left) v[i] = __ldcs(reinterpret_cast<const uint4 *>(from + o));
        }
#pragma unroll
        for (int i = 0; i < CP_DEPTH; ++i) {
            const int o = (i * CP_THREADS + tid) * 16;
            if (o < left) __stcs(reinterpret_cast<uint4 *>(to + o), v[i]);
        }
    }
}

// With `moved` the block table follows first.
__global__ void __launch_bounds__(CP_THREADS) k_pages_copy(PagesArgs a, PoolArgs pl, int moved) {
    pdl_trigger();
    pdl_wait();
    const int n = a.work[PW_COPIES];
    if (moved && n > 0) {
        const int64_t live = a.work[PW_LIVE], entries = (int64_t)a.batch * a.pps;
        for (int64_t i = blockIdx.x * (int64_t)CP_THREADS + threadIdx.x; i < entries; i += (int64_t)gridDim.x * CP_THREADS) {
            const int p = a.table[i];
            if (p == -1) continue;
            bool bad = (unsigned)p >= (unsigned)a.n_pages;
            if (!bad) {
                const int c = a.map()[p];
                const bool listed = (unsigned)c < (unsigned)n;
                const int from = listed ? a.src()[c] : -1, to = listed ? a.dst()[c] : -1;
                if (from == p) a.table[i] = to;
                else bad = p == to || p >= live;  // refs had it free: nothing is counted to hold it
            }
            if (bad) atomicOr(a.work + PW_STATUS, PAGES_BAD_INDEX);  // (the entry stays)
        }
    }
    copy_pages(a, pl, n, blockIdx.x, gridDim.x, threadIdx.x);
}

__global__ void __launch_bounds__(PL_THREADS) k_pages_grow(PagesArgs a, const int *n_new, int *pos, int *granted) {
    pdl_trigger();
    grow_plan(a, n_new, pos, granted);
}

// Plan and copies in one launch, where the copies cannot be more than GROW_BYTES: a cluster of
// GROW_CTAS, whose first CTA plans and all of which copy.  It saves the caller a launch: eight
// samples forked and grown, 512 KB copied, take 16.6 us with it and 18.7 without; without copies (the
// usual step) the kernels take the same, with those 512 KB 1.6 us more.
constexpr int GROW_CTAS = 8;
constexpr int64_t GROW_BYTES = 1 << 20;
__global__ void __launch_bounds__(PL_THREADS) __cluster_dims__(GROW_CTAS, 1, 1)
k_pages_grow_copy(PagesArgs a, PoolArgs pl, const int *n_new, int *pos, int *granted) {
    if (blockIdx.x == 0) grow_plan(a, n_new, pos, granted);
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    constexpr int GROUPS = PL_THREADS / CP_THREADS;
    copy_pages(a, pl, __ldcg(a.work + PW_COPIES), blockIdx.x * GROUPS + threadIdx.x / CP_THREADS,
               GROW_CTAS * GROUPS, threadIdx.x % CP_THREADS);
}

static PagesArgs pages_args(const mog_pages *p) {
    return PagesArgs{p->n_pages, log2_exact(p->page_rows), p->batch, p->pages_per_seq, p->block_table, p->lengths,
                     p->refs, static_cast<int *>(p->work)};
}

// The next pools, MOG_MAX_POOLS at most, from k on.
static PoolArgs pool_args(const mog_pages *p, int &k) {
    PoolArgs pl{};
    for (; k < p->n_pools && pl.n < MOG_MAX_POOLS; ++k, ++pl.n) {
        pl.base[pl.n] = static_cast<uint8_t *>(p->pools[k].base);
        pl.stride[pl.n] = p->pools[k].page_stride;
        pl.bytes[pl.n] = p->pools[k].page_bytes;
        const int64_t ch = ceil_div64(pl.bytes[pl.n], CP_UNIT);
        pl.chunks = ch > pl.chunks ? ch : pl.chunks;
    }
    return pl;
}

static cudaError_t launch_copies(const mog_pages *p, const PagesArgs &a, int64_t most, int moved, cudaStream_t s) {
    const int sms = num_sms();
    int k = 0;
    do {
        const PoolArgs pl = pool_args(p, k);
        // no more than the plan may need
        int64_t grid = most * pl.n * pl.chunks;
        if (moved) grid = grid > 32 ? grid : 32;
        grid = grid < 1 ? 1 : grid < 16LL * sms ? grid : 16LL * sms;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(CP_THREADS);
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, k_pages_copy, a, pl, moved);
        if (e != cudaSuccess) return e;
        moved = 0;
    } while (k < p->n_pools);
    return cudaSuccess;
}

cudaError_t launch_pages_assign(const mog_pages *p, const int32_t *src, cudaStream_t s) {
    const PagesArgs a = pages_args(p);
    const size_t smem = (size_t)p->batch * (AS_COLS + 1) * 4;
    const cudaError_t e = ensure_smem((const void *)k_pages_assign, smem);
    if (e != cudaSuccess) return e;
    k_pages_assign<<<(unsigned)ceil_div64(p->pages_per_seq, AS_COLS), AS_THREADS, smem, s>>>(a, src);
    return cudaGetLastError();
}

cudaError_t launch_pages_grow(const mog_pages *p, const int32_t *n_new, int32_t *pos, int32_t *granted, cudaStream_t s) {
    const PagesArgs a = pages_args(p);
    const size_t smem = (2 * (size_t)p->batch + 1) * 4;
    int64_t bytes = 0;  // of every sequence's last page in every pool
    for (int i = 0; i < p->n_pools; ++i) bytes += p->pools[i].page_bytes;
    if (p->n_pools <= MOG_MAX_POOLS && bytes * p->batch <= GROW_BYTES) {
        int k = 0;
        const PoolArgs pl = pool_args(p, k);
        k_pages_grow_copy<<<GROW_CTAS, PL_THREADS, smem, s>>>(a, pl, n_new, pos, granted);
        return cudaGetLastError();
    }
    k_pages_grow<<<1, PL_THREADS, smem, s>>>(a, n_new, pos, granted);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_copies(p, a, p->batch, 0, s);
}

cudaError_t launch_pages_compact(const mog_pages *p, cudaStream_t s) {
    const PagesArgs a = pages_args(p);
    k_pages_plan<<<1, PL_THREADS, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_copies(p, a, p->n_pages / 2 + 1, 1, s);
}

}  // namespace mog
