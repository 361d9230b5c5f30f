// gdn_pages.cu -- the page pool of the attention layers' cache, for sm_103a: pages reserved,
// shared by forks, copied and released, all on the device.  C ABI: include/gdnattn.h.
//
// Each bookkeeping call is one CTA, or one thread-block cluster of eight where it may touch many
// pages' entries (a cluster's barriers cost about a microsecond more per call).  Every CTA
// makes the same plan (what each row needs, prefix sums over the rows), the pages' entries are
// spread over the cluster's threads, and the per-row words that the plan was read from
// (lengths, owned pages, the free count) are written by one CTA after a barrier.  Results do
// not depend on the order in which threads run.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_common.h"

namespace gdn {
namespace {

constexpr int kThreads = 512, kMaxRows = GDN_PAGES_MAX_ROWS;
constexpr int kManyEntries = 4096;              // entries from which on a cluster is worth its barriers

struct PoolArgs {
    int32_t *table, *seq_len, *n_owned, *ref, *free_list, *free_count, *status;
    int n_slot, max_pages, n_page, page_shift;
};

template <int C> __device__ __forceinline__ void cluster_sync() {
    if constexpr (C == 1) __syncthreads();
    else {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}
template <int C> __device__ __forceinline__ int cluster_rank() {
    if constexpr (C == 1) return 0;
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}
// The word at `p` in the shared memory of CTA `rank` of this cluster.
__device__ __forceinline__ int ld_cluster(const int *p, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Inclusive sum over the CTA's threads; every thread also gets the total.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();                                              // the sums of an earlier call have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int s = warp_sums[w];
        if (w < warp) before += s;
        total += s;
    }
    return x + before;
}

// Row of entry e: the last i with excl[i] <= e (excl ascending, excl[0] = 0).
__device__ __forceinline__ int row_of(const int *excl, int n, int e) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (excl[mid] <= e) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The page that entry k of a call takes from the end of the free list, or -1.
__device__ __forceinline__ int take_page(const PoolArgs &a, int free, int k) {
    const int id = a.free_list[free - 1 - k];
    if (id >= 0 && id < a.n_page) return id;
    atomicOr(a.status, GDN_STATUS_BAD_PAGE);
    return -1;
}

__device__ __forceinline__ int checked_free(const PoolArgs &a) {
    const int f = *a.free_count;
    return f < 0 ? 0 : f > a.n_page ? a.n_page : f;
}

template <int C> __global__ void __launch_bounds__(kThreads) __cluster_dims__(C, 1, 1)
reserve_kernel(const PoolArgs a, int n, const int32_t *slots, int extra)
{
    __shared__ int excl[kMaxRows], sums[kThreads / 32];
    const int tid = threadIdx.x, rank = cluster_rank<C>();
    pdl_wait();
    pdl_release();
    const int free = checked_free(a);
    int total = 0, bad = 0;                                       // total: needs of the rows so far
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        int need = 0;
        if (i < n) {
            const int slot = slots[i];
            if (slot < 0 || slot >= a.n_slot) bad |= GDN_STATUS_BAD_SLOT;
            else {
                const int len = a.seq_len[slot], own = a.n_owned[slot];
                const int room = a.max_pages << a.page_shift;
                if (len < 0 || len > room || own < 0 || own > a.max_pages) bad |= GDN_STATUS_BAD_LEN;
                else {
                    const long long want = (static_cast<long long>(len) + extra + (1 << a.page_shift) - 1) >> a.page_shift;
                    if (want > a.max_pages) bad |= GDN_STATUS_NO_ROOM;
                    else need = want > own ? static_cast<int>(want) - own : 0;
                }
            }
        }
        int sum;
        const int incl = block_scan(need, sums, sum);
        if (i < n) excl[i] = total + incl - need;
        total += sum;
        if (total > free) total = free + 1;                       // no overflow; all later rows fail
        if (i < n && excl[i] > free) excl[i] = free + 1;
    }
    __syncthreads();
    // the entries taken: those of the rows that fit whole
    const bool all = total <= free;
    int given = total;
    if (!all) {
        bad |= GDN_STATUS_NO_PAGES;
        given = 0;
        int lo = 0, hi = n - 1;                                   // the last row that starts within the list
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (excl[mid] <= free) lo = mid;
            else hi = mid - 1;
        }
        given = excl[lo];                                         // that row did not fit
    }
    for (int e = rank * kThreads + tid; e < given; e += C * kThreads) {
        const int i = row_of(excl, n, e), slot = slots[i], own = a.n_owned[slot];
        const int id = take_page(a, free, e);
        a.table[static_cast<size_t>(slot) * a.max_pages + own + (e - excl[i])] = id;
        if (id >= 0) a.ref[id] = 1;
    }
    cluster_sync<C>();
    if (rank == 0) {
        for (int i = tid; i < n; i += kThreads) {
            const int next = i + 1 < n ? excl[i + 1] : total;
            if (next > excl[i] && next <= given) a.n_owned[slots[i]] += next - excl[i];
        }
        if (tid == 0) *a.free_count = free - given;
        if (bad) atomicOr(a.status, bad);
    }
}

template <int C> __global__ void __launch_bounds__(kThreads) __cluster_dims__(C, 1, 1)
fork_kernel(const PoolArgs a, int n, const int32_t *src, const int32_t *dst, int32_t *copies)
{
    // of each row: full pages shared before it, and the page it takes (-1: none, -2: skipped)
    __shared__ int excl[kMaxRows], taken[kMaxRows], sums[kThreads / 32];
    const int tid = threadIdx.x, rank = cluster_rank<C>(), page = 1 << a.page_shift;
    pdl_wait();
    pdl_release();
    const int free = checked_free(a);
    int tails = 0, shared = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        int tail = 0, full = 0;
        bool ok = false;
        if (i < n) {
            const int s = src[i], t = dst[i];
            if (s < 0 || s >= a.n_slot || t < 0 || t >= a.n_slot || a.n_owned[t] != 0) bad |= GDN_STATUS_BAD_SLOT;
            else {
                const int len = a.seq_len[s], own = a.n_owned[s];
                if (len < 0 || own < 0 || own > a.max_pages || len > (own << a.page_shift)) bad |= GDN_STATUS_BAD_LEN;
                else {
                    ok = true;
                    full = len >> a.page_shift;
                    tail = len & (page - 1) ? 1 : 0;
                }
            }
        }
        int sum;
        const int at = tails + block_scan(tail, sums, sum) - tail;
        if (tail && at >= free) {
            bad |= GDN_STATUS_NO_PAGES;
            ok = false;
            full = 0;
        }
        tails += sum;
        const int before = shared + block_scan(full, sums, sum) - full;
        shared += sum;
        if (i < n) {
            excl[i] = before;
            taken[i] = !ok ? -2 : tail ? at : -1;
        }
    }
    __syncthreads();
    for (int e = rank * kThreads + tid; e < shared; e += C * kThreads) {
        const int i = row_of(excl, n, e), c = e - excl[i];
        const int id = a.table[static_cast<size_t>(src[i]) * a.max_pages + c];
        a.table[static_cast<size_t>(dst[i]) * a.max_pages + c] = id;
        if (id >= 0 && id < a.n_page) atomicAdd(&a.ref[id], 1);
        else atomicOr(a.status, GDN_STATUS_BAD_PAGE);
    }
    for (int i = rank * kThreads + tid; i < n; i += C * kThreads) {
        int from = -1, to = -1;
        if (taken[i] >= 0) {
            const int full = a.seq_len[src[i]] >> a.page_shift;
            from = a.table[static_cast<size_t>(src[i]) * a.max_pages + full];
            to = take_page(a, free, taken[i]);
            a.table[static_cast<size_t>(dst[i]) * a.max_pages + full] = to;
            if (to >= 0) a.ref[to] = 1;
        }
        copies[2 * i] = from;
        copies[2 * i + 1] = to;
    }
    cluster_sync<C>();
    if (rank == 0) {
        for (int i = tid; i < n; i += kThreads) {
            if (taken[i] == -2) continue;
            const int len = a.seq_len[src[i]];
            a.seq_len[dst[i]] = len;
            a.n_owned[dst[i]] = (len >> a.page_shift) + (taken[i] >= 0 ? 1 : 0);
        }
        if (tid == 0) *a.free_count = free - min(tails, free);
    }
    if (rank == 0 && bad) atomicOr(a.status, bad);
}

// A page's count while it is being released: positive (still held), 0 (nobody claims it
// yet), kClaim - e (claimed by entry e; the largest entry wins), or a small negative (released
// more often than shared).
constexpr int kClaim = -(1 << 30);

template <int C> __global__ void __launch_bounds__(kThreads) __cluster_dims__(C, 1, 1)
release_kernel(const PoolArgs a, int n, const int32_t *slots)
{
    __shared__ int excl[kMaxRows], sums[kThreads / 32], wins;
    const int tid = threadIdx.x, rank = cluster_rank<C>();
    pdl_wait();
    pdl_release();
    const int free = checked_free(a);
    int total = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        int own = 0;
        if (i < n) {
            const int slot = slots[i];
            if (slot < 0 || slot >= a.n_slot) bad |= GDN_STATUS_BAD_SLOT;
            else {
                own = a.n_owned[slot];
                if (own < 0 || own > a.max_pages) bad |= GDN_STATUS_BAD_LEN, own = 0;
            }
        }
        int sum;
        const int incl = block_scan(own, sums, sum);
        if (i < n) excl[i] = total + incl - own;
        total += sum;
    }
    __syncthreads();
    // this CTA's entries, in order
    const int e0 = static_cast<int>(static_cast<long long>(total) * rank / C);
    const int e1 = static_cast<int>(static_cast<long long>(total) * (rank + 1) / C);
    auto page_at = [&](int e) {
        const int i = row_of(excl, n, e);
        return a.table[static_cast<size_t>(slots[i]) * a.max_pages + (e - excl[i])];
    };
    for (int e = e0 + tid; e < e1; e += kThreads) {
        const int id = page_at(e);
        if (id >= 0 && id < a.n_page) atomicSub(&a.ref[id], 1);
        else bad |= GDN_STATUS_BAD_PAGE;
    }
    cluster_sync<C>();
    for (int e = e0 + tid; e < e1; e += kThreads) {
        const int id = page_at(e);
        if (id < 0 || id >= a.n_page) continue;
        const int r = *const_cast<volatile int32_t *>(&a.ref[id]);
        if (r == 0 || r <= kClaim) atomicMin(&a.ref[id], kClaim - e);
    }
    cluster_sync<C>();
    int mine = 0;
    for (int e = e0 + tid; e < e1; e += kThreads) {
        const int id = page_at(e);
        if (id >= 0 && id < a.n_page && *const_cast<volatile int32_t *>(&a.ref[id]) == kClaim - e) ++mine;
    }
    int cta;
    block_scan(mine, sums, cta);
    if (tid == 0) wins = cta;
    cluster_sync<C>();
    int at = free, all = 0;
    for (int r = 0; r < C; ++r) {
        const int w = C == 1 ? wins : ld_cluster(&wins, r);
        if (r < rank) at += w;
        all += w;
    }
    for (int b0 = e0; b0 < e1; b0 += kThreads) {
        const int e = b0 + tid;
        int id = -1;
        bool win = false;
        if (e < e1) {
            id = page_at(e);
            if (id >= 0 && id < a.n_page) {
                const int r = *const_cast<volatile int32_t *>(&a.ref[id]);
                win = r == kClaim - e;
                if (r < 0 && r > kClaim) {                        // released too often
                    bad |= GDN_STATUS_BAD_PAGE;
                    a.ref[id] = 0;
                }
            }
        }
        int sum;
        const int incl = block_scan(win ? 1 : 0, sums, sum);
        if (win) {
            const int p = at + incl - 1;
            if (p < a.n_page) a.free_list[p] = id;
            else bad |= GDN_STATUS_BAD_PAGE;
            a.ref[id] = 0;
        }
        at += sum;
    }
    if (bad) atomicOr(a.status, bad);
    cluster_sync<C>();                                            // also: every read of `wins` is done
    if (rank == 0) {
        for (int i = tid; i < n; i += kThreads) {
            const int next = i + 1 < n ? excl[i + 1] : total;
            const int slot = slots[i];
            if (slot >= 0 && slot < a.n_slot && (next > excl[i] || a.n_owned[slot] == 0)) {
                a.seq_len[slot] = 0;
                a.n_owned[slot] = 0;
            }
        }
        if (tid == 0) *a.free_count = min(free + all, a.n_page);
    }
}

// One CTA per (pair, layer, k or v): a page of one layer is contiguous.
__global__ void __launch_bounds__(256) copy_pages_kernel(void *k, void *v, const int32_t *copies, int n_page,
                                                         int page_vecs, int32_t *status)
{
    pdl_wait();
    pdl_release();
    const int from = copies[2 * blockIdx.x], to = copies[2 * blockIdx.x + 1];
    if (from == -1 && to == -1) return;
    if (from < 0 || from >= n_page || to < 0 || to >= n_page) {
        if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(status, GDN_STATUS_BAD_PAGE);
        return;
    }
    uint4 *base = static_cast<uint4 *>(blockIdx.y & 1 ? v : k) + static_cast<size_t>(blockIdx.y >> 1) * n_page * page_vecs;
    const uint4 *src = base + static_cast<size_t>(from) * page_vecs;
    uint4 *dst = base + static_cast<size_t>(to) * page_vecs;
    // eight vectors in flight per thread (one: 0.73 of the bandwidth)
    int i = threadIdx.x;
    for (; i + 7 * 256 < page_vecs; i += 8 * 256) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __ldcs(src + i + j * 256);
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[i + j * 256] = x[j];
    }
    for (; i < page_vecs; i += 256) dst[i] = src[i];
}

int check_pool(const gdn_page_cache *c, int n) {
    if (const int rc = check_cache(c)) return rc;
    return n < 0 || n > kMaxRows ? GDN_ERR_DIMS : GDN_OK;
}
bool many(int rows, int pages) { return static_cast<long long>(rows) * pages > kManyEntries; }
bool has_pool(const gdn_page_cache *c) {
    return c->block_table && c->seq_len && c->n_owned && c->ref && c->free_list && c->free_count;
}
PoolArgs pool_args(const gdn_page_cache *c, int32_t *status) {
    return PoolArgs{c->block_table, c->seq_len, c->n_owned, c->ref, c->free_list, c->free_count, status,
                    c->n_slot, c->max_pages, c->n_page, page_shift(c->page)};
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_pages_reserve(const gdn_page_cache *c, int32_t n, const int32_t *slots, int32_t extra, int32_t *status,
                      cudaStream_t stream)
{
    if (const int rc = check_pool(c, n)) return rc;
    if (extra < 0) return GDN_ERR_DIMS;
    if (n == 0) return GDN_OK;
    if (!has_pool(c) || !slots || !status) return GDN_ERR_NULL;
    const int pages = std::min(c->max_pages, extra / c->page + 2);                          // most that a row takes
    const cudaError_t err = many(n, pages)
        ? launch_pdl(reserve_kernel<8>, dim3(8), dim3(kThreads), 0, stream, pool_args(c, status), n, slots, extra)
        : launch_pdl(reserve_kernel<1>, dim3(1), dim3(kThreads), 0, stream, pool_args(c, status), n, slots, extra);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_pages_fork(const gdn_page_cache *c, int32_t n, const int32_t *src, const int32_t *dst, int32_t *copies,
                   int32_t *status, cudaStream_t stream)
{
    if (const int rc = check_pool(c, n)) return rc;
    if (n == 0) return GDN_OK;
    if (!has_pool(c) || !src || !dst || !copies || !status) return GDN_ERR_NULL;
    const cudaError_t err = many(n, c->max_pages)
        ? launch_pdl(fork_kernel<8>, dim3(8), dim3(kThreads), 0, stream, pool_args(c, status), n, src, dst, copies)
        : launch_pdl(fork_kernel<1>, dim3(1), dim3(kThreads), 0, stream, pool_args(c, status), n, src, dst, copies);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_pages_copy(const gdn_page_cache *c, int32_t n, const int32_t *copies, int32_t *status, cudaStream_t stream)
{
    if (const int rc = check_pool(c, n)) return rc;
    if (n == 0) return GDN_OK;
    if (!c->k || !c->v || !copies || !status) return GDN_ERR_NULL;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return GDN_ERR_DIMS;
    const int vecs = c->Hkv * c->page * (c->d * elem_size(c->dtype) / 16);
    return launch_pdl(copy_pages_kernel, dim3(n, 2 * c->n_layer), dim3(256), 0, stream, c->k, c->v, copies, c->n_page,
                      vecs, status) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int gdn_pages_release(const gdn_page_cache *c, int32_t n, const int32_t *slots, int32_t *status, cudaStream_t stream)
{
    if (const int rc = check_pool(c, n)) return rc;
    if (n == 0) return GDN_OK;
    if (!has_pool(c) || !slots || !status) return GDN_ERR_NULL;
    const cudaError_t err = many(n, c->max_pages)
        ? launch_pdl(release_kernel<8>, dim3(8), dim3(kThreads), 0, stream, pool_args(c, status), n, slots)
        : launch_pdl(release_kernel<1>, dim3(1), dim3(kThreads), 0, stream, pool_args(c, status), n, slots);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
