// kda_pages.cu -- page operations: alloc, free, fork, compact (one planning launch each) and
// the copy of page contents.
//
// Planning is whole-number work on the tables (rows x width entries) and the reference counts
// (pages): a few passes with a prefix sum between them, bound by the latency of dependent
// memory accesses, not by bytes (0.5 MB for the largest tables that occur).  One cluster of
// 8 CTAs runs all passes in one launch, separated by cluster barriers; up to 4096 entries and
// pages one CTA does.  The counts and lists live in the CTAs' shared memory, each CTA holding
// a contiguous power-of-two range of the pages, and are reached by the others through
// distributed shared memory (19.8 us for 16384 entries and 2288 pages with them in global
// memory and a fence at each barrier).  Pools of more than 131072 pages keep them in global
// memory.  Free pages are handed out lowest first to entries in row-major order, from prefix
// sums over contiguous ranges, so the result does not depend on the order in which CTAs or
// atomics run (the atomics add whole numbers and take minima).  A fork of 128 rows of a cache takes
// 14.3 us with its copies (10 MB); with one CTA up to 16384 entries it was 57.  Alloc and free of
// 128 rows of 128 entries and 16384 pages take 9.0 and 7.6 us, of 64 rows of one entry 3.8 and 4.0.
//
// The copies are bound by HBM: a fork that copies states of 64 KiB (402 MB read and written) takes
// 70 us, 54 of them the copies (0.84 of the copy rate with the plan), compaction of a cache 55 us
// (292 MB, 0.77), a copy of 256 pages of 1 MiB 87 us (0.91).
#include <cooperative_groups.h>
#include <limits.h>

#include "kda_internal.cuh"
#include "kda_ptx.cuh"
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;
constexpr int kPlanOneCta = 4096;  // entries and pages up to which one CTA plans
constexpr int kPlanPages = 16384;  // pages of a CTA's shared memory
constexpr int kKeep = 4;           // entries of a thread that stay in registers

// Barrier over the CTAs of the plan (one cluster); kGlobal: orders global memory between them.
template <bool kGlobal>
__device__ __forceinline__ void plan_sync() {
    if (kGlobal) __threadfence();
    ptx::cluster_sync();
}

template <typename T>
__device__ __forceinline__ T* at_cta(T* p, int cta) {
    return cooperative_groups::this_cluster().map_shared_rank(p, cta);
}

// One whole number for every page: in the shared memory of the CTA that owns the page (a range
// of 2^shift pages), or in global memory.
template <bool kGlobal>
struct PageArray {
    int32_t* p;
    int shift;
    __device__ __forceinline__ int32_t* at(int x) const {
        return kGlobal ? p + x : at_cta(p + (x & ((1 << shift) - 1)), x >> shift);
    }
    __device__ __forceinline__ int32_t get(int x) const { return kGlobal ? __ldcg(p + x) : *at(x); }
    // A page of this CTA's own range.
    __device__ __forceinline__ int32_t& own(int x) const { return kGlobal ? p[x] : p[x & ((1 << shift) - 1)]; }
};

// Counts of all CTAs, written by each to all.
struct Counts {
    int n[2][kPlanCtas];
};
__device__ __forceinline__ void tell(Counts& c, int which, int value, int cta, int ctas) {
    if ((int)threadIdx.x < ctas) at_cta(&c.n[which][cta], threadIdx.x)[0] = value;
}
// Sum before this CTA, and of all.
__device__ __forceinline__ int before(const Counts& c, int which, int cta, int ctas, int& all) {
    int x = 0;
    all = 0;
    for (int i = 0; i < ctas; ++i) {
        if (i < cta) x += c.n[which][i];
        all += c.n[which][i];
    }
    return x;
}
// Number r of the lists that the CTAs hold one after the other.
__device__ __forceinline__ int32_t listed(int32_t* list, const Counts& c, int which, int r) {
    int cta = 0;
    while (r >= c.n[which][cta]) r -= c.n[which][cta++];
    return at_cta(list, cta)[r];
}

// This CTA's contiguous share [lo, hi) of n things.
__device__ __forceinline__ void share(int n, int cta, int ctas, int& lo, int& hi) {
    const int per = (n + ctas - 1) / ctas;
    lo = min(n, cta * per);
    hi = min(n, lo + per);
}

// Exclusive prefix of `flag` over the CTA's threads; total in `total`.  s: 33 ints.
__device__ __forceinline__ int block_rank(bool flag, int* s, int& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned m = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) s[warp] = __popc(m);
    __syncthreads();
    if (warp == 0) {
        const int c = s[lane];
        int x = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        s[lane] = x - c;
        if (lane == 31) s[32] = x;
    }
    __syncthreads();
    const int r = s[warp] + __popc(m & ((1u << lane) - 1));
    total = s[32];
    __syncthreads();
    return r;
}

struct Entry {
    int32_t page;   // the page the new entry comes from, -1 for none
    bool whole;     // shared (fork), or kept
};

// What new entry e comes from.  Fork: the parent's entry; alloc and free: the row's own.
template <int kMode>
__device__ __forceinline__ Entry source_of(const PagePlan& p, int e) {
    const int r = e / p.width, j = e - r * p.width;
    Entry x{-1, true};
    int row = r;
    if constexpr (kMode == kPagesFork) {
        row = p.parents[r];
        if (row < 0) return x;
        if (row >= p.rows) {
            if (j == 0) report(p.status, kStatusBadIndex);
            return x;
        }
        const int full = p.page_tokens > 0 ? p.lens[row] / p.page_tokens : 0;
        x.whole = j < full;
    } else if constexpr (kMode == kPagesFree) {
        if (p.drop[r]) return x;
    }
    x.page = p.tables[(int64_t)row * p.width + j];
    if (x.page >= p.pages) {
        report(p.status, kStatusBadIndex);
        x.page = -1;
    }
    if (x.page < 0) x.page = -1;
    return x;
}

template <int kMode, bool kGlobal>
__global__ void __launch_bounds__(kPlanThreads, 1) page_plan_kernel(const __grid_constant__ PagePlan p, int shift) {
    extern __shared__ int32_t s_pages[];
    __shared__ int s[33];
    __shared__ Counts counts;
    follow_stream();
    const int cta = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x;
    const int entries = p.rows * p.width;
    const PageArray<kGlobal> held{kGlobal ? p.held : s_pages, shift}, first{kGlobal ? p.first : s_pages + (1 << shift), shift};
    int32_t* list = s_pages + (kGlobal ? 0 : 2 << shift);
    int plo, phi, elo, ehi;
    if (kGlobal) {
        share(p.pages, cta, ctas, plo, phi);
    } else {
        plo = min(p.pages, cta << shift);
        phi = min(p.pages, (cta + 1) << shift);
    }
    share(entries, cta, ctas, elo, ehi);

    for (int x = plo + tid; x < phi; x += kPlanThreads) {
        held.own(x) = max(p.refs[x], 0);
        first.own(x) = INT_MAX;
    }
    // The entries of this thread: kept where they fit, else worked out again in each pass.
    const int tiles = (ehi - elo + kPlanThreads - 1) / kPlanThreads;
    Entry kept[kKeep];
    int32_t old[kKeep];
    const bool small = tiles <= kKeep;
    if (small) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int e = elo + i * kPlanThreads + tid;
            kept[i] = e < ehi ? source_of<kMode>(p, e) : Entry{-1, true};
            old[i] = kMode != kPagesAlloc && e < ehi ? p.tables[e] : -1;
        }
    }
    auto for_entries = [&](auto f) {  // f(e, entry, old): all threads of the CTA in step
        if (small) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (i < tiles) f(elo + i * kPlanThreads + tid, kept[i], old[i]);
        } else {
            for (int i = 0; i < tiles; ++i) {
                const int e = elo + i * kPlanThreads + tid;
                f(e, e < ehi ? source_of<kMode>(p, e) : Entry{-1, true}, kMode != kPagesAlloc && e < ehi ? p.tables[e] : -1);
            }
        }
    };
    plan_sync<kGlobal>();

    // References after the step: old entries give theirs up, kept ones take them again; the
    // first private entry of every page is noted.  An entry that keeps its page changes nothing
    // (rows of one prompt: almost all of them).
    if (kMode != kPagesAlloc) {
        for_entries([&](int e, const Entry& x, int32_t was) {
            if (x.whole && x.page == was) return;
            if (was >= 0 && was < p.pages) atomicSub(held.at(was), 1);
            if (x.page < 0) return;
            if (x.whole)
                atomicAdd(held.at(x.page), 1);
            else
                atomicMin(first.at(x.page), e);
        });
        plan_sync<kGlobal>();
    }

    // Counts of free pages and of entries that need one, in this CTA's contiguous shares.
    auto is_free = [&](int x) { return (kGlobal ? __ldcg(p.held + x) : held.own(x)) <= 0 && (kGlobal ? __ldcg(p.first + x) : first.own(x)) == INT_MAX; };
    auto needs = [&](int e, const Entry& x) {
        if (e >= ehi) return false;
        if (kMode == kPagesAlloc) {
            const int r = e / p.width, j = e - r * p.width;
            const int want = p.want[r];
            if (want > p.width && j == 0) report(p.status, kStatusBadIndex);
            return x.page < 0 && j < want;
        }
        if (kMode == kPagesFree || x.page < 0 || x.whole) return false;
        return held.get(x.page) > 0 || first.get(x.page) != e;
    };
    int nfree = 0, nneed = 0;
    for (int b = plo; b < phi; b += kPlanThreads) {
        const int x = b + tid;
        nfree += __syncthreads_count(x < phi && is_free(x));
    }
    for_entries([&](int e, const Entry& x, int32_t) { nneed += __syncthreads_count(needs(e, x)); });
    tell(counts, 0, nfree, cta, ctas);
    tell(counts, 1, nneed, cta, ctas);
    plan_sync<kGlobal>();
    int free_all, need_all;
    int free_at = before(counts, 0, cta, ctas, free_all), need_at = before(counts, 1, cta, ctas, need_all);
    const int given = min(free_all, need_all);
    // The list of free pages, and the reference counts; the first `given` free pages go out.
    int mine = 0;
    for (int b = plo; b < phi; b += kPlanThreads) {
        const int x = b + tid;
        const bool f = x < phi && is_free(x);
        int total;
        const int r = mine + block_rank(f, s, total);
        if (f) (kGlobal ? p.list + free_at : list)[r] = x;
        if (x < phi) p.new_refs[x] = f ? (free_at + r < given ? 1 : 0) : max(kGlobal ? __ldcg(p.held + x) : held.own(x), 1);
        mine += total;
    }
    if (cta == 0 && tid == 0) {
        *p.copies = kMode == kPagesFork ? given : 0;
        if (need_all > free_all) report(p.status, kStatusNoFreePage);
    }
    plan_sync<kGlobal>();
    for_entries([&](int e, const Entry& x, int32_t) {
        const bool n = needs(e, x);
        int total;
        const int r = need_at + block_rank(n, s, total);
        need_at += total;
        if (e >= ehi) return;
        int32_t page = x.page;
        if (n) {
            page = r >= given ? -1 : kGlobal ? __ldcg(p.list + r) : listed(list, counts, 0, r);
            if (page >= 0 && kMode == kPagesFork) {
                p.src[r] = x.page;
                p.dst[r] = page;
            }
        }
        p.new_tables[e] = page;
    });
    if (!kGlobal) ptx::cluster_sync();  // shared memory stays until all have read it
}

// Exclusive prefix of a thread's value over the CTA; total in `total`.  s: 33 ints.
__device__ __forceinline__ int block_prefix(int value, int* s, int& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = value;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int c = s[lane];
        int y = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        s[lane] = y - c;
        if (lane == 31) s[32] = y;
    }
    __syncthreads();
    total = s[32];
    return s[warp] + x - value;
}

// With n pages in use and r(x) of them below page x: a free page x < n is hole number x - r(x), a
// page x >= n in use is mover number r(x) - r(n), and mover m goes to hole m.  One prefix sum, over
// the runs of pages that the threads hold, gives all ranks.
template <bool kGlobal>
__global__ void __launch_bounds__(kPlanThreads, 1) page_compact_kernel(const __grid_constant__ PagePlan p, int shift) {
    extern __shared__ int32_t s_pages[];
    __shared__ int s[33], s_below;  // r(n)
    __shared__ Counts counts;
    follow_stream();
    const int cta = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x, mask = (1 << shift) - 1;
    const int entries = p.rows * p.width;
    const PageArray<kGlobal> map{kGlobal ? p.page_map : s_pages, shift}, holes{kGlobal ? p.list : s_pages + (1 << shift), shift};
    int32_t* refs_here = s_pages + (2 << shift);
    int lo, hi;
    if (kGlobal) {
        share(p.pages, cta, ctas, lo, hi);
    } else {
        lo = min(p.pages, cta << shift);
        hi = min(p.pages, (cta + 1) << shift);
        for (int x = lo + tid; x < hi; x += kPlanThreads) refs_here[x & mask] = p.refs[x];
        __syncthreads();
    }
    auto refs_of = [&](int x) { return kGlobal ? p.refs[x] : refs_here[x & mask]; };
    const int run = (hi - lo + kPlanThreads - 1) / kPlanThreads;
    const int x0 = min(hi, lo + tid * run), x1 = min(hi, x0 + run);
    int mine = 0, total, n;
    for (int x = x0; x < x1; ++x) mine += refs_of(x) > 0;
    mine = block_prefix(mine, s, total);
    plan_sync<kGlobal>();  // every CTA runs: shared memory may be written
    tell(counts, 0, total, cta, ctas);
    plan_sync<kGlobal>();
    const int r0 = before(counts, 0, cta, ctas, n) + mine;
    int r = r0;
    for (int x = x0; x < x1; ++x) {
        if (x == n)
            for (int c = 0; c < ctas; ++c) *at_cta(&s_below, c) = r;
        if (refs_of(x) > 0) ++r;
        else if (x < n) *holes.at(x - r) = x;
    }
    if (n == p.pages && tid == 0) s_below = n;
    plan_sync<kGlobal>();
    const int below = s_below;
    r = r0;
    for (int x = x0; x < x1; ++x) {
        const int refs = refs_of(x);
        int to = -1;
        if (refs > 0) {
            to = x;
            if (x >= n) {
                const int m = r - below;
                to = holes.get(m);
                p.src[m] = x;
                p.dst[m] = to;
                p.new_refs[to] = refs;
            }
            ++r;
        }
        if (x >= n || refs > 0) p.new_refs[x] = x < n ? refs : 0;
        if (!kGlobal) map.own(x) = to;
        p.page_map[x] = to;
    }
    if (cta == 0 && tid == 0) {
        *p.copies = n - below;
        *p.num_live = n;
    }
    plan_sync<kGlobal>();
    for (int e = cta * kPlanThreads + tid; e < entries; e += ctas * kPlanThreads) {
        const int32_t x = p.tables[e];
        if (x >= p.pages) report(p.status, kStatusBadIndex);
        p.new_tables[e] = x >= 0 && x < p.pages ? map.get(x) : -1;
    }
    if (!kGlobal) ptx::cluster_sync();
}

// Copies: one chunk (up to kCopyChunk bytes) a CTA and step, HBM-bound, each byte read and
// written once.  A pool's chunks go by the widest type that divides all its addresses.
constexpr int kCopyThreads = 256;

template <typename Vec>
__device__ __forceinline__ void copy_chunk(const char* from_bytes, char* to_bytes, int bytes) {
    constexpr int kUnroll = 8;
    const Vec* from = reinterpret_cast<const Vec*>(from_bytes);
    Vec* to = reinterpret_cast<Vec*>(to_bytes);
    const int m = bytes / (int)sizeof(Vec);
    for (int j = threadIdx.x; j < m; j += kCopyThreads * kUnroll) {
        Vec v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (j + u * kCopyThreads < m) v[u] = from[j + u * kCopyThreads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (j + u * kCopyThreads < m) to[j + u * kCopyThreads] = v[u];
    }
}

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ PoolSet pools,
                                                                 int32_t pages, const int32_t* src,
                                                                 const int32_t* dst, const int32_t* count,
                                                                 int32_t limit, int32_t* status) {
    follow_stream();
    const int64_t n = count ? *count : limit;
    for (int64_t w = blockIdx.x; w < n * pools.chunks; w += gridDim.x) {
        const int64_t i = w / pools.chunks;
        int64_t c = w - i * pools.chunks;
        const int32_t a = src[i], b = dst[i];
        if (a < 0 || b < 0) continue;
        if (a >= pages || b >= pages) {
            if (c == 0 && threadIdx.x == 0) report(status, kStatusBadIndex);
            continue;
        }
        int k = 0;
        while (c >= (int64_t)pools.pool[k].layers * pools.pool[k].chunks) {
            c -= (int64_t)pools.pool[k].layers * pools.pool[k].chunks;
            ++k;
        }
        const PoolSet::One& pool = pools.pool[k];
        const int64_t layer = c / pool.chunks, at = (c - layer * pool.chunks) * kCopyChunk;
        char* base = pool.base + layer * pool.layer_stride + at;
        const char* from = base + a * pool.page_stride;
        char* to = base + b * pool.page_stride;
        const int64_t left = pool.page_bytes - at;
        const int bytes = (int)(left < kCopyChunk ? left : kCopyChunk);
        if (pool.unit == 16)
            copy_chunk<uint4>(from, to, bytes);
        else if (pool.unit == 4)
            copy_chunk<uint32_t>(from, to, bytes);
        else
            copy_chunk<uint8_t>(from, to, bytes);
    }
}

// Launches kernel<kGlobal = false>, or `global` where the pages do not fit in shared memory;
// `arrays`: whole numbers of a page in shared memory.
template <typename K>
cudaError_t launch_plan(K shared, K global, int arrays, const PagePlan& p, cudaStream_t stream) {
    const int64_t entries = (int64_t)p.rows * p.width;
    const int ctas = entries > kPlanOneCta || p.pages > kPlanOneCta ? kPlanCtas : 1;
    int shift = 10;
    while (((int64_t)ctas << shift) < p.pages) ++shift;
    const bool fits = (1 << shift) <= kPlanPages;
    K kernel = fits ? shared : global;
    const size_t smem = fits ? ((size_t)arrays * 4) << shift : 0;
    if (smem > 40 * 1024) {  // the static part counts too
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, arrays * 4 * kPlanPages);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, dim3(ctas), kPlanThreads, smem, stream, ctas, p, shift);
}

template <int kMode>
cudaError_t launch_mode(const PagePlan& p, cudaStream_t stream) {
    return launch_plan(page_plan_kernel<kMode, false>, page_plan_kernel<kMode, true>, 3, p, stream);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlan& p, int mode, cudaStream_t stream) {
    if (mode == kPagesFork) return launch_mode<kPagesFork>(p, stream);
    if (mode == kPagesAlloc) return launch_mode<kPagesAlloc>(p, stream);
    return launch_mode<kPagesFree>(p, stream);
}

cudaError_t launch_page_compact(const PagePlan& p, cudaStream_t stream) {
    return launch_plan(page_compact_kernel<false>, page_compact_kernel<true>, 3, p, stream);
}

cudaError_t launch_page_copy(const PoolSet& pools, int32_t pages, const int32_t* src, const int32_t* dst,
                             const int32_t* count, int32_t limit, int32_t* status, int sm_count,
                             cudaStream_t stream) {
    if (limit <= 0 || pools.chunks == 0) return cudaSuccess;
    const int64_t most = (int64_t)limit * pools.chunks;
    const int grid = (int)(most < sm_count * 4ll ? most : sm_count * 4ll);
    return launch_early(page_copy_kernel, dim3(grid), kCopyThreads, 0, stream, 1, pools, pages, src, dst, count, limit, status);
}

}  // namespace kda
