// kda_pages.cu -- page operations: alloc, free, fork, compact (one planning launch each) and
// the copy of page contents.
//
// Planning is whole-number work on the tables (rows x width entries) and the reference counts
// (pages): a few passes with a prefix sum between them, bound by the latency of dependent
// memory accesses, not by bytes (0.5 MB for the largest tables that occur).  One cluster of
// 8 CTAs runs all passes in one launch, separated by cluster barriers; up to 4096 entries and
// pages one CTA does.  Free pages are handed out lowest first to entries in row-major order,
// from prefix sums over contiguous ranges, so the result does not depend on the order in
// which CTAs or atomics run (the atomics add whole numbers and take minima).
#include <limits.h>

#include "kda_internal.cuh"
#include "kda_ptx.cuh"
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;
constexpr int kPlanOneCta = 4096;  // entries and pages up to which one CTA plans

// Barrier over the CTAs of the plan (one cluster); orders global memory between them.
__device__ __forceinline__ void plan_sync() {
    __threadfence();
    ptx::cluster_sync();
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

template <int kMode>
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlan p) {
    __shared__ int s[33];
    const int cta = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x;
    const int entries = p.rows * p.width;
    const int all = ctas * kPlanThreads, me = cta * kPlanThreads + tid;

    for (int x = me; x < p.pages; x += all) {
        p.held[x] = max(p.refs[x], 0);
        p.first[x] = INT_MAX;
    }
    if (me == 0) *p.copies = 0;
    plan_sync();

    // References after the step: old entries give theirs up, kept ones take them again; the
    // first private entry of every page is noted.
    if (kMode != kPagesAlloc) {
        for (int e = me; e < entries; e += all) {
            const int32_t old = p.tables[e];
            if (old >= 0 && old < p.pages) atomicSub(&p.held[old], 1);
            const Entry x = source_of<kMode>(p, e);
            if (x.page < 0) continue;
            if (x.whole)
                atomicAdd(&p.held[x.page], 1);
            else
                atomicMin(&p.first[x.page], e);
        }
        plan_sync();
    }

    // Counts of free pages and of entries that need one, in this CTA's contiguous shares.
    auto is_free = [&](int x) { return __ldcg(&p.held[x]) <= 0 && __ldcg(&p.first[x]) == INT_MAX; };
    auto needs = [&](int e, Entry& x) {
        x = source_of<kMode>(p, e);
        if (kMode == kPagesAlloc) {
            const int r = e / p.width, j = e - r * p.width;
            const int want = p.want[r];
            if (want > p.width && j == 0) report(p.status, kStatusBadIndex);
            return x.page < 0 && j < want;
        }
        if (kMode == kPagesFree || x.page < 0 || x.whole) return false;
        return __ldcg(&p.held[x.page]) > 0 || __ldcg(&p.first[x.page]) != e;
    };
    int plo, phi, elo, ehi;
    share(p.pages, cta, ctas, plo, phi);
    share(entries, cta, ctas, elo, ehi);
    int nfree = 0, nneed = 0;
    for (int b = plo; b < phi; b += kPlanThreads) {
        const int x = b + tid;
        nfree += __syncthreads_count(x < phi && is_free(x));
    }
    Entry src;
    for (int b = elo; b < ehi; b += kPlanThreads) {
        const int e = b + tid;
        nneed += __syncthreads_count(e < ehi && needs(e, src));
    }
    if (tid == 0) {
        p.counts[cta] = nfree;
        p.counts[8 + cta] = nneed;
    }
    plan_sync();
    int free_at = 0, need_at = 0, free_all = 0, need_all = 0;
    for (int c = 0; c < ctas; ++c) {
        const int a = __ldcg(&p.counts[c]), b = __ldcg(&p.counts[8 + c]);
        if (c < cta) {
            free_at += a;
            need_at += b;
        }
        free_all += a;
        need_all += b;
    }
    // The list of free pages, and the reference counts but for the pages about to be given out.
    for (int b = plo; b < phi; b += kPlanThreads) {
        const int x = b + tid;
        const bool f = x < phi && is_free(x);
        int total;
        const int r = block_rank(f, s, total);
        if (f) p.list[free_at + r] = x;
        if (x < phi) {
            const int h = __ldcg(&p.held[x]);
            p.new_refs[x] = f ? 0 : max(h, 1);
        }
        free_at += total;
    }
    if (me == 0) {
        *p.copies = min(need_all, free_all);
        if (need_all > free_all) report(p.status, kStatusNoFreePage);
    }
    plan_sync();
    for (int b = elo; b < ehi; b += kPlanThreads) {
        const int e = b + tid;
        const bool n = e < ehi && needs(e, src);
        int total;
        const int r = need_at + block_rank(n, s, total);
        if (e < ehi) {
            int32_t page = src.page;
            if (n) {
                page = r < free_all ? __ldcg(&p.list[r]) : -1;
                if (page >= 0) {
                    p.new_refs[page] = 1;
                    if (kMode == kPagesFork) {
                        p.src[r] = src.page;
                        p.dst[r] = page;
                    }
                }
            }
            p.new_tables[e] = page;
        }
        need_at += total;
    }
}

__global__ void __launch_bounds__(kPlanThreads) page_compact_kernel(const PagePlan p) {
    __shared__ int s[33];
    const int cta = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x;
    const int entries = p.rows * p.width;
    const int all = ctas * kPlanThreads, me = cta * kPlanThreads + tid;
    int lo, hi;
    share(p.pages, cta, ctas, lo, hi);
    auto live = [&](int x) { return p.refs[x] > 0; };

    int n = 0;
    for (int b = lo; b < hi; b += kPlanThreads) n += __syncthreads_count(b + tid < hi && live(b + tid));
    if (tid == 0) p.counts[cta] = n;
    plan_sync();
    n = 0;
    for (int c = 0; c < ctas; ++c) n += __ldcg(&p.counts[c]);

    // Free pages below n (holes) and pages in use from n on (movers) are equally many.
    int holes = 0, movers = 0;
    for (int b = lo; b < hi; b += kPlanThreads) {
        const int x = b + tid;
        holes += __syncthreads_count(x < hi && x < n && !live(x));
        movers += __syncthreads_count(x < hi && x >= n && live(x));
    }
    if (tid == 0) {
        p.counts[8 + cta] = holes;
        p.counts[16 + cta] = movers;
    }
    plan_sync();
    int hole_at = 0, mover_at = 0, moved = 0;
    for (int c = 0; c < ctas; ++c) {
        const int a = __ldcg(&p.counts[8 + c]);
        if (c < cta) {
            hole_at += a;
            mover_at += __ldcg(&p.counts[16 + c]);
        }
        moved += a;
    }
    for (int b = lo; b < hi; b += kPlanThreads) {
        const int x = b + tid;
        const bool use = x < hi && live(x), hole = x < hi && x < n && !use, mover = use && x >= n;
        int total;
        const int h = block_rank(hole, s, total);
        if (hole) p.dst[hole_at + h] = x;
        hole_at += total;
        const int m = block_rank(mover, s, total);
        if (mover) p.src[mover_at + m] = x;
        mover_at += total;
        if (x < hi) {
            if (!mover) p.page_map[x] = use ? x : -1;
            if (!hole) p.new_refs[x] = use && !mover ? p.refs[x] : 0;
        }
    }
    if (me == 0) {
        *p.copies = moved;
        *p.num_live = n;
    }
    plan_sync();
    for (int i = me; i < moved; i += all) {
        const int from = __ldcg(&p.src[i]), to = __ldcg(&p.dst[i]);
        p.page_map[from] = to;
        p.new_refs[to] = p.refs[from];
    }
    plan_sync();
    for (int e = me; e < entries; e += all) {
        const int32_t x = p.tables[e];
        if (x >= p.pages) report(p.status, kStatusBadIndex);
        p.new_tables[e] = x >= 0 && x < p.pages ? __ldcg(&p.page_map[x]) : -1;
    }
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

template <typename K>
cudaError_t launch_plan(K kernel, const PagePlan& p, cudaStream_t stream) {
    const int64_t entries = (int64_t)p.rows * p.width;
    const int ctas = entries > kPlanOneCta || p.pages > kPlanOneCta ? kPlanCtas : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlan& p, int mode, cudaStream_t stream) {
    if (mode == kPagesFork) return launch_plan(page_plan_kernel<kPagesFork>, p, stream);
    if (mode == kPagesAlloc) return launch_plan(page_plan_kernel<kPagesAlloc>, p, stream);
    return launch_plan(page_plan_kernel<kPagesFree>, p, stream);
}

cudaError_t launch_page_compact(const PagePlan& p, cudaStream_t stream) {
    return launch_plan(page_compact_kernel, p, stream);
}

cudaError_t launch_page_copy(const PoolSet& pools, int32_t pages, const int32_t* src, const int32_t* dst,
                             const int32_t* count, int32_t limit, int32_t* status, int sm_count,
                             cudaStream_t stream) {
    if (limit <= 0 || pools.chunks == 0) return cudaSuccess;
    const int64_t most = (int64_t)limit * pools.chunks;
    const int grid = (int)(most < sm_count * 4ll ? most : sm_count * 4ll);
    page_copy_kernel<<<grid, kCopyThreads, 0, stream>>>(pools, pages, src, dst, count, limit, status);
    return cudaGetLastError();
}

}  // namespace kda
