// kda_kvcache_shared.cu -- which keys the rows of a group have in common, for attention that goes
// through them once for all of the group.
//
// A group's prefix is the longest run of table entries that are the same in all of its rows with new
// tokens, as far as every one of them sees all of its keys (before its first new token), in whole units of
// kSharedUnit tokens: pages and tiles of every kernel end there.  So the result is the attention's,
// whatever the groups are.  A group's tokens lie one after another and no two groups' tokens meet: what comes after
// counts on that, so with malformed offsets of any row nothing is shared.  A cluster has a group; its CTAs look at the
// offsets of a part of all rows each, its warps compare a row with the first one each.
// Bound by the launch and three dependent loads; the tables are read once (8 groups of 8 rows of 261 pages: 4 us).
#include "kda_kvcache_attention.cuh"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kCluster = 8;

__device__ __forceinline__ int32_t load_cluster(uint32_t at) {
    int32_t x;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ SharedPlan p) {
    const CacheParams& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    __shared__ int s_ref, s_active, s_tokens, s_limit, s_equal;
    if (tid == 0) {
        s_ref = INT_MAX;
        s_active = s_tokens = 0;
        s_limit = s_equal = INT_MAX;
    }
    follow_stream();
    bool bad = tid == 0 && (p.cu_rows[0] != 0 || p.cu_rows[p.groups] != c.rows);
    for (int i = tid; i < p.groups; i += kThreads) {
        const int a = p.cu_rows[i], b = p.cu_rows[i + 1];
        bad |= a < 0 || b < a || b > c.rows;
    }
    if (__syncthreads_or(bad)) {  // nothing is shared
        if (tid == 0 && rank == 0) {
            report(c.status, kStatusBadSeqlens);
            p.group[g] = SharedGroup{0, 0, 0, 0, 0};
        }
        for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < c.rows; r += (int64_t)gridDim.x * kThreads) p.from[r] = 0;
        return;
    }
    if (c.cu) {
        bool malformed = rank == 0 && tid == 0 && (c.cu[0] != 0 || c.cu[c.rows] != c.tokens);
        for (int r = rank * kThreads + tid; r < c.rows; r += kCluster * kThreads) {
            const int a = c.cu[r], b = c.cu[r + 1];
            malformed |= a < 0 || b < a || b > c.tokens;
        }
        if (malformed) {
            s_equal = 0;
            report(c.status, kStatusBadSeqlens);
        }
    }
    const int r0 = p.cu_rows[g], r1 = p.cu_rows[g + 1];
    for (int r = r0 + tid; r < r1; r += kThreads) {
        int64_t begin;
        const int n = row_tokens(c, r, begin);
        if (n == 0) continue;
        atomicMin(&s_ref, r);
        atomicAdd(&s_active, 1);
        atomicAdd(&s_tokens, n);
        atomicMin(&s_limit, max(row_length(c, r) - n, 0));
    }
    __syncthreads();
    const int ref = s_ref;
    const int64_t begin = c.cu ? c.cu[r0] : r0, end = c.cu ? c.cu[r1] : r1;
    const bool shares = s_active >= p.least && s_tokens == end - begin;  // (malformed offsets: s_equal is 0 somewhere)
    const int entries = shares ? s_limit / kSharedUnit * kSharedUnit / c.page_tokens : 0;
    if (entries > 0) {
        const int32_t* first = c.tables + (int64_t)ref * c.width;
        for (int r = r0 + rank * kWarps + warp; r < r1; r += kCluster * kWarps) {
            int64_t unused;
            if (r == ref || row_tokens(c, r, unused) == 0) continue;
            const int32_t* table = c.tables + (int64_t)r * c.width;
            constexpr int kAhead = 8;
            for (int i0 = 0; i0 < min(entries, __shfl_sync(0xffffffffu, *(volatile int*)&s_equal, 0)); i0 += 32 * kAhead) {
                int32_t a[kAhead], b[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int i = i0 + 32 * k + lane;
                    a[k] = i < entries ? __ldg(first + i) : 0;
                    b[k] = i < entries ? __ldg(table + i) : 0;
                }
                int at = INT_MAX;
#pragma unroll
                for (int k = kAhead - 1; k >= 0; --k)
                    if (a[k] != b[k]) at = i0 + 32 * k + lane;
                at = __reduce_min_sync(0xffffffffu, at);
                if (at < INT_MAX) {
                    if (lane == 0) atomicMin(&s_equal, at);
                    break;
                }
            }
        }
    }
    ptx::cluster_sync();
    if (rank == 0) {
        if (tid < kCluster) atomicMin(&s_equal, load_cluster(ptx::mapa(ptx::smem_u32(&s_equal), tid)));
        __syncthreads();
        const int shared = (int)((int64_t)min(entries, s_equal) * c.page_tokens / kSharedUnit * kSharedUnit);
        if (tid == 0) p.group[g] = SharedGroup{begin, shared > 0 ? (int)(end - begin) : 0, shared, shared > 0 ? ref : 0, 0};
        for (int r = r0 + tid; r < r1; r += kThreads) p.from[r] = shared;
    }
    ptx::cluster_sync();
}

}  // namespace

// Whether the prefixes' three kernels can be worth their 55 us, if tables were full and rows had them in
// common but for one row a group.  The kernels for few query rows a row read pages at 8 TB/s (of one
// another's out of L2 too); those of many take an SM `cycles` for 64 keys of 128 query rows, of one row there,
// of a group here.  8 heads, dim 128, shared against not (us): 8 rows of 4196 keys 44 and 29, of 16484 63 and 59,
// of 32868 75 and 94; 8 groups of 4 rows of 4196 keys 71 and 51, of 8292 85 and 82, 16 groups of 16684 192
// and 270; 8 rows with 6 tokens of 8292 keys 75 and 70, 64 of 16684 392 and 625; pieces of 64 tokens gain nothing.
// (State and parts past kMostSharedScratch are the caller's to refuse; a state of 2^27 numbers alone is 512 MB.)
bool sharing_pays(const AttentionParams& p, int cols, int32_t least) {
    const CacheParams& c = p.c;
    const int64_t group = p.q_heads / c.heads;
    if (p.groups >= c.rows || c.rows < least || c.tokens < least || c.tokens * p.q_heads * c.dim > (1 << 27)) return false;
    const double keys = (double)c.width * c.page_tokens * c.heads, cycles = c.dim == 64 ? 900 : 1350;
    if (cols < kBlockRows) return (double)(c.rows - p.groups) * keys * 2 * c.dim / 8e6 >= 55;
    const int64_t each = (c.tokens + c.rows - 1) / c.rows * group;
    const int64_t saved = c.rows * ((each + kBlockRows - 1) / kBlockRows) - (c.tokens * group + kBlockRows - 1) / kBlockRows;
    return (double)saved * keys / 64 * cycles / (1900.0 * p.sm_count) >= 55;
}

cudaError_t launch_shared_plan(const SharedPlan& p, cudaStream_t stream) {
    return launch_early(plan_kernel, dim3((unsigned)p.groups * kCluster), kThreads, 0, stream, kCluster, p);
}

}  // namespace kda
