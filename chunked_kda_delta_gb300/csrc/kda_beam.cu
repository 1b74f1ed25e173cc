// kda_beam.cu -- one step of beam search: log-softmax over the vocabulary, the largest
// totals over beams and tokens, in two launches.
//
// Bound by reading the logits once.  beam_scan cuts every row (request, beam) into segments
// of 256 threads x kE values that stay in registers: one load of each value gives the
// segment's maximum and sum of exponentials and its largest k + 1 values.  beam_join, one
// CTA a request, puts the sums together and ranks the candidates.
//
// Selection in one pass: the c-th largest of the threads' own maxima is a lower bound for
// the c-th largest of all values (c threads hold a value at least as large), so only
// values not below it are candidates -- a few more than c for values in no particular order.
// Candidates are 64-bit keys (value, complement of the index), all different: ranking them
// by counting larger keys needs no sort and ties go to the lowest index.  Where more values
// reach the bound than the buffer holds (many equal ones), k + 1 rounds of a block maximum
// give the same keys.
//
// Ranking by totals, not logits: within a row larger logits give totals that are not
// smaller, but rounding can make totals equal whose logits differ, and then the lower index
// wins.  The (k + 1)-th key of a segment bounds what the segment left out; if the next
// smaller logit would still reach the k-th best total, beam_join reads that segment again.
#include <cuda_fp16.h>
#include <math.h>

#include "../../include/kda.h"
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kScanThreads = 256;
constexpr int kJoinThreads = 512;
constexpr int kBuffer = 1024;  // candidate keys of one selection
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;

// Whole number in the order of the float (-0 counts as +0).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
    return ((uint64_t)ordered(x) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xffffffffu - (uint32_t)k; }

// Logits that are not finite count as absent.
__device__ __forceinline__ float usable(float x) { return fabsf(x) < INFINITY ? x : kNegInf; }

template <typename T> struct Logit;
template <> struct Logit<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float from(uint32_t b) { return __uint_as_float(b); }
    static constexpr uint32_t kSign = 0x80000000u;
};
template <> struct Logit<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16(x)); }
    static __device__ __forceinline__ float from(uint32_t b) { return __bfloat162float(__ushort_as_bfloat16((unsigned short)b)); }
    static constexpr uint32_t kSign = 0x8000u;
};
template <> struct Logit<__half> {
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __half_as_ushort(__float2half(x)); }
    static __device__ __forceinline__ float from(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
    static constexpr uint32_t kSign = 0x8000u;
};
// The next smaller value of the logits' type (-inf after the smallest).
template <typename T>
__device__ __forceinline__ float next_below(float x) {
    const uint32_t b = Logit<T>::bits(x);
    if (x == 0.f) return Logit<T>::from(Logit<T>::kSign | 1u);
    return Logit<T>::from(b & Logit<T>::kSign ? b + 1 : b - 1);
}

__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, x, o);
        x = y > x ? y : x;
    }
    return x;
}

template <int kThreads>
struct Select {
    uint64_t top[kThreads];     // the threads' own largest keys
    uint64_t buf[kBuffer];
    uint64_t red[kThreads / 32];
    uint64_t bound;
    int n;
};

// Largest key of the block that is below `under`.
template <int kThreads, typename ForEach>
__device__ uint64_t block_next(Select<kThreads>& s, uint64_t under, ForEach each) {
    uint64_t best = 0;
    each([&](uint64_t k) { best = k < under && k > best ? k : best; });
    best = warp_max(best);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < kThreads / 32; ++w) best = s.red[w] > best ? s.red[w] : best;
    return best;
}

// The c largest keys over all threads, in order, to out(rank, key); missing ones are 0.  `each`
// calls its argument for every key that the thread holds (keys differ, 0 is none).
template <int kThreads, typename ForEach, typename Out>
__device__ void block_select(Select<kThreads>& s, int c, ForEach each, Out out) {
    const int tid = threadIdx.x;
    uint64_t top = 0;
    each([&](uint64_t k) { top = k > top ? k : top; });
    s.top[tid] = top;
    if (tid == 0) {
        s.bound = 1;  // fewer than c threads hold a key: every key is a candidate
        s.n = 0;
    }
    __syncthreads();
    if (top) {
        int larger = 0;
#pragma unroll 8
        for (int i = 0; i < kThreads; ++i) larger += s.top[i] > top;
        if (larger == c - 1) s.bound = top;
    }
    __syncthreads();
    const uint64_t bound = s.bound;
    if (top >= bound)
        each([&](uint64_t k) {
            if (k >= bound) {
                const int at = atomicAdd(&s.n, 1);
                if (at < kBuffer) s.buf[at] = k;
            }
        });
    __syncthreads();
    const int n = s.n;
    if (n <= kBuffer) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = s.buf[i];
            int larger = 0;
            for (int j = 0; j < n; ++j) larger += s.buf[j] > k;
            if (larger < c) out(larger, k);
        }
        for (int r = n + tid; r < c; r += kThreads) out(r, 0);
    } else {
        uint64_t under = ~0ull;
        for (int r = 0; r < c; ++r) {
            const uint64_t k = under ? block_next(s, under, each) : 0;
            if (tid == 0) out(r, k);
            under = k;
        }
    }
    __syncthreads();
}

// One segment of one row.  kE values a thread; 16-byte loads where the address allows, element
// loads at the row's ends and in rows that are not aligned to the element size's multiple.
template <typename T, int kE>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamParams p) {
    constexpr int kVec = 16 / sizeof(T), kN = kE / kVec;
    __shared__ Select<kScanThreads> s;
    __shared__ float red[2][kScanThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int seg = blockIdx.x;
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * 32768;
    if (row >= (int64_t)p.batch * p.beams) return;
    if (p.done && p.done[row]) return;  // beam_join takes its one candidate from the scores
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // Vector i of the row starts at element i * kVec - skew: aligned.
    const int skew = (int)(((uintptr_t)x % 16) / sizeof(T));

    float v[kE];
    auto index = [&](int n, int e) { return (seg * kN * kScanThreads + n * kScanThreads + tid) * kVec + e - skew; };
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int at = index(n, 0);
        if (at >= 0 && at + kVec <= p.vocab) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4*>(x + at));
            const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[n * kVec + e] = usable(Logit<T>::get(t[e]));
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                v[n * kVec + e] = at + e >= 0 && at + e < p.vocab ? usable(Logit<T>::get(x[at + e])) : kNegInf;
        }
    }
    cudaTriggerProgrammaticLaunchCompletion();

    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < kE; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = red[0][0];
#pragma unroll
    for (int w = 1; w < kScanThreads / 32; ++w) m = fmaxf(m, red[0][w]);
    float sum = 0.f;
    if (m > kNegInf) {
#pragma unroll
        for (int i = 0; i < kE; ++i) sum += exp2f((v[i] - m) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0.f;
        for (int w = 0; w < kScanThreads / 32; ++w) sum += red[1][w];
        p.part[row * p.segs + seg] = make_float2(m, sum);
    }
    uint64_t* cand = p.cand + (row * p.segs + seg) * (p.k + 1);
    block_select(
        s, p.k + 1,
        [&](auto f) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (v[n * kVec + e] > kNegInf) f(key_of(v[n * kVec + e], (uint32_t)index(n, e)));
        },
        [&](int r, uint64_t k) { cand[r] = k; });
}

constexpr int kMaxBeams = 64;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamParams p) {
    __shared__ Select<kJoinThreads> s;
    __shared__ uint64_t best[kMaxBeams];
    __shared__ float lse[kMaxBeams], score[kMaxBeams];
    __shared__ bool done[kMaxBeams];
    __shared__ int found;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t b = blockIdx.x, row0 = b * p.beams;
    const int c1 = p.k + 1;

    for (int w = tid; w < p.beams; w += kJoinThreads) {
        score[w] = p.scores[row0 + w];
        done[w] = p.done && p.done[row0 + w];
    }
    cudaGridDependencySynchronize();
    // lse of each beam: the segments' maxima and sums put together, one warp a beam.
    for (int w = warp; w < p.beams; w += kJoinThreads / 32) {
        if (p.done && p.done[row0 + w]) continue;
        const float2* part = p.part + (row0 + w) * p.segs;
        float m = kNegInf, sum = 0.f;
        for (int i = lane; i < p.segs; i += 32) m = fmaxf(m, part[i].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int i = lane; i < p.segs; i += 32)
            if (part[i].x > kNegInf) sum += part[i].y * exp2f((part[i].x - m) * kLog2e);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) lse[w] = m + logf(sum);  // no finite logit: there are no candidates
    }
    __syncthreads();

    const uint32_t lists = (uint32_t)p.beams * p.segs;
    auto total_key = [&](int w, float x, uint32_t t) -> uint64_t {
        const float total = score[w] + (x - lse[w]);
        return total > kNegInf ? key_of(total, (uint32_t)w * p.vocab + t) : 0;
    };
    auto each = [&](auto f) {
        for (uint32_t i = tid; i < lists * c1; i += kJoinThreads) {
            const uint32_t list = i / c1;
            const int w = list / p.segs;
            if (done[w]) continue;
            const uint64_t k = p.cand[row0 * p.segs * c1 + i];
            if (k) f(total_key(w, key_value(k), key_index(k)));
        }
        if (tid < p.beams && done[tid] && score[tid] > kNegInf)
            f(key_of(score[tid], (uint32_t)tid * p.vocab + p.eos));
    };
    block_select(s, p.k, each, [&](int r, uint64_t k) { best[r] = k; });

    // What the segments left out (see the head of this file): any total that would still
    // come before the k-th best is put in its place, largest first.
    uint64_t under = ~0ull;
    for (int round = 0; round < p.k && under; ++round) {
        const uint64_t last = best[p.k - 1];
        uint64_t more = 0;
        for (uint32_t list = 0; list < lists; ++list) {
            const int w = list / p.segs, seg = list - w * p.segs;
            if (done[w]) continue;
            const uint64_t edge = p.cand[(row0 * p.segs + list) * c1 + p.k];
            if (!edge) continue;  // nothing was left out
            const float next = next_below<T>(key_value(edge));
            const uint64_t could = total_key(w, next, 0);
            if ((could | 0xffffffffu) <= last) continue;  // no index can bring it before the last
            if (could == 0) continue;
            const T* x = static_cast<const T*>(p.logits) + (row0 + w) * p.stride;
            const int skew = (int)(((uintptr_t)x % 16) / sizeof(T));
            const int lo = max(0, seg * p.seg_len - skew), hi = min(p.vocab, (seg + 1) * p.seg_len - skew);
            for (int t = lo + tid; t < hi; t += kJoinThreads) {
                const float v = usable(Logit<T>::get(x[t]));
                if (!(v > kNegInf) || key_of(v, (uint32_t)t) >= edge) continue;
                const uint64_t k = total_key(w, v, (uint32_t)t);
                if (k > last && k < under && k > more) more = k;
            }
        }
        more = warp_max(more);
        __syncthreads();
        if (lane == 0) s.red[warp] = more;
        __syncthreads();
        more = 0;
        for (int w = 0; w < kJoinThreads / 32; ++w) more = s.red[w] > more ? s.red[w] : more;
        under = more;
        if (more && tid == 0) {
            int r = p.k - 1;
            for (; r > 0 && best[r - 1] < more; --r) best[r] = best[r - 1];
            best[r] = more;
        }
        __syncthreads();
    }

    for (int r = tid; r < p.k; r += kJoinThreads) {
        const uint64_t k = best[r];
        const int64_t o = b * p.k + r;
        const uint32_t at = key_index(k);
        const int w = k ? at / p.vocab : 0, t = k ? (int)(at - (uint32_t)w * p.vocab) : -1;
        p.new_scores[o] = k ? key_value(k) : kNegInf;
        p.tokens[o] = t;
        p.parents[o] = k ? (int32_t)(row0 + w) : -1;
        if (p.new_done) p.new_done[o] = !k || t == p.eos || done[w];
    }
}

template <typename T, int kE>
cudaError_t launch_both(const BeamParams& p, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.batch * p.beams;
    const dim3 grid(p.segs, (unsigned)(rows < 32768 ? rows : 32768), (unsigned)((rows + 32767) / 32768));
    beam_scan_kernel<T, kE><<<grid, kScanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.batch);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, beam_join_kernel<T>, p);
}

constexpr int kFew = 8, kMany = 32;  // values a thread

template <typename T>
cudaError_t launch_type(const BeamParams& p, cudaStream_t stream) {
    if (p.seg_len == kFew * kScanThreads) return launch_both<T, kFew>(p, stream);
    return launch_both<T, kMany>(p, stream);
}

}  // namespace

// 32 values a thread (four or eight 16-byte loads in flight); 8 where that would leave SMs
// without a CTA.
int beam_seg_len(int64_t rows, int32_t vocab, int sm_count) {
    const int many = kMany * kScanThreads;
    return rows * ((vocab + many - 1) / many) < 2 * sm_count ? kFew * kScanThreads : many;
}

cudaError_t launch_beam(const BeamParams& p, cudaStream_t stream) {
    if (p.batch == 0) return cudaSuccess;
    if (p.dtype == KDA_LOGITS_F32) return launch_type<float>(p, stream);
    if (p.dtype == KDA_LOGITS_BF16) return launch_type<__nv_bfloat16>(p, stream);
    return launch_type<__half>(p, stream);
}

}  // namespace kda
