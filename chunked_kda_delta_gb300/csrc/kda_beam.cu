// kda_beam.cu -- one step of beam search: log-softmax over the vocabulary, the largest
// totals over beams and tokens, in two launches.
//
// Bound by reading the logits once.  beam_scan gives every warp a segment of a row (request,
// beam), which it reads in steps of four 16-byte loads a lane, the next step's loads under way
// while it works on this one.  Warps share nothing, so no barrier holds up the loads.  A lane
// keeps its own running sum of exponentials; the warp keeps the segment's k + 1 largest
// logits as a sorted list spread over its lanes, and only values not below the list's last
// take the path that inserts them (about (k + 1) ln(n) of n values in no particular order).
// The first step's list starts from a bound: the (k + 1)-th largest of the lanes' (or of the
// loads') own maxima is not above the (k + 1)-th largest value.  beam_join, one CTA a request,
// puts the sums together and ranks the candidates.
//
// Candidates are 64-bit keys (value, complement of the index), all different: ranking them
// by counting larger keys needs no sort and ties go to the lowest index.
//
// Sums are relative to 2^c with whole c, so exp2(x log2 e - c) takes one fused multiply-add and
// the reference is exact.  Logits of 1e30 and more (the type's lowest value as a mask) have
// a sum of their own, relative to their maximum; steps with such logits, NaN or
// infinities take a slower path.
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

constexpr int kScanWarps = 4;
constexpr int kJoinThreads = 512, kGroups = 128;
constexpr int kBuffer = 512;  // candidate keys of one selection
constexpr int kLoads = 4;     // 16-byte loads of a lane and step
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHuge = 1e30f;

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
    static __device__ __forceinline__ void unpack(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
    static __device__ __forceinline__ float get(float x) { return x; }
    static constexpr uint32_t kNone = 0xff800000u;  // -inf
    static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float from(uint32_t b) { return __uint_as_float(b); }
    static constexpr uint32_t kSign = 0x80000000u;
};
template <> struct Logit<__nv_bfloat16> {
    static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    }
    static constexpr uint32_t kNone = 0xff80u;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16(x)); }
    static __device__ __forceinline__ float from(uint32_t b) { return __bfloat162float(__ushort_as_bfloat16((unsigned short)b)); }
    static constexpr uint32_t kSign = 0x8000u;
};
template <> struct Logit<__half> {
    static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        v[0] = f.x;
        v[1] = f.y;
    }
    static constexpr uint32_t kNone = 0xfc00u;
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

// 16 bytes of a row from element `at` on; -inf outside [0, vocab).
template <typename T>
__device__ __forceinline__ uint4 load16(const T* x, int at, int vocab) {
    constexpr int kVec = 16 / sizeof(T);
    if (at >= 0 && at + kVec <= vocab) return __ldcs(reinterpret_cast<const uint4*>(x + at));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = at + i >= 0 && at + i < vocab ? reinterpret_cast<const uint32_t*>(x)[at + i] : Logit<T>::kNone;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(x);
            const int a = at + 2 * i;
            const uint32_t lo = a >= 0 && a < vocab ? h[a] : Logit<T>::kNone;
            const uint32_t hi = a + 1 >= 0 && a + 1 < vocab ? h[a + 1] : Logit<T>::kNone;
            w[i] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest keys of a warp, in order: number r of them in lane r % 32, register r / 32.
template <int kRegs>
struct TopList {
    uint64_t key[kRegs];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kRegs; ++i) key[i] = 0;
    }
    // The r-th key, for all lanes.
    __device__ __forceinline__ uint64_t at(int r) const {
        uint64_t k = key[0];
#pragma unroll
        for (int i = 1; i < kRegs; ++i) k = (r >> 5) == i ? key[i] : k;
        return __shfl_sync(0xffffffffu, k, r & 31);
    }
    // Puts k (the same in all lanes) in its place.
    __device__ __forceinline__ void insert(uint64_t k, int lane) {
        uint64_t carry = k;  // what enters register i at its first lane from its place on
        int before = 0;
#pragma unroll
        for (int i = 0; i < kRegs; ++i) before += __popc(__ballot_sync(0xffffffffu, key[i] > k));
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, key[i], 1), last = __shfl_sync(0xffffffffu, key[i], 31);
            const int r = 32 * i + lane;
            if (r > before) key[i] = lane == 0 ? carry : up;
            if (r == before) key[i] = k;
            carry = last;
        }
    }
};

template <typename T, int kRegs>
__global__ void __launch_bounds__(kScanWarps * 32) beam_scan_kernel(const BeamParams p) {
    constexpr int kVec = 16 / sizeof(T);
    cudaTriggerProgrammaticLaunchCompletion();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kScanWarps + (threadIdx.x >> 5);
    const int64_t row = unit / p.segs;
    if (row >= (int64_t)p.batch * p.beams) return;
    if (p.done && p.done[row]) return;  // beam_join takes its one candidate from the scores
    const int seg = (int)(unit - row * p.segs), c1 = p.k + 1;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // Loads are aligned: the row's first lies up to kVec - 1 elements before it.
    const int skew = (int)(((uintptr_t)x % 16) / sizeof(T));
    const int begin = seg * p.seg_len - skew;
    const int end = min(p.vocab, begin + p.seg_len);
    constexpr int kStep = kLoads * 32 * kVec;

    TopList<kRegs> top;
    top.clear();
    uint64_t worst = 1;            // keys below it are not wanted; the list's last once it is full
    float worst_value = kNegInf;
    float c = kNegInf, sum = 0.f;  // sum of 2^(x log2 e - c) of this lane's logits
    float huge = kNegInf, huge_sum = 0.f;

    uint4 next[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) next[i] = load16(x, begin + (i * 32 + lane) * kVec, p.vocab);
    for (int at = begin; at < end; at += kStep) {
        float v[kLoads][kVec];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t w[4] = {next[i].x, next[i].y, next[i].z, next[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) Logit<T>::unpack(w[k], &v[i][k * (kVec / 4)]);
        }
        if (at + kStep < end) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) next[i] = load16(x, at + kStep + (i * 32 + lane) * kVec, p.vocab);
        }
        float most[kLoads];  // of each load
        float part = 0.f;
        auto take = [&]() {
            float m = kNegInf;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                most[i] = v[i][0];
#pragma unroll
                for (int e = 1; e < kVec; ++e) most[i] = fmaxf(most[i], v[i][e]);
                m = fmaxf(m, most[i]);
            }
            return m;
        };
        float m = take();
        float c_new = fmaxf(c, ceilf(m * kLog2e));
        float ref = c_new == kNegInf ? 0.f : c_new;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) part += exp2f(fmaf(v[i][e], kLog2e, -ref));
        if (__any_sync(0xffffffffu, !(m < kHuge) || part != part || (m < -kHuge && m > kNegInf))) {
            // Something is not finite, or huge.
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[i][e] = usable(v[i][e]);
            m = take();
            float rest = kNegInf, high = kNegInf;  // largest of the others, and of the huge ones
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float y = v[i][e];
                    if (fabsf(y) < kHuge) rest = fmaxf(rest, y);
                    else high = fmaxf(high, y);
                }
            c_new = fmaxf(c, ceilf(rest * kLog2e));
            ref = c_new == kNegInf ? 0.f : c_new;
            const float h_new = fmaxf(huge, high);
            if (huge > kNegInf) huge_sum *= exp2f((huge - h_new) * kLog2e);
            huge = h_new;
            part = 0.f;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float y = v[i][e];
                    if (fabsf(y) < kHuge) part += exp2f(fmaf(y, kLog2e, -ref));
                    else if (y > kNegInf) huge_sum += exp2f((y - huge) * kLog2e);
                }
        }
        if (c > kNegInf) sum *= exp2f(c - ref);
        c = c_new;
        sum += part;

        if (at == begin) {
            // A bound for the list's last value from maxima of disjoint parts of this step.
            if (kRegs == 1) {
                int larger = 0;
#pragma unroll 8
                for (int i = 0; i < 32; ++i) {
                    const float y = __shfl_sync(0xffffffffu, m, i);
                    larger += y > m || (y == m && i < lane);
                }
                const unsigned who = __ballot_sync(0xffffffffu, larger == c1 - 1);
                if (who) worst_value = __shfl_sync(0xffffffffu, m, __ffs(who) - 1);
            } else {
                int larger[kLoads] = {};
                for (int i = 0; i < 32; ++i)
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        const float y = __shfl_sync(0xffffffffu, most[j], i);
#pragma unroll
                        for (int k = 0; k < kLoads; ++k) larger[k] += y > most[k] || (y == most[k] && (i < lane || (i == lane && j < k)));
                    }
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const unsigned who = __ballot_sync(0xffffffffu, larger[k] == c1 - 1);
                    if (who) worst_value = __shfl_sync(0xffffffffu, most[k], __ffs(who) - 1);
                }
            }
            if (worst_value > kNegInf) worst = (uint64_t)ordered(worst_value) << 32;
        }
        if (!__any_sync(0xffffffffu, m >= worst_value && m > kNegInf)) continue;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (!__any_sync(0xffffffffu, most[i] >= worst_value)) continue;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const uint64_t k = v[i][e] > kNegInf ? key_of(v[i][e], (uint32_t)(at + (i * 32 + lane) * kVec + e)) : 0;
                unsigned who = __ballot_sync(0xffffffffu, k > worst);
                while (who) {
                    const uint64_t one = __shfl_sync(0xffffffffu, k, __ffs(who) - 1);
                    top.insert(one, lane);
                    const uint64_t last = top.at(c1 - 1);
                    if (last > worst) worst = last;
                    who &= who - 1;
                    who &= __ballot_sync(0xffffffffu, k > worst);
                }
            }
            worst_value = worst >> 32 ? key_value(worst) : kNegInf;
        }
    }

    // The lanes' sums put together.
    float c_all = c, h_all = huge;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        c_all = fmaxf(c_all, __shfl_xor_sync(0xffffffffu, c_all, o));
        h_all = fmaxf(h_all, __shfl_xor_sync(0xffffffffu, h_all, o));
    }
    sum = c > kNegInf ? sum * exp2f(c - c_all) : 0.f;
    huge_sum = huge > kNegInf ? huge_sum * exp2f((huge - h_all) * kLog2e) : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        huge_sum += __shfl_xor_sync(0xffffffffu, huge_sum, o);
    }
    if (lane == 0) p.part[unit] = make_float4(c_all, sum, h_all, huge_sum);
#pragma unroll
    for (int i = 0; i < kRegs; ++i)
        if (32 * i + lane < c1) p.cand[unit * c1 + 32 * i + lane] = top.key[i];
}

struct Select {
    uint64_t top[kGroups];  // largest keys of groups of threads
    uint64_t buf[kBuffer];
    uint64_t red[kJoinThreads / 32];
    uint64_t bound;
    int n;
};

// Largest key of the block.
__device__ __forceinline__ uint64_t block_max(Select& s, uint64_t best) {
    best = warp_max(best);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < kJoinThreads / 32; ++w) best = s.red[w] > best ? s.red[w] : best;
    return best;
}

// The c (<= kGroups) largest keys over all threads, in order, to out[]; missing ones are 0.
// `each` calls its argument for every key that the thread holds (keys differ, 0 is none).
// Where more keys reach the bound than the buffer holds, c rounds of a block maximum do.
template <typename ForEach>
__device__ void block_select(Select& s, int c, ForEach each, uint64_t* out) {
    const int tid = threadIdx.x;
    constexpr int kLanes = kJoinThreads / kGroups;
    uint64_t top = 0;
    each([&](uint64_t k) { top = k > top ? k : top; });
    uint64_t group = top;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, group, o);
        group = y > group ? y : group;
    }
    if (tid % kLanes == 0) s.top[tid / kLanes] = group;
    if (tid == 0) {
        s.bound = 1;  // fewer than c groups hold a key: every key is a candidate
        s.n = 0;
    }
    __syncthreads();
    if (tid < kGroups && s.top[tid]) {
        const uint64_t mine = s.top[tid];
        int larger = 0;
#pragma unroll 16
        for (int i = 0; i < kGroups; ++i) larger += s.top[i] > mine;
        if (larger == c - 1) s.bound = mine;
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
        for (int i = tid; i < n; i += kJoinThreads) {
            const uint64_t k = s.buf[i];
            int larger = 0;
            for (int j = 0; j < n; ++j) larger += s.buf[j] > k;
            if (larger < c) out[larger] = k;
        }
        for (int r = n + tid; r < c; r += kJoinThreads) out[r] = 0;
    } else {
        uint64_t under = ~0ull;
        for (int r = 0; r < c; ++r) {
            uint64_t best = 0;
            each([&](uint64_t k) { best = k < under && k > best ? k : best; });
            best = block_max(s, best);
            if (tid == 0) out[r] = best;
            under = best;
        }
    }
    __syncthreads();
}

constexpr int kMaxBeams = 64;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamParams p) {
    __shared__ Select s;
    __shared__ uint64_t best[kMaxBeams];
    __shared__ int again[kJoinThreads], agains;
    __shared__ float lse[kMaxBeams], score[kMaxBeams];
    __shared__ bool done[kMaxBeams];
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
        const float4* part = p.part + (row0 + w) * p.segs;
        float c = kNegInf, h = kNegInf, sum = 0.f, huge = 0.f;
        for (int i = lane; i < p.segs; i += 32) {
            c = fmaxf(c, part[i].x);
            h = fmaxf(h, part[i].z);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
            h = fmaxf(h, __shfl_xor_sync(0xffffffffu, h, o));
        }
        for (int i = lane; i < p.segs; i += 32) {
            const float4 y = part[i];
            if (y.x > kNegInf) sum += y.y * exp2f(y.x - c);
            if (y.z > kNegInf) huge += y.w * exp2f((y.z - h) * kLog2e);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            huge += __shfl_xor_sync(0xffffffffu, huge, o);
        }
        // Huge logits matter alone, or where they are positive.  With no finite logit at all
        // there are no candidates either.
        if (lane == 0)
            lse[w] = h > 0.f || c == kNegInf ? h + logf(huge) : (float)(((double)c + log2f(sum)) * 0.6931471805599453);
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
    block_select(s, p.k, each, best);

    // What the segments left out (see the head of this file): any total that would still
    // come before the k-th best is put in its place, largest first.
    for (uint32_t list0 = 0; list0 < lists; list0 += kJoinThreads) {
        if (tid == 0) agains = 0;
        __syncthreads();
        if (list0 + tid < lists) {
            const int w = (list0 + tid) / p.segs;
            const uint64_t edge = done[w] ? 0 : p.cand[(row0 * p.segs + list0 + tid) * c1 + p.k];
            if (edge) {  // else nothing was left out
                const uint64_t could = total_key(w, next_below<T>(key_value(edge)), 0);
                // Whatever its index, it may come before the last.
                if (could && (could | 0xffffffffu) > best[p.k - 1]) again[atomicAdd(&agains, 1)] = list0 + tid;
            }
        }
        __syncthreads();
        uint64_t under = ~0ull;
        for (int round = 0; agains && round < p.k && under; ++round) {
            const uint64_t last = best[p.k - 1];
            uint64_t more = 0;
            for (int a = 0; a < agains; ++a) {
                const int list = again[a], w = list / p.segs, seg = list - w * p.segs;
                const uint64_t edge = p.cand[(row0 * p.segs + list) * c1 + p.k];
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
            under = more = block_max(s, more);
            if (more && tid == 0) {
                int r = p.k - 1;
                for (; r > 0 && best[r - 1] < more; --r) best[r] = best[r - 1];
                best[r] = more;
            }
            __syncthreads();
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

template <typename T>
cudaError_t launch_type(const BeamParams& p, cudaStream_t stream) {
    const int64_t warps = (int64_t)p.batch * p.beams * p.segs;
    const dim3 grid((unsigned)((warps + kScanWarps - 1) / kScanWarps));
    if (p.k < 32)
        beam_scan_kernel<T, 1><<<grid, kScanWarps * 32, 0, stream>>>(p);
    else
        beam_scan_kernel<T, 3><<<grid, kScanWarps * 32, 0, stream>>>(p);
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

}  // namespace

// Values of a warp's segment: whole steps, the fewest with which all warps are resident at
// once (five CTAs of four warps an SM by their registers), at most 16.
int beam_seg_len(int64_t rows, int32_t vocab, int elem, int sm_count) {
    const int step = kLoads * 32 * 16 / elem;
    const int64_t steps = (vocab + step - 1) / step;
    int each = 1;
    while (each < 16 && rows * ((steps + each - 1) / each) > 20ll * sm_count) ++each;
    return step * each;
}

cudaError_t launch_beam(const BeamParams& p, cudaStream_t stream) {
    if (p.batch == 0) return cudaSuccess;
    if (p.dtype == KDA_LOGITS_F32) return launch_type<float>(p, stream);
    if (p.dtype == KDA_LOGITS_BF16) return launch_type<__nv_bfloat16>(p, stream);
    return launch_type<__half>(p, stream);
}

}  // namespace kda
