// kda_beam.cu -- one step of beam search: log-softmax over the vocabulary, the largest
// totals over beams and tokens, in two launches.
//
// Bound by reading the logits once.  beam_scan gives every CTA a segment of a row (request,
// beam).  Its warps stream it in steps of four 16-byte loads a lane, the next step's loads
// under way while they work on this one; a lane keeps a running sum of exponentials and
// notes the largest value of each of its steps, nothing else.  Selection comes after the stream:
// the values form 32 groups by lane (128 by lane and load where k + 1 does not fit), and the
// (k + 1)-th largest of the groups' maxima is not above the segment's (k + 1)-th largest value.
// (Groups of neighbouring lanes of one warp are empty in short segments, the last of most
// rows: without a bound all of their values are candidates, too many for the buffer, and the
// rounds that are left then took 40 us for 16 beams of 1326 or 9077 logits instead of 10.)  Only the steps of lanes
// whose noted maximum reaches that bound are read again, a few dozen bytes each and little
// more than k + 1 of them, and their values that reach it are the candidates.  (Keeping sorted
// lists while streaming, with a bound that rises, took 12 us more on 256 rows of 131072: some
// warp always has a value to insert.)  beam_join, one CTA a request, puts the sums together and
// ranks the candidates.  32 x 8 beams of 131072 bf16 logits: 21 us (0.48 of the 67 MB at the copy
// rate), 15 for the stream alone, with or without the exponentials; 4 beams of 32001: 8 us, the
// latency of two launches.
//
// Candidates are 64-bit keys (value, complement of the index), all different: ranking them
// by counting larger keys needs no sort and ties go to the lowest index.
//
// Sums are relative to 2^c with whole c, so exp2(x log2 e - c) takes one fused multiply-add and
// the reference is exact.  c is made from the rounded product, which for |x| below 2^30 is off by up to
// 2^6: terms stay below 2^65.  Logits of 2^30 and more (large numbers and the type's lowest value as
// masks) have a sum of their own, relative to their maximum; steps with such logits, NaN
// or infinities take a slower path.  One of 2^30 and more is at least 64 away from the largest of
// the others: the lower of the two sums does not count.
//
// Ranking by totals, not logits: within a row larger logits give totals that are not
// smaller, but rounding can make totals equal whose logits differ, and then the lower index
// wins.  The (k + 1)-th key of a segment, its edge, bounds what the segment left out: the edge's
// logit at higher indexes, and smaller logits anywhere.  If the edge's logit at the next index, or the
// next smaller logit at any, would come before the k-th best total, beam_join reads that
// segment again.
#include <cuda_fp16.h>
#include <math.h>

#include "../../include/kda.h"
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kScanWarps = 8, kScanThreads = kScanWarps * 32;
constexpr int kJoinThreads = 512, kGroups = 128;
constexpr int kBuffer = 512;  // candidate keys of one selection
constexpr int kLoads = 4;     // 16-byte loads of a lane and step
constexpr int kMaxSteps = 16; // of a warp
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHuge = 0x1p30f;

// 2^x by the hardware's instruction (results below 2^-126 are 0, which sums of a largest
// term near 1 do not notice).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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
    static constexpr int kPer = 1;  // values of a 32-bit word
    static __device__ __forceinline__ void unpack(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
    static __device__ __forceinline__ float get(float x) { return x; }
    // Largest of two words, by values; NaN loses.
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static constexpr uint32_t kNone = 0xff800000u;  // -inf
    static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float from(uint32_t b) { return __uint_as_float(b); }
    static constexpr uint32_t kSign = 0x80000000u;
};
template <> struct Logit<__nv_bfloat16> {
    static constexpr int kPer = 2;
    static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static constexpr uint32_t kNone = 0xff80u;
    static __device__ __forceinline__ uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16(x)); }
    static __device__ __forceinline__ float from(uint32_t b) { return __bfloat162float(__ushort_as_bfloat16((unsigned short)b)); }
    static constexpr uint32_t kSign = 0x8000u;
};
template <> struct Logit<__half> {
    static constexpr int kPer = 2;
    static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        v[0] = f.x;
        v[1] = f.y;
    }
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static constexpr uint32_t kNone = 0xfc00u;
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

// A step's values that are not finite, or huge: sums of the others and of the huge ones.
struct Sums {
    float c, sum;      // sum of 2^(x log2 e - c)
    float huge, huge_sum;  // sum of exp(x - huge) over |x| >= kHuge
};
template <typename T>
__device__ __noinline__ float slow_sums(const T* x, int at, int vocab, Sums& s) {
    uint32_t words[kLoads * 4];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint4 w = load16(x, at + i * 32 * (int)(16 / sizeof(T)), vocab);
        words[4 * i] = w.x; words[4 * i + 1] = w.y; words[4 * i + 2] = w.z; words[4 * i + 3] = w.w;
    }
    float rest = kNegInf, high = kNegInf;
    constexpr int kPer = Logit<T>::kPer;
#pragma unroll
    for (int i = 0; i < kLoads * 4; ++i) {
        float v[kPer];
        Logit<T>::unpack(words[i], v);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float y = usable(v[e]);
            if (fabsf(y) < kHuge) rest = fmaxf(rest, y);
            else high = fmaxf(high, y);
        }
    }
    const float c_new = fmaxf(s.c, ceilf(rest * kLog2e)), h_new = fmaxf(s.huge, high);
    if (s.c > kNegInf) s.sum *= exp2_fast(s.c - c_new);
    if (s.huge > kNegInf) s.huge_sum *= exp2_fast((s.huge - h_new) * kLog2e);
    s.c = c_new;
    s.huge = h_new;
#pragma unroll
    for (int i = 0; i < kLoads * 4; ++i) {
        float v[kPer];
        Logit<T>::unpack(words[i], v);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float y = usable(v[e]);
            if (fabsf(y) < kHuge) s.sum += exp2_fast(fmaf(y, kLog2e, -c_new));
            else if (y > kNegInf) s.huge_sum += exp2_fast((y - h_new) * kLog2e);
        }
    }
    return fmaxf(rest, high);
}

// kBound groups of lanes give the bound; kBound >= k + 1.
template <typename T, int kBound>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const BeamParams p) {
    constexpr int kVec = 16 / sizeof(T), kPer = Logit<T>::kPer;
    constexpr int kStep = kLoads * 32 * kVec;
    constexpr int kGroupsOf = kBound / 32;  // groups that a lane adds to: one, or one for each of its loads
    static_assert(kGroupsOf == 1 || kGroupsOf == kLoads, "groups");
    __shared__ float s_most[kMaxSteps][kScanThreads];
    __shared__ float s_group[kScanWarps][kBound];
    __shared__ float4 s_sums[kScanWarps];
    __shared__ uint64_t s_key[kBuffer], s_red[kScanWarps];
    __shared__ int s_keys, s_found, s_step[kBuffer];
    follow_stream();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / p.segs;
    if (p.done && p.done[row]) return;  // beam_join takes its one candidate from the scores
    const int seg = (int)(blockIdx.x - row * p.segs), c1 = p.k + 1;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // Loads are aligned: the row's first lies up to kVec - 1 elements before it.
    const int skew = (int)(((uintptr_t)x % 16) / sizeof(T));
    const int begin = seg * p.seg_len - skew;
    const int end = p.vocab - begin < p.seg_len ? p.vocab : begin + p.seg_len;
    const int first = begin + warp * kStep;  // steps of the warps take turns
    constexpr int kTurn = kScanWarps * kStep;

    Sums s{kNegInf, 0.f, kNegInf, 0.f};
    float mine = kNegInf;  // the largest of this lane
    float group[kGroupsOf];
#pragma unroll
    for (int i = 0; i < kGroupsOf; ++i) group[i] = kNegInf;
    if (tid == 0) s_keys = s_found = 0;

    uint4 next[kLoads];
    auto load = [&](int at) {
        if (at >= 0 && at + kStep <= p.vocab) {
            const uint4* src = reinterpret_cast<const uint4*>(x + at) + lane;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) next[i] = __ldcs(src + 32 * i);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) next[i] = load16(x, at + (i * 32 + lane) * kVec, p.vocab);
        }
    };
    if (first < end) load(first);
    int steps = 0;
    for (int at = first; at < end; at += kTurn, ++steps) {
        uint32_t w[kLoads * 4];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            w[4 * i] = next[i].x; w[4 * i + 1] = next[i].y; w[4 * i + 2] = next[i].z; w[4 * i + 3] = next[i].w;
        }
        if (at + kTurn < end) load(at + kTurn);
        const auto value = [](uint32_t word) {
            float v[kPer];
            Logit<T>::unpack(word, v);
            return kPer == 2 ? fmaxf(v[0], v[kPer - 1]) : v[0];
        };
        uint32_t ml[kLoads], mw;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            ml[i] = Logit<T>::larger(Logit<T>::larger(w[4 * i], w[4 * i + 1]), Logit<T>::larger(w[4 * i + 2], w[4 * i + 3]));
            mw = i ? Logit<T>::larger(mw, ml[i]) : ml[i];
        }
        float m = value(mw);
        const float c_new = fmaxf(s.c, ceilf(m * kLog2e));
        const float ref = c_new == kNegInf ? 0.f : c_new;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kLoads * 4; ++i) {
            float v[kPer];
            Logit<T>::unpack(w[i], v);
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[(i * kPer + e) & 3] += exp2_fast(fmaf(v[e], kLog2e, -ref));
        }
        const float part = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if (!(m < kHuge) || part != part || (m < -kHuge && m > kNegInf)) {
            m = slow_sums<T>(x, at + lane * kVec, p.vocab, s);
            group[0] = fmaxf(group[0], m);  // (of any one group)
        } else {
            if constexpr (kGroupsOf == 1) {
                group[0] = fmaxf(group[0], m);
            } else {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) group[i] = fmaxf(group[i], value(ml[i]));
            }
            if (s.c > kNegInf) s.sum *= exp2_fast(s.c - ref);
            s.c = c_new;
            s.sum += part;
        }
        s_most[steps][tid] = m;
        mine = fmaxf(mine, m);
    }

    // Sums and group maxima put together.
#pragma unroll
    for (int i = 0; i < kGroupsOf; ++i) s_group[warp][32 * i + lane] = group[i];
    float c_all = s.c, h_all = s.huge;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        c_all = fmaxf(c_all, __shfl_xor_sync(0xffffffffu, c_all, o));
        h_all = fmaxf(h_all, __shfl_xor_sync(0xffffffffu, h_all, o));
    }
    float sum = s.c > kNegInf ? s.sum * exp2_fast(s.c - c_all) : 0.f;
    float huge_sum = s.huge > kNegInf ? s.huge_sum * exp2_fast((s.huge - h_all) * kLog2e) : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        huge_sum += __shfl_xor_sync(0xffffffffu, huge_sum, o);
    }
    if (lane == 0) s_sums[warp] = make_float4(c_all, sum, h_all, huge_sum);
    __syncthreads();
    if (tid == 0) {
        float4 a = s_sums[0];
        for (int i = 1; i < kScanWarps; ++i) {
            const float4 y = s_sums[i];
            const float c = fmaxf(a.x, y.x), h = fmaxf(a.z, y.z);
            a.y = (a.x > kNegInf ? a.y * exp2_fast(a.x - c) : 0.f) + (y.x > kNegInf ? y.y * exp2_fast(y.x - c) : 0.f);
            a.w = (a.z > kNegInf ? a.w * exp2_fast((a.z - h) * kLog2e) : 0.f) + (y.z > kNegInf ? y.w * exp2_fast((y.z - h) * kLog2e) : 0.f);
            a.x = c;
            a.z = h;
        }
        p.part[blockIdx.x] = a;
    }
    if (tid < kBound) {
        float g = s_group[0][tid];
#pragma unroll
        for (int w = 1; w < kScanWarps; ++w) g = fmaxf(g, s_group[w][tid]);
        s_group[0][tid] = g;
    }
    __syncthreads();
    // The c1-th largest group maximum; every warp finds it for itself.
    float bound = kNegInf;
#pragma unroll
    for (int r = 0; r < kBound / 32; ++r) {
        const int me = r * 32 + lane;
        const float g = s_group[0][me];
        int larger = 0;
#pragma unroll 8
        for (int i = 0; i < kBound; ++i) {
            const float y = s_group[0][i];
            larger += y > g || (y == g && i < me);
        }
        const unsigned who = __ballot_sync(0xffffffffu, larger == c1 - 1);
        if (who) bound = __shfl_sync(0xffffffffu, g, __ffs(who) - 1);
    }
    // The values of this lane that reach the bound (where there are too many for the buffers).
    auto each = [&](auto f) {
        if (mine < bound || mine == kNegInf) return;
        for (int t = 0; t < steps; ++t) {
            if (s_most[t][tid] < bound) continue;
            const int at = first + t * kTurn + lane * kVec;
            uint4 u[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) u[i] = load16(x, at + i * 32 * kVec, p.vocab);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t q[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[kPer];
                    Logit<T>::unpack(q[j], v);
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        if (v[e] >= bound && fabsf(v[e]) < INFINITY)
                            f(key_of(v[e], (uint32_t)(at + i * 32 * kVec + j * kPer + e)));
                }
            }
        }
    };
    // The steps that hold them are shared out to all threads, four to a step: a warp that held
    // several would read them one after the other (5 us at the end of 32 x 8 rows of 131072).
    if (mine >= bound && mine > kNegInf)
        for (int t = 0; t < steps; ++t)
            if (s_most[t][tid] >= bound && s_most[t][tid] > kNegInf) {
                const int place = atomicAdd(&s_found, 1);
                if (place < kBuffer) s_step[place] = t << 8 | tid;
            }
    __syncthreads();
    const int found = s_found;
    for (int i = tid / kLoads; i < min(found, kBuffer); i += kScanThreads / kLoads) {
        const int t = s_step[i] >> 8, who = s_step[i] & 255;
        const int at = begin + (who >> 5) * kStep + t * kTurn + ((tid % kLoads) * 32 + (who & 31)) * kVec;
        const uint4 u = load16(x, at, p.vocab);
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[kPer];
            Logit<T>::unpack(q[j], v);
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (v[e] >= bound && fabsf(v[e]) < INFINITY) {
                    const int place = atomicAdd(&s_keys, 1);
                    if (place < kBuffer) s_key[place] = key_of(v[e], (uint32_t)(at + j * kPer + e));
                }
        }
    }
    __syncthreads();
    uint64_t* cand = p.cand + (int64_t)blockIdx.x * c1;
    const int n = s_keys;
    if (found <= kBuffer && n <= kBuffer) {
        for (int i = tid; i < n; i += kScanThreads) {
            const uint64_t k = s_key[i];
            int larger = 0;
            for (int j = 0; j < n; ++j) larger += s_key[j] > k;
            if (larger < c1) cand[larger] = k;
        }
        for (int r = n + tid; r < c1; r += kScanThreads) cand[r] = 0;
    } else {
        // Many equal values: c1 rounds of the largest key below the last one.
        uint64_t under = ~0ull;
        for (int r = 0; r < c1; ++r) {
            uint64_t best = 0;
            each([&](uint64_t k) { best = k < under && k > best ? k : best; });
            best = warp_max(best);
            __syncthreads();
            if (lane == 0) s_red[warp] = best;
            __syncthreads();
            best = 0;
            for (int i = 0; i < kScanWarps; ++i) best = s_red[i] > best ? s_red[i] : best;
            if (tid == 0) cand[r] = best;
            under = best;
        }
    }
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
    const uint32_t lists = (uint32_t)p.beams * p.segs, keys = lists * c1, per_beam = (uint32_t)p.segs * c1;
    const uint64_t* cand = p.cand + row0 * p.segs * c1;
    constexpr int kKeep = 4;  // keys of a thread that stay in registers

    for (int w = tid; w < p.beams; w += kJoinThreads) {
        score[w] = p.scores[row0 + w];
        done[w] = p.done && p.done[row0 + w];
    }
    follow_stream();
    uint64_t keep[kKeep];
    const bool kept = keys <= kKeep * kJoinThreads;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) keep[i] = kept && tid + i * kJoinThreads < keys ? cand[tid + i * kJoinThreads] : 0;
    const uint64_t edge0 = (uint32_t)tid < lists ? cand[(uint32_t)tid * c1 + p.k] : 0;
    // lse of each beam: the segments' sums put together, one warp a beam.
    for (int w = warp; w < p.beams; w += kJoinThreads / 32) {
        if (p.done && p.done[row0 + w]) continue;
        const float4* part = p.part + (row0 + w) * p.segs;
        const float4 none = make_float4(kNegInf, 0.f, kNegInf, 0.f);
        const float4 mine = lane < p.segs ? part[lane] : none;
        float c = mine.x, h = mine.z, sum = 0.f, huge = 0.f;
        for (int i = lane + 32; i < p.segs; i += 32) {
            const float4 y = part[i];
            c = fmaxf(c, y.x);
            h = fmaxf(h, y.z);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
            h = fmaxf(h, __shfl_xor_sync(0xffffffffu, h, o));
        }
        for (int i = lane; i < p.segs; i += 32) {
            const float4 y = i == lane ? mine : part[i];
            if (y.x > kNegInf) sum += y.y * exp2f(y.x - c);
            if (y.z > kNegInf) huge += y.w * exp2f((y.z - h) * kLog2e);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            huge += __shfl_xor_sync(0xffffffffu, huge, o);
        }
        // Huge logits matter alone, or where they are positive.  With no finite logit at all
        // there are no candidates either.  (The scan's rounded factor is divided out again, not
        // log2 e: they differ by 1.3e-8 of a logit, 13 for one of 1e9.)
        if (lane == 0)
            lse[w] = h > 0.f || c == kNegInf ? h + logf(huge) : (float)(((double)c + log2f(sum)) * (1.0 / (double)kLog2e));
    }
    __syncthreads();

    auto total_key = [&](int w, float x, uint32_t t) -> uint64_t {
        const float total = score[w] + (x - lse[w]);
        return total > kNegInf ? key_of(total, (uint32_t)w * p.vocab + t) : 0;
    };
    auto total_of = [&](uint32_t i, uint64_t k) -> uint64_t {  // key number i as a total
        const int w = i / per_beam;
        return k && !done[w] ? total_key(w, key_value(k), key_index(k)) : 0;
    };
    const uint64_t ended = tid < p.beams && done[tid] && score[tid] > kNegInf
                               ? key_of(score[tid], (uint32_t)tid * p.vocab + p.eos) : 0;
    if (kept) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) keep[i] = total_of(tid + i * kJoinThreads, keep[i]);
        block_select(s, p.k, [&](auto f) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (keep[i]) f(keep[i]);
            if (ended) f(ended);
        }, best);
    } else {
        block_select(s, p.k, [&](auto f) {
            for (uint32_t i = tid; i < keys; i += kJoinThreads) {
                const uint64_t k = total_of(i, cand[i]);
                if (k) f(k);
            }
            if (ended) f(ended);
        }, best);
    }

    // What the segments left out (see the head of this file): any total that would still
    // come before the k-th best is put in its place, largest first.
    for (uint32_t list0 = 0; list0 < lists; list0 += kJoinThreads) {
        if (tid == 0) agains = 0;
        __syncthreads();
        if (list0 + tid < lists) {
            const int w = (list0 + tid) / p.segs;
            const uint64_t edge = done[w] ? 0 : list0 == 0 ? edge0 : cand[(list0 + tid) * c1 + p.k];
            if (edge) {  // else nothing was left out
                const uint64_t last = best[p.k - 1], same = total_key(w, key_value(edge), key_index(edge) + 1);
                const uint64_t could = total_key(w, next_below<T>(key_value(edge)), 0);  // whatever its index
                if (same > last || (could && (could | 0xffffffffu) > last)) again[atomicAdd(&agains, 1)] = list0 + tid;
            }
        }
        __syncthreads();
        uint64_t under = ~0ull;
        for (int round = 0; agains && round < p.k && under; ++round) {
            const uint64_t last = best[p.k - 1];
            uint64_t more = 0;
            for (int a = 0; a < agains; ++a) {
                const int list = again[a], w = list / p.segs, seg = list - w * p.segs;
                const uint64_t edge = cand[(uint32_t)list * c1 + p.k];
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
    const dim3 grid((unsigned)((int64_t)p.batch * p.beams * p.segs));
    const cudaError_t e = launch_early(p.k < 32 ? beam_scan_kernel<T, 32> : beam_scan_kernel<T, 128>, grid, kScanThreads, 0, stream, 1, p);
    if (e != cudaSuccess) return e;
    return launch_early(beam_join_kernel<T>, dim3(p.batch), kJoinThreads, 0, stream, 1, p);
}

}  // namespace

// Values of a CTA's segment: whole steps of all its warps.  The fullest SM has n = ceil(CTAs /
// SMs) CTAs, each as long as its steps and about three more at its ends, and issues 0.036 of
// its peak for each resident warp up to 0.8 of it (measured on 32 x 8 rows of 131072 bf16
// values).
int beam_seg_len(int64_t rows, int32_t vocab, int elem, int sm_count) {
    const int turn = kScanWarps * kLoads * 32 * 16 / elem;
    int best = 1;
    double least = 1e30;
    for (int each = 1; each <= kMaxSteps; ++each) {
        const int64_t segs = (vocab + (int64_t)each * turn - 1) / ((int64_t)each * turn), ctas = rows * segs;
        const int64_t n = (ctas + sm_count - 1) / sm_count;
        const double rate = 0.036 * kScanWarps * (double)(n < 4 ? n : 4);
        const double cost = (double)n * (each + 3) / (rate < 0.8 ? rate : 0.8);
        if (cost < least) {
            least = cost;
            best = each;
        }
    }
    return turn * best;
}

cudaError_t launch_beam(const BeamParams& p, cudaStream_t stream) {
    if (p.batch == 0) return cudaSuccess;
    if (p.dtype == KDA_LOGITS_F32) return launch_type<float>(p, stream);
    if (p.dtype == KDA_LOGITS_BF16) return launch_type<__nv_bfloat16>(p, stream);
    return launch_type<__half>(p, stream);
}

}  // namespace kda
