// kda_kvcache_attention.cuh -- what the attention kernels over the 8-bit cache share:
// activation types, widening of codes, rows of a batch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include "kda_serving.cuh"

namespace kda {

constexpr float kNegInf = -INFINITY;
constexpr float kBlockLift = 7.f;  // log2 of a weight at its reference, in the block kernel and the state

__device__ __forceinline__ uint32_t widen2(uint32_t codes) {  // two e4m3 codes (low 16 bits)
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}
// Codes are read once by an SM: kept out of L1 (133 -> 128 us for 64 rows of up to 8192 tokens).
__device__ __forceinline__ uint4 load_codes16(const uint8_t* p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p) {
    uint2 v;
    asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T> struct Act;
template <> struct Act<__nv_bfloat16> {
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <> struct Act<__half> {
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_half2(a, b); }
};

// The power of two that brings a row of q with largest magnitude a into [2^14, 2^15); the
// exponent is limited so that this factor and its inverse are normal.
__device__ __forceinline__ int row_exponent(float a) {
    return max(a > 0.f && a < INFINITY ? ilogbf(a) : 0, -100);
}

// New tokens of row r: [begin, begin + n); n = 0 for malformed offsets.
__device__ __forceinline__ int row_tokens(const CacheParams& c, int r, int64_t& begin) {
    if (!c.cu) {
        begin = r;
        return 1;
    }
    begin = c.cu[r];
    const int64_t end = c.cu[r + 1];
    if (begin < 0 || end < begin || end > c.tokens || (r == 0 && begin != 0)) {
        report(c.status, kStatusBadSeqlens);
        return 0;
    }
    if (r == c.rows - 1 && end != c.tokens) report(c.status, kStatusBadSeqlens);
    return (int)(end - begin);
}
// Softmax weights carry the scale of their v in the exponent, and what is largest of weight and scale
// together, m, is the reference: so a weight's rounding to fp16 is relative to the row's largest
// contributions, whatever the scales.  The sum of the weights takes the scale out again, and there a
// block counts whose contributions are nothing: 2^(s + log2 v - m) must not fall out of fp32 where
// 2^s matters.  So in m and in the sum no block's log2 v counts as less than the largest met so far less
// kScaleSpan (m is at most max s + that largest, and 2^-126 is 36 bits below max s then), nor as less
// than kScaleLeast, which holds sums of 2^31 weights in fp32.  The weights for the product are
// brought down again to what the scale is.
constexpr float kScaleSpan = 90.f, kScaleLeast = -80.f;
__device__ __forceinline__ uint32_t brought_down(uint32_t half2, float by) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&half2), __float2half2_rn(by));
    return *reinterpret_cast<const uint32_t*>(&h);
}
// l 2^d for d <= 0 in two steps, h = 2^(d / 2): a sum of small scales is as large as 2^125, and 2^d alone
// may lie below fp32's range.
__device__ __forceinline__ float rescaled(float l, float h) { return l * h * h; }
// 2^x by the hardware's instruction (results below 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Cached tokens of row r that its table has places for, and key numbers: those of the tiles, pages and scales
// that are looked at ahead fit in 31 bits too.
constexpr int kMaxLength = INT_MAX - 4095;
__device__ __forceinline__ int row_length(const CacheParams& c, int r) {
    const int len = c.lens[r];
    const int64_t room = min((int64_t)c.width * c.page_tokens, (int64_t)kMaxLength);
    if (len < 0 || len > room) report(c.status, kStatusBadIndex);
    return len < 0 ? 0 : len > room ? (int)room : len;
}

// first[r] = work of the rows before r, first[rows] = all, with work(r) for each row.  The whole
// block of kThreads calls it; s: one value a warp.
template <int kThreads, typename Work>
__device__ __forceinline__ void scan_rows(int rows, int64_t* first, int64_t* s, Work work) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t base = 0;
    for (int r0 = 0; r0 < rows; r0 += kThreads) {
        const int r = r0 + tid;
        const int64_t w = work(r);
        int64_t x = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s[warp] = x;
        __syncthreads();
        int64_t before = base;
        for (int i = 0; i < warp; ++i) before += s[i];
        if (r < rows) first[r] = before + x - w;
        for (int i = 0; i < kThreads / 32; ++i) base += s[i];
        __syncthreads();
    }
    if (tid == 0) first[rows] = base;
}

// The row that work number w belongs to: the last with first[row] <= w (rows without work
// share their number with the next).
__device__ __forceinline__ int row_of(const int64_t* first, int rows, int64_t w) {
    int lo = 0, hi = rows;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= w) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What a launch's rows have: all of their keys, or those behind a prefix that is shared (kda_kvcache_shared.cu),
// which go on from the state (maximum, sum, least scale, output) that the prefix left for each query row.
enum { kKindRows = 0, kKindSuffix = 1 };
// A row's first key (a multiple of kSharedUnit).
template <int kKind>
__device__ __forceinline__ int unit_from(const AttentionParams& p, int r) { return kKind == kKindSuffix ? p.from[r] : 0; }

// Work of one share.
__device__ __forceinline__ int64_t share_of(int64_t all, int shares) { return (all + shares - 1) / shares; }

// The row that item number i of the joining launch belongs to, and the item's number in it.
// Items are counted by an upper bound: row r's first is number (cu[r] * group / cols + r) *
// heads, as its column blocks are at most n * group / cols + 1.  False: no such item.
__device__ __forceinline__ bool joined_item(const CacheParams& c, int group, int cols, int64_t& i, int& row) {
    if (!c.cu) {
        const int64_t each = (int64_t)c.heads * ((group + cols - 1) / cols);
        row = (int)(i / each);
        i -= row * each;
    } else {
        int lo = 0, hi = c.rows;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (((int64_t)c.cu[mid] * group / cols + mid) * c.heads <= i) lo = mid;
            else hi = mid;
        }
        row = lo;
        i -= ((int64_t)c.cu[row] * group / cols + row) * c.heads;
    }
    return row < c.rows && i >= 0;
}
inline int64_t joined_items(const CacheParams& c, int64_t group, int cols) {
    return c.cu ? (c.tokens * group / cols + c.rows) * c.heads : (int64_t)c.rows * c.heads * ((group + cols - 1) / cols);
}

}  // namespace kda
