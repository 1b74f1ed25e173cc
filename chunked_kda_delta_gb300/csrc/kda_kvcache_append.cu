// kda_kvcache_append.cu -- new keys and values into the 8-bit paged cache.
//
// Per touched page and head: a = max |x| of the new tokens, scale s = a / 448 for a page that
// starts here, else max(s, a / 448) with the page's older codes rounded again where s grew;
// codes = e4m3(x / s).  HBM-bound: 2 bytes read and 1 written per value.  The new values stay
// in registers between the maximum and the quotients, so they are read once.  A block owns a
// (page, head) of k or v, so no two write the same scale.
//
// The definition's quotient is the correctly rounded one.  Values of a block share their
// divisor, so it is formed from the correctly rounded reciprocal r by Markstein's theorem
// (IBM J. Res. Dev. 34, 1990): q = rn(x r), then rn(q + rn(x - q s) r) is the correctly rounded
// x / s wherever no intermediate leaves the normal range and s's fraction is not all
// ones -- three operations a value instead of a full division (86 us for 30.7k tokens of 8
// heads with divisions, where instructions and not bytes were the bound; now 34, 0.81 of its bytes
// at the copy rate, with 71% of the issue slots taken).  Other scales, and blocks with values that
// are not finite, take the division.  One token of 256 rows, 8 heads: 5.1 us, a launch and a chain of
// dependent loads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr float kCodeMax = 448.f;

template <typename T> struct Act;
template <> struct Act<__nv_bfloat16> {
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    }
};
template <> struct Act<__half> {
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Act<T>::two(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Two codes; saturating, round to nearest even.
__device__ __forceinline__ uint32_t code2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 values2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Largest magnitude of eight values as packed; +inf or NaN patterns compare above all finite ones.
template <typename T>
__device__ __forceinline__ uint32_t largest2(const uint4& w) {  // halves: largest of the even and the odd values
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
}
template <typename T>
__device__ __forceinline__ float top_of(uint32_t halves) {  // as a float: inf or NaN where some value is
    const uint32_t u = max(halves & 0xffffu, halves >> 16);
    return Act<T>::two(u).x;
}
// Largest finite magnitude.
__device__ __forceinline__ float largest(const float (&x)[8]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[i]);
        if (m < INFINITY) a = fmaxf(a, m);
    }
    return a;
}

// Quotient of the definition: 0 for NaN and for a scale of 0, infinities saturate.
__device__ __forceinline__ float quotient(float x, float s) {
    if (x != x) return 0.f;
    if (fabsf(x) == INFINITY) return copysignf(kCodeMax, x);
    return s > 0.f ? __fdiv_rn(x, s) : 0.f;
}
// Whether the short quotient is exact for every finite |x| <= 448 s: quotients too small for it
// (|x| below 2^-100, or x / s below the least code) round to the code 0 all the same.
__device__ __forceinline__ bool short_division(float s) {
    return s > 0x1p-80f && s < 0x1p80f && (__float_as_uint(s) & 0x7fffffu) != 0x7fffffu;
}
__device__ __forceinline__ float short_quotient(float x, float s, float r) {
    const float q = __fmul_rn(x, r), y = fmaf(fmaf(-q, s, x), r, q);
    return __uint_as_float(__float_as_uint(y) | (__float_as_uint(x) & 0x80000000u));  // -0 / s is -0
}
__device__ __forceinline__ uint2 encode(const float (&x)[8], float s) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = code2(quotient(x[2 * i], s), quotient(x[2 * i + 1], s));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
__device__ __forceinline__ uint2 encode_short(const float (&x)[8], float s, float r) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = code2(short_quotient(x[2 * i], s, r), short_quotient(x[2 * i + 1], s, r));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// Rounds `bytes` older codes (a multiple of 16) of scale `was` again for the larger scale s; by
// kThreads threads, four 16-byte loads of each in flight.
template <int kThreads>
__device__ __forceinline__ void grade_again(uint8_t* codes, int bytes, float was, float s, int tid) {
    const bool quick = short_division(s);
    const float r = __frcp_rn(s);
    auto again = [&](uint32_t two) {
        const float2 f = values2(two);
        const float a = __fmul_rn(f.x, was), b = __fmul_rn(f.y, was);
        return quick ? code2(short_quotient(a, s, r), short_quotient(b, s, r)) : code2(quotient(a, s), quotient(b, s));
    };
    for (int at = tid * 16; at < bytes; at += kThreads * 64) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i * kThreads * 16 < bytes) w[i] = *reinterpret_cast<const uint4*>(codes + at + i * kThreads * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (at + i * kThreads * 16 >= bytes) continue;
            uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = again(u[k] & 0xffffu) | again(u[k] >> 16) << 16;
            *reinterpret_cast<uint4*>(codes + at + i * kThreads * 16) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
}

// One token a row (the decode step): a warp per (row, head, k or v).  An open page whose scale
// grows has its older codes rounded again by the whole block (by its warp alone the step took
// 40 us where half of 256 x 8 pages grew, now 10; 6 where 7% grow, 4 where none does).
constexpr int kStepWarps = 4;

template <typename T, int kDim>
__global__ void __launch_bounds__(kStepWarps * 32) append_step_kernel(const __grid_constant__ AppendParams p) {
    follow_stream();
    const CacheParams& c = p.c;
    struct Growth {
        uint8_t* codes;
        int bytes;  // 0: none
        float was, now;
    };
    __shared__ Growth s_growth[kStepWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kStepWarps + warp;
    Growth growth{nullptr, 0, 0.f, 0.f};
    if (w < 2 * c.tokens * c.heads) {
        const int which = (int)(w & 1), head = (int)((w >> 1) % c.heads);
        const int64_t row = (w >> 1) / c.heads;
        const int32_t len = c.lens[row];
        const int64_t slot = len < 0 ? c.width : len / c.page_tokens;
        const int32_t page = slot < c.width ? c.tables[row * c.width + slot] : -1;
        if (page < 0 || page >= c.pages) {
            if (lane == 0) report(c.status, kStatusBadIndex);
        } else {
            constexpr int kLanes = kDim / 8;
            const bool mine = lane < kLanes;
            float x[8];
            const T* src = static_cast<const T*>(p.x[which]) + row * p.stride[which] + (int64_t)head * kDim;
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (mine) raw = reinterpret_cast<const uint4*>(src)[lane];
            unpack<T>(raw, x);
            if (!(top_of<T>(largest2<T>(raw)) < INFINITY)) report(c.status, kStatusNonfinite);
            float a = largest(x);
#pragma unroll
            for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));

            const int off = len % c.page_tokens;
            const int64_t block = (int64_t)page * c.heads + head;
            float* scale = (which ? c.v_scale : c.k_scale) + block;
            uint8_t* codes = (which ? c.v_codes : c.k_codes) + block * c.page_tokens * kDim;
            float s = __fdiv_rn(a, kCodeMax);
            if (off > 0) {
                const float was = *scale;
                if (s > was) growth = Growth{codes, off * kDim, was, s};
                else s = was;
                __syncwarp();  // every lane has read the scale
            }
            if (lane == 0) *scale = s;
            if (mine) reinterpret_cast<uint2*>(codes + (int64_t)off * kDim)[lane] = encode(x, s);
        }
    }
    if (lane == 0) s_growth[warp] = growth;
    if (!__syncthreads_or(growth.bytes)) return;
#pragma unroll 1
    for (int i = 0; i < kStepWarps; ++i) {
        const Growth g = s_growth[i];
        if (g.bytes) grade_again<kStepWarps * 32>(g.codes, g.bytes, g.was, g.now, threadIdx.x);
    }
}

// Several tokens a row: a block of 128 threads per (touched page, head, k or v).  Row r's i-th
// touched page has number cu[r] / page_tokens + 2 r + i: n tokens touch at most
// n / page_tokens + 2 pages, so the numbers of different rows do not meet.
constexpr int kAppendThreads = 128;

template <typename T, int kDim, int kPage>
__global__ void __launch_bounds__(kAppendThreads, kDim * kPage <= 8192 ? 8 : 4) append_kernel(const __grid_constant__ AppendParams p) {
    follow_stream();
    const CacheParams& c = p.c;
    __shared__ float red[kAppendThreads / 32];
    constexpr int kLanes = kDim / 8, kRows = kAppendThreads / kLanes;  // tokens a pass
    constexpr int kPasses = (kPage + kRows - 1) / kRows;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t unit = blockIdx.x;
    const int head = blockIdx.y >> 1, which = blockIdx.y & 1;

    // The last row whose numbers start at or before this unit; all warps search alike.
    int lo = 0, hi = c.rows;  // first number of lo <= unit < first number of hi
    while (hi - lo > 1) {
        const int step = (hi - lo + 32) / 33, r = lo + step * (lane + 1);
        const bool below = r < hi && c.cu[r] / kPage + 2ll * r <= unit;
        const int n = __popc(__ballot_sync(0xffffffffu, below));
        const int next = lo + step * (n + 1);
        lo += step * n;
        if (next < hi) hi = next;
    }
    const int row = lo;
    const int64_t begin = c.cu[row], end = c.cu[row + 1];
    if (begin < 0 || end < begin || end > c.tokens || (row == 0 && begin != 0) ||
        (row == c.rows - 1 && end != c.tokens)) {
        if (tid == 0) report(c.status, kStatusBadSeqlens);
        return;
    }
    const int64_t i = unit - (begin / kPage + 2ll * row);
    const int32_t len = c.lens[row];
    if (i < 0 || len < 0) {
        if (len < 0 && tid == 0) report(c.status, kStatusBadIndex);
        return;
    }
    const int64_t slot = len / kPage + i;               // of the row's table
    const int64_t p0 = slot * kPage;                    // position of the page's first token
    const int64_t first = p0 > len ? p0 : len;          // first new position in the page
    const int64_t last = min(p0 + kPage, len + (end - begin));
    if (first >= last) return;
    const int32_t page = slot < c.width ? c.tables[(int64_t)row * c.width + slot] : -1;
    if (page < 0 || page >= c.pages) {
        if (tid == 0) report(c.status, kStatusBadIndex);
        return;
    }
    const int n = (int)(last - first), off = (int)(first - p0);
    const int64_t stride = p.stride[which];
    const T* src = static_cast<const T*>(p.x[which]) + (begin + first - len) * stride + (int64_t)head * kDim;
    const int at = tid % kLanes, t0 = tid / kLanes;

    bool finite = true;  // all values of this thread
    uint4 raw[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int t = t0 + k * kRows;
        raw[k] = t < n ? __ldcs(reinterpret_cast<const uint4*>(src + t * stride) + at) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) most = __vmaxu2(most, largest2<T>(raw[k]));
    float a = top_of<T>(most);
    if (!(a < INFINITY)) {
        report(c.status, kStatusNonfinite);
        a = 0.f;
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            float x[8];
            unpack<T>(raw[k], x);
            a = fmaxf(a, largest(x));
        }
        finite = false;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) red[tid >> 5] = a;
    const int64_t block = (int64_t)page * c.heads + head;
    float* scale = (which ? c.v_scale : c.k_scale) + block;
    uint8_t* codes = (which ? c.v_codes : c.k_codes) + block * kPage * kDim;
    const float was = off > 0 ? *scale : 0.f;
    __syncthreads();  // the maxima are there, and every thread has read the scale
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) a = fmaxf(a, red[w]);
    float s = __fdiv_rn(a, kCodeMax);
    const bool grown = off > 0 && s > was;
    if (off > 0 && !grown) s = was;
    if (tid == 0) *scale = s;
    if (finite && short_division(s)) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const int t = t0 + k * kRows;
            float x[8];
            unpack<T>(raw[k], x);
            if (t < n) reinterpret_cast<uint2*>(codes + (int64_t)(off + t) * kDim)[at] = encode_short(x, s, r);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const int t = t0 + k * kRows;
            float x[8];
            unpack<T>(raw[k], x);
            if (t < n) reinterpret_cast<uint2*>(codes + (int64_t)(off + t) * kDim)[at] = encode(x, s);
        }
    }
    if (grown) grade_again<kAppendThreads>(codes, off * kDim, was, s, tid);  // the registers are free now
}

template <typename T, int kDim>
cudaError_t launch_dim(const AppendParams& p, cudaStream_t stream) {
    const CacheParams& c = p.c;
    if (!c.cu) {
        const int64_t warps = 2 * c.tokens * c.heads;
        return launch_early(append_step_kernel<T, kDim>, dim3((unsigned)((warps + kStepWarps - 1) / kStepWarps)), kStepWarps * 32, 0, stream, 1, p);
    }
    const dim3 grid((unsigned)(c.tokens / c.page_tokens + 2ll * c.rows), 2 * c.heads);
    const auto kernel = c.page_tokens == 16   ? append_kernel<T, kDim, 16>
                        : c.page_tokens == 32 ? append_kernel<T, kDim, 32>
                        : c.page_tokens == 64 ? append_kernel<T, kDim, 64>
                                              : append_kernel<T, kDim, 128>;
    return launch_early(kernel, grid, kAppendThreads, 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool f16, cudaStream_t stream) {
    if (p.c.tokens == 0 || p.c.rows == 0) return cudaSuccess;
    if (p.c.dim == 64) return f16 ? launch_dim<__half, 64>(p, stream) : launch_dim<__nv_bfloat16, 64>(p, stream);
    return f16 ? launch_dim<__half, 128>(p, stream) : launch_dim<__nv_bfloat16, 128>(p, stream);
}

}  // namespace kda
