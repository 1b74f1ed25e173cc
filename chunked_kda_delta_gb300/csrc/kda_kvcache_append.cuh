// kda_kvcache_append.cuh -- what the two appends to the 8-bit cache share: exact quotients and codes,
// the rounding again of pages whose scale grows.
#pragma once

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

}  // namespace
}  // namespace kda
