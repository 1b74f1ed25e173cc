// kda_logits.cu -- penalties for repeated tokens, biases and grammar masks on logits.
//
// Per row and token t, with `seen` the tokens of the row's history and c(t) how often t is in it
// behind the prompt:
//   x = x > 0 ? x / r : x r   where seen;  x = x - f c(t) - p [c(t) > 0];  x = x + b(t);
//   x = -inf                  where the row's mask has no bit.
// fp32, rounded once; a token that nothing applies to keeps its bits.
//
// HBM-bound: the logits are read and written once, mask bits and histories beside them.  A CTA has a
// segment of a row's vocabulary.  It counts the row's history tokens that fall into it, and adds up the
// biases, in shared memory (a word a token), while its share of the logits is on the way to registers.
// Counts are whole numbers, so their order does not matter; biases of one token are added in the
// order of the list by one warp.  In place, a load of 16 bytes that nothing applies to is neither read nor
// written, and one that the mask takes whole is not read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t kBiased = 1u << 31, kPrompt = 1u << 30, kCount = kPrompt - 1;

// A type's bits, and its values in a 16-byte load.
template <typename T> struct Logit;
template <> struct Logit<float> {
    using Raw = uint32_t;
    static __device__ __forceinline__ float value(Raw x) { return __uint_as_float(x); }
    static __device__ __forceinline__ Raw rounded(float x) { return __float_as_uint(x); }
};
template <> struct Logit<__nv_bfloat16> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float value(Raw x) { return __bfloat162float(__ushort_as_bfloat16(x)); }
    static __device__ __forceinline__ Raw rounded(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <> struct Logit<__half> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float value(Raw x) { return __half2float(__ushort_as_half(x)); }
    static __device__ __forceinline__ Raw rounded(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
template <typename Raw>
__device__ __forceinline__ Raw get(const uint4& v, int i) {
    const int word = i * (int)sizeof(Raw) / 4;
    const uint32_t u = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
    return sizeof(Raw) == 4 ? (Raw)u : (Raw)(u >> (16 * (i & 1)));
}
template <typename Raw>
__device__ __forceinline__ void set(uint4& v, int i, Raw x) {
    const int word = i * (int)sizeof(Raw) / 4;
    uint32_t& u = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
    if (sizeof(Raw) == 4) u = x;
    else u = i & 1 ? (u & 0xffffu) | (uint32_t)x << 16 : (u & 0xffff0000u) | x;
}

struct Penalties {
    float repetition, presence, frequency;
    __device__ __forceinline__ float apply(float x, uint32_t word, float bias) const {
        if (word & ~kBiased) {
            x = x > 0.f ? __fdiv_rn(x, repetition) : x * repetition;
            const uint32_t n = word & kCount;
            if (n) x = x - frequency * (float)n - presence;
        }
        if (word & kBiased) x += bias;
        return x;
    }
};

// kVecs: 16-byte loads of a thread.  kWords: there are histories or biases.
template <typename T, int kVecs, bool kWords>
__global__ void __launch_bounds__(kThreads) penalize_kernel(const __grid_constant__ LogitsParams p) {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    constexpr int kEach = 16 / sizeof(Raw), kSeg = kVecs * kThreads * kEach;
    extern __shared__ __align__(16) uint32_t s_word[];   // [kSeg], then the biases where there are any
    float* s_bias = reinterpret_cast<float*>(s_word + kSeg);
    const int tid = threadIdx.x;
    follow_stream();
    const int64_t row = blockIdx.x / p.segs;
    const Raw* src = static_cast<const Raw*>(p.logits) + row * p.stride;
    Raw* dst = static_cast<Raw*>(p.out) + row * p.out_stride;
    const bool place = src == dst;
    // Segments begin at 16-byte boundaries of dst; the first may begin before the row.
    const int before = (int)(((uintptr_t)dst & 15) / sizeof(Raw));
    const int t0 = (int)(blockIdx.x % p.segs) * kSeg - before;   // (vocab is at most 2^30)
    if (t0 >= p.vocab) return;
    const bool even = (((uintptr_t)src ^ (uintptr_t)dst) & 15) == 0;  // src has those boundaries too
    const uint32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;

    // Bits of the tokens of a load that the mask lets through (of those in the row).
    auto allowed = [&](int t) {
        uint32_t bits = (1u << kEach) - 1;
        if (t < 0) bits = bits >> -t << -t;
        if (t + kEach > p.vocab) bits &= t < p.vocab ? (1u << (p.vocab - t)) - 1 : 0u;
        if (mask && bits) {
            const int at = max(t, 0), word = at >> 5, shift = at & 31;
            const uint32_t lo = __ldg(mask + word), hi = shift + kEach > 32 && (word + 1) * 32 < p.vocab ? __ldg(mask + word + 1) : 0u;
            bits &= __funnelshift_r(lo, hi, shift) << (at - t);
        }
        return bits;
    };
    auto inside = [&](int t) {  // bits of the tokens in the row
        uint32_t bits = (1u << kEach) - 1;
        if (t < 0) bits = bits >> -t << -t;
        if (t + kEach > p.vocab) bits &= t < p.vocab ? (1u << (p.vocab - t)) - 1 : 0u;
        return bits;
    };
    auto read = [&](int t, uint32_t in) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (even && in == (1u << kEach) - 1) return *reinterpret_cast<const uint4*>(src + t);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (in >> i & 1) set<Raw>(v, i, src[t + i]);
        return v;
    };

    uint32_t in[kVecs], pass[kVecs];
    uint4 x[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int t = t0 + (k * kThreads + tid) * kEach;
        in[k] = inside(t);
        pass[k] = allowed(t);
    }
    if (!place) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            if (pass[k]) x[k] = read(t0 + (k * kThreads + tid) * kEach, in[k]);
    }

    Penalties rules{1.f, 0.f, 0.f};
    if constexpr (kWords) {
        for (int i = tid; i < kSeg / 4; i += kThreads) reinterpret_cast<uint4*>(s_word)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.repetition) rules.repetition = p.repetition[row];
        if (p.presence) rules.presence = p.presence[row];
        if (p.frequency) rules.frequency = p.frequency[row];
        if (!(rules.repetition > 0.f && rules.repetition < INFINITY && fabsf(rules.presence) < INFINITY && fabsf(rules.frequency) < INFINITY)) {
            if (tid == 0) report(p.status, kStatusBadIndex);
            rules = Penalties{1.f, 0.f, 0.f};
        }
        __syncthreads();
        if (p.width > 0) {
            int len = p.lens ? p.lens[row] : p.width;
            if ((len < 0 || len > p.width) && tid == 0) report(p.status, kStatusBadIndex);
            len = max(0, min(len, p.width));
            const int prompt = p.prompt_lens ? max(0, min(p.prompt_lens[row], len)) : 0;
            const int32_t* history = p.history + row * p.width;
            bool bad = false;
            auto count = [&](int i, int32_t token) {
                bad |= token >= p.vocab;
                const int at = token - t0;
                if (token < 0 || token >= p.vocab || at < 0 || at >= kSeg) return;
                if (i < prompt) atomicOr(s_word + at, kPrompt);
                else atomicAdd(s_word + at, 1u);
            };
            // Loads of 16 bytes where the rows have their boundaries.
            const int head = min(len, (int)((16 - ((uintptr_t)history & 15)) % 16 / 4));
            if (tid < head) count(tid, history[tid]);
            const int4* body = reinterpret_cast<const int4*>(history + head);
            const int quads = (len - head) / 4;
#pragma unroll 4
            for (int i = tid; i < quads; i += kThreads) {
                const int4 q = __ldg(body + i);
                const int at = head + 4 * i;
                count(at, q.x);
                count(at + 1, q.y);
                count(at + 2, q.z);
                count(at + 3, q.w);
            }
            const int rest = head + 4 * quads + tid;
            if (rest < len) count(rest, history[rest]);
            if (bad) report(p.status, kStatusBadIndex);
        }
        if (p.num_bias > 0) {
            __syncthreads();
            if (tid < 32) {
                const int32_t* tokens = p.bias_tokens + row * p.num_bias;
                const float* values = p.bias + row * p.num_bias;
                for (int i0 = 0; i0 < p.num_bias; i0 += 32) {
                    const int i = i0 + tid;
                    const int32_t token = i < p.num_bias ? tokens[i] : -1;
                    const float value = i < p.num_bias ? values[i] : 0.f;
                    if (token >= p.vocab) report(p.status, kStatusBadIndex);
                    const int at = token - t0;
                    const bool ours = token >= 0 && token < p.vocab && at >= 0 && at < kSeg;
                    const uint32_t some = __ballot_sync(0xffffffffu, ours);
                    if (!some) continue;
                    const uint32_t same = __match_any_sync(0xffffffffu, ours ? at : -1 - tid);
                    const bool first = ours && __ffs(same) - 1 == tid;
                    float sum = first && (s_word[at] & kBiased) ? s_bias[at] : 0.f;
                    for (uint32_t left = some; left; left &= left - 1) {
                        const int from = __ffs(left) - 1;
                        const float y = __shfl_sync(0xffffffffu, value, from);
                        if (same >> from & 1) sum += y;
                    }
                    if (first) {
                        s_bias[at] = sum;
                        s_word[at] |= kBiased;
                    }
                    __syncwarp();
                }
            }
        }
        __syncthreads();
    }

#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int i0 = (k * kThreads + tid) * kEach, t = t0 + i0;
        if (!in[k]) continue;
        uint32_t word[kEach], any = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) word[i] = 0;
        if constexpr (kWords) {
#pragma unroll
            for (int i = 0; i < kEach; i += 4) {
                const uint4 w = reinterpret_cast<const uint4*>(s_word + i0)[i / 4];
                word[i] = w.x, word[i + 1] = w.y, word[i + 2] = w.z, word[i + 3] = w.w;
                any |= w.x | w.y | w.z | w.w;
            }
        }
        if (place) {
            if (pass[k] == in[k] && !any) continue;
            if (pass[k]) x[k] = read(t, in[k]);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (!(pass[k] >> i & 1)) set<Raw>(x[k], i, L::rounded(-INFINITY));
            else if (word[i]) set<Raw>(x[k], i, L::rounded(rules.apply(L::value(get<Raw>(x[k], i)), word[i], word[i] & kBiased ? s_bias[i0 + i] : 0.f)));
        }
        if (in[k] == (1u << kEach) - 1) {
            *reinterpret_cast<uint4*>(dst + t) = x[k];
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (in[k] >> i & 1) dst[t + i] = get<Raw>(x[k], i);
        }
    }
}

template <typename T, int kVecs, bool kWords>
cudaError_t launch_one(const LogitsParams& p, cudaStream_t stream) {
    constexpr int kSeg = kVecs * kThreads * (16 / (int)sizeof(T));
    const size_t smem = kWords ? (size_t)kSeg * 4 * (p.num_bias > 0 ? 2 : 1) : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(penalize_kernel<T, kVecs, kWords>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_early(penalize_kernel<T, kVecs, kWords>, dim3((unsigned)(p.rows * p.segs)), kThreads, smem, stream, 1, p);
}
template <typename T, int kVecs>
cudaError_t launch_words(const LogitsParams& p, cudaStream_t stream) {
    return p.width > 0 || p.num_bias > 0 ? launch_one<T, kVecs, true>(p, stream) : launch_one<T, kVecs, false>(p, stream);
}
template <typename T>
cudaError_t launch_type(LogitsParams& p, cudaStream_t stream) {
    constexpr int kEach = 16 / sizeof(T);
    const bool even = ((uintptr_t)p.out & 15) == 0 && (p.out_stride * sizeof(T) & 15) == 0;
    // The longest segments that still give every SM a few CTAs.
    int vecs = 4;
    auto segs = [&](int v) { return (int)(((int64_t)p.vocab + (even ? 0 : kEach - 1) + v * kThreads * kEach - 1) / (v * kThreads * kEach)); };
    while (vecs > 1 && p.rows * segs(vecs) < 4ll * p.sm_count) vecs /= 2;
    p.segs = segs(vecs);
    if (p.rows * p.segs > 0x7fffffffll) return cudaErrorInvalidValue;
    return vecs == 4 ? launch_words<T, 4>(p, stream) : vecs == 2 ? launch_words<T, 2>(p, stream) : launch_words<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_penalize(LogitsParams p, int dtype, cudaStream_t stream) {
    if (dtype == 0) return launch_type<float>(p, stream);
    return dtype == 1 ? launch_type<__nv_bfloat16>(p, stream) : launch_type<__half>(p, stream);
}

}  // namespace kda
