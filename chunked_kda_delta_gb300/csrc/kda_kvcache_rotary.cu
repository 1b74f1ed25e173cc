// kda_kvcache_rotary.cu -- new keys and values into the 8-bit paged cache, the rotation of their
// positions applied on the way, and the rotated queries.
//
// Each pair (a, b) of a head's first `rot` channels turns by its token's angle:
//   a' = a cos - b sin,  b' = b cos + a sin,
// in fp32 with the error of one product put back (Kahan's a b - c d: within 1.5 units in the last
// place also where the two terms cancel); an infinite product makes the result infinite, or NaN where two
// cancel.  Rotated keys go to the cache's quantisation as they are,
// without a rounding to 16 bits between; queries are rounded once.  Quantisation as in
// kda_kvcache_append.cu; for finite values a table of cosines 1 and sines 0 gives its codes, but for the sign of
// zeros (a' is +0 for a = -0 and b < 0).
//
// A thread has an item: the 16 channels of eight pairs, with their eight cosines and sines.
// HBM-bound: 2 bytes read and 2 written for a value of q, 2 and 1 for k and v.  The table's rows
// (4 rot bytes a token, twice a head's values) come from L2; a thread turns several heads of q
// with the angles it holds, so that they are not read for each: four, two of them loaded at a time, so that
// four blocks fit an SM (5 prompts of up to 8191 tokens, 32 heads over 8 of 128, bf16: 140.4 us, 5.0 TB/s, 60% of the
// issue slots; eight heads, four at a time 146, two heads 142; three blocks 151, five 172).  One token a row
// (256 rows, 64 heads over 8 of 128) takes 7.5 us, a chain of length -> table -> page -> scale -> store; one
// row 4.8.
#include "kda_kvcache_append.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kQHeads = 4;  // of a block, for each set of threads that has its own tokens
constexpr int kStepWarps = 4;

__device__ __forceinline__ float minus_products(float a, float c, float b, float s) {  // a c - b s
    // (An infinite product has no error to put back: inf - inf would be NaN.  To look at the results instead and work out
    // again what is NaN spills: 191 us for the prompts above.)
    const float w = __fmul_rn(b, s), e = fabsf(w) < INFINITY ? fmaf(b, s, -w) : 0.f;
    return __fadd_rn(fmaf(a, c, -w), -e);
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// The two runs of 8 channels of item j, in units of 8 channels: pairs lie rot / 2 channels apart,
// or side by side; items past the rotated channels are as they come.
struct Item {
    int lo, hi;
    bool turns, side;
    __device__ __forceinline__ Item(int j, int rot, bool interleaved) {
        turns = j < rot / 16;
        side = !turns || interleaved;
        lo = side ? 2 * j : j;
        hi = side ? 2 * j + 1 : j + rot / 16;
    }
};
struct Angles {
    float c[8], s[8];
    __device__ __forceinline__ void read(const float* row, int rot, int j) {
        const float4* p = reinterpret_cast<const float4*>(row + 8 * j);
        const float4* q = reinterpret_cast<const float4*>(row + rot / 2 + 8 * j);
        const float4 a = __ldg(p), b = __ldg(p + 1), x = __ldg(q), y = __ldg(q + 1);
        c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
        s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w, s[4] = y.x, s[5] = y.y, s[6] = y.z, s[7] = y.w;
    }
    // lo and hi: the item's runs; pair i is (lo[i], hi[i]), or side by side (2 i, 2 i + 1) through both.
    __device__ __forceinline__ void turn(float (&lo)[8], float (&hi)[8], bool side) const {
        if (side) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a = lo[2 * i], b = lo[2 * i + 1];
                lo[2 * i] = minus_products(a, c[i], b, s[i]);
                lo[2 * i + 1] = minus_products(b, c[i], a, -s[i]);
                a = hi[2 * i], b = hi[2 * i + 1];
                hi[2 * i] = minus_products(a, c[4 + i], b, s[4 + i]);
                hi[2 * i + 1] = minus_products(b, c[4 + i], a, -s[4 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = lo[i], b = hi[i];
                lo[i] = minus_products(a, c[i], b, s[i]);
                hi[i] = minus_products(b, c[i], a, -s[i]);
            }
        }
    }
};

// The table's row for a token, or null (recorded): such tokens are not turned.
__device__ __forceinline__ const float* table_row(const RotaryParams& p, int64_t token, int64_t place) {
    const int64_t at = p.positions ? p.positions[token] : place;
    if (at >= 0 && at < p.num_positions) return p.table + at * p.rot;
    report(p.c.status, kStatusBadIndex);
    return nullptr;
}

// All values of an item finite?
__device__ __forceinline__ bool finite16(const float (&lo)[8], const float (&hi)[8]) {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) ok &= fabsf(lo[i]) < INFINITY && fabsf(hi[i]) < INFINITY;
    return ok;
}

// Item j of one head of q, from src to dst (which may be the same).
template <typename T>
__device__ __forceinline__ void turn_q(const uint4& a, const uint4& b, uint4* dst, const Item& it, const Angles& angles, bool turns) {
    if (turns) {
        float lo[8], hi[8];
        unpack<T>(a, lo);
        unpack<T>(b, hi);
        angles.turn(lo, hi, it.side);
        dst[it.lo] = pack8<T>(lo);
        dst[it.hi] = pack8<T>(hi);
    } else {
        dst[it.lo] = a;
        dst[it.hi] = b;
    }
}

// One token a row (the decode step).  Warps of the first blocks have a (row, head, k or v) each, as in
// kda_kvcache_append.cu; then a warp has a row and as many heads of q as it has lanes for.
template <typename T, int kDim>
__global__ void __launch_bounds__(kStepWarps * 32) rotary_step_kernel(const __grid_constant__ RotaryParams p) {
    follow_stream();
    const CacheParams& c = p.c;
    constexpr int kItems = kDim / 16, kHeads = 32 / kItems;
    struct Growth {
        uint8_t* codes;
        int bytes;  // 0: none
        float was, now;
    };
    __shared__ Growth s_growth[kStepWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % kItems;
    const int64_t first_q = (2 * c.tokens * c.heads + kStepWarps - 1) / kStepWarps;  // block
    if (blockIdx.x >= first_q) {
        const int sets = (p.q_heads + kHeads - 1) / kHeads;
        const int64_t w = (blockIdx.x - first_q) * kStepWarps + warp;
        const int64_t row = w / sets;
        const int head = (int)(w % sets) * kHeads + lane / kItems;
        if (row >= c.tokens || head >= p.q_heads) return;
        const Item it(j, p.rot, p.interleaved);
        const float* angle_row = table_row(p, row, c.lens[row]);
        const bool turns = it.turns && angle_row;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + row * p.q_stride + (int64_t)head * kDim);
        const uint4 a = src[it.lo], b = src[it.hi];
        Angles angles;
        if (turns) angles.read(angle_row, p.rot, j);
        turn_q<T>(a, b, reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + row * p.out_stride + (int64_t)head * kDim), it, angles, turns);
        return;
    }
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
            const bool mine = lane < kItems;
            const Item it(j, which ? 0 : p.rot, p.interleaved);
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x[which]) + row * p.stride[which] + (int64_t)head * kDim);
            uint4 a4 = make_uint4(0u, 0u, 0u, 0u), b4 = a4;
            if (mine) a4 = src[it.lo], b4 = src[it.hi];
            float lo[8], hi[8];
            unpack<T>(a4, lo);
            unpack<T>(b4, hi);
            if (mine && it.turns) {
                const float* angle_row = table_row(p, row, len);
                if (angle_row) {
                    Angles angles;
                    angles.read(angle_row, p.rot, j);
                    angles.turn(lo, hi, it.side);
                }
            }
            if (!finite16(lo, hi)) report(c.status, kStatusNonfinite);
            float a = fmaxf(largest(lo), largest(hi));
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
            if (mine) {
                uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)off * kDim);
                dst[it.lo] = encode(lo, s);
                dst[it.hi] = encode(hi, s);
            }
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

// Several tokens a row: blocks of a page as in kda_kvcache_append.cu (row r's i-th touched page has
// number cu[r] / page_tokens + 2 r + i), blockIdx.y: heads of k, heads of v, then sets of q's heads for the
// same tokens.
template <typename T, int kDim, int kPage>
__global__ void __launch_bounds__(kThreads, kDim * kPage <= 8192 ? 4 : 2) rotary_kernel(const __grid_constant__ RotaryParams p) {
    follow_stream();
    const CacheParams& c = p.c;
    constexpr int kItems = kDim / 16;
    constexpr int kTokens = kPage < kThreads / kItems ? kPage : kThreads / kItems;  // of a pass
    constexpr int kSets = kThreads / (kItems * kTokens);  // sets of threads that have the same tokens
    constexpr int kPasses = kPage / kTokens;
    __shared__ float red[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, j = tid % kItems, set = tid / (kItems * kTokens), t0 = tid / kItems % kTokens;
    const int64_t unit = blockIdx.x;

    // The last row whose numbers start at or before this unit; all warps search alike.
    int lo_row = 0, hi_row = c.rows;
    while (hi_row - lo_row > 1) {
        const int step = (hi_row - lo_row + 32) / 33, r = lo_row + step * (lane + 1);
        const bool below = r < hi_row && c.cu[r] / kPage + 2ll * r <= unit;
        const int n = __popc(__ballot_sync(0xffffffffu, below));
        const int next = lo_row + step * (n + 1);
        lo_row += step * n;
        if (next < hi_row) hi_row = next;
    }
    const int row = lo_row;
    const int64_t begin = c.cu[row], end = c.cu[row + 1];
    if (begin < 0 || end < begin || end > c.tokens || (row == 0 && begin != 0) || (row == c.rows - 1 && end != c.tokens)) {
        if (tid == 0) report(c.status, kStatusBadSeqlens);
        return;
    }
    const int64_t i = unit - (begin / kPage + 2ll * row);
    const int32_t len = c.lens[row];
    const bool is_q = (int)blockIdx.y >= 2 * c.heads;
    // (Tokens of a row of negative length have no pages; their queries are turned by their places from 0 on.)
    if (len < 0 && tid == 0) report(c.status, kStatusBadIndex);
    if (i < 0 || (len < 0 && !is_q)) return;
    const int32_t held = max(len, 0);
    const int64_t slot = held / kPage + i;               // of the row's table
    const int64_t p0 = slot * kPage;                     // position of the page's first token
    const int64_t first = p0 > held ? p0 : held;         // first new position in the page
    const int64_t last = min(p0 + kPage, held + (end - begin));
    if (first >= last) return;
    const int n = (int)(last - first), off = (int)(first - p0);
    const int64_t token0 = begin + first - held, place0 = first - held + len;

    if (is_q) {
        const Item it(j, p.rot, p.interleaved);
        const int head0 = ((int)blockIdx.y - 2 * c.heads) * kQHeads * kSets, head1 = min(p.q_heads, head0 + kQHeads * kSets);
        for (int t = t0; t < n; t += kTokens) {
            const int64_t token = token0 + t;
            const float* angle_row = table_row(p, token, place0 + t);
            const bool turns = it.turns && angle_row;
            Angles angles;
            if (turns) angles.read(angle_row, p.rot, j);
            const T* src = static_cast<const T*>(p.q) + token * p.q_stride;
            T* dst = static_cast<T*>(p.q_out) + token * p.out_stride;
            constexpr int kAhead = 2;  // heads whose loads are under way
            for (int h0 = head0 + set; h0 < head1; h0 += kAhead * kSets) {
                uint4 a[kAhead], b[kAhead];
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    const int h = h0 + x * kSets;
                    if (h >= head1) continue;
                    const uint4* s = reinterpret_cast<const uint4*>(src + (int64_t)h * kDim);
                    a[x] = __ldcs(s + it.lo);
                    b[x] = __ldcs(s + it.hi);
                }
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    const int h = h0 + x * kSets;
                    if (h < head1) turn_q<T>(a[x], b[x], reinterpret_cast<uint4*>(dst + (int64_t)h * kDim), it, angles, turns);
                }
            }
        }
        return;
    }

    const int which = (int)blockIdx.y >= c.heads, head = (int)blockIdx.y - which * c.heads;
    const int32_t page = slot < c.width ? c.tables[(int64_t)row * c.width + slot] : -1;
    if (page < 0 || page >= c.pages) {
        if (tid == 0) report(c.status, kStatusBadIndex);
        return;
    }
    const Item it(j, which ? 0 : p.rot, p.interleaved);
    const int64_t stride = p.stride[which];
    const T* src = static_cast<const T*>(p.x[which]) + token0 * stride + (int64_t)head * kDim;
    const bool works = set == 0;  // (of small pages half the threads have none of the values)
    float lo[kPasses][8], hi[kPasses][8];
    uint4 ra[kPasses], rb[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int t = t0 + k * kTokens;
        const uint4* s = reinterpret_cast<const uint4*>(src + t * stride);
        const bool there = works && t < n;
        ra[k] = there ? __ldcs(s + it.lo) : make_uint4(0u, 0u, 0u, 0u);
        rb[k] = there ? __ldcs(s + it.hi) : make_uint4(0u, 0u, 0u, 0u);
    }
    float a = 0.f;
    bool finite = true;  // all values of this thread
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int t = t0 + k * kTokens;
        unpack<T>(ra[k], lo[k]);
        unpack<T>(rb[k], hi[k]);
        if (it.turns && works && t < n) {
            const float* angle_row = table_row(p, token0 + t, first + t);
            if (angle_row) {
                Angles angles;
                angles.read(angle_row, p.rot, j);
                angles.turn(lo[k], hi[k], it.side);
            }
        }
        finite &= finite16(lo[k], hi[k]);
        a = fmaxf(a, fmaxf(largest(lo[k]), largest(hi[k])));
    }
    if (!finite) report(c.status, kStatusNonfinite);
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) red[tid >> 5] = a;
    const int64_t block = (int64_t)page * c.heads + head;
    float* scale = (which ? c.v_scale : c.k_scale) + block;
    uint8_t* codes = (which ? c.v_codes : c.k_codes) + block * kPage * kDim;
    const float was = off > 0 ? *scale : 0.f;
    __syncthreads();  // the maxima are there, and every thread has read the scale
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a = fmaxf(a, red[w]);
    float s = __fdiv_rn(a, kCodeMax);
    const bool grown = off > 0 && s > was;
    if (off > 0 && !grown) s = was;
    if (tid == 0) *scale = s;
    const bool quick = finite && short_division(s);
    const float r = __frcp_rn(s);
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int t = t0 + k * kTokens;
        if (!works || t >= n) continue;
        uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)(off + t) * kDim);
        dst[it.lo] = quick ? encode_short(lo[k], s, r) : encode(lo[k], s);
        dst[it.hi] = quick ? encode_short(hi[k], s, r) : encode(hi[k], s);
    }
    if (grown) grade_again<kThreads>(codes, off * kDim, was, s, tid);
}

template <typename T, int kDim>
cudaError_t launch_dim(const RotaryParams& p, cudaStream_t stream) {
    const CacheParams& c = p.c;
    constexpr int kItems = kDim / 16;
    if (!c.cu) {
        const int64_t kv = (2 * c.tokens * c.heads + kStepWarps - 1) / kStepWarps;
        const int64_t sets = (p.q_heads + 32 / kItems - 1) / (32 / kItems);
        const int64_t q = (c.tokens * sets + kStepWarps - 1) / kStepWarps;
        return launch_early(rotary_step_kernel<T, kDim>, dim3((unsigned)(kv + q)), kStepWarps * 32, 0, stream, 1, p);
    }
    const int sets = c.page_tokens < kThreads / kItems ? kThreads / (kItems * c.page_tokens) : 1;
    const dim3 grid((unsigned)(c.tokens / c.page_tokens + 2ll * c.rows), 2 * c.heads + (p.q_heads + kQHeads * sets - 1) / (kQHeads * sets));
    const auto kernel = c.page_tokens == 16   ? rotary_kernel<T, kDim, 16>
                        : c.page_tokens == 32 ? rotary_kernel<T, kDim, 32>
                        : c.page_tokens == 64 ? rotary_kernel<T, kDim, 64>
                                              : rotary_kernel<T, kDim, 128>;
    return launch_early(kernel, grid, kThreads, 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryParams& p, bool f16, cudaStream_t stream) {
    if (p.c.tokens == 0 || p.c.rows == 0) return cudaSuccess;
    if (p.c.dim == 64) return f16 ? launch_dim<__half, 64>(p, stream) : launch_dim<__nv_bfloat16, 64>(p, stream);
    return f16 ? launch_dim<__half, 128>(p, stream) : launch_dim<__nv_bfloat16, 128>(p, stream);
}

}  // namespace kda
