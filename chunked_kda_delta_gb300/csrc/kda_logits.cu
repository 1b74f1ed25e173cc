// kda_logits.cu -- penalties for repeated tokens, biases and grammar masks on logits.
//
// Per row and token t, with `seen` the tokens of the row's history and c(t) how often t is in it
// behind the prompt:
//   x = x > 0 ? x / r : x r   where seen;  x = x - f c(t) - p [c(t) > 0];  x = x + b(t);
//   x = -inf                  where the row's mask has no bit.
// fp32, rounded once; a token that nothing applies to keeps its bits.
//
// HBM-bound: the logits are read and written once, mask bits and histories beside them.  Few tokens of
// a vocabulary are touched by histories and biases, so two kinds of warps share a CTA's segment of a row:
//   half of them copy the segment and put -inf where the mask says so (in place they read only loads of 16 bytes
//   that the mask takes in part, and write none that it leaves alone);
//   the others count the touched tokens in shared memory, by their place in the segment or, in long segments
//   with short histories, in a hash table (linear probing, a third of it free), work them out from the logits as
//   they came, and store them when the copy is done.
// Counts are whole numbers, so their order does not matter; biases of one token are added in the order of
// the list.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "kda_ptx.cuh"
#include "kda_serving.cuh"

namespace kda {
namespace {

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

// Bits of the tokens t .. t + kEach - 1 that lie in a row of the vocabulary.
template <int kEach>
__device__ __forceinline__ uint32_t inside(int t, int vocab) {
    uint32_t bits = (1u << kEach) - 1;
    if (t < 0) bits = bits >> -t << -t;
    if (t + kEach > vocab) bits &= t < vocab ? (1u << (vocab - t)) - 1 : 0u;
    return bits;
}
// The lowest value where a token's bit is not set.
template <typename T>
__device__ __forceinline__ void take_out(uint4& v, uint32_t pass) {
    if constexpr (sizeof(T) == 4) {
        if (!(pass & 1)) v.x = Logit<T>::rounded(-INFINITY);
        if (!(pass & 2)) v.y = Logit<T>::rounded(-INFINITY);
        if (!(pass & 4)) v.z = Logit<T>::rounded(-INFINITY);
        if (!(pass & 8)) v.w = Logit<T>::rounded(-INFINITY);
    } else {
        const uint32_t low = Logit<T>::rounded(-INFINITY) * 0x10001u;
        auto two = [&](uint32_t& u, uint32_t bits) {
            const uint32_t keep = ((bits & 1) | (bits & 2) << 15) * 0xffffu;
            u = (u & keep) | (low & ~keep);
        };
        two(v.x, pass);
        two(v.y, pass >> 2);
        two(v.z, pass >> 4);
        two(v.w, pass >> 6);
    }
}

constexpr int kHalf = 256, kThreads = 2 * kHalf;  // threads of a kind
constexpr int kVecs = 4;                            // 16-byte loads of a thread under way
constexpr int kResident = 2;                        // CTAs an SM
constexpr uint32_t kBarTable = 1;

constexpr int kRing = 3;                            // chunks of a longer segment under way
constexpr uint32_t kBarCopy = 2;
constexpr int64_t kWaitLimit = 1ll << 20;

// The tokens of a segment: [t0, t0 + reach) as far as they lie in the row.
template <typename Raw>
struct Segment {
    const Raw* src;
    Raw* dst;
    const uint32_t* mask;
    int t0, reach, vocab;
};

// Bits of the tokens t .. t + kEach - 1, some in the row (`in`), that the mask lets through.
template <int kEach>
__device__ __forceinline__ uint32_t allowed(const uint32_t* mask, int t, uint32_t in, int vocab) {
    if (!mask || !in) return in;
    if (t >= 0 && t % kEach == 0) return __ldg(reinterpret_cast<const uint8_t*>(mask) + t / 8) >> (t % 8) & in;
    const int from = max(t, 0), word = from >> 5, shift = from & 31;
    const uint32_t lo = __ldg(mask + word), hi = shift + kEach > 32 && (word + 1) * 32 < vocab ? __ldg(mask + word + 1) : 0u;
    return __funnelshift_r(lo, hi, shift) << (from - t) & in;
}

// The copy of the tokens [at, at + kVecs * kCopy loads) of a segment, by kCopy threads; through registers.
template <typename T, int kCopy, typename Raw>
__device__ __forceinline__ void copy_piece(const Segment<Raw>& g, int at, int end, int tid) {
    constexpr int kEach = 16 / sizeof(Raw), kUnit = kCopy * kEach;
    constexpr uint32_t kAll = (1u << kEach) - 1;
    const bool place = g.src == g.dst;
    const bool even = (((uintptr_t)g.src ^ (uintptr_t)g.dst) & 15) == 0;  // src has dst's 16-byte boundaries too
    uint32_t in[kVecs], pass[kVecs];
    uint4 x[kVecs];
    const bool whole = g.t0 + at >= 0 && at + kVecs * kUnit <= end;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int t = g.t0 + at + k * kUnit + tid * kEach;
        in[k] = whole ? kAll : at + k * kUnit < end ? inside<kEach>(t, g.vocab) : 0u;
        pass[k] = allowed<kEach>(g.mask, t, in[k], g.vocab);
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int t = g.t0 + at + k * kUnit + tid * kEach;
        if (place && pass[k] == in[k]) in[k] = 0;  // nothing to do
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (!in[k] || !pass[k]) continue;
        if (even && in[k] == kAll) {
            x[k] = *reinterpret_cast<const uint4*>(g.src + t);
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (in[k] >> i & 1) set<Raw>(x[k], i, g.src[t + i]);
        }
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int t = g.t0 + at + k * kUnit + tid * kEach;
        if (!in[k]) continue;
        if (pass[k] != kAll) take_out<T>(x[k], pass[k]);
        if (in[k] == kAll) {
            *reinterpret_cast<uint4*>(g.dst + t) = x[k];
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (in[k] >> i & 1) g.dst[t + i] = get<Raw>(x[k], i);
        }
    }
}

// The copy of a segment by kCopy threads.  Longer ones come through a ring of chunks in shared memory, as many
// bytes under way as HBM wants without a register for each.
template <typename T, int kCopy, typename Raw>
__device__ __forceinline__ void copy_segment(const Segment<Raw>& g, unsigned char* ring, uint64_t* s_bar, int32_t* status, int tid) {
    constexpr int kEach = 16 / sizeof(Raw), kUnit = kCopy * kEach, kChunk = kVecs * kUnit;
    if (g.src == g.dst && !g.mask) return;
    const int end = min(g.reach, g.vocab - g.t0);
    const bool even = (((uintptr_t)g.src ^ (uintptr_t)g.dst) & 15) == 0;
    if (!ring || g.src == g.dst || !even) {
        for (int at = 0; at < end; at += kChunk) copy_piece<T, kCopy>(g, at, end, tid);
        return;
    }
    // Whole loads of 16 bytes in the row: [first, last) of the segment; what is left has less than a load at
    // either end.
    const int first = g.t0 < 0 ? kEach : 0, last = end / kEach * kEach, chunks = (last - first + kChunk - 1) / kChunk;
    if (tid < 2 * kEach) {
        const int t = tid < kEach ? (first ? g.t0 + tid : -1) : (g.t0 + last + tid - kEach < g.t0 + end ? g.t0 + last + tid - kEach : -1);
        if (t >= 0) g.dst[t] = allowed<1>(g.mask, t, 1u, g.vocab) ? g.src[t] : Logit<T>::rounded(-INFINITY);
    }
    const uint32_t ring_at = ptx::smem_u32(ring), bar = ptx::smem_u32(s_bar);
    auto request = [&](int c) {
        const uint32_t bytes = (uint32_t)min(kChunk, last - first - c * kChunk) * sizeof(Raw), slot = c % kRing;
        ptx::mbar_arrive_expect_tx(bar + 8 * slot, bytes);
        ptx::bulk_load(ring_at + slot * (kChunk * sizeof(Raw)), g.src + g.t0 + first + c * kChunk, bytes, bar + 8 * slot);
    };
    if (tid == 0)
        for (int c = 0; c < min(kRing, chunks); ++c) request(c);
    uint32_t pass[kVecs], next[kVecs];
    auto masks = [&](int c, uint32_t (&bits)[kVecs]) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int at = first + c * kChunk + k * kUnit + tid * kEach;
            bits[k] = at < last ? allowed<kEach>(g.mask, g.t0 + at, (1u << kEach) - 1, g.vocab) : 0u;
        }
    };
    masks(0, next);
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
        const uint32_t slot = c % kRing;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) pass[k] = next[k];
        if (c + 1 < chunks) masks(c + 1, next);
        // (After a wait that ran out nothing more is asked for, and what follows is garbage.)
        ok = ptx::mbar_wait_now(bar + 8 * slot, c / kRing & 1, ok ? kWaitLimit : 1024) && ok;
        uint4 x[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) x[k] = reinterpret_cast<const uint4*>(ring + slot * (kChunk * sizeof(Raw)))[k * kCopy + tid];
        if (c + kRing < chunks) {
            ptx::named_bar_sync(kBarCopy, kCopy);  // everyone has read the slot
            if (tid == 0 && ok) request(c + kRing);
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int at = first + c * kChunk + k * kUnit + tid * kEach;
            if (at >= last) continue;
            if (pass[k] != (1u << kEach) - 1) take_out<T>(x[k], pass[k]);
            *reinterpret_cast<uint4*>(g.dst + g.t0 + at) = x[k];
        }
    }
    if (!ok) report(status, kStatusTimeout);
}

// The touched tokens, in entries of shared memory: by their place in the segment (p.direct), or hashed.
struct Table {
    int32_t* key;     // tokens, -1 where there is none
    uint32_t* word;   // counts, later the logit's bits
    float* sum;       // of the biases
    int entries, shift, t0;
    bool direct;
    __device__ __forceinline__ uint32_t entry(int32_t token) const {
        if (direct) {
            key[token - t0] = token;
            return token - t0;
        }
        uint32_t at = (uint32_t)token * 0x9e3779b1u >> shift;
        for (;; at = (at + 1) & (entries - 1)) {  // (ends: a third of the entries stays free)
            const int32_t k = key[at];
            if (k == token) return at;
            if (k >= 0) continue;
            const int32_t old = atomicCAS(key + at, -1, token);
            if (old < 0 || old == token) return at;
        }
    }
};
// What a thread reads of its row before it does anything else: loads take a microsecond and more while the
// copies keep the memory busy, so none waits for another.
struct Touches {
    static constexpr int kKept = 2;
    int len, prompt, head;
    const int32_t* history;
    int4 quad[kKept];        // of the history, whatever its length
    int32_t edge[2];         // before and behind the loads of 16 bytes
    int32_t bias_token;
    float bias_value;
    Penalties rules;
    template <int kCount>
    __device__ __forceinline__ void read(const LogitsParams& p, int64_t row, int tid) {
        len = p.width > 0 && p.lens ? p.lens[row] : p.width;
        prompt = p.width > 0 && p.prompt_lens ? p.prompt_lens[row] : 0;
        history = p.history + row * p.width;
        // Loads of 16 bytes where the rows have their boundaries.
        head = min(p.width, (int)((16 - ((uintptr_t)history & 15)) % 16 / 4));
        const int quads = (p.width - head) / 4, tail = head + 4 * quads + tid;
        edge[0] = tid < head ? __ldg(history + tid) : -1;
        edge[1] = tail < p.width ? __ldg(history + tail) : -1;
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            quad[k] = k * kCount + tid < quads ? __ldg(reinterpret_cast<const int4*>(history + head) + k * kCount + tid) : make_int4(-1, -1, -1, -1);
        bias_token = tid < p.num_bias ? p.bias_tokens[row * p.num_bias + tid] : -1;
        bias_value = tid < p.num_bias ? p.bias[row * p.num_bias + tid] : 0.f;
        rules = Penalties{p.repetition ? p.repetition[row] : 1.f, p.presence ? p.presence[row] : 0.f, p.frequency ? p.frequency[row] : 0.f};
    }
};

// Counts them and works them out, by kCount threads.
template <typename T, int kCount, typename Raw>
__device__ __forceinline__ void touch_segment(const LogitsParams& p, const Segment<Raw>& g, const Table& table, Touches& own, int64_t row, int tid) {
    using L = Logit<T>;
    __shared__ int32_t s_token[kCount];
    __shared__ float s_value[kCount];
    __shared__ int s_counts[kCount / 32];
    const int lane = tid & 31, warp = tid >> 5;
    auto sync = [] { ptx::named_bar_sync(kBarTable, kCount); };
    bool bad = false;
    auto ours = [&](int32_t token) {
        bad |= token >= p.vocab;
        return token >= max(g.t0, 0) && token < p.vocab && token - g.t0 < g.reach;
    };
    // The few logits of a hash table are asked for right away.
    auto entry = [&](int32_t token) {
        if (!table.direct) asm volatile("prefetch.global.L2 [%0];" ::"l"(g.src + token));
        return table.entry(token);
    };
    if ((own.len < 0 || own.len > p.width) && tid == 0) report(p.status, kStatusBadIndex);
    const int len = max(0, min(own.len, p.width)), prompt = max(0, min(own.prompt, len));
    auto count = [&](int32_t token, int i) {
        if (i >= len || !ours(token)) return;
        uint32_t* word = table.word + entry(token);
        if (i < prompt) atomicOr(word, kPrompt);
        else atomicAdd(word, 1u);
    };
    auto count4 = [&](const int4& q, int i) {
        count(q.x, i);
        count(q.y, i + 1);
        count(q.z, i + 2);
        count(q.w, i + 3);
    };
    if (len > 0) {
        const int quads = (p.width - own.head) / 4;
        count(own.edge[0], tid);
        count(own.edge[1], own.head + 4 * quads + tid);
#pragma unroll
        for (int k = 0; k < Touches::kKept; ++k) count4(own.quad[k], own.head + 4 * (k * kCount + tid));
        constexpr int kAhead = 4;
        const int used = min(quads, (len - own.head + 3) / 4);
        for (int i0 = Touches::kKept * kCount + tid; i0 < used; i0 += kAhead * kCount) {
            int4 q[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                q[k] = i0 + k * kCount < used ? __ldg(reinterpret_cast<const int4*>(own.history + own.head) + i0 + k * kCount) : make_int4(-1, -1, -1, -1);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) count4(q[k], own.head + 4 * (i0 + k * kCount));
        }
    }
    // Biases, as many at a time as there are threads: those of this segment side by side, in order; the first of
    // each token adds up all of them.
    for (int i0 = 0; i0 < p.num_bias; i0 += kCount) {
        int32_t token = own.bias_token;
        float value = own.bias_value;
        if (i0 > 0) {
            token = i0 + tid < p.num_bias ? p.bias_tokens[row * p.num_bias + i0 + tid] : -1;
            value = i0 + tid < p.num_bias ? p.bias[row * p.num_bias + i0 + tid] : 0.f;
        }
        const bool mine = ours(token);
        const uint32_t some = __ballot_sync(0xffffffffu, mine);
        if (i0 > 0) sync();  // (the round before is over)
        if (lane == 0) s_counts[warp] = __popc(some);
        sync();
        int slot = __popc(some & ((1u << lane) - 1)), n = 0;
#pragma unroll
        for (int w = 0; w < kCount / 32; ++w) {
            if (w < warp) slot += s_counts[w];
            n += s_counts[w];
        }
        if (mine) {
            s_token[slot] = token;
            s_value[slot] = value;
        }
        sync();
        if (tid < n) {
            const int32_t t = s_token[tid];
            bool leads = true;  // the first with this token
#pragma unroll 8
            for (int i = 0; i < tid; ++i) leads &= s_token[i] != t;
            if (leads) {
                const uint32_t at = entry(t);
                float sum = table.word[at] & kBiased ? table.sum[at] + s_value[tid] : s_value[tid];
#pragma unroll 8
                for (int i = tid + 1; i < n; ++i) sum = s_token[i] == t ? sum + s_value[i] : sum;
                table.sum[at] = sum;
                atomicOr(table.word + at, kBiased);
            }
        }
    }
    if (bad) report(p.status, kStatusBadIndex);
    Penalties rules = own.rules;
    if (!(rules.repetition > 0.f && rules.repetition < INFINITY && fabsf(rules.presence) < INFINITY && fabsf(rules.frequency) < INFINITY)) {
        if (tid == 0) report(p.status, kStatusBadIndex);
        rules = Penalties{1.f, 0.f, 0.f};
    }
    sync();
    // The touched logits, which take their words' place; those that the mask takes are left out.
    constexpr int kTouched = 8;
    for (int i0 = tid; i0 < table.entries; i0 += kTouched * kCount) {
        int32_t token[kTouched];
        Raw y[kTouched];
        uint32_t bits[kTouched];
#pragma unroll
        for (int k = 0; k < kTouched; ++k) {
            const int i = i0 + k * kCount;
            token[k] = i < table.entries ? table.key[i] : -1;
            bits[k] = ~0u;
            if (token[k] < 0) continue;
            y[k] = g.src[token[k]];
            if (g.mask) bits[k] = __ldg(g.mask + (token[k] >> 5));
        }
#pragma unroll
        for (int k = 0; k < kTouched; ++k) {
            const int i = i0 + k * kCount;
            if (token[k] < 0) continue;
            const uint32_t word = table.word[i];
            if (bits[k] >> (token[k] & 31) & 1) table.word[i] = L::rounded(rules.apply(L::value(y[k]), word, word & kBiased ? table.sum[i] : 0.f));
            else table.key[i] = -1;
        }
    }
}

// kTouches 1: each half of the threads has its kind of work; 2 (segments of few loads): all do the one, then the
// other.
template <typename T, int kTouches>
__global__ void __launch_bounds__(kThreads, kResident) penalize_kernel(const __grid_constant__ LogitsParams p) {
    using Raw = typename Logit<T>::Raw;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(8) uint64_t s_bar[kRing];
    const int tid = threadIdx.x;
    const size_t table_bytes = (size_t)p.entries * (p.num_bias > 0 ? 12 : 8);
    Table table{reinterpret_cast<int32_t*>(smem), reinterpret_cast<uint32_t*>(smem) + p.entries, reinterpret_cast<float*>(smem) + 2 * p.entries,
                p.entries, p.shift, 0, p.direct};
    if (kTouches)
        for (int i = tid; i < p.entries / 4; i += kThreads) {
            reinterpret_cast<int4*>(table.key)[i] = make_int4(-1, -1, -1, -1);
            reinterpret_cast<uint4*>(table.word)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) ptx::mbar_init(ptx::smem_u32(s_bar + i), 1);
        ptx::fence_mbar_init();
    }
    follow_stream();
    const int64_t row = blockIdx.x / p.segs;
    Segment<Raw> g;
    g.src = static_cast<const Raw*>(p.logits) + row * p.stride;
    g.dst = static_cast<Raw*>(p.out) + row * p.out_stride;
    g.mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
    g.reach = p.seg_len;
    g.vocab = p.vocab;
    // Segments begin at 16-byte boundaries of dst; the first may begin before the row.
    g.t0 = (int)(blockIdx.x % p.segs) * p.seg_len - (int)(((uintptr_t)g.dst & 15) / sizeof(Raw));
    if (g.t0 >= p.vocab) return;
    table.t0 = g.t0;
    unsigned char* ring = p.ring ? smem + table_bytes : nullptr;
    Touches own;
    if (kTouches == 2 || (kTouches == 1 && tid < kHalf)) own.read<kTouches == 1 ? kHalf : kThreads>(p, row, tid);
    __syncthreads();
    if constexpr (kTouches != 1) copy_segment<T, kThreads>(g, ring, s_bar, p.status, tid);
    if constexpr (kTouches == 1) {
        if (tid >= kHalf) copy_segment<T, kHalf>(g, ring, s_bar, p.status, tid - kHalf);
        else touch_segment<T, kHalf>(p, g, table, own, row, tid);
    } else if constexpr (kTouches == 2) {
        touch_segment<T, kThreads>(p, g, table, own, row, tid);
    }
    if constexpr (kTouches != 0) {
        __syncthreads();
        for (int i = 4 * tid; i < p.entries; i += 4 * kThreads) {
            const int4 keys = *reinterpret_cast<const int4*>(table.key + i);
            const uint4 words = *reinterpret_cast<const uint4*>(table.word + i);
            if (keys.x >= 0) g.dst[keys.x] = (Raw)words.x;
            if (keys.y >= 0) g.dst[keys.y] = (Raw)words.y;
            if (keys.z >= 0) g.dst[keys.z] = (Raw)words.z;
            if (keys.w >= 0) g.dst[keys.w] = (Raw)words.w;
        }
    }
}

constexpr int kMostEntries = 8192;  // of a table: 96 KB with biases

template <typename T>
cudaError_t launch_type(LogitsParams& p, cudaStream_t stream) {
    const int64_t touches = (int64_t)p.width + p.num_bias;
    const bool place = p.out == p.logits;
    if (place && !p.mask && touches == 0) return cudaSuccess;
    const int each = 16 / sizeof(T), unit = kHalf * each;
    const bool even = ((uintptr_t)p.out & 15) == 0 && (p.out_stride * sizeof(T) & 15) == 0;
    // Segments of whole units, as few as fill the CTAs' places well; in place, where it is the chain of loads that
    // counts, of a chunk.
    const int64_t span = (int64_t)p.vocab + (even ? 0 : each - 1), units = (span + unit - 1) / unit, places = (int64_t)kResident * p.sm_count;
    int64_t segs = 1;
    double best = 0;
    for (int64_t n = 1; n <= units && (n == 1 || p.rows * n <= 8 * places) && best < 0.8; ++n) {
        const double waves = (double)(p.rows * n) / places, use = waves / ceil(waves);
        if (use > best) best = use, segs = n;
    }
    int64_t len = (units + segs - 1) / segs * unit;
    if (place && !touches && len > 2 * kVecs * unit) len = 2 * kVecs * unit;
    // A table holds the most tokens that a segment can have touched: hashed with a third of it free.
    const bool hashed = 3 * touches <= 2 * kMostEntries;
    if (!hashed && len > kMostEntries) len = kMostEntries;
    p.seg_len = (int32_t)len;
    p.segs = (int32_t)((span + len - 1) / len);
    p.entries = 0;
    if (touches > 0) {
        int log = 8;
        while (hashed && (int64_t)2 << log < 3 * touches) ++log;
        p.shift = 32 - log;
        p.direct = !hashed || len <= (int64_t)1 << log;
        p.entries = p.direct ? (int32_t)len : 1 << log;
    }
    // With touched tokens, halves of the threads where the copy is long enough to hide the other half's work.
    const int chunk = kVecs * unit * (touches ? 1 : 2);
    p.ring = !place && len > chunk;
    const auto kernel = !touches ? penalize_kernel<T, 0> : p.ring ? penalize_kernel<T, 1> : penalize_kernel<T, 2>;
    const size_t smem = (size_t)p.entries * (p.num_bias > 0 ? 12 : 8) + (p.ring ? (size_t)kRing * chunk * sizeof(T) : 0);
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, dim3((unsigned)(p.rows * p.segs)), kThreads, smem, stream, 1, p);
}

}  // namespace

cudaError_t launch_penalize(LogitsParams p, int dtype, cudaStream_t stream) {
    if (dtype == 0) return launch_type<float>(p, stream);
    return dtype == 1 ? launch_type<__nv_bfloat16>(p, stream) : launch_type<__half>(p, stream);
}

}  // namespace kda
