// kda_logits.cu -- penalties for repeated tokens, biases and grammar masks on logits.
//
// Per row and token t, with `seen` the tokens of the row's history and c(t) how often t is in it
// behind the prompt:
//   x = x > 0 ? x / r : x r   where seen;  x = x - f c(t) - p [c(t) > 0];  x = x + b(t);
//   x = -inf                  where the row's mask has no bit.
// fp32, rounded once; a token that nothing applies to keeps its bits.
//
// HBM-bound: the logits are read and written once, mask bits and histories beside them.  Few tokens of
// a vocabulary are touched by histories and biases: a CTA counts those of its segment of a row in shared memory,
// by their place in the segment or, in long segments with short histories, in a hash table (linear probing, a
// third of it free), while bulk copies bring the first chunks of the segment; touched and masked logits are
// changed in the chunks, which leave by bulk copies.  (To fetch and store them one by one beside the copy is
// a memory request each: for 256 rows of 131072 bf16 with 2000 tokens each, 100 biases and a mask 42.8 us.  So it
// is 34.4, 3.9 TB/s: the copy alone takes 24.6, the count before it, in which only the first chunks come, most
// of the rest, latency of shared memory and of first instructions.)  In place, and
// where out's 16-byte boundaries are not those of the logits, through registers: in place only loads of 16
// bytes that the mask takes in part are read, and none written that it leaves alone.
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

constexpr int kThreads = 512;
constexpr int kUnitLoads = 256;                     // segments are whole multiples of as many loads of 16 bytes
constexpr int kVecs = 4;                            // 16-byte loads of a thread under way
constexpr int kResident = 2;                        // CTAs an SM
constexpr int kRing = 3, kChunkBytes = 16384;       // chunks of a segment under way
constexpr int kMostChunks = 64;                     // of a segment
constexpr int64_t kWaitLimit = 1ll << 14;

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

// The copy of the tokens [at, at + kVecs * kThreads loads) of a segment, through registers.
template <typename T, typename Raw>
__device__ __forceinline__ void copy_piece(const Segment<Raw>& g, int at, int end, int tid) {
    constexpr int kEach = 16 / sizeof(Raw), kUnit = kThreads * kEach;
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

template <typename T, typename Raw>
__device__ __forceinline__ void copy_segment(const Segment<Raw>& g, int tid) {
    if (g.src == g.dst && !g.mask) return;
    const int end = min(g.reach, g.vocab - g.t0);
    for (int at = 0; at < end; at += kVecs * kThreads * (16 / (int)sizeof(Raw))) copy_piece<T>(g, at, end, tid);
}

// The touched tokens, in entries of shared memory: by their place in the segment (p.direct), or hashed.
struct Table {
    int32_t* key;     // tokens, -1 where there is none
    uint32_t* word;   // counts, later the logit's bits
    float* sum;       // of the biases
    int entries, shift, t0;
    bool direct;
    int* tokens;      // touched ones of each chunk; NULL: not counted
    int first, last, log_chunk;
    // 0 for the tokens before the chunks, kMostChunks + 1 for those behind.
    __device__ __forceinline__ int chunk_of(int32_t token) const {
        const int at = token - t0;
        return at < first ? 0 : at >= last ? kMostChunks + 1 : 1 + ((at - first) >> log_chunk);
    }
    __device__ __forceinline__ uint32_t entry(int32_t token) const {
        if (direct) {
            if (tokens) {
                if (atomicExch(key + token - t0, token) < 0) atomicAdd(tokens + chunk_of(token), 1);
            } else {
                key[token - t0] = token;
            }
            return token - t0;
        }
        uint32_t at = (uint32_t)token * 0x9e3779b1u >> shift;
        for (;; at = (at + 1) & (entries - 1)) {  // (ends: a third of the entries stays free)
            const int32_t old = atomicCAS(key + at, -1, token);
            if (old < 0 && tokens) atomicAdd(tokens + chunk_of(token), 1);
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
            quad[k] = k * kThreads + tid < quads ? __ldg(reinterpret_cast<const int4*>(history + head) + k * kThreads + tid) : make_int4(-1, -1, -1, -1);
        bias_token = tid < p.num_bias ? p.bias_tokens[row * p.num_bias + tid] : -1;
        bias_value = tid < p.num_bias ? p.bias[row * p.num_bias + tid] : 0.f;
        rules = Penalties{p.repetition ? p.repetition[row] : 1.f, p.presence ? p.presence[row] : 0.f, p.frequency ? p.frequency[row] : 0.f};
    }
};

// Counts them and adds up their biases; returns the row's rules.
template <typename Raw>
__device__ __forceinline__ Penalties count_touched(const LogitsParams& p, const Segment<Raw>& g, const Table& table, Touches& own, int64_t row, int tid) {
    __shared__ int32_t s_token[kThreads];
    __shared__ float s_value[kThreads];
    int32_t most = -1;
    const int32_t low = max(g.t0, 0);
    const uint32_t length = min(p.vocab, g.t0 + min(g.reach, p.vocab - g.t0)) - low;
    auto ours = [&](int32_t token) {
        most = max(most, token);
        return (uint32_t)(token - low) < length;
    };
    if ((own.len < 0 || own.len > p.width) && tid == 0) report(p.status, kStatusBadIndex);
    const int len = max(0, min(own.len, p.width)), prompt = max(0, min(own.prompt, len));
    auto count = [&](int32_t token, int i) {
        if (i >= len || !ours(token)) return;
        uint32_t* word = table.word + table.entry(token);
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
        for (int k = 0; k < Touches::kKept; ++k) count4(own.quad[k], own.head + 4 * (k * kThreads + tid));
        constexpr int kQuads = 4;
        const int used = min(quads, (len - own.head + 3) / 4);
        for (int i0 = Touches::kKept * kThreads + tid; i0 < used; i0 += kQuads * kThreads) {
            int4 q[kQuads];
#pragma unroll
            for (int k = 0; k < kQuads; ++k)
                q[k] = i0 + k * kThreads < used ? __ldg(reinterpret_cast<const int4*>(own.history + own.head) + i0 + k * kThreads) : make_int4(-1, -1, -1, -1);
#pragma unroll
            for (int k = 0; k < kQuads; ++k) count4(q[k], own.head + 4 * (i0 + k * kThreads));
        }
    }
    // Biases, as many at a time as there are threads.
    for (int i0 = 0; i0 < p.num_bias; i0 += kThreads) {
        int32_t token = own.bias_token;
        float value = own.bias_value;
        if (i0 > 0) {
            token = i0 + tid < p.num_bias ? p.bias_tokens[row * p.num_bias + i0 + tid] : -1;
            value = i0 + tid < p.num_bias ? p.bias[row * p.num_bias + i0 + tid] : 0.f;
        }
        const bool mine = ours(token);
        const uint32_t at = mine ? table.entry(token) : 0;
        const bool again = mine && atomicOr(table.word + at, kBiased) & kBiased;
        if (!__syncthreads_or(again)) {
            if (mine) table.sum[at] = value;
        } else {  // a token several times: its first thread adds up all of them, in order
            s_token[tid] = mine ? token : -1;
            s_value[tid] = value;
            __syncthreads();
            bool leads = mine;
            for (int i = 0; i < tid && leads; ++i) leads = s_token[i] != token;
            if (leads) {
                float sum = table.sum[at];
                for (int i = tid; i < kThreads; ++i)
                    if (s_token[i] == token) sum += s_value[i];
                table.sum[at] = sum;
            }
            __syncthreads();
        }
    }
    if (most >= p.vocab) report(p.status, kStatusBadIndex);
    Penalties rules = own.rules;
    if (!(rules.repetition > 0.f && rules.repetition < INFINITY && fabsf(rules.presence) < INFINITY && fabsf(rules.frequency) < INFINITY)) {
        if (tid == 0) report(p.status, kStatusBadIndex);
        rules = Penalties{1.f, 0.f, 0.f};
    }
    __syncthreads();
    return rules;
}

// The touched logits, out of memory and into it.
template <typename T, typename Raw>
__device__ __forceinline__ void change_in_memory(const Segment<Raw>& g, const Table& table, const Penalties& rules, int tid) {
    using L = Logit<T>;
    // The touched logits, which take their words' place; those that the mask takes are left out.
    constexpr int kTouched = 8;
    for (int i0 = tid; i0 < table.entries; i0 += kTouched * kThreads) {
        int32_t token[kTouched];
        Raw y[kTouched];
        uint32_t bits[kTouched];
#pragma unroll
        for (int k = 0; k < kTouched; ++k) {
            const int i = i0 + k * kThreads;
            token[k] = i < table.entries ? table.key[i] : -1;
            bits[k] = ~0u;
            if (token[k] < 0) continue;
            y[k] = g.src[token[k]];
            if (g.mask) bits[k] = __ldg(g.mask + (token[k] >> 5));
        }
#pragma unroll
        for (int k = 0; k < kTouched; ++k) {
            const int i = i0 + k * kThreads;
            if (token[k] < 0) continue;
            const uint32_t word = table.word[i];
            if (bits[k] >> (token[k] & 31) & 1) table.word[i] = L::rounded(rules.apply(L::value(y[k]), word, word & kBiased ? table.sum[i] : 0.f));
            else table.key[i] = -1;
        }
    }
}

// A segment through the ring: touched tokens and then the mask's are changed in its chunks.
template <typename T, bool kTouched, typename Raw>
__device__ __forceinline__ void through_ring(const LogitsParams& p, const Segment<Raw>& g, Table table, uint16_t* list, unsigned char* ring, uint64_t* s_bar, int64_t row, int tid) {
    using L = Logit<T>;
    constexpr int kEach = 16 / sizeof(Raw), kChunk = kChunkBytes / sizeof(Raw), kUnit = kThreads * kEach, kLoads = kChunk / kUnit;
    constexpr uint32_t kAll = (1u << kEach) - 1;
    // Whole loads of 16 bytes in the row: [first, last) of the segment; what is left has less than a load at
    // either end.
    const int end = min(g.reach, g.vocab - g.t0), first = g.t0 < 0 ? kEach : 0, last = max(first, end / kEach * kEach);
    const int chunks = (last - first + kChunk - 1) / kChunk;
    const uint32_t ring_at = ptx::smem_u32(ring), bar = ptx::smem_u32(s_bar);
    auto bytes_of = [&](int c) { return (uint32_t)min(kChunk, last - first - c * kChunk) * (uint32_t)sizeof(Raw); };
    auto request = [&](int c) {
        const uint32_t slot = c % kRing;
        ptx::mbar_arrive_expect_tx(bar + 8 * slot, bytes_of(c));
        ptx::bulk_load(ring_at + slot * kChunkBytes, g.src + g.t0 + first + c * kChunk, bytes_of(c), bar + 8 * slot);
    };
    if (tid == 0)
        for (int c = 0; c < min(kRing, chunks); ++c) request(c);
    // Each chunk has a list of its touched tokens' entries, behind one another.
    __shared__ int s_tokens[kMostChunks + 2], s_begin[kMostChunks + 3];
    Touches own;
    if constexpr (kTouched) {
        own.read(p, row, tid);
        table.first = first;
        table.last = last;
        table.log_chunk = 31 - __clz(kChunk);
        table.tokens = s_tokens;
        if (tid < kMostChunks + 2) s_tokens[tid] = 0;
    }
    const int edge = tid < kEach ? tid : last + tid - kEach;  // of the tokens outside of whole loads
    if (tid < 2 * kEach && (tid < kEach ? first > 0 : true) && g.t0 + edge >= 0 && edge < end)
        g.dst[g.t0 + edge] = allowed<1>(g.mask, g.t0 + edge, 1u, g.vocab) ? g.src[g.t0 + edge] : L::rounded(-INFINITY);
    uint32_t even[kLoads], odd[kLoads];  // mask bits of chunks, asked for two chunks ahead
    auto masks = [&](int c, uint32_t (&bits)[kLoads]) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int at = first + c * kChunk + k * kUnit + tid * kEach;
            bits[k] = at < last ? allowed<kEach>(g.mask, g.t0 + at, kAll, g.vocab) : kAll;
        }
    };
    if (g.mask) masks(0, even), masks(1, odd);
    __syncthreads();
    Penalties rules;
    if constexpr (kTouched) rules = count_touched(p, g, table, own, row, tid);
    else if (!g.mask && tid) return;  // (nothing to change)
    if constexpr (kTouched) {
        if (tid < 32) {
            constexpr int kMine = (kMostChunks + 2 + 31) / 32;
            int n[kMine], sum = 0;
#pragma unroll
            for (int k = 0; k < kMine; ++k) sum += n[k] = kMine * tid + k < kMostChunks + 2 ? s_tokens[kMine * tid + k] : 0;
            int at = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, at, o);
                if (tid >= o) at += u;
            }
            at -= sum;
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                if (kMine * tid + k < kMostChunks + 3) s_begin[kMine * tid + k] = at;
                if (kMine * tid + k < kMostChunks + 2) s_tokens[kMine * tid + k] = at;
                at += n[k];
            }
        }
        __syncthreads();
        for (int i = 4 * tid; i < p.entries; i += 4 * kThreads) {
            const int4 keys = *reinterpret_cast<const int4*>(table.key + i);
            auto add = [&](int32_t token, int at) {
                if (token >= 0) list[atomicAdd(s_tokens + table.chunk_of(token), 1)] = (uint16_t)at;
            };
            add(keys.x, i);
            add(keys.y, i + 1);
            add(keys.z, i + 2);
            add(keys.w, i + 3);
        }
        __syncthreads();
    }
    auto changed = [&](Raw x, int at) {
        const uint32_t word = table.word[at];
        return L::rounded(rules.apply(L::value(x), word, word & kBiased ? table.sum[at] : 0.f));
    };
    bool ok = true;
    auto step = [&](int c, uint32_t (&bits)[kLoads]) {
        const uint32_t slot = c % kRing;
        unsigned char* chunk = ring + slot * kChunkBytes;
        // (After a wait that ran out nothing more is asked for; what is under way is waited for, and what follows is garbage.)
        ok = ptx::mbar_wait(bar + 8 * slot, c / kRing & 1, ok ? kWaitLimit : 64) && ok;
        if constexpr (kTouched) {
            const int from = g.t0 + first + c * kChunk;
            for (int i = s_begin[c + 1] + tid; i < s_begin[c + 2]; i += kThreads) {
                Raw* x = reinterpret_cast<Raw*>(chunk) + (table.key[list[i]] - from);
                *x = changed(*x, list[i]);
            }
            if (g.mask) __syncthreads();
        }
        if (g.mask) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                if (bits[k] == kAll) continue;
                uint4* at = reinterpret_cast<uint4*>(chunk) + k * kThreads + tid;
                uint4 x = *at;
                take_out<T>(x, bits[k]);
                *at = x;
            }
            masks(c + 2, bits);
        }
        if (kTouched || g.mask) {
            ptx::fence_proxy_async_smem();
            __syncthreads();
        }
        if (tid == 0 && ok) {
            ptx::bulk_store(g.dst + g.t0 + first + c * kChunk, ring_at + slot * kChunkBytes, bytes_of(c));
            ptx::bulk_commit();
            if (c > 0 && c - 1 + kRing < chunks) {
                ptx::bulk_wait_read<1>();  // the chunk before has left its slot
                request(c - 1 + kRing);
            }
        }
    };
    for (int c = 0; c < chunks; c += 2) {
        step(c, even);
        if (c + 1 < chunks) step(c + 1, odd);
    }
    if constexpr (kTouched) {
        auto edge_list = [&](int i0, int i1) {
            for (int i = i0 + tid; i < i1; i += kThreads) {
                const int32_t token = table.key[list[i]];
                if (allowed<1>(g.mask, token, 1u, g.vocab)) g.dst[token] = changed(g.src[token], list[i]);
            }
        };
        edge_list(0, s_begin[1]);
        edge_list(s_begin[kMostChunks + 1], s_begin[kMostChunks + 2]);
    }
    if (tid == 0) ptx::bulk_wait_read0();
    if (!ok) report(p.status, kStatusTimeout);
}

template <typename T, bool kThroughRing, bool kTouched>
__global__ void __launch_bounds__(kThreads, kResident) penalize_kernel(const __grid_constant__ LogitsParams p) {
    using Raw = typename Logit<T>::Raw;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(8) uint64_t s_bar[kRing];
    const int tid = threadIdx.x;
    const size_t table_bytes = (size_t)p.entries * (p.num_bias > 0 ? 12 : 8), list_bytes = (size_t)p.entries * 2;
    Table table{reinterpret_cast<int32_t*>(smem), reinterpret_cast<uint32_t*>(smem) + p.entries, reinterpret_cast<float*>(smem) + 2 * p.entries,
                p.entries, p.shift, 0, p.direct, nullptr, 0, 0, 0};
    if (kTouched)
        for (int i = tid; i < p.entries / 4; i += kThreads) {
            reinterpret_cast<int4*>(table.key)[i] = make_int4(-1, -1, -1, -1);
            reinterpret_cast<uint4*>(table.word)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (p.num_bias > 0) reinterpret_cast<float4*>(table.sum)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    if (kThroughRing && tid == 0) {
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
    if constexpr (kThroughRing) {
        through_ring<T, kTouched>(p, g, table, reinterpret_cast<uint16_t*>(smem + table_bytes), smem + table_bytes + list_bytes, s_bar, row, tid);
    } else {
        Touches own;
        if constexpr (kTouched) own.read(p, row, tid);
        copy_segment<T>(g, tid);
        if constexpr (kTouched) {
            __syncthreads();
            const Penalties rules = count_touched(p, g, table, own, row, tid);
            change_in_memory<T>(g, table, rules, tid);
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
}

constexpr int kMostEntries = 8192;  // of a table: 96 KB with biases

template <typename T>
cudaError_t launch_type(LogitsParams& p, cudaStream_t stream) {
    const int64_t touches = (int64_t)p.width + p.num_bias;
    const bool place = p.out == p.logits;
    if (place && !p.mask && touches == 0) return cudaSuccess;
    const int each = 16 / sizeof(T), unit = kUnitLoads * each;
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
    if (len > kMostChunks * (kChunkBytes / (int)sizeof(T))) len = kMostChunks * (kChunkBytes / (int)sizeof(T));
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
    // Through the ring where a segment has more than a chunk (16 rows of 50257 fp32 with 32768 tokens each, 16 KB
    // a segment, so just not: 16.6 us through it, 15.3 through registers) and rows of out have the boundaries of the logits'.
    const bool ring = !place && len * (int64_t)sizeof(T) > kChunkBytes && (((uintptr_t)p.out ^ (uintptr_t)p.logits) & 15) == 0 && (p.rows == 1 || ((p.out_stride ^ p.stride) * sizeof(T) & 15) == 0);
    const auto kernel = ring ? (touches ? penalize_kernel<T, true, true> : penalize_kernel<T, true, false>)
                             : (touches ? penalize_kernel<T, false, true> : penalize_kernel<T, false, false>);
    const int64_t chunks = (len * (int64_t)sizeof(T) + kChunkBytes - 1) / kChunkBytes;
    const size_t smem = (size_t)p.entries * (p.num_bias > 0 ? 12 : 8) + (ring ? (size_t)p.entries * 2 + (size_t)(chunks < kRing ? chunks : kRing) * kChunkBytes : 0);
    if (smem > 40 * 1024) {
        // (The most that any call needs, not this one: the limit is the kernel's, for calls of other threads too.)
        const int most = ring ? kMostEntries * 14 + kRing * kChunkBytes : kMostEntries * 12;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
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
