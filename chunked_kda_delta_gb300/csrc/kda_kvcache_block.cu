// kda_kvcache_block.cu -- causal attention over the 8-bit paged cache for many new tokens a row
// (pieces of prompts): the products on tcgen05.
//
// An item is 128 query rows (token, query head of a group) of one row and key/value head; they
// are the 128 rows of the tensor core's tile.  For every 64 keys:
//   S = Q K^T       both operands in shared memory, K widened there from its codes (e4m3 is
//                   exact in fp16), S in one of two buffers in tensor memory;
//   softmax         a thread has a row: nothing is exchanged;
//   O += P V        P in fp16 in tensor memory where its S was, V widened into shared memory with
//                   its rows as they come (channel-major, 128-byte swizzle), O in tensor memory.
// Four warps do the softmax, four read and widen codes (each the tile's 16 keys of one page), the
// first of which issues the matrix instructions as well (a ninth warp for that left 96 registers
// a thread and spills); two CTAs an SM.  S(j + 1) is computed and V(j) widened while the softmax
// of tile j runs.  (One kind of warps for everything, two threads a row, took 4300 cycles a tile:
// 1000 of them issuing, the rest waiting for each other at three barriers; 159 us instead of 88 for 8 pieces of up to 512
// tokens, 16 heads of 64 over 4, 4096 cached.  Eight widening warps: 102; two softmax groups: 105
// and 108.)
// O is rescaled only when a row's maximum has grown by more than 2^8 over the one in use (a published
// method), whose weight is 2^7: weights stay below 2^15 in fp16, which is normal down to 2^-21 of the
// largest, and the sums are the same.  The v scale enters the exponent, also for the
// maximum, and leaves the sum again by blocks of 16 keys.
//
// Bound by issue and latency: a tile takes each of an SM's two CTAs 2700 cycles (head_dim 128: 4700),
// nearly all of them work of both kinds of warps, 55% of the issue slots and 21% of the tensor
// cores' cycles.  The call above takes 88 us, 393 TFLOP/s; with heads of 128 151 us, 456.
//
// Work split as in kda_kvcache_attention.cu, by tiles that are seen: the CTAs (two an SM) take
// equal contiguous shares of all tiles of all items, and the parts are joined by a second launch.
// q's and the scales' handling is that file's too.
#include "kda_kvcache_attention.cuh"
#include "kda_ptx.cuh"

namespace kda {
namespace {

using namespace ptx;

constexpr int kRows = kBlockRows, kKeys = 64, kBlocks = kKeys / 16;
constexpr int kSoft = 128, kWiden = 128;          // threads of the softmax, of the widening
constexpr int kThreads = kSoft + kWiden;
constexpr int kMaxListed = 512;           // rows whose prefix fits in shared memory
constexpr float kGrowth = 8.f, kLift = 7.f; // log2 of how far a maximum may grow, of the weight at it
constexpr uint32_t kColS = 0, kColO = 128, kColumns = 256;  // tensor memory: S and P twice, O
constexpr int64_t kWaitLimit = 1ll << 20;
// Two CTAs an SM and no third: the tensor memory is for two.
constexpr size_t kSmemBytes = 80 * 1024;

// Two floats side by side: one instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Matrix instructions by one thread of a converged warp: the election is part of each, so that
// the descriptors stay in uniform registers (issued under `if (lane == 0)` four of them took 500
// cycles).
__device__ __forceinline__ void mma_ss_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Named barriers for the issuing warp: K is widened; V is, and P is written; q is there.
constexpr uint32_t kBarK = 1, kBarP = 2, kBarQ = 3;

// fp16 operands, fp32 result; `b_rows`: B's rows are the reduction (channel-major).
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_rows) {
    return (1u << 4) | ((uint32_t)b_rows << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

// Keys that column block `block` of a row sees, and its tiles (at least one).  (The host sees to it
// that tokens times group fits in 31 bits.)
__device__ __forceinline__ int block_seen(int n, int len, int group, int block) {
    const int last = min(n * group - block * kRows, kRows) - 1 + block * kRows;
    return min(len, max(0, len - n + last / group + 1));
}
__device__ __forceinline__ int tiles_of(int seen) { return seen > kKeys ? (seen + kKeys - 1) / kKeys : 1; }
__device__ __forceinline__ int blocks_of(int n, int group) { return (n * group + kRows - 1) / kRows; }
// Tiles of the blocks before `block`, a lane each; the same in all lanes.
__device__ __forceinline__ int64_t tiles_before(int n, int len, int group, int block) {
    int64_t x = 0;
    for (int b = threadIdx.x & 31; b < block; b += 32) x += tiles_of(block_seen(n, len, group, b));
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// An item that lies in the shares [its own, last] of several CTAs; last < 0: none.
struct alignas(16) SplitItem {
    int begin, n, head, block, slot, last, unused[2];  // first token and tokens of its row; slot of its first part
};

struct Meta {  // scales of 16 keys, of v in shared memory its log2 (-inf for 0); k negative where the page is missing
    float k, v;
};

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, 2) block_attention_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kLoads = kDim / 32;                 // 16-byte loads of a thread for a tile of K (and V)
    constexpr uint32_t kLbo = 128, kSbo = kDim * 16;  // K-major core matrices: along the reduction, along rows
    constexpr uint32_t kBoxBytes = kKeys * 128;       // 64 channels of V
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ int64_t s_first[kMaxListed + 1], s_scan[kThreads / 32], s_tiles[kThreads / 32];
    __shared__ __align__(16) Meta s_meta[4][kBlocks];
    __shared__ volatile int s_bad;  // a wait ran out
    __shared__ __align__(8) uint64_t s_bar[3];
    __shared__ uint32_t s_tmem;
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* v_sm = smem;
    unsigned char* k_sm = v_sm + kKeys * kDim * 2;
    unsigned char* q_sm = k_sm + kKeys * kDim * 2;

    const CacheParams& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool soft = tid < kSoft, issuer = warp == kSoft / 32;
    const int group = p.q_heads / c.heads;
    const int page_shift = __ffs(c.page_tokens) - 1;
    const int64_t block_bytes = (int64_t)c.page_tokens * kDim;
    // S of a tile is there (one barrier for each buffer: S(j + 1) may be done before the softmax has
    // seen S(j), and a barrier must not run two phases ahead of a waiter); O += P V is done.
    const uint32_t bar_s = smem_u32(&s_bar[0]), bar_o = smem_u32(&s_bar[2]);
    auto bar_of = [&](int j) { return bar_s + 8 * (j & 1); };  // j: tiles of the item so far

    if (tid == 0) {
        mbar_init(bar_of(0), 1 + kBlocks);  // S is computed, and the widening warps' scales are there
        mbar_init(bar_of(1), 1 + kBlocks);
        mbar_init(bar_o, 1);
        fence_mbar_init();
        s_bad = 0;
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&s_tmem), kColumns);
        tmem_relinquish();
    }
    follow_stream();
    int64_t* first = c.rows <= kMaxListed ? s_first : p.first_work;
    // Tiles of the rows.  As many rows as warps: a warp each.  More: a thread each, where a row has few
    // blocks, else its warp for it.
    constexpr int kFewBlocks = 4;
    if (c.rows <= kThreads / 32) {
        int64_t begin;
        const int n = warp < c.rows ? row_tokens(c, warp, begin) : 0, len = warp < c.rows ? row_length(c, warp) : 0;
        const int64_t tiles = tiles_before(n, len, group, blocks_of(n, group));
        if (lane == 0) s_tiles[warp] = tiles;
        __syncthreads();
    }
    scan_rows<kThreads>(c.rows, first, s_scan, [&](int r) {
        int64_t tiles = 0;
        if (c.rows <= kThreads / 32) {
            if (r < c.rows) tiles = s_tiles[r];
        } else {
            int64_t begin;
            const int n = r < c.rows ? row_tokens(c, r, begin) : 0, len = r < c.rows ? row_length(c, r) : 0, blocks = blocks_of(n, group);
            for (int x = 0; x < blocks && blocks <= kFewBlocks; ++x) tiles += tiles_of(block_seen(n, len, group, x));
            for (unsigned many = __ballot_sync(0xffffffffu, blocks > kFewBlocks); many; many &= many - 1) {
                const int from = __ffs(many) - 1;
                const int64_t t = tiles_before(__shfl_sync(0xffffffffu, n, from), __shfl_sync(0xffffffffu, len, from), group,
                                               __shfl_sync(0xffffffffu, blocks, from));
                if (lane == from) tiles = t;
            }
        }
        return tiles * c.heads;
    });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (blockIdx.x == 0 && c.rows <= kMaxListed)
        for (int r = tid; r <= c.rows; r += kThreads) p.first_work[r] = s_first[r];
    const uint32_t tmem = s_tmem, lanes = (uint32_t)(32 * (warp % 4)) << 16;
    const int64_t per = share_of(first[c.rows], p.ctas);
    const int64_t w_begin = per * blockIdx.x, w_end = min(first[c.rows], w_begin + per);
    uint32_t phase_s = 0, phase_o = 0;  // (phase_s: a bit for each buffer)
    // After a wait that ran out, all others end at once and what follows is garbage.
    auto wait = [&](uint32_t bar, uint32_t phase) {
        if (!mbar_try_wait_now(bar, phase) && !mbar_wait_now(bar, phase, s_bad ? 1 : kWaitLimit)) s_bad = 1;
    };
    auto wait_s = [&](int j) {
        wait(bar_of(j), (phase_s >> (j & 1)) & 1);
        phase_s ^= 1u << (j & 1);
    };
    auto wait_o = [&]() {
        wait(bar_o, phase_o);
        phase_o ^= 1;
    };

    // The item that begins in this share and ends in another: none yet.
    if (tid == 0) reinterpret_cast<SplitItem*>(p.split_items)[blockIdx.x].last = -1;
    for (int64_t w = w_begin; w < w_end;) {
        const int row = row_of(first, c.rows, w);
        int64_t begin;
        const int n = row_tokens(c, row, begin), len = row_length(c, row);
        const int64_t each = (first[row + 1] - first[row]) / c.heads;  // tiles of a head's blocks
        const int head = (int)((w - first[row]) / each);
        int64_t item = first[row] + head * each;
        int block = 0, tiles = 0;
        for (int b0 = 0;; b0 += 32) {  // 32 blocks at a time: the one that w falls into
            const int mine = tiles_of(block_seen(n, len, group, b0 + lane));
            int64_t end = mine;  // of the blocks up to this lane's
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += y;
            }
            const unsigned behind = __ballot_sync(0xffffffffu, item + end > w);
            if (behind) {
                const int at = __ffs(behind) - 1;
                block = b0 + at;
                tiles = __shfl_sync(0xffffffffu, mine, at);
                item += __shfl_sync(0xffffffffu, end, at) - tiles;
                break;
            }
            item += __shfl_sync(0xffffffffu, end, 31);
        }
        const int64_t item_end = item + tiles;
        const int rows_all = n * group, row0 = block * kRows, f = row0 + tid % 128;
        const bool there = f < rows_all;
        const int seen_max = block_seen(n, len, group, block);
        const int seen_min = max(0, min(len, len - n + row0 / group + 1));
        const int seen = there ? max(0, min(len, len - n + f / group + 1)) : 0;
        const int tile0 = (int)(w - item);
        const int tile1 = min((int)(min(item_end, w_end) - item), (seen_max + kKeys - 1) / kKeys);

        const int32_t* table = c.tables + (int64_t)row * c.width;
        // This thread's row of q as fp16 into shared memory.
        float factor = 0.f;
        if (soft) {
            const T* src = static_cast<const T*>(p.q) + (begin + (there ? f / group : 0)) * p.q_stride +
                           (int64_t)(head * group + (there ? f % group : 0)) * kDim;
            // 64 channels in registers at a time; of 128 the first half is read again (L1).
            uint4 raw[8];
            auto read = [&](int half) {
#pragma unroll
                for (int i = 0; i < 8; ++i) raw[i] = there ? reinterpret_cast<const uint4*>(src)[8 * half + i] : make_uint4(0u, 0u, 0u, 0u);
            };
            float a = 0.f;
#pragma unroll
            for (int half = 0; half < kDim / 64; ++half) {
                read(half);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 y = Act<T>::two(u[k]);
                        a = fmaxf(a, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
            }
            const int e = row_exponent(a);
            // The sign of the scale goes with q, so that factors are not negative.
            const float up = copysignf(exp2f((float)(14 - e)), p.scale);
            factor = exp2f((float)(e - 14)) * fabsf(p.scale);
#pragma unroll
            for (int half = kDim / 64 - 1; half >= 0; --half) {
                if (half < kDim / 64 - 1) read(half);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 y = Act<T>::two(u[k]);
                        u[k] = pack_half2(y.x * up, y.y * up);
                    }
                    *reinterpret_cast<uint4*>(q_sm + (tid / 8) * kSbo + (8 * half + i) * kLbo + (tid % 8) * 16) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            fence_proxy_async_smem();
            named_bar_arrive(kBarQ, kSoft + 32);
        }

        // Matrix instructions of the issuing warp: S of a tile into its buffer, O += P V.
        const uint64_t qd = sdesc(smem_u32(q_sm), kLbo, kSbo), kd = sdesc(smem_u32(k_sm), kLbo, kSbo);
        const uint64_t vd = sdesc(smem_u32(v_sm), kBoxBytes, 1024) | ((uint64_t)2 << 61);
        auto issue_s = [&](int tile) {
            const uint32_t d = tmem + kColS + ((tile - tile0) & 1) * kKeys;
#pragma unroll
            for (int kk = 0; kk < kDim / 16; ++kk)  // (a step is 2 core matrices: 16 units of 16 bytes)
                mma_ss_one(d, qd + kk * (2 * kLbo / 16), kd + kk * (2 * kLbo / 16), idesc_f16(kKeys, false), kk > 0);
            commit_one(bar_of(tile - tile0));
        };
        auto issue_o = [&](int tile) {
            const uint32_t a = tmem + kColS + ((tile - tile0) & 1) * kKeys;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts_one(tmem + kColO, a + kk * 8, vd + kk * (2048 / 16), idesc_f16(kDim, true), tile > tile0 || kk > 0);
            commit_one(bar_o);
        };

        float m = kNegInf, l = 0.f;
        if (!soft) {
            // This warp's 16 keys of each tile lie in one page.  Load number i of a lane: key
            // 8 (i % 2) + lane % 8, channels 16 (4 (i / 2) + lane / 8).
            const int mine = warp - kSoft / 32;
            auto needed = [&](int tile) { return tile < tile1 && tile * kKeys + mine * 16 < seen_max; };
            auto entry_at = [&](int tile) { return needed(tile) ? table[(tile * kKeys + mine * 16) >> page_shift] : -1; };
            // (Looked at a tile after it was read: the wait for the table would hold up the loop.)
            auto checked = [&](int32_t x, int tile) {
                if (x >= 0 && x < c.pages) return x;
                if (lane == 0 && needed(tile)) report(c.status, kStatusBadIndex);
                return -1;
            };
            auto meta_of = [&](int32_t page) {
                const int64_t at = (int64_t)max(page, 0) * c.heads + head;
                return page < 0 ? Meta{-1.f, 1.f} : Meta{c.k_scale[at], c.v_scale[at]};
            };
            // What no row sees, and V of a scale of 0, is to leave no trace: zero.
            auto load = [&](uint4 (&raw)[kLoads], const uint8_t* codes, int tile, int32_t page, int keys) {
                const uint8_t* src = codes + ((int64_t)max(page, 0) * c.heads + head) * block_bytes +
                                     (((tile * kKeys + mine * 16) & (c.page_tokens - 1)) + lane % 8) * kDim + lane / 8 * 16;
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
                    raw[i] = page >= 0 && lane % 8 + 8 * (i % 2) < keys ? load_codes16(src + i % 2 * 8 * kDim + i / 2 * 64)
                                                                        : make_uint4(0u, 0u, 0u, 0u);
            };
            auto widen = [](const uint4& r, uint4& lo, uint4& hi) {
                lo = make_uint4(widen2(r.x), widen2(r.x >> 16), widen2(r.y), widen2(r.y >> 16));
                hi = make_uint4(widen2(r.z), widen2(r.z >> 16), widen2(r.w), widen2(r.w >> 16));
            };
            unsigned char* k_dst = k_sm + mine * 2 * kSbo + lane / 8 * 2 * kLbo + lane % 8 * 16;
            unsigned char* v_dst = v_sm + (mine * 16 + lane % 8) * 128;
            const int v_lo = ((lane / 8 * 2) ^ (lane % 8)) * 16, v_hi = ((lane / 8 * 2 + 1) ^ (lane % 8)) * 16;

            auto put_k = [&](const uint4 (&raw)[kLoads], int tile, const Meta& meta) {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    uint4 lo, hi;
                    widen(raw[i], lo, hi);
                    unsigned char* dst = k_dst + i % 2 * kSbo + i / 2 * 8 * kLbo;
                    *reinterpret_cast<uint4*>(dst) = lo;
                    *reinterpret_cast<uint4*>(dst + kLbo) = hi;
                }
                if (lane == 0) {
                    s_meta[tile & 3][mine] = Meta{meta.k, log2f(meta.v)};
                    mbar_arrive(bar_of(tile - tile0));
                }
                fence_proxy_async_smem();
                if (issuer) named_bar_sync(kBarK, kWiden);
                else named_bar_arrive(kBarK, kWiden);
            };

            // Pages, scales and codes are read a tile or two ahead.
            int32_t page0 = entry_at(tile0), page1 = entry_at(tile0 + 1), page2 = entry_at(tile0 + 2);
            page0 = checked(page0, tile0);
            page1 = checked(page1, tile0 + 1);
            Meta meta1 = meta_of(page1);  // of tile + 1
            uint4 kr[kLoads], vr[kLoads];
            if (tile0 < tile1) {
                const Meta meta = meta_of(page0);
                load(kr, c.k_codes, tile0, page0, 16);
                load(vr, c.v_codes, tile0, page0, meta.v > 0.f ? seen_max - tile0 * kKeys - mine * 16 : 0);
                put_k(kr, tile0, meta);
                load(kr, c.k_codes, tile0 + 1, page1, 16);
            }
            if (issuer) {
                named_bar_sync(kBarQ, kSoft + 32);
                tc_fence_after();
                if (tile0 < tile1) issue_s(tile0);
            }
            for (int tile = tile0; tile < tile1; ++tile) {
                wait_s(tile - tile0);  // K's shared memory is free
                if (tile + 1 < tile1) put_k(kr, tile + 1, meta1);
                // V's is, and the place of P(tile - 1), which S(tile + 1) takes: matrix instructions
                // with different results are not ordered by themselves.
                if (tile > tile0) wait_o();
                if (issuer && tile + 1 < tile1) {
                    tc_fence_after();
                    issue_s(tile + 1);
                }
                page2 = checked(page2, tile + 2);
                load(kr, c.k_codes, tile + 2, page2, 16);
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    uint4 lo, hi;
                    widen(vr[i], lo, hi);
                    unsigned char* dst = v_dst + i % 2 * 8 * 128 + i / 2 * kBoxBytes;
                    *reinterpret_cast<uint4*>(dst + v_lo) = lo;
                    *reinterpret_cast<uint4*>(dst + v_hi) = hi;
                }
                fence_proxy_async_smem();
                load(vr, c.v_codes, tile + 1, page1, meta1.v > 0.f ? seen_max - (tile + 1) * kKeys - mine * 16 : 0);
                page1 = page2;
                meta1 = meta_of(page1);
                page2 = entry_at(tile + 3);
                if (issuer) {
                    named_bar_sync(kBarP, kThreads);
                    tc_fence_after();
                    issue_o(tile);
                } else {
                    named_bar_arrive(kBarP, kThreads);
                }
            }
            if (tile0 < tile1) wait_o();
        } else {
            float least = kScaleLeast;  // that a log2 of v's scale counts as
            for (int tile = tile0; tile < tile1; ++tile) {
                wait_s(tile - tile0);
                tc_fence_after();
                const uint32_t t_s = tmem + kColS + ((tile - tile0) & 1) * kKeys + lanes;
                uint32_t sr[kKeys];
                tmem_ld32(t_s, sr);
                tmem_ld32(t_s + 32, sr + 32);
                Meta meta[kBlocks];
                bool missing = false, low = false;
#pragma unroll
                for (int x = 0; x < kBlocks; ++x) {
                    meta[x] = s_meta[tile & 3][x];
                    missing |= meta[x].k < 0.f;
                    least = fmaxf(least, meta[x].v - kScaleSpan);
                }
#pragma unroll
                for (int x = 0; x < kBlocks; ++x) {
                    low |= meta[x].v < least;
                    meta[x].v = fmaxf(meta[x].v, least);
                }
                tmem_wait_ld_regs<kKeys>(sr);
                const int key0 = tile * kKeys;
                if (key0 + kKeys > seen_min || missing) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i)
                        if (key0 + i >= seen || meta[i / 16].k < 0.f) sr[i] = __float_as_uint(kNegInf);
                }
                float top = kNegInf;
#pragma unroll
                for (int x = 0; x < kBlocks; ++x) {
                    float y = max3(__uint_as_float(sr[16 * x]), __uint_as_float(sr[16 * x + 1]), __uint_as_float(sr[16 * x + 2]));
                    float z = max3(__uint_as_float(sr[16 * x + 3]), __uint_as_float(sr[16 * x + 4]), __uint_as_float(sr[16 * x + 5]));
#pragma unroll
                    for (int i = 6; i < 14; i += 4) {
                        y = max3(y, __uint_as_float(sr[16 * x + i]), __uint_as_float(sr[16 * x + i + 1]));
                        z = max3(z, __uint_as_float(sr[16 * x + i + 2]), __uint_as_float(sr[16 * x + i + 3]));
                    }
                    y = fmaxf(max3(y, z, __uint_as_float(sr[16 * x + 14])), __uint_as_float(sr[16 * x + 15]));
                    top = fmaxf(top, y == kNegInf ? kNegInf : fmaf(y, meta[x].k * factor, meta[x].v));  // (a scale of 0 makes scores 0)
                }
                // The reference of the weights.
                const float m_new = top > m + kGrowth || m == kNegInf ? fmaxf(m, top) : m;
                const float m_use = m_new == kNegInf ? 0.f : m_new;
                const float half = m == kNegInf ? (m_new == kNegInf ? 1.f : 0.f) : exp2_fast(0.5f * (m - m_use)), fix = half * half;
                m = m_new;
                l = rescaled(l, half);
#pragma unroll
                for (int x = 0; x < kBlocks; ++x) {
                    // (A factor of 0 must not make masked scores NaN.)
                    const float k = meta[x].k * factor > 0.f ? meta[x].k * factor : 0x1p-126f;
                    const float bias = meta[x].v - m_use + kLift;
                    const uint64_t k2 = pair(k, k), bias2 = pair(bias, bias);
                    uint64_t acc[2] = {0, 0};  // (+0, +0)
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float a, b;
                        unpair(fma2(pair(__uint_as_float(sr[16 * x + i]), __uint_as_float(sr[16 * x + i + 1])), k2, bias2), a, b);
                        a = exp2_fast(a);
                        b = exp2_fast(b);
                        acc[i / 2 % 2] = add2(acc[i / 2 % 2], pair(a, b));
                        sr[8 * x + i / 2] = pack_half2(a, b);  // P takes S's registers
                    }
                    float sum[2];
                    unpair(add2(acc[0], acc[1]), sum[0], sum[1]);
                    l += (sum[0] + sum[1]) * exp2_fast(-meta[x].v);
                }
                if (low) {
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) {
                        const float by = exp2_fast(fminf(s_meta[tile & 3][x].v - least, 0.f));
#pragma unroll
                        for (int i = 0; i < 8; ++i) sr[8 * x + i] = brought_down(sr[8 * x + i], by);
                    }
                }
                if (tile > tile0) {  // O += P V of the tile before is done
                    wait_o();
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, fix != 1.f)) {
#pragma unroll
                        for (int q = 0; q < kDim; q += 16) {
                            uint32_t o[16];
                            tmem_ld16(tmem + kColO + lanes + q, o);
                            tmem_wait_ld_regs<16>(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
                            tmem_st8(tmem + kColO + lanes + q, *reinterpret_cast<uint32_t(*)[8]>(o));
                            tmem_st8(tmem + kColO + lanes + q + 8, *reinterpret_cast<uint32_t(*)[8]>(o + 8));
                        }
                    }
                }
                tmem_st32(t_s, sr);
                tmem_wait_st();
                tc_fence_before();
                named_bar_arrive(kBarP, kThreads);
            }
            if (tile0 < tile1) wait_o();
            tc_fence_after();
        }

        const bool whole = w == item && item_end <= w_end;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (w == w_begin ? 0 : 1);
        if (tid == 0 && w == item && item_end > w_end)
            reinterpret_cast<SplitItem*>(p.split_items)[blockIdx.x] = SplitItem{(int)begin, n, head, block, (int)slot, (int)((item_end - 1) / per), 0, 0};
        const float by = l > 0.f ? 1.f / l : 0.f;
        T* out = static_cast<T*>(p.out) + (begin + (there ? f / group : 0)) * p.out_stride +
                 (int64_t)(head * group + (there ? f % group : 0)) * kDim;
        if (!whole && soft) {
            p.part_ml[(slot * 2 + 0) * kRows + tid] = m;
            p.part_ml[(slot * 2 + 1) * kRows + tid] = l;
        }
#pragma unroll
        for (int q = 0; q < kDim && soft; q += 16) {
            uint32_t o[16];
            if (tile0 < tile1) {
                tmem_ld16(tmem + kColO + lanes + q, o);
                tmem_wait_ld_regs<16>(o);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0u;
            }
            if (whole) {
                if (there) {
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            u[k] = Act<T>::pack(__uint_as_float(o[i + 2 * k]) * by, __uint_as_float(o[i + 2 * k + 1]) * by);
                        *reinterpret_cast<uint4*>(out + q + i) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) p.part_o[(slot * kDim + q + i) * kRows + tid] = __uint_as_float(o[i]);
            }
        }
        tc_fence_before();
        __syncthreads();  // tensor memory, pages and q are used anew
        tc_fence_after();
        w = item_end;
    }
    if (s_bad && tid == 0) report(c.status, kStatusTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kColumns);
}

// Joins the parts of the items that lie in several CTAs' shares: blockIdx.y counts channels, a
// thread has one query row.  kShares 1: blockIdx.x is the share that the item begins in, at most
// as many as there are CTAs, however many items there are.  kShares > 1 (few items, of many
// parts): blockIdx.x counts items, and that many threads have a row's parts in turn.  (One thread
// after the other through 91 parts took 65 of 73 us for 34 tokens of 3 heads over 5670 keys; a
// CTA for each of 2560 items and 16 channels 80 of 672 us for 64 rows of 64 tokens, 32 heads.)
template <typename T, int kDim, int kShares>
__global__ void __launch_bounds__(kRows * kShares, kShares == 4 ? 2 : 1) block_join_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kCh = kShares == 8 ? 4 : kShares == 4 ? 8 : 16, kAhead = kShares == 8 ? 6 : kShares == 4 ? 3 : 1;  // channels, parts under way
    __shared__ float s_part[kShares > 1 ? kShares - 1 : 1][kCh + 2][kShares > 1 ? kRows : 1];
    const CacheParams& c = p.c;
    const int group = p.q_heads / c.heads, tid = threadIdx.x % kRows, share = threadIdx.x / kRows, d0 = blockIdx.y * kCh;
    int64_t begin, u0, u1, slot0;
    int n, head, block;
    if constexpr (kShares == 1) {
        follow_stream();
        const SplitItem x = reinterpret_cast<const SplitItem*>(p.split_items)[blockIdx.x];
        if (x.last < 0) return;
        begin = x.begin, n = x.n, head = x.head, block = x.block, slot0 = x.slot, u0 = blockIdx.x, u1 = x.last;
    } else {
        int64_t i = blockIdx.x;
        int row;
        const bool there = joined_item(c, group, kRows, i, row);
        begin = n = 0;
        if (there) n = row_tokens(c, row, begin);
        const int len = there ? row_length(c, row) : 0, blocks = blocks_of(n, group);
        const bool ours = blocks > 0 && i < (int64_t)blocks * c.heads;
        head = ours ? (int)(i / blocks) : 0, block = ours ? (int)(i % blocks) : 0;
        const int64_t before = tiles_before(n, len, group, block);
        const int tiles = ours ? tiles_of(block_seen(n, len, group, block)) : 0;
        follow_stream();
        if (!ours) return;
        const int64_t per = share_of(p.first_work[c.rows], p.ctas);
        const int64_t each = (p.first_work[row + 1] - p.first_work[row]) / c.heads;
        const int64_t w0 = p.first_work[row] + head * each + before, w1 = w0 + tiles;
        u0 = w0 / per, u1 = (w1 - 1) / per, slot0 = 2 * u0 + (u0 * per >= w0 ? 0 : 1);
        if (u0 == u1) return;
    }
    const int f = block * kRows + tid;
    const bool mine = f < n * group;
    float top = kNegInf, sum = 0.f, acc[kCh];
#pragma unroll
    for (int d = 0; d < kCh; ++d) acc[d] = 0.f;
    auto add = [&](float mk, float lk, const float* o) {
        const float m = fmaxf(top, mk), use = m == kNegInf ? 0.f : m;
        const float ha = exp2_fast(0.5f * (top - use)), hb = exp2_fast(0.5f * (mk - use)), a = ha * ha, b = hb * hb;
        top = m;
        sum = rescaled(sum, ha) + rescaled(lk, hb);
#pragma unroll
        for (int d = 0; d < kCh; ++d) acc[d] = acc[d] * a + o[d] * b;
    };
    for (int64_t k = u0 + share; mine && k <= u1; k += kAhead * kShares) {
        float mk[kAhead], lk[kAhead], o[kAhead][kCh];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int64_t u = k + x * kShares;
            if (u > u1) continue;
            const int64_t slot = u == u0 ? slot0 : 2 * u;
            mk[x] = p.part_ml[(slot * 2 + 0) * kRows + tid];
            lk[x] = p.part_ml[(slot * 2 + 1) * kRows + tid];
#pragma unroll
            for (int d = 0; d < kCh; ++d) o[x][d] = p.part_o[(slot * kDim + d0 + d) * kRows + tid];
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            if (k + x * kShares <= u1) add(mk[x], lk[x], o[x]);
    }
    if constexpr (kShares > 1) {
        if (share) {
            s_part[share - 1][kCh][tid] = top;
            s_part[share - 1][kCh + 1][tid] = sum;
#pragma unroll
            for (int d = 0; d < kCh; ++d) s_part[share - 1][d][tid] = acc[d];
        }
        __syncthreads();
        if (share) return;
        for (int x = 0; x < kShares - 1; ++x) {
            float o[kCh];
#pragma unroll
            for (int d = 0; d < kCh; ++d) o[d] = s_part[x][d][tid];
            add(s_part[x][kCh][tid], s_part[x][kCh + 1][tid], o);
        }
    }
    if (!mine) return;
    const float by = sum > 0.f ? 1.f / sum : 0.f;
    T* out = static_cast<T*>(p.out) + (begin + f / group) * p.out_stride + (int64_t)(head * group + f % group) * kDim + d0;
#pragma unroll
    for (int d = 0; d < kCh; d += 4)
        *reinterpret_cast<uint2*>(out + d) = make_uint2(Act<T>::pack(acc[d] * by, acc[d + 1] * by), Act<T>::pack(acc[d + 2] * by, acc[d + 3] * by));
}

template <typename T, int kDim>
cudaError_t launch_dim(const AttentionParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(block_attention_kernel<T, kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_early(block_attention_kernel<T, kDim>, dim3(p.ctas), kThreads, kSmemBytes, stream, 1, p);
    if (e != cudaSuccess) return e;
    // As many threads to a row as one wave holds: few items have many parts each.
    const int64_t items = joined_items(p.c, p.q_heads / p.c.heads, kRows);
    if (items * (kDim / 4) <= 2 * p.sm_count)
        return launch_early(block_join_kernel<T, kDim, 8>, dim3((unsigned)items, kDim / 4), kRows * 8, 0, stream, 1, p);
    if (items * (kDim / 8) <= 4 * p.sm_count)
        return launch_early(block_join_kernel<T, kDim, 4>, dim3((unsigned)items, kDim / 8), kRows * 4, 0, stream, 1, p);
    return launch_early(block_join_kernel<T, kDim, 1>, dim3((unsigned)p.ctas, kDim / 16), kRows, 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_block_attention(const AttentionParams& p, bool f16, cudaStream_t stream) {
    if (p.c.dim == 64) return f16 ? launch_dim<__half, 64>(p, stream) : launch_dim<__nv_bfloat16, 64>(p, stream);
    return f16 ? launch_dim<__half, 128>(p, stream) : launch_dim<__nv_bfloat16, 128>(p, stream);
}

}  // namespace kda
