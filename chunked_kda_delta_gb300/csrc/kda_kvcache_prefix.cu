// kda_kvcache_prefix.cu -- attention of groups of rows to the keys that all of a group's rows share, for the
// state that the rows go on from (kda_kvcache_attention.cu, kda_kvcache_block.cu): products on tcgen05.
//
// Every query row of a group sees every key of its prefix, so nothing is masked but what is missing.  One CTA an SM,
// three kinds of warps:
//   two softmax groups of 128 threads, a thread a query row;
//   for each of them a warp that issues its matrix instructions: S = Q K^T for tiles of 64 keys into one of two
//   buffers in tensor memory, O += P V with P in fp16 where its S was; S of the next tile is computed while the
//   weights of this one are worked out.  (Issuing S blocks a warp for the 384 cycles that its operands take to be read:
//   too long for a softmax warp's chain, and for a warp that the other group waits for too);
//   six that widen codes (e4m3 is exact in fp16) into the operands' layouts in shared memory, each the tiles of
//   one of three places of K or of V, from a place of its own that bulk copies fill.  Lanes take pieces of 16 bytes along
//   diagonals of keys and channels, so that neither side has bank conflicts.
// A barrier's waiters tell its phases apart by their parity alone, so everyone who waits for a place of the ring waits
// for each of its tiles: a widening warp has one place, and an issuing warp passes the other group's tiles too.  What a
// softmax group does not wait for in every step has a barrier for each of S's buffers: S of a step is computed after O
// has taken the step before the last.
// Items of more than 128 query rows (token, query head of the group) give each softmax group 128 of 256, and every
// widened tile is used twice; smaller items give the softmax groups alternate tiles, and the rows stand twice
// or four times among the 128, each time for a part of the tile's keys (the others' weights are 0): a thread
// then has 32 or 16 scores of a tile to exponentiate.
//
// Softmax as in kda_kvcache_block.cu: O is rescaled only when a row's maximum has grown by more than 2^8 over
// the one in use; v's scale enters the exponent and leaves the sum again by blocks of 16 keys; q's and the
// scales' handling is kda_kvcache_attention.cu's.  The maximum holds the prefix's largest scale, so what a scale counts
// as at least goes into the state with it.
//
// What bounds it: for items of up to 128 rows shared memory, where a widened tile of head_dim 128 is written and read
// for 1024 cycles (codes in, out, operands in, K and V by the matrix instructions); it takes 1250.  For wider ones the
// softmax's instructions with 1536 cycles of shared memory behind them; 2600.  8 groups of 8 rows and
// 8 key/value heads with 8 query heads each, 16384 keys, take 84 us (29% of the tensor pipes, 45% of the issue slots), one
// of 64 rows, 32768 keys, 86 (40%, 52%); 10 to 15 us of it are an item's beginning, a chain of loads (table, codes, scales, q, 2 to 3 us each while all CTAs
// begin), and its part's way out.
//
// Work split: the CTAs take equal contiguous shares of all tiles of all items, an item of 256 rows counted
// twice; what a share has of an item is a part, and a second launch joins them.
#include <type_traits>

#include "kda_kvcache_attention.cuh"
#include "kda_ptx.cuh"
#include "kda_tcgen05.cuh"

namespace kda {
namespace {

using namespace ptx;

constexpr int kRows = 128, kKeys = 64, kBlocks = kKeys / 16, kLanes = 2 * kRows;
constexpr int kSoftWarps = 8, kIssuer = 8, kWidenFirst = 10, kSlots = 3, kWidenWarps = 2 * kSlots;  // places of K and of V, a warp for each
constexpr int kThreads = 16 * 32;  // (a seventeenth warp would leave 96 registers a thread)
constexpr int kMaxListed = 128;  // groups whose prefix sums fit in shared memory
constexpr float kGrowth = 8.f, kLift = kBlockLift;
constexpr int64_t kWaitLimit = 1ll << 20;
constexpr uint32_t kBarSoft = 1, kBarGroup = 2;  // among the softmax groups; q of one of them is there (and the next number)
constexpr int kMetaTiles = 16, kBatch = 8;       // tiles whose scales are kept; of a widening warp's, whose pages it holds
constexpr int kPrefetch = 2;                     // of its tiles ahead that L2 is asked for
template <int kDim> constexpr int kTileBytes = kKeys * kDim * 2;
template <int kDim> constexpr int kQBytes = kRows * kDim * 2;
template <int kDim> constexpr size_t kSmemBytes = (size_t)2 * kSlots * kTileBytes<kDim> + 2 * kQBytes<kDim> + kWidenWarps * kKeys * kDim + 1024;

struct Meta {  // scale of k and log2 of v's for 16 keys; k negative where the page is missing
    float k, v;
};

// An item's place: group, head, block of query rows, and what its share is counted in.
struct Item {
    int group, head, block, rows;  // query rows of the block
    bool wide;                     // more than kRows of them: both softmax groups have every tile
    int tiles;
    int64_t first;                 // of its work
    int64_t number;
    __device__ __forceinline__ int64_t work() const { return (int64_t)tiles * (wide ? 2 : 1); }
    // Steps of a softmax group in so many tiles: its tile number i is tile i, or 2 i + group.
    __device__ __forceinline__ int steps(int tiles, int grp) const { return wide ? tiles : (tiles + 1 - grp) / 2; }
    __device__ __forceinline__ int tile_of(int grp, int i) const { return wide ? i : 2 * i + grp; }
    __device__ __forceinline__ int tile_at(int64_t offset) const { return (int)(wide ? (offset + 1) / 2 : offset); }
};
// Work and items of one key/value head of a group.
__device__ __forceinline__ int64_t head_work(const SharedGroup& g, int heads) {  // heads: query heads of a key/value head
    const uint32_t rows = (uint32_t)(g.tokens * heads), tail = rows % kLanes;  // (the host sees to it that they fit)
    return (int64_t)(rows / kLanes * 2 + (tail > kRows ? 2 : tail > 0 ? 1 : 0)) * (g.shared / kKeys);
}
__device__ __forceinline__ int head_items(const SharedGroup& g, int heads) { return (int)(((uint32_t)(g.tokens * heads) + kLanes - 1) / kLanes); }
// Quotients of numbers that hardly ever need 64 bits (whose division takes some 700 cycles).
__device__ __noinline__ int64_t long_quotient(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) { return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : long_quotient(a, b); }
// The item of a group that work number w belongs to.
__device__ __forceinline__ Item item_at(const SharedGroup& g, int group, int heads, int64_t w, int64_t first, int64_t first_item) {
    Item it;
    const int64_t each = head_work(g, heads), per = (int64_t)g.shared / kKeys * 2;
    const int blocks = head_items(g, heads);
    it.group = group;
    it.head = (int)quotient(w - first, each);
    const int64_t off = w - first - it.head * each;
    it.block = (int)min(quotient(off, per), (int64_t)blocks - 1);
    it.rows = min(g.tokens * heads - it.block * kLanes, kLanes);
    it.wide = it.rows > kRows;
    it.tiles = g.shared / kKeys;
    it.first = first + it.head * each + it.block * per;
    it.number = first_item + (int64_t)it.head * blocks + it.block;
    return it;
}

// 16 bytes of codes widened.
__device__ __forceinline__ void widen(const uint4& r, uint4& lo, uint4& hi) {
    lo = make_uint4(widen2(r.x), widen2(r.x >> 16), widen2(r.y), widen2(r.y >> 16));
    hi = make_uint4(widen2(r.z), widen2(r.z >> 16), widen2(r.w), widen2(r.w >> 16));
}

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ AttentionParams p) {
    constexpr uint32_t kLbo = 128, kSbo = kDim * 16;  // K-major core matrices: along the reduction, along rows
    constexpr uint32_t kBoxBytes = kKeys * 128;       // 64 channels of V
    constexpr uint32_t kColO = 128, kColGroup = 256;  // tensor memory of a softmax group: S and P, O
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ int64_t s_first[kMaxListed + 1], s_item[kMaxListed + 1], s_scan[kThreads / 32];
    __shared__ float s_ml[3][kLanes];
    __shared__ __align__(16) Meta s_meta[kMetaTiles][kBlocks];
    __shared__ volatile int s_bad;  // a wait ran out
    __shared__ __align__(8) uint64_t s_bar[4 * kSlots + 12 + 2 * kWidenWarps + 2];
    __shared__ uint32_t s_tmem;
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* v_sm = smem;
    unsigned char* k_sm = v_sm + kSlots * kTileBytes<kDim>;
    unsigned char* q_sm = k_sm + kSlots * kTileBytes<kDim>;
    unsigned char* raw_sm = q_sm + 2 * kQBytes<kDim>;

    const CacheParams& c = p.c;
    // (Of a value from a shuffle the compiler knows that it is the same for the warp.)
    auto uniform = [](auto x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int heads = p.q_heads / c.heads;
    const int page_shift = __ffs(c.page_tokens) - 1;
    const int64_t block_bytes = (int64_t)c.page_tokens * kDim;
    const uint32_t bars = smem_u32(s_bar);
    auto k_full = [&](uint32_t n) { return bars + 8 * (n % kSlots); };
    auto k_empty = [&](uint32_t n) { return bars + 8 * (kSlots + n % kSlots); };
    auto v_full = [&](uint32_t n) { return bars + 8 * (2 * kSlots + n % kSlots); };
    auto v_empty = [&](uint32_t n) { return bars + 8 * (3 * kSlots + n % kSlots); };
    auto s_full = [&](int grp, uint32_t n) { return bars + 8 * (4 * kSlots + 2 * grp + (n & 1)); };  // S of a step is there
    auto o_done = [&](int grp, uint32_t n) { return bars + 8 * (4 * kSlots + 4 + 2 * grp + (n & 1)); };  // O += P V of a step is done
    auto p_full = [&](int grp, uint32_t n) { return bars + 8 * (4 * kSlots + 8 + 2 * grp + (n & 1)); };  // P of a step is there
    const uint32_t raw_full = bars + 8 * (4 * kSlots + 12);  // codes of half a tile of a widening warp
    const uint32_t drained = raw_full + 8 * 2 * kWidenWarps;  // after a wait that ran out: an issuing warp's products

    if (tid == 0) {
        for (uint32_t i = 0; i < kSlots; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(v_full(i), 1);
            mbar_init(k_empty(i), 2);  // both groups' issuing warps, also of tiles that one has alone
            mbar_init(v_empty(i), 2);
        }
        for (int grp = 0; grp < 2; ++grp) {
            mbar_init(s_full(grp, 0), 2);  // the product, and the issuing warp, which has seen the tile's scales
            mbar_init(s_full(grp, 1), 2);
            mbar_init(o_done(grp, 0), 1);
            mbar_init(o_done(grp, 1), 1);
            mbar_init(p_full(grp, 0), 4);
            mbar_init(p_full(grp, 1), 4);
        }
        for (int i = 0; i < 2 * kWidenWarps; ++i) mbar_init(raw_full + 8 * i, 2);
        for (int grp = 0; grp < 2; ++grp) mbar_init(drained + 8 * grp, 1);
        fence_mbar_init();
        s_bad = 0;
    }
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    follow_stream();
    const bool listed = p.groups <= kMaxListed;
    int64_t* first = listed ? s_first : p.first_work;
    int64_t* first_item = listed ? s_item : p.first_item;
    if (p.groups <= 32) {  // (a warp's work, without the blocks' barriers)
        if (warp == 0) {
            const SharedGroup sg = lane < p.groups ? p.group[lane] : SharedGroup{0, 0, 0, 0, 0};
            const int64_t work = head_work(sg, heads) * c.heads, items = (int64_t)head_items(sg, heads) * c.heads;
            int64_t x = work, y = items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) x += u, y += v;
            }
            if (lane < p.groups) first[lane + 1] = x, first_item[lane + 1] = y;
            if (lane == 0) first[0] = 0, first_item[0] = 0;
        }
    } else {
        scan_rows<kThreads>(p.groups, first, s_scan, [&](int g) -> int64_t { return g < p.groups ? head_work(p.group[g], heads) * c.heads : 0; });
        __syncthreads();
        scan_rows<kThreads>(p.groups, first_item, s_scan, [&](int g) -> int64_t { return g < p.groups ? (int64_t)head_items(p.group[g], heads) * c.heads : 0; });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (blockIdx.x == 0 && listed)
        for (int g = tid; g <= p.groups; g += kThreads) p.first_work[g] = s_first[g], p.first_item[g] = s_item[g];
    const uint32_t tmem = uniform(s_tmem);
    const int64_t all = first[p.groups], per = quotient(all + p.ctas - 1, p.ctas);
    const int64_t w_begin = per * blockIdx.x, w_end = min(all, w_begin + per);
    // After a wait that ran out, all others end at once and what follows is garbage; but what is under way, codes on
    // their way into shared memory and products, is waited for before the CTA gives its memory back.
    auto wait = [&](uint32_t bar, uint32_t phase) {
        if (!mbar_try_wait(bar, phase & 1) && !mbar_wait(bar, phase & 1, s_bad ? 1 : kWaitLimit)) s_bad = 1;
    };
    // For several barriers at once, a lane each (a wait costs 150 cycles also where it is over).
    auto wait_lanes = [&](bool some, uint32_t bar, uint32_t phase) {
        bool done = !some || mbar_test(bar, phase & 1);
        // (Each lane counts for itself and all leave together: they need not have seen the same of s_bad.)
        for (int64_t i = s_bad ? 1 : 64 * kWaitLimit; !__all_sync(0xffffffffu, done || i <= 0); --i)
            if (!done) done = mbar_test(bar, phase & 1);
        if (!done) s_bad = 1;
        __syncwarp();
    };
    uint32_t base = 0;           // tiles before this item
    uint32_t steps[2] = {0, 0};  // steps of the softmax groups before this item

    uint32_t raw_base = 0;       // blocks of a widening warp before this item
    bool stuck = false;          // its codes did not come: it asks for no more
    // Every kind of warps goes through the share's items by itself: body(group, item, its first tile, its tiles).
    auto each_item = [&](auto&& body) {
        for (int64_t w = w_begin; w < w_end;) {
            const int g = row_of(first, p.groups, w);
            const SharedGroup sg = p.group[g];
            const Item it = item_at(sg, g, heads, w, first[g], first_item[g]);
            const int64_t item_end = it.first + it.work();
            const int tile0 = it.tile_at(w - it.first), tiles = it.tile_at(min(item_end, w_end) - it.first) - tile0;
            body(sg, it, tile0, tiles);
            base += tiles;
            steps[0] += it.steps(tiles, 0);
            steps[1] += it.steps(tiles, 1);
            w = item_end;
        }
    };

    if (warp < kSoftWarps) {
        each_item([&](const SharedGroup& sg, const Item& it, int tile0, int tiles) {
            const int grp = warp / 4, t = tid % kRows;
            if (tiles == 0) {  // (half of a wide item's tile)
                float* part_ml = p.part_ml + (it.number + blockIdx.x) * 3 * kLanes + tid;
                part_ml[0] = kNegInf;
                part_ml[kLanes] = 0.f;
                part_ml[2 * kLanes] = kScaleLeast;
                return;
            }
            // Rows of a narrow item stand `copies` times among the 128.
            const int log_spread = it.wide || it.rows > 64 ? 7 : it.rows > 32 ? 6 : 5, spread = 1 << log_spread;
            const int block0 = (t >> log_spread) * (spread / 32);  // its first 16 keys of a tile
            const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16, t_s = tmem + grp * kColGroup + lanes, t_o = t_s + kColO;
            float factor = 0.f;  // of this thread's scores

            // The warp's rows of q as fp16 into shared memory: a load has 8 rows, 64 bytes of each.
            {
                constexpr int kQ = kDim / 32;  // loads of 8 rows
                auto read = [&](int x, uint4 (&to)[kQ]) {
                    const int row = 32 * (warp % 4) + 8 * x + lane % 8, f = it.block * kLanes + (it.wide ? grp * kRows + row : row & (spread - 1));
                    const bool some = f < sg.tokens * heads;
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (sg.begin + (some ? f / heads : 0)) * p.q_stride +
                                                                      (int64_t)(it.head * heads + (some ? f % heads : 0)) * kDim) + lane / 8;
#pragma unroll
                    for (int k = 0; k < kQ; ++k) to[k] = some ? __ldg(src + 4 * k) : make_uint4(0u, 0u, 0u, 0u);
                };
                // (All of them at once: each chain of loads is 2000 cycles and more here.)
                uint4 r[4][kQ];
#pragma unroll
                for (int x = 0; x < 4; ++x) read(x, r[x]);
                unsigned char* dst = q_sm + grp * kQBytes<kDim> + 4 * (warp % 4) * kSbo + lane % 8 * 16 + lane / 8 * kLbo;
                // (Loops that run once or a few times are not unrolled: their instructions come from memory.)
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {
                    float a = 0.f;
#pragma unroll
                    for (int k = 0; k < kQ; ++k) {
                        const uint32_t u[4] = {r[0][k].x, r[0][k].y, r[0][k].z, r[0][k].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float2 v = Act<T>::two(u[y]);
                            a = max3(a, fabsf(v.x), fabsf(v.y));
                        }
                    }
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
                    const int e = row_exponent(a);
                    // The sign of the scale goes with q, so that factors are not negative.
                    const float up = copysignf(exp2f((float)(14 - e)), p.scale);
#pragma unroll
                    for (int k = 0; k < kQ; ++k) {
                        uint32_t u[4] = {r[0][k].x, r[0][k].y, r[0][k].z, r[0][k].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float2 v = Act<T>::two(u[y]);
                            u[y] = pack_half2(v.x * up, v.y * up);
                        }
                        *reinterpret_cast<uint4*>(dst + x * kSbo + 4 * k * kLbo) = make_uint4(u[0], u[1], u[2], u[3]);
                        r[0][k] = r[1][k], r[1][k] = r[2][k], r[2][k] = r[3][k];
                    }
                    const float mine = __shfl_sync(0xffffffffu, exp2f((float)(e - 14)) * fabsf(p.scale), lane % 8);
                    if (lane / 8 == x) factor = mine;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                // (A group without steps does not wait for its issuing warp, so it must not be counted twice by it.)
                if (it.steps(tiles, grp) > 0) named_bar_arrive(kBarGroup + grp, kRows + 32);
            }

            float m = kNegInf, l = 0.f, least = kScaleLeast;  // least: that a log2 of v's scale counts as
            const int n = it.steps(tiles, grp);
            // A tile's scores of this thread, 16 kMine of them.
            auto step = [&](auto count, int i) {
                constexpr int kMine = decltype(count)::value;
                const uint32_t u = steps[grp] + i, t_b = t_s + (u & 1) * kKeys;
                wait(s_full(grp, u), u >> 1);
                tc_fence_after();
                uint32_t sr[16 * kMine];
                if constexpr (kMine == 1) tmem_ld16(t_b + 16 * block0, sr);
                else {
                    tmem_ld32(t_b + 16 * block0, sr);
                    if constexpr (kMine == 4) tmem_ld32(t_b + 32, sr + 32);
                }
                const Meta* metas = s_meta[(base + it.tile_of(grp, i)) % kMetaTiles] + block0;  // (in registers they would spill)
#pragma unroll
                for (int x = 0; x < kMine; ++x) {
                    least = fmaxf(least, metas[x].v - kScaleSpan);
                }
                tmem_wait_ld_regs<16 * kMine>(sr);
                float top = kNegInf;
#pragma unroll
                for (int x = 0; x < kMine; ++x) {
                    const Meta b = metas[x];
                    float y = max3(__uint_as_float(sr[16 * x]), __uint_as_float(sr[16 * x + 1]), __uint_as_float(sr[16 * x + 2]));
                    float z = max3(__uint_as_float(sr[16 * x + 3]), __uint_as_float(sr[16 * x + 4]), __uint_as_float(sr[16 * x + 5]));
#pragma unroll
                    for (int k = 6; k < 14; k += 4) {
                        y = max3(y, __uint_as_float(sr[16 * x + k]), __uint_as_float(sr[16 * x + k + 1]));
                        z = max3(z, __uint_as_float(sr[16 * x + k + 2]), __uint_as_float(sr[16 * x + k + 3]));
                    }
                    y = fmaxf(max3(y, z, __uint_as_float(sr[16 * x + 14])), __uint_as_float(sr[16 * x + 15]));
                    top = fmaxf(top, b.k < 0.f ? kNegInf : fmaf(y, b.k * factor, fmaxf(b.v, least)));  // (not of a missing page)
                }
                // The reference of the weights.
                const float m_new = top > m + kGrowth || m == kNegInf ? fmaxf(m, top) : m;
                const float m_use = m_new == kNegInf ? 0.f : m_new;
                const float half = m == kNegInf ? (m_new == kNegInf ? 1.f : 0.f) : exp2_fast(0.5f * (m - m_use)), fix = half * half;
                m = m_new;
                l = rescaled(l, half);
#pragma unroll
                for (int x = 0; x < kMine; ++x) {
                    const Meta b = metas[x];
                    // (Scores are finite, those of a missing page 0: its weights are 0 by -inf.)
                    const float k = b.k * factor, lv = fmaxf(b.v, least), bias = b.k < 0.f ? kNegInf : lv - m_use + kLift;
                    const uint64_t k2 = pair(k, k), bias2 = pair(bias, bias);
                    uint64_t acc[2] = {0, 0};  // (+0, +0)
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float a, d;
                        unpair(fma2(pair(__uint_as_float(sr[16 * x + j]), __uint_as_float(sr[16 * x + j + 1])), k2, bias2), a, d);
                        a = exp2_fast(a);
                        d = exp2_fast(d);
                        acc[j / 2 % 2] = add2(acc[j / 2 % 2], pair(a, d));
                        sr[8 * x + j / 2] = pack_half2(a, d);  // the weights take the scores' registers
                    }
                    float sum[2];
                    unpair(add2(acc[0], acc[1]), sum[0], sum[1]);
                    l += (sum[0] + sum[1]) * exp2_fast(-lv);
                }
#pragma unroll
                for (int x = 0; x < kMine; ++x) tmem_st8(t_b + 8 * (block0 + x), *reinterpret_cast<uint32_t(*)[8]>(sr + 8 * x));
                // Rare, so taken once more from tensor memory: held in registers until here it cost a step 8%.
                if (fminf(fminf(metas[0].v, metas[kMine > 1].v), fminf(metas[kMine / 2].v, metas[kMine - 1].v)) < least) {
                    tmem_wait_st();
#pragma unroll 1
                    for (int x = 0; x < kMine; ++x) {
                        const float by = exp2_fast(fminf(metas[x].v - least, 0.f));
                        uint32_t w[8];
                        tmem_ld8(t_b + 8 * (block0 + x), w);
                        tmem_wait_ld_regs<8>(w);
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = brought_down(w[j], by);
                        tmem_st8(t_b + 8 * (block0 + x), w);
                    }
                }
                if constexpr (kMine < 4) {  // the other copies' keys
                    const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                    for (int x = 0; x < 4 - kMine; ++x) tmem_st8(t_b + 8 * (x < block0 ? x : x + kMine), zero);
                }
                if (i > 0 && __any_sync(0xffffffffu, fix != 1.f)) {
                    wait(o_done(grp, u - 1), (u - 1) >> 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < kDim; q += 32) {
                        uint32_t o[32];
                        tmem_ld32(t_o + q, o);
                        tmem_wait_ld_regs<32>(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fix);
                        tmem_st32(t_o + q, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(grp, u));
            };
            auto steps_of = [&](auto count) {
                for (int i = 0; i < n; ++i) step(count, i);
            };
            if (log_spread == 7) steps_of(std::integral_constant<int, 4>{});
            else if (log_spread == 6) steps_of(std::integral_constant<int, 2>{});
            else steps_of(std::integral_constant<int, 1>{});
            if (n > 0) {
                wait(o_done(grp, steps[grp] + n - 1), (steps[grp] + n - 1) >> 1);
                tc_fence_after();
            }
            // The part: of a wide item 256 rows as they are; of the others the lanes that stand for the same row are
            // joined in shared memory first, in q's place.
            const int64_t slot = it.number + blockIdx.x;
            const int at = grp * kRows + t;
            float* part_ml = p.part_ml + slot * 3 * kLanes;
            float scale = 1.f;
            if (!it.wide) {
                named_bar_sync(kBarSoft, kLanes);  // both groups are done with q
                s_ml[0][at] = m, s_ml[1][at] = l, s_ml[2][at] = least;
                named_bar_sync(kBarSoft, kLanes);
                const int mine = at & (spread - 1);
                float top = kNegInf, sum = 0.f;
#pragma unroll 1
                for (int x = mine; x < kLanes; x += spread) top = fmaxf(top, s_ml[0][x]), least = fmaxf(least, s_ml[2][x]);
                const float use = top == kNegInf ? 0.f : top;
#pragma unroll 1
                for (int x = mine; x < kLanes; x += spread) sum += rescaled(s_ml[1][x], exp2_fast(0.5f * (s_ml[0][x] - use)));
                scale = exp2_fast(0.5f * (m - use));
                scale *= scale;
                m = top, l = sum;
            }
            if (it.wide || at < spread) {
                part_ml[at] = m;
                part_ml[kLanes + at] = l;
                part_ml[2 * kLanes + at] = least;
            }
            float* part_o = p.part_o + slot * kDim * kLanes;
            if (it.wide) {
#pragma unroll 1
                for (int q = 0; q < kDim; q += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_o + q, o);
                    tmem_wait_ld_regs<32>(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) part_o[(q + k) * kLanes + at] = __uint_as_float(o[k]);
                }
            } else {
                constexpr int kPass = kDim / 2;                      // channels that q's place holds for 256 lanes
                float* s_o = reinterpret_cast<float*>(q_sm);
                const int mine = at & (spread - 1), copies = kLanes >> log_spread, first_ch = at >> log_spread;
#pragma unroll 1
                for (int pass = 0; pass < kDim; pass += kPass) {
                    if (pass > 0) named_bar_sync(kBarSoft, kLanes);
#pragma unroll 1
                    for (int q = 0; q < kPass; q += 32) {
                        uint32_t o[32];
                        if (n > 0) {
                            tmem_ld32(t_o + pass + q, o);
                            tmem_wait_ld_regs<32>(o);
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) s_o[(q + k) * kLanes + at] = n > 0 ? __uint_as_float(o[k]) * scale : 0.f;
                    }
                    named_bar_sync(kBarSoft, kLanes);
                    constexpr int kMost = 8;  // copies of 32 rows
#pragma unroll 2
                    for (int k = first_ch; k < kPass; k += copies) {
                        float o[kMost];
#pragma unroll
                        for (int x = 0; x < kMost; ++x) o[x] = x < copies ? s_o[k * kLanes + mine + (x << log_spread)] : 0.f;
                        part_o[(pass + k) * kLanes + mine] = ((o[0] + o[1]) + (o[2] + o[3])) + ((o[4] + o[5]) + (o[6] + o[7]));
                    }
                }
            }
            tc_fence_before();  // (the next S and O follow on this thread's arrivals)
            named_bar_sync(kBarSoft, kLanes);  // q's place is free
        });
    } else if (warp < kWidenFirst) {
        const int grp = warp - kIssuer;
        each_item([&](const SharedGroup&, const Item& it, int tile0, int tiles_any) {
            const int tiles = uniform(tiles_any);
            if (tiles == 0) return;
            const bool wide = uniform((int)it.wide);
            const int n = it.steps(tiles, grp);
            const uint32_t t_grp = tmem + grp * kColGroup;
            const uint64_t qd = sdesc(smem_u32(q_sm + grp * kQBytes<kDim>), kLbo, kSbo);
            // Waits for the tile, and for the one before it, which the other group has alone, and passes that one.
            auto wait_tile = [&](uint32_t full, uint32_t empty, int tile, bool also, uint32_t bar, uint32_t phase) {
                const uint32_t number = base + tile, before = number - 1;
                const bool passes = !wide && tile > 0;
                wait_lanes(lane == 0 ? also : lane == 1 ? tile < tiles : lane == 2 && passes, lane == 0 ? bar : full + 8 * ((lane == 1 ? number : before) % kSlots),
                           lane == 0 ? phase : (lane == 1 ? number : before) / kSlots);
                if (lane == 2 && passes) mbar_arrive(empty + 8 * (before % kSlots));
            };
            auto issue_s = [&](int i) {
                const int tile = wide ? i : 2 * i + grp;
                const uint32_t number = uniform(base + tile), u = uniform(steps[grp] + i);
                wait_tile(k_full(0), k_empty(0), tile, i > 1, o_done(grp, u), (u - 2) >> 1);  // S takes the place of its weights
                tc_fence_after();
                const uint64_t kd = sdesc(smem_u32(k_sm + number % kSlots * kTileBytes<kDim>), kLbo, kSbo);
#pragma unroll
                for (int kk = 0; kk < kDim / 16; ++kk)  // (a step is 2 core matrices: 16 units of 16 bytes)
                    mma_ss_one(t_grp + (u & 1) * kKeys, qd + kk * (2 * kLbo / 16), kd + kk * (2 * kLbo / 16), idesc_f16(kKeys, false), kk > 0);
                commit_one(s_full(grp, u));
                commit_one(k_empty(number));
                if (lane == 1) mbar_arrive(s_full(grp, u));  // (the lane that has waited for the tile)
            };
            if (n > 0) {
                named_bar_sync(kBarGroup + grp, kRows + 32);
                tc_fence_after();
                issue_s(0);
            }
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const uint32_t number = uniform(base + (wide ? i : 2 * i + grp)), u = uniform(steps[grp] + i);
                if (i + 1 < n) issue_s(i + 1);
                wait_tile(v_full(0), v_empty(0), wide ? i : 2 * i + grp, true, p_full(grp, u), u >> 1);
                tc_fence_after();
                const uint64_t vd = sdesc(smem_u32(v_sm + number % kSlots * kTileBytes<kDim>), kBoxBytes, 1024) | ((uint64_t)2 << 61);
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_ts_one(t_grp + kColO, t_grp + (u & 1) * kKeys + kk * 8, vd + kk * (2048 / 16), idesc_f16(kDim, true), i > 0 || kk > 0);
                commit_one(o_done(grp, u));
                commit_one(v_empty(number));
            }
            // A last tile of the other group.
            const int last = 2 * n + grp - 1;  // (n tiles of this group were 2 i + grp, i < n)
            if (!wide && last >= 0 && last < tiles && (last & 1) != grp) {
                wait_lanes(lane < 2, lane == 0 ? k_full(base + last) : v_full(base + last), (base + last) / kSlots);
                if (lane < 2) mbar_arrive(lane == 0 ? k_empty(base + last) : v_empty(base + last));
            }
        });
    } else {
        each_item([&](const SharedGroup& sg, const Item& it, int tile0, int tiles) {
            // This warp's tiles: those whose numbers fall on its place.  A lane has the page (of 16 keys) and the scales of block
            // lane % 4 of one of a batch of them.
            const int mine = warp - kWidenFirst, place = mine % kSlots;
            const bool v = mine >= kSlots;
            const int j0 = (place + kSlots - (int)(base % kSlots)) % kSlots, own = (tiles - j0 + kSlots - 1) / kSlots;
            if (own <= 0) return;
            const int32_t* table = c.tables + (int64_t)sg.row * c.width;
            auto first_key = [&](int n) { return (tile0 + j0 + n * kSlots) * kKeys; };
            auto entry_of = [&](int batch) {
                const int n = batch * kBatch + lane / kBlocks;
                return n < own ? table[(first_key(n) + lane % kBlocks * 16) >> page_shift] : -1;
            };
            auto checked = [&](int32_t x, int batch) {
                if (x >= 0 && x < c.pages) return x;
                if (batch * kBatch + lane / kBlocks < own) report(c.status, kStatusBadIndex);
                return -1;
            };
            auto meta_of = [&](int32_t page) {
                const int64_t at = (int64_t)max(page, 0) * c.heads + it.head;
                return page < 0 ? Meta{-1.f, 1.f} : Meta{c.k_scale[at], c.v_scale[at]};
            };
            int32_t pages = checked(entry_of(0), 0), pages_next = -1;
            Meta meta = meta_of(pages), meta_next = Meta{-1.f, 1.f};
            const uint8_t* codes = v ? c.v_codes : c.k_codes;
            auto page_of = [&](int n, int batch) {  // for the first lanes, of this batch or the next
                return __shfl_sync(0xffffffffu, n / kBatch > batch ? pages_next : pages, (n % kBatch * kBlocks + lane) & 31);
            };
            auto codes_of = [&](int n, int32_t page) {
                return codes + ((int64_t)page * c.heads + it.head) * block_bytes + ((first_key(n) + lane * 16) & (c.page_tokens - 1)) * kDim;
            };
            unsigned char* own_raw = raw_sm + mine * kKeys * kDim;
            // This warp's own copies, which wait for nobody: with the whole limit also after another wait ran out.
            auto wait_codes = [&](uint32_t bar, uint32_t phase) {
                const bool done = stuck || mbar_try_wait(bar, phase & 1) || mbar_wait(bar, phase & 1, kWaitLimit);
                if (!__all_sync(0xffffffffu, done)) s_bad = 1, stuck = true;
            };
            // Asks for the codes of half a tile, a lane for 16 keys.
            auto request = [&](int n, int half, int batch) {
                const int32_t page = page_of(n, batch);
                if (lane / 2 == half) {
                    const uint32_t bar = raw_full + 8 * (2 * mine + half);
                    if (page >= 0) {
                        mbar_arrive_expect_tx(bar, 16 * kDim);
                        bulk_load(smem_u32(own_raw) + lane * 16 * kDim, codes_of(n, page), 16 * kDim, bar);
                    } else {
                        mbar_arrive(bar);
                    }
                }
            };
            if (!stuck) {
                request(0, 0, 0);
                request(0, 1, 0);
            }
            // A lane's pieces of 32 keys: key lane % 8 and every eighth from it, and of them the 16 channels that go with lane / 8 and
            // h: a diagonal, eight lanes have eight keys, and together all banks of what is read and of what is written.
            const int key = lane % 8;
            auto channels = [&](int h) {
                const int turn = lane / 8 + 4 * h;
                if (kDim == 128) return (key + turn) % 8;
                const int r = key >> 1;
                return ((r << 1) ^ ((r >> 1) * 3) ^ turn) & 3;
            };
            const uint32_t row8 = v ? 8 * 128 : kSbo;
            unsigned char* dst = (v ? v_sm + key * 128 : k_sm + key * 16) + place * kTileBytes<kDim>;
#pragma unroll 1
            for (int n = 0; n < own; ++n) {
                const int inside = n % kBatch, batch = n / kBatch;
                if (inside == 0) pages_next = entry_of(batch + 1);
                if (inside == kBatch / 2) {
                    pages_next = checked(pages_next, batch + 1);
                    meta_next = meta_of(pages_next);
                }
                if (n + kPrefetch < own && (inside + kPrefetch < kBatch || inside >= kBatch / 2)) {
                    const int32_t ahead = page_of(n + kPrefetch, batch);
                    if (lane < kBlocks && ahead >= 0) bulk_prefetch(codes_of(n + kPrefetch, ahead), 16 * kDim);
                }
                const uint32_t number = base + j0 + n * kSlots;
                // What is missing is zero, and what a scale of 0 makes of V, to leave no trace.  (K does without the scales until its
                // codes are widened: the first ones are 3 us on their way.)
                const int block = inside * kBlocks + lane % kBlocks;
                const bool there = __shfl_sync(0xffffffffu, pages, block) >= 0;
                unsigned some = __ballot_sync(0xffffffffu, there);
                if (v) {  // (the whole warp)
                    const float vs = __shfl_sync(0xffffffffu, meta.v, block);
                    some &= __ballot_sync(0xffffffffu, vs > 0.f);
                }
                wait(v ? v_empty(number) : k_empty(number), (number / kSlots & 1) ^ 1);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    wait_codes(raw_full + 8 * (2 * mine + half), raw_base + n);
                    const unsigned char* src = own_raw + half * 32 * kDim + key * kDim;
                    uint4 raw[kDim / 64][4];
#pragma unroll
                    for (int h = 0; h < kDim / 64; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            raw[h][i] = some >> (2 * half + i / 2) & 1 ? *reinterpret_cast<const uint4*>(src + i * 8 * kDim + channels(h) * 16) : make_uint4(0u, 0u, 0u, 0u);
                    // K: core matrices of 8 keys and 16 bytes; V: rows of 128 bytes, 64 channels, their 16-byte pieces in the order that the
                    // 128-byte swizzle wants.
#pragma unroll
                    for (int h = 0; h < kDim / 64; ++h) {
                        const int ch = channels(h);
                        unsigned char* lo_at = dst + half * 4 * row8 + (v ? ch / 4 * kBoxBytes + ((2 * ch % 8) ^ key) * 16 : 2 * ch * kLbo);
                        unsigned char* hi_at = dst + half * 4 * row8 + (v ? ch / 4 * kBoxBytes + ((2 * ch % 8 + 1) ^ key) * 16 : (2 * ch + 1) * kLbo);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint4 lo, hi;
                            widen(raw[h][i], lo, hi);
                            *reinterpret_cast<uint4*>(lo_at + i * row8) = lo;
                            *reinterpret_cast<uint4*>(hi_at + i * row8) = hi;
                        }
                    }
                    if (half && !v) {
                        const Meta of{__shfl_sync(0xffffffffu, meta.k, block), __shfl_sync(0xffffffffu, meta.v, block)};
                        if (lane < kBlocks) s_meta[number % kMetaTiles][lane] = Meta{of.k, log2f(of.v)};
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (half && lane == 0) mbar_arrive(v ? v_full(number) : k_full(number));
                    if (n + 1 < own && !stuck) request(n + 1, half, batch);
                }
                if (inside == kBatch - 1) {
                    pages = pages_next;
                    meta = meta_next;
                }
            }
            raw_base += own;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (s_bad) {  // (the same for all from here on)
        if (tid == 0) report(c.status, kStatusTimeout);
        if (warp == kIssuer || warp == kIssuer + 1) {
            commit_one(drained + 8 * (warp - kIssuer));
            mbar_wait(drained + 8 * (warp - kIssuer), 0, kWaitLimit);
        }
        __syncthreads();
    }
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

// Joins an item's parts into the state: blockIdx.x counts items, blockIdx.y kJoinCh channels.  A thread has a query
// row, for some of the parts.
constexpr int kJoinThreads = 256, kJoinCh = 16;

template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ AttentionParams p) {
    __shared__ float s_part[kJoinCh + 3][kJoinThreads];
    const int tid = threadIdx.x, d0 = blockIdx.y * kJoinCh, heads = p.q_heads / p.c.heads;
    follow_stream();
    const int64_t number = blockIdx.x, all = p.first_work[p.groups];
    if (number >= p.first_item[p.groups]) return;
    const int g = row_of(p.first_item, p.groups, number);
    const SharedGroup sg = p.group[g];
    const int64_t first_item = p.first_item[g], first_work = p.first_work[g];
    const int blocks = head_items(sg, heads);
    const int64_t head = quotient(number - first_item, blocks), block = number - first_item - head * blocks;
    const Item it = item_at(sg, g, heads, first_work + head * head_work(sg, heads) + block * (sg.shared / kKeys * 2), first_work, first_item);
    const int64_t per = quotient(all + p.ctas - 1, p.ctas), u0 = quotient(it.first, per), u1 = quotient(it.first + it.work() - 1, per);
    const int log_lanes = it.rows > 128 ? 8 : it.rows > 64 ? 7 : it.rows > 32 ? 6 : 5, shares = kJoinThreads >> log_lanes;
    const int lane = tid & ((1 << log_lanes) - 1), share = tid >> log_lanes;

    float top = kNegInf, sum = 0.f, least = kScaleLeast, acc[kJoinCh];
#pragma unroll
    for (int d = 0; d < kJoinCh; ++d) acc[d] = 0.f;
    auto add = [&](float mk, float lk, float least_k, const float* o) {
        least = fmaxf(least, least_k);
        const float m = fmaxf(top, mk), use = m == kNegInf ? 0.f : m;
        const float ha = exp2_fast(0.5f * (top - use)), hb = exp2_fast(0.5f * (mk - use)), a = ha * ha, b = hb * hb;
        top = m;
        sum = rescaled(sum, ha) + rescaled(lk, hb);
#pragma unroll
        for (int d = 0; d < kJoinCh; ++d) acc[d] = acc[d] * a + (mk == kNegInf ? 0.f : o[d] * b);
    };
    constexpr int kAhead = 3;
    for (int64_t u = u0 + share; u <= u1; u += kAhead * shares) {
        float mk[kAhead], lk[kAhead], least_k[kAhead], o[kAhead][kJoinCh];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int64_t at = u + x * shares, slot = it.number + at;
            if (at > u1) continue;
            mk[x] = p.part_ml[slot * 3 * kLanes + lane];
            lk[x] = p.part_ml[slot * 3 * kLanes + kLanes + lane];
            least_k[x] = p.part_ml[slot * 3 * kLanes + 2 * kLanes + lane];
#pragma unroll
            for (int d = 0; d < kJoinCh; ++d) o[x][d] = p.part_o[(slot * kDim + d0 + d) * kLanes + lane];
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            if (u + x * shares <= u1) add(mk[x], lk[x], least_k[x], o[x]);
    }
    const int used = (int)min((int64_t)shares, u1 - u0 + 1);  // shares that have a part
    if (share && share < used) {
        s_part[kJoinCh][tid] = top;
        s_part[kJoinCh + 1][tid] = sum;
        s_part[kJoinCh + 2][tid] = least;
#pragma unroll
        for (int d = 0; d < kJoinCh; ++d) s_part[d][tid] = acc[d];
    }
    if (used > 1) __syncthreads();
    if (share || lane >= it.rows) return;
    for (int x = 1; x < used; ++x) {
        float o[kJoinCh];
#pragma unroll
        for (int d = 0; d < kJoinCh; ++d) o[d] = s_part[d][(x << log_lanes) + lane];
        add(s_part[kJoinCh][(x << log_lanes) + lane], s_part[kJoinCh + 1][(x << log_lanes) + lane], s_part[kJoinCh + 2][(x << log_lanes) + lane], o);
    }
    const int f = it.block * kLanes + lane;
    const int64_t state = (sg.begin + f / heads) * p.q_heads + it.head * heads + f % heads;
    if (d0 == 0) p.state_ml[state] = make_float4(top, sum, least, 0.f);
#pragma unroll
    for (int d = 0; d < kJoinCh; d += 4) *reinterpret_cast<float4*>(p.state_o + state * kDim + d0 + d) = make_float4(acc[d], acc[d + 1], acc[d + 2], acc[d + 3]);
}

template <typename T, int kDim>
cudaError_t launch_dim(const AttentionParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(prefix_kernel<T, kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<kDim>);
    if (e != cudaSuccess) return e;
    e = launch_early(prefix_kernel<T, kDim>, dim3(p.ctas), kThreads, kSmemBytes<kDim>, stream, 1, p);
    if (e != cudaSuccess) return e;
    return launch_early(prefix_join_kernel<kDim>, dim3((unsigned)prefix_items(p, p.least), kDim / kJoinCh), kJoinThreads, 0, stream, 1, p);
}

}  // namespace

// (Groups that share have at least `least` rows with tokens each.)
int64_t prefix_items(const AttentionParams& p, int32_t least) {
    const int64_t most = (p.c.tokens < p.c.rows ? p.c.tokens : p.c.rows) / least;
    return (p.c.tokens * (p.q_heads / p.c.heads) / kLanes + (most < p.groups ? most : p.groups)) * p.c.heads;
}
cudaError_t launch_prefix(const AttentionParams& p, bool f16, cudaStream_t stream) {
    if (p.c.dim == 64) return f16 ? launch_dim<__half, 64>(p, stream) : launch_dim<__nv_bfloat16, 64>(p, stream);
    return f16 ? launch_dim<__half, 128>(p, stream) : launch_dim<__nv_bfloat16, 128>(p, stream);
}

}  // namespace kda
