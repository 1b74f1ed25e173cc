// kda_kvcache_attention.cu -- causal attention over the 8-bit paged cache, for one or a few
// new tokens a row.
//
// Query rows (token, query head of a group) that share a key/value head go through the cache
// together: an item is kCols = 8 kNT such rows of one (row, key/value head), so the codes are
// read once for a whole group.  HBM-bound for single tokens: 2 dim bytes per cached token and
// key/value head, each read once.
//
// Both products run on m16n8k16 matrix instructions with the keys (then the channels) as the
// 16-row side and the query rows as the 8-column side: groups of up to 8 heads waste nothing,
// and S^T's fragments become the second product's operand after an 8 x 8 transpose in
// registers.  Codes go from global memory to registers in 16-byte loads and are widened there
// (e4m3 is exact in fp16); the order of the channels within the reduction is free as long as
// q has the same one, so the loads need no shared memory and warps run without barriers:
//   S^T = K Q^T     thread (g, t) loads 16 channels at 16 t (and 64 + 16 t) of keys g, g + 8
//   O^T = V^T P^T   thread (g, t) loads 16 channels at 16 g of keys 2t, 2t + 1, 2t + 8, 2t + 9
// The tcgen05 path would need the codes widened through shared memory for a 128-row operand
// that single tokens cannot fill; the loads, not the products, are the bound here.
//
// q is scaled by a power of two per row so that its largest magnitude is in [2^14, 2^15) and
// becomes fp16 without loss (bf16 has fewer bits; what falls below fp16's range is 2^-38 of the
// largest).  Softmax weights are fp16 relative to the running maximum; each page's v scale
// enters as its ratio to the largest one met, so weights stay in [0, 1].  Running maximum,
// sums, outputs and the joined parts are fp32.
//
// Work split: every item has one tile (128 keys, 32 a warp) per 128 cached tokens; the CTAs
// take equal contiguous shares of all tiles of all items in order, however long the rows
// are.  An item that lies in one share is written at once; the parts of the others are joined
// by a second launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kTile = 128, kSlab = 32;  // keys of a tile, and of a warp in it
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ uint32_t widen2(uint32_t codes) {  // two e4m3 codes (low 16 bits)
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T> struct Act;
template <> struct Act<__nv_bfloat16> {
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Act<__half> {
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};

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
// Cached tokens of row r that its table has places for.
__device__ __forceinline__ int row_length(const CacheParams& c, int r) {
    const int len = c.lens[r];
    const int64_t room = (int64_t)c.width * c.page_tokens;
    if (len < 0 || len > room) report(c.status, kStatusBadIndex);
    return len < 0 ? 0 : len > room ? (int)room : len;
}
__device__ __forceinline__ int row_tiles(int len) { return len > kTile ? (len + kTile - 1) / kTile : 1; }

// first[r] = tiles of all items of the rows before r; first[rows] = all.  Items of a row: column
// blocks (kCols query rows each) by key/value heads.  The whole block calls it; s: 5 values.
__device__ void scan_rows(const AttentionParams& p, int cols, int64_t* first, int64_t* s) {
    const CacheParams& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = p.q_heads / c.heads;
    int64_t base = 0;
    for (int r0 = 0; r0 < c.rows; r0 += kThreads) {
        const int r = r0 + tid;
        int64_t w = 0;
        if (r < c.rows) {
            int64_t begin;
            const int n = row_tokens(c, r, begin);
            w = ((int64_t)n * group + cols - 1) / cols * c.heads * row_tiles(row_length(c, r));
        }
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
        if (r < c.rows) first[r] = before + x - w;
        for (int i = 0; i < kWarps; ++i) base += s[i];
        __syncthreads();
    }
    if (tid == 0) first[c.rows] = base;
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

struct Item {
    int row, head, block;  // cache row, key/value head, column block
    int n, len, tiles;     // new tokens, cached tokens and tiles of the row
    int64_t begin;         // first new token
    int64_t first;         // first work number
};
__device__ __forceinline__ Item item_of(const AttentionParams& p, const int64_t* first, int64_t w) {
    Item it;
    it.row = row_of(first, p.c.rows, w);
    it.n = row_tokens(p.c, it.row, it.begin);
    it.len = row_length(p.c, it.row);
    it.tiles = row_tiles(it.len);
    const int64_t i = (w - first[it.row]) / it.tiles;
    it.head = (int)(i % p.c.heads);
    it.block = (int)(i / p.c.heads);
    it.first = first[it.row] + i * it.tiles;
    return it;
}

// Largest share of one CTA, and the CTA that work number w falls to.
__device__ __forceinline__ int64_t share_of(int64_t all, int ctas) { return (all + ctas - 1) / ctas; }

template <typename T, int kDim, int kNT>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttentionParams p) {
    constexpr int kCols = 8 * kNT;
    constexpr int kHalves = kDim / 64;   // 16-byte loads of a key by a thread
    constexpr int kSteps = kDim / 16;    // reduction steps of S^T
    constexpr int kMT = kDim / 16;       // 16-channel tiles of O^T
    constexpr int kVWords = kDim / 32;   // 4-byte words of a V load
    constexpr int kPad = kDim + 4;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float* s_o = reinterpret_cast<float*>(smem_raw);                 // [warps][kCols][kPad]
    float* s_ml = s_o + kWarps * kCols * kPad;                       // [warps][kCols][2]
    __shared__ int64_t s_scan[kWarps];

    const CacheParams& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int group = p.q_heads / c.heads;
    const int page_shift = __ffs(c.page_tokens) - 1;

    // Every CTA needs the rows' prefix; each one writes the same values.
    scan_rows(p, kCols, p.first_work, s_scan);
    __syncthreads();
    const int64_t all = p.first_work[c.rows];
    const int64_t per = share_of(all, p.ctas);
    int64_t w = per * blockIdx.x;
    const int64_t w_end = min(all, w + per);
    const int64_t w_begin = w;

    while (w < w_end) {
        const Item it = item_of(p, p.first_work, w);
        const int64_t item_end = it.first + it.tiles;
        const int tile0 = (int)(w - it.first);
        int tile1 = (int)(min(item_end, w_end) - it.first);

        // Columns of this thread: kNT pairs (8 nt + 2 t, + 1) for S^T and O^T, rows g for q.
        const int rows_all = it.n * group, row0 = it.block * kCols;
        // Last key any column of this block sees, plus one.
        const int last_token = (min(rows_all, row0 + kCols) - 1) / group;
        const int seen_max = min(it.len, max(0, it.len - it.n + last_token + 1));
        tile1 = min(tile1, (seen_max + kTile - 1) / kTile);
        const int first_token = row0 / group;
        const int seen_min = max(0, min(it.len, it.len - it.n + first_token + 1));

        uint32_t q[kNT][kSteps][2];
        float q_scale[kNT];  // of column 8 nt + g
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int f = row0 + nt * 8 + g;
            const bool there = f < rows_all;
            const T* src = static_cast<const T*>(p.q) + (it.begin + (there ? f / group : 0)) * p.q_stride +
                           (int64_t)(it.head * group + (there ? f % group : 0)) * kDim;
            float x[kHalves][16];
            float a = 0.f;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = there ? reinterpret_cast<const uint4*>(src + 64 * h + 16 * t)[i] : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 y = Act<T>::two(u[k]);
                        x[h][8 * i + 2 * k] = y.x;
                        x[h][8 * i + 2 * k + 1] = y.y;
                        a = fmaxf(a, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            // a in [2^e, 2^(e+1)): times 2^(14 - e); e limited so that both factors are normal.
            int e = a > 0.f && a < INFINITY ? ilogbf(a) : 0;
            e = max(e, -100);
            const float up = exp2f((float)(14 - e));
            q_scale[nt] = exp2f((float)(e - 14)) * p.scale;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q[nt][4 * h + j][0] = pack_half2(x[h][4 * j] * up, x[h][4 * j + 1] * up);
                    q[nt][4 * h + j][1] = pack_half2(x[h][4 * j + 2] * up, x[h][4 * j + 3] * up);
                }
        }
        // What each column sees and its factor, for this thread's column pairs.
        int seen[kNT][2];
        float factor[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int f = row0 + nt * 8 + 2 * t + i;
                seen[nt][i] = f < rows_all ? max(0, min(it.len, it.len - it.n + f / group + 1)) : 0;
                factor[nt][i] = __shfl_sync(0xffffffffu, q_scale[nt], (2 * t + i) * 4);
            }

        float o[kNT][kMT][4], m[kNT][2], l[kNT][2], ref = 0.f;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            m[nt][0] = m[nt][1] = kNegInf;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < kMT; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }

        const int32_t* table = c.tables + (int64_t)it.row * c.width;
        // Page of the 16 keys from `key` on; -1 past what any column sees.
        auto page_at = [&](int key) {
            if (key >= seen_max) return -1;
            const int32_t x = table[key >> page_shift];
            if (x < 0 || x >= c.pages) {
                if (lane == 0) report(c.status, kStatusBadIndex);
                return -1;
            }
            return x;
        };
        auto block_of = [&](int32_t page, int key) {  // element offset of `key`'s codes
            return (((int64_t)page * c.heads + it.head) * c.page_tokens + (key & (c.page_tokens - 1))) * kDim;
        };
        int32_t pg[2];
        uint4 kr[2][2][kHalves];  // [16-key tile][key g, g + 8][channel half]
        auto load_k = [&](int key0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                pg[i] = page_at(key0 + 16 * i);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint8_t* src = pg[i] < 0 ? nullptr : c.k_codes + block_of(pg[i], key0 + 16 * i + 8 * r + g) + 16 * t;
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        kr[i][r][h] = src ? __ldg(reinterpret_cast<const uint4*>(src + 64 * h)) : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        };
        int key0 = tile0 * kTile + warp * kSlab;
        if (tile0 < tile1) load_k(key0);
        for (int tile = tile0; tile < tile1; ++tile, key0 += kTile) {
            const int32_t cur[2] = {pg[0], pg[1]};
            // V of this slab: keys 2t, 2t + 1, 2t + 8, 2t + 9 of each 16, zero where unseen.
            uint32_t vr[2][4][kVWords];
            float ks[2], vs[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t s_at = cur[i] < 0 ? 0 : (int64_t)cur[i] * c.heads + it.head;
                ks[i] = cur[i] < 0 ? 0.f : c.k_scale[s_at];
                vs[i] = cur[i] < 0 ? 0.f : c.v_scale[s_at];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = key0 + 16 * i + 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
                    for (int x = 0; x < kVWords; ++x) vr[i][r][x] = 0u;
                    if (cur[i] >= 0 && key < seen_max) {
                        const uint8_t* src = c.v_codes + block_of(cur[i], key) + kVWords * 4 * g;
                        if constexpr (kVWords == 4) {
                            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
                            vr[i][r][0] = v.x; vr[i][r][1] = v.y; vr[i][r][2] = v.z; vr[i][r][3] = v.w;
                        } else {
                            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
                            vr[i][r][0] = v.x; vr[i][r][1] = v.y;
                        }
                    }
                }
            }
            float sc[kNT][2][4];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[nt][i][0] = sc[nt][i][1] = sc[nt][i][2] = sc[nt][i][3] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const uint32_t a[4] = {kr[i][0][h].x, kr[i][0][h].y, kr[i][0][h].z, kr[i][0][h].w};
                    const uint32_t b[4] = {kr[i][1][h].x, kr[i][1][h].y, kr[i][1][h].z, kr[i][1][h].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t a0 = widen2(a[j]), a2 = widen2(a[j] >> 16), a1 = widen2(b[j]), a3 = widen2(b[j] >> 16);
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma16816(sc[nt][i], a0, a1, a2, a3, q[nt][4 * h + j][0], q[nt][4 * h + j][1]);
                    }
                }
            if (tile + 1 < tile1) load_k(key0 + kTile);

            // Running maximum of each column over this slab's 32 keys.
            const bool edge = key0 + kSlab > seen_min || cur[0] < 0 || cur[1] < 0;
            const float ref_new = fmaxf(ref, fmaxf(vs[0], vs[1]));
            const float ref_inv = ref_new > 0.f ? 1.f / ref_new : 0.f;
            const float wv[2] = {vs[0] * ref_inv, vs[1] * ref_inv}, shrink = ref * ref_inv;
            ref = ref_new;
            uint32_t pf[kNT][2][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                float top[2] = {kNegInf, kNegInf};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int col = x & 1, key = key0 + 16 * i + g + 8 * (x >> 1);
                        float y = sc[nt][i][x] * (factor[nt][col] * ks[i]);
                        if (edge && (cur[i] < 0 || key >= seen[nt][col])) y = kNegInf;
                        sc[nt][i][x] = y;
                        top[col] = fmaxf(top[col], y);
                    }
                float fix[2];
#pragma unroll
                for (int col = 0; col < 2; ++col) {
#pragma unroll
                    for (int s = 4; s <= 16; s <<= 1) top[col] = fmaxf(top[col], __shfl_xor_sync(0xffffffffu, top[col], s));
                    const float m_new = fmaxf(m[nt][col], top[col]);
                    const float m_use = m_new == kNegInf ? 0.f : m_new;
                    fix[col] = exp2f(m[nt][col] - m_use);
                    m[nt][col] = m_new;
                    l[nt][col] *= fix[col];
                    top[col] = m_use;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        e[x] = exp2f(sc[nt][i][x] - top[x & 1]);
                        l[nt][x & 1] += e[x];
                        e[x] *= wv[i];
                    }
                    pf[nt][i][0] = transpose8x8(pack_half2(e[0], e[1]));
                    pf[nt][i][1] = transpose8x8(pack_half2(e[2], e[3]));
                }
                const float f0 = fix[0] * shrink, f1 = fix[1] * shrink;
                if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
                    for (int j = 0; j < kMT; ++j) {
                        o[nt][j][0] *= f0;
                        o[nt][j][1] *= f1;
                        o[nt][j][2] *= f0;
                        o[nt][j][3] *= f1;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < kVWords; ++x) {
                    // Codes of channels d, d + 1 (then d + 2, d + 3) of two neighbouring keys.
                    const uint32_t lo0 = __byte_perm(vr[i][0][x], vr[i][1][x], 0x5140), lo1 = __byte_perm(vr[i][0][x], vr[i][1][x], 0x7362);
                    const uint32_t hi0 = __byte_perm(vr[i][2][x], vr[i][3][x], 0x5140), hi1 = __byte_perm(vr[i][2][x], vr[i][3][x], 0x7362);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t lo = y ? lo1 : lo0, hi = y ? hi1 : hi0;
                        const uint32_t a0 = widen2(lo), a1 = widen2(lo >> 16), a2 = widen2(hi), a3 = widen2(hi >> 16);
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) mma16816(o[nt][2 * x + y], a0, a1, a2, a3, pf[nt][i][0], pf[nt][i][1]);
                    }
                }
        }

        // The four warps' parts into shared memory, then joined by columns.
        // o[nt][j][x] is channel 4 kVWords g + 2 j + x / 2 of column 8 nt + 2 t + x % 2.
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int col = 0; col < 2; ++col) {
#pragma unroll
                for (int s = 4; s <= 16; s <<= 1) l[nt][col] += __shfl_xor_sync(0xffffffffu, l[nt][col], s);
                float* ml = s_ml + (warp * kCols + nt * 8 + 2 * t + col) * 2;
                if (g == 0) {
                    ml[0] = m[nt][col];
                    ml[1] = l[nt][col];
                }
                float* dst = s_o + (warp * kCols + nt * 8 + 2 * t + col) * kPad + kVWords * 4 * g;
#pragma unroll
                for (int j = 0; j < kMT; ++j)
                    *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[nt][j][col] * ref, o[nt][j][2 + col] * ref);
            }
        }
        __syncthreads();
        const bool whole = w == it.first && item_end <= w_end;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (w == w_begin ? 0 : 1);
        for (int x = tid; x < kCols * kDim; x += kThreads) {
            const int col = x / kDim, d = x % kDim, f = row0 + col;
            if (f >= rows_all) break;
            float top = kNegInf, sum = 0.f, acc = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_ml[(k * kCols + col) * 2]);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float mk = s_ml[(k * kCols + col) * 2];
                const float e = mk == kNegInf ? 0.f : exp2f(mk - top);
                sum += e * s_ml[(k * kCols + col) * 2 + 1];
                if (e > 0.f) acc += e * s_o[(k * kCols + col) * kPad + d];
            }
            if (whole) {
                T* out = static_cast<T*>(p.out) + (it.begin + f / group) * p.out_stride + (int64_t)(it.head * group + f % group) * kDim;
                out[d] = Act<T>::from(sum > 0.f ? acc / sum : 0.f);
            } else {
                p.part_o[(slot * kCols + col) * kDim + d] = acc;
                if (d == 0) {
                    p.part_ml[(slot * kCols + col) * 2] = top;
                    p.part_ml[(slot * kCols + col) * 2 + 1] = sum;
                }
            }
        }
        __syncthreads();  // shared memory is written again for the next item
        w = item_end;
    }
}

// Joins the parts of the items that lie in several CTAs' shares: blockIdx.x counts items,
// blockIdx.y columns.
template <typename T, int kDim, int kCols>
__global__ void __launch_bounds__(kDim) attention_join_kernel(const AttentionParams p) {
    cudaGridDependencySynchronize();
    const CacheParams& c = p.c;
    const int group = p.q_heads / c.heads;
    const int64_t all = p.first_work[c.rows], per = share_of(all, p.ctas);
    // Items are counted as rows * heads * blocks when every row has the same number of column
    // blocks (one token a row), else by walking the rows.
    int64_t i = blockIdx.x;
    int row = 0;
    if (!c.cu) {
        const int blocks = (group + kCols - 1) / kCols;
        row = (int)(i / ((int64_t)c.heads * blocks));
        i -= (int64_t)row * c.heads * blocks;
    } else {
        // Item numbers by an upper bound: row r's first item is number
        // (cu[r] * group / kCols + r) * heads (its blocks are at most n * group / kCols + 1).
        int lo = 0, hi = c.rows;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (((int64_t)c.cu[mid] * group / kCols + mid) * c.heads <= i) lo = mid;
            else hi = mid;
        }
        row = lo;
        i -= ((int64_t)c.cu[row] * group / kCols + row) * c.heads;
    }
    if (row >= c.rows || i < 0) return;
    int64_t begin;
    const int n = row_tokens(c, row, begin);
    const int tiles = row_tiles(row_length(c, row));
    const int64_t w0 = p.first_work[row] + i * tiles, w1 = w0 + tiles;
    if (w1 > p.first_work[row + 1]) return;
    const int64_t c0 = w0 / per, c1 = (w1 - 1) / per;
    if (c0 == c1) return;
    const int head = (int)(i % c.heads), block = (int)(i / c.heads);
    const int col = blockIdx.y, f = block * kCols + col, d = threadIdx.x;
    if (f >= n * group) return;
    float top = kNegInf, sum = 0.f, acc = 0.f;
    for (int64_t k = c0; k <= c1; ++k) {
        const int64_t slot = 2 * k + (k * per >= w0 ? 0 : 1);
        const float mk = p.part_ml[(slot * kCols + col) * 2], lk = p.part_ml[(slot * kCols + col) * 2 + 1];
        const float ok = p.part_o[(slot * kCols + col) * kDim + d];
        if (mk == kNegInf) continue;
        const float m = fmaxf(top, mk), a = exp2f(top - m), b = exp2f(mk - m);
        top = m;
        sum = sum * a + lk * b;
        acc = acc * a + ok * b;
    }
    T* out = static_cast<T*>(p.out) + (begin + f / group) * p.out_stride + (int64_t)(head * group + f % group) * kDim;
    out[d] = Act<T>::from(sum > 0.f ? acc / sum : 0.f);
}

template <int kDim, int kNT>
constexpr size_t smem_bytes() {
    return (size_t)kWarps * 8 * kNT * (kDim + 4 + 2) * sizeof(float);
}

template <typename T, int kDim, int kNT>
cudaError_t launch_one(const AttentionParams& p, cudaStream_t stream) {
    const CacheParams& c = p.c;
    constexpr int kCols = 8 * kNT;
    attention_kernel<T, kDim, kNT><<<p.ctas, kThreads, smem_bytes<kDim, kNT>(), stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t group = p.q_heads / c.heads;
    const int64_t items = c.cu ? (c.tokens * group / kCols + c.rows) * c.heads
                               : (int64_t)c.rows * c.heads * ((group + kCols - 1) / kCols);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)items, kCols);
    cfg.blockDim = dim3(kDim);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, kDim, kCols>, p);
}

template <typename T, int kDim, int kNT>
int resident() {
    int n = 0;
    if (cudaFuncSetAttribute(attention_kernel<T, kDim, kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<kDim, kNT>()) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attention_kernel<T, kDim, kNT>, kThreads,
                                                      smem_bytes<kDim, kNT>()) != cudaSuccess ||
        n < 1) {
        cudaGetLastError();
        n = 1;
    }
    return n;
}

template <typename T, int kDim>
cudaError_t launch_cols(const AttentionParams& p, int cols, cudaStream_t stream) {
    if (cols == 8) return launch_one<T, kDim, 1>(p, stream);
    if (cols == 16) return launch_one<T, kDim, 2>(p, stream);
    return launch_one<T, kDim, 4>(p, stream);
}
template <typename T, int kDim>
int resident_cols(int cols) {
    if (cols == 8) return resident<T, kDim, 1>();
    if (cols == 16) return resident<T, kDim, 2>();
    return resident<T, kDim, 4>();
}

}  // namespace

// Query rows of an item: as few of 8, 16 and 32 as hold one row's (token, head) pairs.
int attention_cols(int64_t tokens, int32_t rows, int32_t group) {
    const int64_t each = (tokens + rows - 1) / rows * group;
    return each <= 8 ? 8 : each <= 16 ? 16 : 32;
}

size_t attention_scratch(int32_t rows, int32_t dim, int cols, int ctas) {
    return ((size_t)rows + 1) * 8 + 16 + (size_t)2 * ctas * cols * (dim + 2) * 4;
}

int attention_ctas(int32_t dim, int cols, bool f16, int sm_count) {
    int n;
    if (dim == 64) n = f16 ? resident_cols<__half, 64>(cols) : resident_cols<__nv_bfloat16, 64>(cols);
    else n = f16 ? resident_cols<__half, 128>(cols) : resident_cols<__nv_bfloat16, 128>(cols);
    return n * sm_count;
}

cudaError_t launch_attention(const AttentionParams& p, int cols, bool f16, cudaStream_t stream) {
    if (p.c.dim == 64)
        return f16 ? launch_cols<__half, 64>(p, cols, stream) : launch_cols<__nv_bfloat16, 64>(p, cols, stream);
    return f16 ? launch_cols<__half, 128>(p, cols, stream) : launch_cols<__nv_bfloat16, 128>(p, cols, stream);
}

}  // namespace kda
