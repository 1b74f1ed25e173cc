// kda_kvcache_attention.cu -- causal attention over the 8-bit paged cache, for one or a few
// new tokens a row (up to 32 query rows for a key/value head, and small calls with more;
// kda_kvcache_block.cu takes the others).
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
// largest).  Weights times their page's v scale are fp16 relative to the running maximum of
// that product, which becomes 2^14, so they use fp16's whole range: a long row's weights may all be
// 2^-20 of one key's and less and hold a large part of the sum together.  The sum of the weights divides
// the scale out again by blocks of 16 keys.  Running maximum, sums, outputs and the joined parts are fp32.
//
// Work split: warps work alone.  The items' cached tokens, cut into slabs, are numbered
// through all items; every resident warp takes an equal contiguous share, however long the rows
// are.  An item inside one share is written at once; the parts of the others, in the layout of
// the product's fragments, are joined by a second launch.  (With four warps sharing each tile
// and joining in shared memory at every item's end the loads paused there: 147 us instead of
// 133 for 64 rows of up to 8192 tokens, 8 heads.  Asking L2 for codes two to eight slabs ahead
// made it 1 to 35% slower, slabs of 16 keys with four CTAs an SM 5%, two CTAs without spills
// 10%.)  Bound by HBM: that call takes 127 us, 0.83 of its bytes at the copy rate (718 MB), the join
// and its tail with it; 4 rows of up to 131072 tokens, 4 heads, 68 us, 0.78; one row of 1000
// tokens 8 us, two launches' latency.  16 columns, and head_dim 64, are bound by latency: the codes under
// way are in registers, of which 16 columns leave eight warps an SM (85 rows of up to 7582 tokens, 32 heads
// of 64 over 2: 51 us, 0.32 of its bytes; 64 rows of up to 8192, 64 heads of 64 over 8: 79 us, 0.67).
#include "kda_kvcache_attention.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr float kLift = 14.f;     // log2 of the largest weight: fp16 is normal down to 2^-28 of it
constexpr int kMaxListed = 1024;  // rows whose prefix fits in shared memory
// Keys of a slab: 4 KB of codes of K, so that as many bytes are under way for head_dim 64 as for
// 128 (64 keys against 32 there: 85 rows of up to 7582 tokens, 32 heads over 2, 51 against 65 us; one
// row of 130878, 9 over 3, 26 against 34).
template <int kDim>
constexpr int kSlabKeys = 4096 / kDim;

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

template <int kDim>
__device__ __forceinline__ int row_slabs(int len) {
    constexpr int kKeys = kSlabKeys<kDim>;
    return len > kKeys ? (len + kKeys - 1) / kKeys : 1;
}
// Codes of 16 keys, widened, against the query rows: acc += K Q^T.  q(step, nt) gives the two
// registers of a reduction step.
template <int kHalves, int kNT, typename Q>
__device__ __forceinline__ void product_k(float (&acc)[kNT][4], const uint4 (&k)[2][kHalves], Q q) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
        const uint32_t a[4] = {k[0][h].x, k[0][h].y, k[0][h].z, k[0][h].w};
        const uint32_t b[4] = {k[1][h].x, k[1][h].y, k[1][h].z, k[1][h].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = widen2(a[j]), a2 = widen2(a[j] >> 16), a1 = widen2(b[j]), a3 = widen2(b[j] >> 16);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const uint2 y = q(4 * h + j, nt);
                mma16816(acc[nt], a0, a1, a2, a3, y.x, y.y);
            }
        }
    }
}

template <typename T, int kDim, int kNT, int kKind>
__global__ void __launch_bounds__(kThreads, kNT == 1 ? 3 : 2) attention_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kCols = 8 * kNT, kKeys = kSlabKeys<kDim>, kBlk = kKeys / 16;  // (blocks of 16 keys)
    constexpr int kHalves = kDim / 64;   // 16-byte loads of a key by a thread
    constexpr int kSteps = kDim / 16;    // reduction steps of S^T
    constexpr int kMT = kDim / 16;       // 16-channel tiles of O^T
    constexpr int kVWords = kDim / 32;   // 4-byte words of a V load
    __shared__ int64_t s_first[kMaxListed + 1], s_scan[kWarps];

    follow_stream();
    const CacheParams& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int group = p.q_heads / c.heads;
    const int page_shift = __ffs(c.page_tokens) - 1;
    const int64_t block_bytes = (int64_t)c.page_tokens * kDim;

    // Every CTA needs the rows' prefix; past kMaxListed rows all write the same values to the
    // scratch.
    int64_t* first = c.rows <= kMaxListed ? s_first : p.first_work;
    scan_rows<kThreads>(c.rows, first, s_scan, [&](int r) -> int64_t {  // items: column blocks by key/value heads
        if (r >= c.rows) return 0;
        int64_t begin;
        const int n = row_tokens(c, r, begin);
        return ((int64_t)n * group + kCols - 1) / kCols * c.heads * row_slabs<kDim>(row_length(c, r) - unit_from<kKind>(p, r));
    });
    __syncthreads();
    if (blockIdx.x == 0 && c.rows <= kMaxListed)
        for (int r = tid; r <= c.rows; r += kThreads) p.first_work[r] = s_first[r];
    const int64_t all = first[c.rows];
    const int64_t per = share_of(all, p.ctas * kWarps);
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t w_begin = per * unit, w_end = min(all, w_begin + per);

    for (int64_t w = w_begin; w < w_end;) {
        const int row = row_of(first, c.rows, w);
        int64_t begin;
        const int n = row_tokens(c, row, begin), len = row_length(c, row), from = unit_from<kKind>(p, row), slabs = row_slabs<kDim>(len - from);
        const int64_t i_row = (w - first[row]) / slabs, item = first[row] + i_row * slabs, item_end = item + slabs;
        const int head = (int)(i_row % c.heads), block = (int)(i_row / c.heads);
        const int slab0 = (int)(w - item) + from / kKeys;

        const int rows_all = n * group, row0 = block * kCols;
        // Keys that any, and that every, column of this block sees.
        const int seen_max = min(len, max(0, len - n + (min(rows_all, row0 + kCols) - 1) / group + 1));
        const int seen_min = max(0, min(len, len - n + row0 / group + 1));
        const int slab1 = min((int)(min(item_end, w_end) - item) + from / kKeys, (seen_max + kKeys - 1) / kKeys);

        // Page and scales of the 16 keys of block number b; lane l holds block b0 + l.
        const int32_t* table = c.tables + (int64_t)row * c.width;
        auto page_at = [&](int b) {
            const int key = b * 16;
            if (key >= seen_max) return -1;
            const int32_t x = table[key >> page_shift];
            if (x < 0 || x >= c.pages) {
                report(c.status, kStatusBadIndex);
                return -1;
            }
            return x;
        };
        constexpr int kBatch = 32 / kBlk;  // slabs whose pages a warp holds
        int32_t pages = page_at(slab0 * kBlk + lane), pages_next = -1;

        uint32_t q[kNT][kSteps][2];
        float q_scale[kNT];  // of column 8 nt + g
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int f = row0 + nt * 8 + g;
            const bool there = f < rows_all;
            const T* src = static_cast<const T*>(p.q) + (begin + (there ? f / group : 0)) * p.q_stride +
                           (int64_t)(head * group + (there ? f % group : 0)) * kDim;
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
            const int e = row_exponent(a);
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
        auto q_at = [&](int step, int nt) { return make_uint2(q[nt][step][0], q[nt][step][1]); };
        // What each column sees and its factor, for this thread's column pairs.
        int seen[kNT][2];
        float factor[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int f = row0 + nt * 8 + 2 * t + i;
                seen[nt][i] = f < rows_all ? max(0, min(len, len - n + f / group + 1)) : 0;
                factor[nt][i] = __shfl_sync(0xffffffffu, q_scale[nt], (2 * t + i) * 4);
            }

        float o[kNT][kMT][4], m[kNT][2], l[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            m[nt][0] = m[nt][1] = kNegInf;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < kMT; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }
        float least = kScaleLeast;  // that a log2 of v's scale counts as: the same for the warp
        if (kKind == kKindSuffix && w == item && from > 0) {  // on from the prefix
            least = p.state_ml[(begin + row0 / group) * p.q_heads + head * group + row0 % group].z;  // (as in all of its rows)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    const int f = row0 + nt * 8 + 2 * t + col;
                    if (f >= rows_all) continue;
                    const int64_t at = (begin + f / group) * p.q_heads + head * group + f % group;
                    const float4 ml = p.state_ml[at];
                    m[nt][col] = ml.x + (kLift - kBlockLift);
                    l[nt][col] = g == 0 ? ml.y : 0.f;  // (summed over the lanes in the end)
                    const float2* src = reinterpret_cast<const float2*>(p.state_o + at * kDim + kVWords * 4 * g);
#pragma unroll
                    for (int j = 0; j < kMT; ++j) {
                        const float2 y = src[j];
                        o[nt][j][col] = y.x;
                        o[nt][j][2 + col] = y.y;
                    }
                }
        }

        auto scale_of = [&](const float* scales, int32_t page) { return page < 0 ? 0.f : scales[(int64_t)page * c.heads + head]; };
        auto log_of = [&](int32_t page) { return page < 0 ? 0.f : log2f(scale_of(c.v_scale, page)); };
        float k_scales = scale_of(c.k_scale, pages), v_logs = log_of(pages);
        int b0 = slab0 * kBlk;  // block of lane 0

        uint4 kr[kBlk][2][kHalves];  // [16 keys][key g, g + 8][channel half]
        uint32_t vr[kBlk][4][kVWords];  // keys 2t, 2t + 1, 2t + 8, 2t + 9 of each 16
        auto load_k = [&](int slab) {
#pragma unroll
            for (int i = 0; i < kBlk; ++i) {
                const int b = slab * kBlk + i;
                const int32_t page = __shfl_sync(0xffffffffu, pages, b - b0);
                if (page >= 0) {
                    const uint8_t* src = c.k_codes + ((int64_t)page * c.heads + head) * block_bytes +
                                         ((b * 16 & (c.page_tokens - 1)) + g) * kDim + 16 * t;
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) kr[i][r][h] = load_codes16(src + 8 * r * kDim + 64 * h);
                } else {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) kr[i][r][h] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        };
        auto load_v = [&](int slab) {
#pragma unroll
            for (int i = 0; i < kBlk; ++i) {
                const int b = slab * kBlk + i, key0 = b * 16;
                const int32_t page = __shfl_sync(0xffffffffu, pages, b - b0);
                const uint8_t* src = c.v_codes + ((int64_t)max(page, 0) * c.heads + head) * block_bytes +
                                     ((key0 & (c.page_tokens - 1)) + 2 * t) * kDim + kVWords * 4 * g;
                const bool whole = page >= 0 && key0 + 16 <= seen_max;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = 2 * t + (r & 1) + 8 * (r >> 1), off = ((r & 1) + 8 * (r >> 1)) * kDim;
#pragma unroll
                    for (int x = 0; x < kVWords; ++x) vr[i][r][x] = 0u;  // what no column sees stays out
                    if (whole || (page >= 0 && key0 + key < seen_max)) {
                        if constexpr (kVWords == 4) {
                            const uint4 v = load_codes16(src + off);
                            vr[i][r][0] = v.x; vr[i][r][1] = v.y; vr[i][r][2] = v.z; vr[i][r][3] = v.w;
                        } else {
                            const uint2 v = load_codes8(src + off);
                            vr[i][r][0] = v.x; vr[i][r][1] = v.y;
                        }
                    }
                }
            }
        };
        if (slab0 < slab1) {
            load_k(slab0);
            load_v(slab0);
        }
        if (slab1 - slab0 > kBatch) pages_next = page_at(b0 + 32 + lane);
        for (int slab = slab0; slab < slab1; ++slab) {
            float ks[kBlk], lv[kBlk];
            bool missing = false;
#pragma unroll
            for (int i = 0; i < kBlk; ++i) {
                const int from = slab * kBlk + i - b0;
                ks[i] = __shfl_sync(0xffffffffu, k_scales, from);
                lv[i] = __shfl_sync(0xffffffffu, v_logs, from);
                missing |= __shfl_sync(0xffffffffu, pages, from) < 0;
                least = fmaxf(least, lv[i] - kScaleSpan);
            }
            bool low = false;
#pragma unroll
            for (int i = 0; i < kBlk; ++i) {
                low |= lv[i] < least;
                lv[i] = fmaxf(lv[i], least);
            }
            const int32_t pages_now = pages;
            const int b_now = b0;
            float sc[kBlk][kNT][4];
#pragma unroll
            for (int i = 0; i < kBlk; ++i) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) sc[i][nt][0] = sc[i][nt][1] = sc[i][nt][2] = sc[i][nt][3] = 0.f;
                product_k<kHalves, kNT>(sc[i], kr[i], q_at);
            }
            // The next slab's pages, then its K while this one's weights are worked out.
            if (slab + 1 < slab1) {
                if ((slab + 1) * kBlk - b0 == 32) {
                    pages = pages_next;
                    k_scales = scale_of(c.k_scale, pages);
                    v_logs = log_of(pages);
                    b0 += 32;
                    if ((b0 + 32) / kBlk < slab1) pages_next = page_at(b0 + 32 + lane);
                }
                load_k(slab + 1);
            }

            const int key0 = slab * kKeys;
            const bool edge = key0 + kKeys > seen_min || missing;
            uint32_t pf[kBlk][kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                float top[2] = {kNegInf, kNegInf};
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    const float fk[2] = {factor[nt][0] * ks[i], factor[nt][1] * ks[i]};
                    const bool gone = edge && __shfl_sync(0xffffffffu, pages_now, slab * kBlk + i - b_now) < 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float y = fmaf(sc[i][nt][x], fk[x & 1], lv[i]);
                        if (edge && (gone || key0 + 16 * i + g + 8 * (x >> 1) >= seen[nt][x & 1])) y = kNegInf;
                        sc[i][nt][x] = y;
                        top[x & 1] = fmaxf(top[x & 1], y);
                    }
                }
                float down[2];  // log2 of what sums and outputs are rescaled by
#pragma unroll
                for (int col = 0; col < 2; ++col) {
#pragma unroll
                    for (int s = 4; s <= 16; s <<= 1) top[col] = fmaxf(top[col], __shfl_xor_sync(0xffffffffu, top[col], s));
                    const float m_new = fmaxf(m[nt][col], top[col]);
                    const float m_use = m_new == kNegInf ? 0.f : m_new;
                    down[col] = m[nt][col] - m_use;
                    m[nt][col] = m_new;
                    top[col] = m_use - kLift;
                }
                float add[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    const float iv = exp2_fast(-lv[i]);
                    float e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        e[x] = exp2_fast(sc[i][nt][x] - top[x & 1]);
                        add[x & 1] += e[x] * iv;
                    }
                    pf[i][nt][0] = transpose8x8(pack_half2(e[0], e[1]));
                    pf[i][nt][1] = transpose8x8(pack_half2(e[2], e[3]));
                }
                if (__any_sync(0xffffffffu, down[0] != 0.f || down[1] != 0.f)) {
                    const float half[2] = {exp2_fast(0.5f * down[0]), exp2_fast(0.5f * down[1])};
                    const float fix[2] = {half[0] * half[0], half[1] * half[1]};
                    l[nt][0] = rescaled(l[nt][0], half[0]);
                    l[nt][1] = rescaled(l[nt][1], half[1]);
#pragma unroll
                    for (int j = 0; j < kMT; ++j) {
                        o[nt][j][0] *= fix[0];
                        o[nt][j][1] *= fix[1];
                        o[nt][j][2] *= fix[0];
                        o[nt][j][3] *= fix[1];
                    }
                }
                l[nt][0] += add[0];
                l[nt][1] += add[1];
            }
            if (low) {
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    const int32_t page = __shfl_sync(0xffffffffu, pages_now, slab * kBlk + i - b_now);
                    const float by = exp2_fast(fminf(log_of(page) - lv[i], 0.f));
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        pf[i][nt][0] = brought_down(pf[i][nt][0], by);
                        pf[i][nt][1] = brought_down(pf[i][nt][1], by);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kBlk; ++i)
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
                        for (int nt = 0; nt < kNT; ++nt) mma16816(o[nt][2 * x + y], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
                    }
                }
            if (slab + 1 < slab1) load_v(slab + 1);
        }

        // o[nt][j][x] is channel 4 kVWords g + 2 j + x / 2 of column 8 nt + 2 t + x % 2.
        const bool whole = w == item && item_end <= w_end;
        const int64_t slot = 2 * unit + (w == w_begin ? 0 : 1);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int col = 0; col < 2; ++col)
#pragma unroll
                for (int s = 4; s <= 16; s <<= 1) l[nt][col] += __shfl_xor_sync(0xffffffffu, l[nt][col], s);
            if (whole) {
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    const int f = row0 + nt * 8 + 2 * t + col;
                    if (f >= rows_all) continue;
                    const float by = l[nt][col] > 0.f ? 1.f / l[nt][col] : 0.f;
                    T* out = static_cast<T*>(p.out) + (begin + f / group) * p.out_stride + (int64_t)(head * group + f % group) * kDim + kVWords * 4 * g;
#pragma unroll
                    for (int j = 0; j < kMT; ++j)
                        *reinterpret_cast<uint32_t*>(out + 2 * j) = Act<T>::pack(o[nt][j][col] * by, o[nt][j][2 + col] * by);
                }
            } else {
                float4* part = reinterpret_cast<float4*>(p.part_o) + (slot * kNT + nt) * kMT * 32 + lane;
#pragma unroll
                for (int j = 0; j < kMT; ++j)
                    part[32 * j] = make_float4(o[nt][j][0], o[nt][j][1], o[nt][j][2], o[nt][j][3]);
                if (g == 0)
                    reinterpret_cast<float4*>(p.part_ml)[(slot * kNT + nt) * 4 + t] = make_float4(m[nt][0], l[nt][0], m[nt][1], l[nt][1]);
            }
        }
        w = item_end;
    }
}

// Joins the parts of the items that lie in several warps' shares.  blockIdx.x counts items,
// blockIdx.y column tiles; a warp has 16 channels of 8 columns, in the fragments' layout.
// kShares > 1 (items of many parts): blockIdx.z is the channel tile, and that many warps share the
// parts.
template <typename T, int kDim, int kNT, int kShares, int kKind>
__global__ void __launch_bounds__(kShares > 1 ? kShares * 32 : kDim * 2) attention_join_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kCols = 8 * kNT, kMT = kDim / 16, kVWords = kDim / 32;
    constexpr bool kSplit = kShares > 1;
    __shared__ float4 s_o[kShares][32], s_ml[kShares][32];
    const CacheParams& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nt = blockIdx.y, j = kSplit ? blockIdx.z : warp;
    const int group = p.q_heads / c.heads;
    int64_t i = blockIdx.x;
    int row;
    const bool there = joined_item(c, group, kCols, i, row);
    int64_t begin = 0;
    const int n = there ? row_tokens(c, row, begin) : 0;
    const int slabs = there ? row_slabs<kDim>(row_length(c, row) - unit_from<kKind>(p, row)) : 0;
    follow_stream();
    if (!there) return;
    const int64_t all = p.first_work[c.rows], w_row = p.first_work[row], w_next = p.first_work[row + 1];
    const int64_t per = share_of(all, p.ctas * kWarps);
    const int64_t w0 = w_row + i * slabs, w1 = w0 + slabs;
    if (w1 > w_next) return;
    const int64_t u0 = w0 / per, u1 = (w1 - 1) / per;
    if (u0 == u1) return;
    const int head = (int)(i % c.heads), block = (int)(i / c.heads);

    float top[2] = {kNegInf, kNegInf}, sum[2] = {0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float4& ml, const float4& o) {
        const float mk[2] = {ml.x, ml.z}, lk[2] = {ml.y, ml.w}, ok[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            const float m = fmaxf(top[col], mk[col]), use = m == kNegInf ? 0.f : m;
            const float ha = exp2_fast(0.5f * (top[col] - use)), hb = exp2_fast(0.5f * (mk[col] - use)), a = ha * ha, b = hb * hb;
            top[col] = m;
            sum[col] = rescaled(sum[col], ha) + rescaled(lk[col], hb);
            acc[col] = acc[col] * a + ok[col] * b;
            acc[2 + col] = acc[2 + col] * a + ok[2 + col] * b;
        }
    };
    constexpr int kAhead = 8;
    const int64_t step = kShares;
    for (int64_t k = u0 + (kSplit ? warp : 0); k <= u1; k += kAhead * step) {
        float4 ml[kAhead], o[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int64_t u = k + x * step;
            if (u > u1) continue;
            const int64_t slot = 2 * u + (u * per >= w0 ? 0 : 1);
            ml[x] = reinterpret_cast<const float4*>(p.part_ml)[(slot * kNT + nt) * 4 + t];
            o[x] = reinterpret_cast<const float4*>(p.part_o)[((slot * kNT + nt) * kMT + j) * 32 + lane];
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            if (k + x * step <= u1) add(ml[x], o[x]);
    }
    if (kSplit) {
        s_o[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        s_ml[warp][lane] = make_float4(top[0], sum[0], top[1], sum[1]);
        __syncthreads();
        if (warp) return;
        for (int x = 1; x < kShares; ++x) add(s_ml[x][lane], s_o[x][lane]);
    }
#pragma unroll
    for (int col = 0; col < 2; ++col) {
        const int f = block * kCols + nt * 8 + 2 * t + col;
        if (f >= n * group) continue;
        const float by = sum[col] > 0.f ? 1.f / sum[col] : 0.f;
        T* out = static_cast<T*>(p.out) + (begin + f / group) * p.out_stride + (int64_t)(head * group + f % group) * kDim + kVWords * 4 * g + 2 * j;
        *reinterpret_cast<uint32_t*>(out) = Act<T>::pack(acc[col] * by, acc[2 + col] * by);
    }
}

template <typename T, int kDim, int kNT, int kKind>
cudaError_t launch_one(const AttentionParams& p, cudaStream_t stream) {
    const CacheParams& c = p.c;
    constexpr int kCols = 8 * kNT;
    const cudaError_t e = launch_early(attention_kernel<T, kDim, kNT, kKind>, dim3(p.ctas), kThreads, 0, stream, 1, p);
    if (e != cudaSuccess) return e;
    const int64_t group = p.q_heads / c.heads;
    const int64_t items = joined_items(c, group, kCols);
    // As many warps to a part of an item as a wave or two hold: few items have many parts each (2 rows
    // of up to 24086 tokens: 20 us with 16, 29 with 8; 34 rows of 135: 17 us with one, 28 with 16).
    const int64_t tiles = items * kNT * (kDim / 16);
    if (tiles <= 2ll * p.sm_count)
        return launch_early(attention_join_kernel<T, kDim, kNT, 16, kKind>, dim3((unsigned)items, kNT, kDim / 16), 512, 0, stream, 1, p);
    if (tiles <= 5ll * p.sm_count)
        return launch_early(attention_join_kernel<T, kDim, kNT, 4, kKind>, dim3((unsigned)items, kNT, kDim / 16), 128, 0, stream, 1, p);
    return launch_early(attention_join_kernel<T, kDim, kNT, 1, kKind>, dim3((unsigned)items, kNT), kDim * 2, 0, stream, 1, p);
}

// CTAs an SM holds; the same on every device the library runs on.
template <typename T, int kDim, int kNT, int kKind>
int resident() {
    static const int count = [] {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attention_kernel<T, kDim, kNT, kKind>, kThreads, 0) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = 1;
        }
        return n;
    }();
    return count;
}

template <typename T, int kDim, int kKind>
cudaError_t launch_cols(const AttentionParams& p, int cols, cudaStream_t stream) {
    if (cols == 8) return launch_one<T, kDim, 1, kKind>(p, stream);
    return launch_one<T, kDim, 2, kKind>(p, stream);
}
template <typename T, int kDim>
int resident_cols(int cols) {
    if (cols == 8) return resident<T, kDim, 1, kKindRows>();
    return resident<T, kDim, 2, kKindRows>();
}
template <int kKind>
cudaError_t launch_kind(const AttentionParams& p, int cols, bool f16, cudaStream_t stream) {
    if (p.c.dim == 64)
        return f16 ? launch_cols<__half, 64, kKind>(p, cols, stream) : launch_cols<__nv_bfloat16, 64, kKind>(p, cols, stream);
    return f16 ? launch_cols<__half, 128, kKind>(p, cols, stream) : launch_cols<__nv_bfloat16, 128, kKind>(p, cols, stream);
}

}  // namespace

// Query rows of an item: 8 where they hold a row's (token, head) pairs, 16 up to kFewRows pairs or
// where the call is small, else 128 on tcgen05.  Items of 16 against items of 128, us for rows,
// key/value heads and tokens cached at most (a third of it and more): 32 pairs, 16 rows, 4 heads, 2000:
// 20 against 24 (head_dim 64), 24 against 31 (128); 64, 4, 500: 22 / 22, 32 / 35; 1, 8, 30000: 28 / 28,
// 40 / 47.  48 pairs, 64, 4, 500: 24 / 23, 36 / 35; 1, 8, 30000: 40 / 28, 50 / 47.  Small
// calls, with two warps for an item of 16 and at most 256 keys of an item for a warp: 128 pairs, 4, 8,
// 500: 12 / 15, 19 / 21; 96 pairs, 16, 4, 500: 16 / 18, 23 / 27; 128 pairs, 1, 1, 30000: 22 / 22, 25 / 28; with
// more items than that 64 pairs, 111, 2, 40: 14 / 11, 25 / 16.  (Of the cached tokens the host knows what
// the tables have places for: where those are 32768 and more, calls like these small ones take the second
// figure.)
constexpr int kFewRows = 32, kFewKeys = 256;
int attention_cols(const CacheParams& c, int32_t group, int sm_count) {
    const int64_t each = (c.tokens + c.rows - 1) / c.rows * group;
    if (each <= 8) return 8;
    const int64_t items = (c.tokens * group / 16 + c.rows) * c.heads, keys = (int64_t)c.width * c.page_tokens;
    const int64_t warps = 2ll * kWarps * sm_count;
    const bool small = items <= warps / 2 && items * keys <= kFewKeys * warps;
    return each <= kFewRows || small ? 16 : kBlockRows;
}

size_t attention_slots(int ctas) { return (size_t)2 * ctas * kWarps; }

int attention_ctas(int32_t dim, int cols, bool f16, int sm_count) {
    if (cols == kBlockRows) return 2 * sm_count;
    int n;
    if (dim == 64) n = f16 ? resident_cols<__half, 64>(cols) : resident_cols<__nv_bfloat16, 64>(cols);
    else n = f16 ? resident_cols<__half, 128>(cols) : resident_cols<__nv_bfloat16, 128>(cols);
    return n * sm_count;
}

cudaError_t launch_attention(const AttentionParams& p, int cols, bool f16, cudaStream_t stream) {
    if (cols == kBlockRows) return launch_block_attention(p, f16, stream);
    return launch_kind<kKindRows>(p, cols, f16, stream);
}
cudaError_t launch_suffix(const AttentionParams& p, int cols, bool f16, cudaStream_t stream) {
    if (cols == kBlockRows) return launch_block_suffix(p, f16, stream);
    return launch_kind<kKindSuffix>(p, cols, f16, stream);
}

}  // namespace kda
