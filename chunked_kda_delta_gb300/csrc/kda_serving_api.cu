// kda_serving_api.cu -- the C ABI of the serving operators: page operations, the 8-bit
// key/value cache, penalties on logits and beam selection.  Validation, scratch layout and launches; the kernels
// live in kda_pages.cu, kda_kvcache_append.cu, kda_kvcache_rotary.cu, kda_kvcache_attention.cu,
// kda_kvcache_block.cu, kda_kvcache_prefix.cu, kda_kvcache_shared.cu, kda_logits.cu and kda_beam.cu.
#include <math.h>

#include <exception>
#include <initializer_list>

#include "../../include/kda.h"
#include "kda_host.cuh"
#include "kda_internal.cuh"
#include "kda_serving.cuh"

using namespace kda::host;

namespace {

// Runs an entry's body: nothing throws across the ABI.
template <typename F>
kda_status guarded(F body) {
    clear_error();
    try {
        return body();
    } catch (const std::exception& e) {
        return fail(KDA_ERR_OUT_OF_MEMORY, "%s", e.what());
    } catch (...) {
        return fail(KDA_ERR_CUDA, "unknown host exception");
    }
}

struct Buffer {
    const char* name;
    Range r;
};

// Every `out` is clear of every `in` and of the other outs.
kda_status check_overlap(std::initializer_list<Buffer> outs, std::initializer_list<Buffer> ins) {
    for (const Buffer* a = outs.begin(); a != outs.end(); ++a) {
        for (const Buffer* b = a + 1; b != outs.end(); ++b)
            if (overlaps(a->r, b->r)) return fail(KDA_ERR_ALIASING, "%s overlaps %s", a->name, b->name);
        for (const Buffer& b : ins)
            if (overlaps(a->r, b.r)) return fail(KDA_ERR_ALIASING, "%s overlaps %s", a->name, b.name);
    }
    return KDA_OK;
}

kda_status check_pointer(const char* name, const void* p, size_t bytes, size_t align) {
    if (bytes == 0) return KDA_OK;
    if (!p) return fail(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", name);
    if (!aligned(p, align)) return fail(KDA_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", name, align);
    return KDA_OK;
}

kda_status check_page_shape(const kda_page_shape* s) {
    if (!s) return fail(KDA_ERR_INVALID_ARGUMENT, "shape is NULL");
    if (s->rows < 0 || s->width < 1 || (int64_t)s->rows * s->width > (1 << 30))
        return fail(KDA_ERR_INVALID_ARGUMENT, "rows must be >= 0, width >= 1 and their product at most 2^30 (got %d, %d)",
                    s->rows, s->width);
    if (s->pages < 0 || s->pages > (1 << 30))
        return fail(KDA_ERR_INVALID_ARGUMENT, "pages must be in [0, 2^30] (got %d)", s->pages);
    return KDA_OK;
}

// Checks the pools and lays them out for the copy kernel.
kda_status make_pools(const kda_pool* pools, int32_t n, int32_t pages, kda::PoolSet* set) {
    *set = kda::PoolSet{};
    if (n < 0 || n > kda::kMaxPools || (n > 0 && !pools))
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_pools must be in [0, %d], pools not NULL (got %d)", kda::kMaxPools, n);
    static_assert(kda::kMaxPools == KDA_MAX_POOLS, "pool limit");
    set->n = n;
    for (int32_t i = 0; i < n; ++i) {
        const kda_pool& a = pools[i];
        if (a.layers < 0 || a.page_bytes < 0 || a.page_bytes > (int64_t)1 << 40)
            return fail(KDA_ERR_INVALID_ARGUMENT, "pool %d: layers and page_bytes must not be negative", i);
        const bool used = a.layers > 0 && a.page_bytes > 0 && pages > 0;
        if (used && !a.base) return fail(KDA_ERR_INVALID_ARGUMENT, "pool %d: base is NULL", i);
        if (used && (a.page_stride < a.page_bytes || a.page_stride > (int64_t)1 << 40))
            return fail(KDA_ERR_INVALID_ARGUMENT, "pool %d: page_stride is smaller than page_bytes", i);
        // Offsets stay below 2^47.
        if (used && (a.page_stride > ((int64_t)1 << 46) / pages ||
                     (a.layers > 1 && (a.layer_stride < 0 || a.layer_stride > ((int64_t)1 << 46) / a.layers))))
            return fail(KDA_ERR_INVALID_ARGUMENT, "pool %d: page_stride or layer_stride is too large", i);
        const int64_t extent = used ? (int64_t)(pages - 1) * a.page_stride + a.page_bytes : 0;
        // Layers either follow one another or lie inside each other's page stride.
        if (used && a.layers > 1 && a.layer_stride < extent &&
            (a.layer_stride < a.page_bytes || (int64_t)a.layers * a.layer_stride > a.page_stride))
            return fail(KDA_ERR_INVALID_ARGUMENT, "pool %d: layers overlap (layer_stride)", i);
        kda::PoolSet::One& o = set->pool[i];
        o.base = static_cast<char*>(a.base);
        o.page_bytes = a.page_bytes;
        o.page_stride = a.page_stride;
        o.layer_stride = a.layers > 1 ? a.layer_stride : 0;
        o.layers = used ? a.layers : 0;
        const int64_t chunks = (a.page_bytes + kda::kCopyChunk - 1) / kda::kCopyChunk;
        if (chunks > 0x7fffffff) return fail(KDA_ERR_INVALID_ARGUMENT, "pool %d: page_bytes is too large", i);
        o.chunks = (int32_t)chunks;
        const uintptr_t bits = (uintptr_t)o.base | (uintptr_t)o.page_bytes | (uintptr_t)o.page_stride | (uintptr_t)o.layer_stride;
        o.unit = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
        set->chunks += (int64_t)o.layers * o.chunks;
    }
    if (set->chunks > (int64_t)1 << 31) return fail(KDA_ERR_INVALID_ARGUMENT, "the pools' pages are too large");
    return KDA_OK;
}

// Bytes of a pool from its base on.
Range pool_range(const kda::PoolSet::One& o, int32_t pages) {
    if (o.layers == 0 || pages == 0) return {nullptr, 0};
    return {o.base, (size_t)((o.layers - 1) * o.layer_stride + (int64_t)(pages - 1) * o.page_stride + o.page_bytes)};
}

kda_status check_pool_overlap(const kda::PoolSet& set, int32_t pages, std::initializer_list<Buffer> others) {
    for (int i = 0; i < set.n; ++i)
        for (const Buffer& b : others)
            if (overlaps(pool_range(set.pool[i], pages), b.r))
                return fail(KDA_ERR_ALIASING, "pool %d overlaps %s", i, b.name);
    return KDA_OK;
}

// The planning step that alloc, free, fork and compact share, then the copies.
kda_status run_plan(kda::PagePlan p, int mode, bool compact, const kda::PoolSet& pools, void* stream) {
    int dev = 0;
    DeviceInfo* di = nullptr;
    kda_status st = current_device(&dev, &di);
    if (st != KDA_OK) return st;
    const size_t entries = (size_t)p.rows * p.width;
    if (entries == 0 && p.pages == 0 && !compact) return KDA_OK;
    const size_t pairs = compact ? (size_t)p.pages : mode == kda::kPagesFork ? entries : 0;
    Scratch ws;
    if ((st = ws.take(dev, stream, (64 + 3 * (size_t)p.pages + 2 * pairs) * 4)) != KDA_OK) return st;
    int32_t* at = reinterpret_cast<int32_t*>(ws.base);
    p.copies = at;
    p.held = at + 64;
    p.first = p.held + p.pages;
    p.list = p.first + p.pages;
    p.src = p.list + p.pages;
    p.dst = p.src + pairs;
    p.status = di->status;
    cudaError_t e = compact ? kda::launch_page_compact(p, (cudaStream_t)stream)
                            : kda::launch_page_plan(p, mode, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "page plan launch");
    const int32_t most = (int32_t)(pairs < (size_t)p.pages ? pairs : (size_t)p.pages);
    if ((e = kda::launch_page_copy(pools, p.pages, p.src, p.dst, p.copies, most, di->status, di->sm_count,
                                   (cudaStream_t)stream)) != cudaSuccess)
        return cuda_fail(e, "page copy launch");
    return KDA_OK;
}

// Checks shared by the plans; `extra` is the operation's own input.
kda_status check_plan(const kda_page_shape* s, const int32_t* tables, const int32_t* refs, Buffer extra, size_t extra_align,
                      Buffer extra2, const int32_t* new_tables, const int32_t* new_refs) {
    kda_status st = check_page_shape(s);
    if (st != KDA_OK) return st;
    const size_t tb = (size_t)s->rows * s->width * 4, rb = (size_t)s->pages * 4;
    if ((st = check_pointer("tables", tables, tb, 4)) || (st = check_pointer("refs", refs, rb, 4)) ||
        (st = check_pointer("new_tables", new_tables, tb, 4)) || (st = check_pointer("new_refs", new_refs, rb, 4)) ||
        (st = check_pointer(extra.name, extra.r.p, extra.r.bytes, extra_align)) ||
        (st = check_pointer(extra2.name, extra2.r.p, extra2.r.bytes, 4)))
        return st;
    return check_overlap({{"new_tables", {new_tables, tb}}, {"new_refs", {new_refs, rb}}},
                         {{"tables", {tables, tb}}, {"refs", {refs, rb}}, extra, extra2});
}

kda::PagePlan plan_of(const kda_page_shape* s, const int32_t* tables, const int32_t* refs, int32_t* new_tables,
                      int32_t* new_refs) {
    kda::PagePlan p{};
    p.tables = tables;
    p.refs = refs;
    p.rows = s->rows;
    p.width = s->width;
    p.pages = s->pages;
    p.new_tables = new_tables;
    p.new_refs = new_refs;
    return p;
}

// Bytes a strided [n][inner] activation spans.
size_t span(int64_t n, int64_t stride, int64_t inner) { return n > 0 ? (size_t)((n - 1) * stride + inner) * 2 : 0; }

// Strided activations [n][inner] that share memory.  Those of one stride, heads of a fused projection
// for instance, may lie between each other.
bool strided_overlap(const void* a, int64_t a_stride, int64_t a_inner, const void* b, int64_t b_stride, int64_t b_inner, int64_t n) {
    if (!overlaps({a, span(n, a_stride, a_inner)}, {b, span(n, b_stride, b_inner)})) return false;
    if (a_stride != b_stride) return true;
    const int64_t step = a_stride * 2;
    int64_t d = ((int64_t)(uintptr_t)b - (int64_t)(uintptr_t)a) % step;  // b's rows start here within a's
    if (d < 0) d += step;
    return d < a_inner * 2 || d + b_inner * 2 > step;
}

kda_status check_cache(const kda_kvcache* c, int64_t num_tokens, const int32_t* lens, const int32_t* cu) {
    if (!c) return fail(KDA_ERR_INVALID_ARGUMENT, "cache is NULL");
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return fail(KDA_ERR_INVALID_ARGUMENT, "page_tokens must be 16, 32, 64 or 128 (got %d)", c->page_tokens);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(KDA_ERR_INVALID_ARGUMENT, "head_dim must be 64 or 128 (got %d)", c->head_dim);
    if (c->num_kv_heads < 1 || c->num_kv_heads > 1024)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_kv_heads must be in [1, 1024] (got %d)", c->num_kv_heads);
    if (c->pages < 0 || c->pages > (1 << 30)) return fail(KDA_ERR_INVALID_ARGUMENT, "pages must be in [0, 2^30] (got %d)", c->pages);
    if (c->rows < 0 || c->width < 1 || (int64_t)c->rows * c->width > (1 << 30))
        return fail(KDA_ERR_INVALID_ARGUMENT, "rows must be >= 0, width >= 1 and their product at most 2^30 (got %d, %d)",
                    c->rows, c->width);
    if (num_tokens < 0 || num_tokens > (1 << 30))
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_tokens must be in [0, 2^30] (got %lld)", (long long)num_tokens);
    if (!cu && num_tokens != c->rows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_tokens every row has one token: num_tokens must be %d (got %lld)",
                    c->rows, (long long)num_tokens);
    if (num_tokens > 0 && c->rows == 0) return fail(KDA_ERR_INVALID_ARGUMENT, "tokens without rows");
    kda_status st;
    const size_t blocks = (size_t)c->pages * c->num_kv_heads, codes = blocks * c->page_tokens * c->head_dim;
    if ((st = check_pointer("k_codes", c->k_codes, codes, 16)) || (st = check_pointer("v_codes", c->v_codes, codes, 16)) ||
        (st = check_pointer("k_scale", c->k_scale, blocks * 4, 4)) || (st = check_pointer("v_scale", c->v_scale, blocks * 4, 4)) ||
        (st = check_pointer("tables", c->tables, (size_t)c->rows * c->width * 4, 4)) ||
        (st = check_pointer("lens", lens, (size_t)c->rows * 4, 4)))
        return st;
    if (cu && !aligned(cu, 4)) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_tokens is not 4-byte aligned");
    return KDA_OK;
}

kda_status check_act(const char* name, const void* p, int64_t n, int64_t stride, int64_t inner) {
    if (stride < inner || stride % 8 != 0 || stride > (int64_t)1 << 32)
        return fail(KDA_ERR_INVALID_ARGUMENT, "%s: the token stride must be a multiple of 8, at least %lld (got %lld)", name,
                    (long long)inner, (long long)stride);
    return check_pointer(name, p, span(n, stride, inner), 16);
}

kda::CacheParams cache_params(const kda_kvcache* c, int64_t num_tokens, const int32_t* lens, const int32_t* cu, int32_t* status) {
    kda::CacheParams p{};
    p.k_codes = static_cast<uint8_t*>(c->k_codes);
    p.v_codes = static_cast<uint8_t*>(c->v_codes);
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.tables = c->tables;
    p.lens = lens;
    p.cu = cu;
    p.pages = c->pages;
    p.page_tokens = c->page_tokens;
    p.heads = c->num_kv_heads;
    p.dim = c->head_dim;
    p.rows = c->rows;
    p.width = c->width;
    p.tokens = num_tokens;
    p.status = status;
    return p;
}

// Attention over the cache; with cu_rows for groups of rows that share prefixes.
kda_status attend(const kda_kvcache* cache, const void* q, int32_t num_q_heads, int32_t act_dtype, int64_t q_stride, int64_t num_tokens,
                  const int32_t* lens, const int32_t* cu_tokens, const int32_t* cu_rows, int32_t groups, float scale, void* out,
                  int64_t out_stride, void* stream) {
    kda_status st = check_cache(cache, num_tokens, lens, cu_tokens);
    if (st != KDA_OK) return st;
    if (act_dtype != KDA_ACT_BF16 && act_dtype != KDA_ACT_F16)
        return fail(KDA_ERR_INVALID_ARGUMENT, "unknown act_dtype %d", act_dtype);
    if (num_q_heads < 1 || num_q_heads > (1 << 16) || num_q_heads % cache->num_kv_heads != 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_q_heads must be a multiple of num_kv_heads (got %d, %d)", num_q_heads,
                    cache->num_kv_heads);
    if (!isfinite(scale)) return fail(KDA_ERR_INVALID_ARGUMENT, "scale must be finite");
    const int64_t inner = (int64_t)num_q_heads * cache->head_dim;
    if ((st = check_act("q", q, num_tokens, q_stride, inner)) || (st = check_act("out", out, num_tokens, out_stride, inner))) return st;
    const size_t blocks = (size_t)cache->pages * cache->num_kv_heads, codes = blocks * cache->page_tokens * cache->head_dim;
    if ((st = check_overlap({{"out", {out, span(num_tokens, out_stride, inner)}}},
                            {{"q", {q, span(num_tokens, q_stride, inner)}}, {"k_codes", {cache->k_codes, codes}},
                             {"v_codes", {cache->v_codes, codes}}, {"k_scale", {cache->k_scale, blocks * 4}},
                             {"v_scale", {cache->v_scale, blocks * 4}},
                             {"tables", {cache->tables, (size_t)cache->rows * cache->width * 4}},
                             {"lens", {lens, (size_t)cache->rows * 4}},
                             {"cu_tokens", {cu_tokens, ((size_t)cache->rows + 1) * 4}},
                             {"cu_rows", {cu_rows, ((size_t)groups + 1) * 4}}})) != KDA_OK)
        return st;
    const int32_t group = num_q_heads / cache->num_kv_heads;
    if (num_tokens * group > 0x7fffff00 || (num_tokens * group / 8 + cache->rows) * cache->num_kv_heads > 0x7fffffff)
        return fail(KDA_ERR_INVALID_ARGUMENT, "too many tokens for one launch");
    int dev = 0;
    DeviceInfo* di = nullptr;
    if ((st = current_device(&dev, &di)) != KDA_OK) return st;
    if (num_tokens == 0) return KDA_OK;
    const bool f16 = act_dtype == KDA_ACT_F16;
    kda::AttentionParams p{};
    p.c = cache_params(cache, num_tokens, lens, cu_tokens, di->status);
    const int cols = kda::attention_cols(p.c, group, di->sm_count);
    p.sm_count = di->sm_count;
    p.ctas = kda::attention_ctas(cache->head_dim, cols, f16, di->sm_count);
    // With shared prefixes the parts' place is the prefixes' first, then the rows'.
    p.q_heads = num_q_heads;
    p.groups = groups;
    // (A tile of the prefixes' kernel is 1.3 us of an SM, as much as two rows' with few query rows each: 32 pairs of
    // rows of 16684 keys took 308 us with shared prefixes and 274 without, 21 groups of three 226 and 268.)
    const int32_t least = cols == 8 ? 3 : 2;
    if (cu_rows && !kda::sharing_pays(p, cols, least)) cu_rows = nullptr;
    const size_t units = (size_t)cache->rows;
    size_t bytes, at_o, at_ml, at_split, at_first, at_group, at_from, at_state, at_state_ml, at_item;
    auto place = [&](size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    };
    for (;;) {
        size_t parts = (cols == kda::kBlockRows ? (size_t)2 * p.ctas : kda::attention_slots(p.ctas)) * cols;
        size_t part_ml = parts * 2;
        if (cu_rows) {
            const size_t prefix = (size_t)(kda::prefix_items(p, least) + di->sm_count) * kda::kPrefixLanes;
            if (prefix > parts) parts = prefix;
            if (3 * prefix > part_ml) part_ml = 3 * prefix;
        }
        const size_t query_rows = cu_rows ? (size_t)num_tokens * num_q_heads : 0;
        bytes = 0;
        at_o = place(parts * cache->head_dim * 4), at_ml = place(part_ml * 4), at_split = place((size_t)p.ctas * 32);
        at_first = place((units + 1) * 8), at_group = place(cu_rows ? (size_t)groups * sizeof(kda::SharedGroup) : 0);
        at_from = place(cu_rows ? units * 4 : 0), at_state = place(query_rows * cache->head_dim * 4);
        at_state_ml = place(query_rows * 16), at_item = place(cu_rows ? (units + 1) * 8 : 0);
        if (!cu_rows || bytes <= kda::kMostSharedScratch) break;
        cu_rows = nullptr;  // worked out without shared prefixes
    }
    Scratch ws;
    if ((st = ws.take(dev, stream, bytes)) != KDA_OK) return st;
    p.part_o = reinterpret_cast<float*>(ws.base + at_o);
    p.part_ml = reinterpret_cast<float*>(ws.base + at_ml);
    p.split_items = ws.base + at_split;
    p.first_work = reinterpret_cast<int64_t*>(ws.base + at_first);
    p.q = q;
    p.out = out;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.scale = scale * 1.4426950408889634f;
    const cudaStream_t on = (cudaStream_t)stream;
    if (!cu_rows) {
        const cudaError_t e = kda::launch_attention(p, cols, f16, on);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "cache attention launch");
    }
    kda::SharedPlan plan{p.c, cu_rows, groups, least, reinterpret_cast<kda::SharedGroup*>(ws.base + at_group), reinterpret_cast<int32_t*>(ws.base + at_from)};
    p.group = plan.group;
    p.from = plan.from;
    p.state_o = reinterpret_cast<float*>(ws.base + at_state);
    p.state_ml = reinterpret_cast<float4*>(ws.base + at_state_ml);
    p.first_item = reinterpret_cast<int64_t*>(ws.base + at_item);
    kda::AttentionParams prefix = p;
    prefix.ctas = di->sm_count;
    prefix.least = least;
    cudaError_t e = kda::launch_shared_plan(plan, on);
    if (e == cudaSuccess) e = kda::launch_prefix(prefix, f16, on);
    if (e == cudaSuccess) e = kda::launch_suffix(p, cols, f16, on);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "shared attention launch");
}

}  // namespace

extern "C" {

kda_status kda_pages_alloc(const kda_page_shape* shape, const int32_t* tables, const int32_t* refs,
                           const int32_t* want, int32_t* new_tables, int32_t* new_refs, void* stream) {
    return guarded([&] {
        const size_t n = shape && shape->rows > 0 ? (size_t)shape->rows * 4 : 0;
        kda_status st = check_plan(shape, tables, refs, {"want", {want, n}}, 4, {"", {nullptr, 0}}, new_tables, new_refs);
        if (st != KDA_OK) return st;
        kda::PagePlan p = plan_of(shape, tables, refs, new_tables, new_refs);
        p.want = want;
        return run_plan(p, kda::kPagesAlloc, false, kda::PoolSet{}, stream);
    });
}

kda_status kda_pages_free(const kda_page_shape* shape, const int32_t* tables, const int32_t* refs,
                          const uint8_t* drop, int32_t* new_tables, int32_t* new_refs, void* stream) {
    return guarded([&] {
        const size_t n = shape && shape->rows > 0 ? (size_t)shape->rows : 0;
        kda_status st = check_plan(shape, tables, refs, {"drop", {drop, n}}, 1, {"", {nullptr, 0}}, new_tables, new_refs);
        if (st != KDA_OK) return st;
        kda::PagePlan p = plan_of(shape, tables, refs, new_tables, new_refs);
        p.drop = drop;
        return run_plan(p, kda::kPagesFree, false, kda::PoolSet{}, stream);
    });
}

kda_status kda_pages_fork(const kda_page_shape* shape, const int32_t* tables, const int32_t* refs,
                          const int32_t* parents, const int32_t* lens, int32_t page_tokens,
                          const kda_pool* pools, int32_t num_pools, int32_t* new_tables,
                          int32_t* new_refs, void* stream) {
    return guarded([&] {
        if (page_tokens < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "page_tokens must be >= 0 (got %d)", page_tokens);
        const size_t n = shape && shape->rows > 0 ? (size_t)shape->rows * 4 : 0;
        kda_status st = check_plan(shape, tables, refs, {"parents", {parents, n}}, 4,
                                   {"lens", {lens, page_tokens > 0 ? n : 0}}, new_tables, new_refs);
        if (st != KDA_OK) return st;
        kda::PoolSet set;
        if ((st = make_pools(pools, num_pools, shape->pages, &set)) != KDA_OK) return st;
        const size_t tb = n * shape->width, rb = (size_t)shape->pages * 4;
        if ((st = check_pool_overlap(set, shape->pages,
                                     {{"tables", {tables, tb}}, {"refs", {refs, rb}}, {"parents", {parents, n}}, {"lens", {lens, n}},
                                      {"new_tables", {new_tables, tb}}, {"new_refs", {new_refs, rb}}})) != KDA_OK)
            return st;
        kda::PagePlan p = plan_of(shape, tables, refs, new_tables, new_refs);
        p.parents = parents;
        p.lens = lens;
        p.page_tokens = page_tokens;
        return run_plan(p, kda::kPagesFork, false, set, stream);
    });
}

kda_status kda_pages_compact(const kda_page_shape* shape, const int32_t* tables, const int32_t* refs,
                             const kda_pool* pools, int32_t num_pools, int32_t* new_tables,
                             int32_t* new_refs, int32_t* page_map, int32_t* num_live, void* stream) {
    return guarded([&] {
        kda_status st = check_plan(shape, tables, refs, {"", {nullptr, 0}}, 1, {"", {nullptr, 0}}, new_tables, new_refs);
        if (st != KDA_OK) return st;
        const size_t tb = (size_t)shape->rows * shape->width * 4, rb = (size_t)shape->pages * 4;
        if ((st = check_pointer("page_map", page_map, rb, 4)) || (st = check_pointer("num_live", num_live, 4, 4)) ||
            (st = check_overlap({{"page_map", {page_map, rb}}, {"num_live", {num_live, 4}}},
                                {{"tables", {tables, tb}}, {"refs", {refs, rb}}, {"new_tables", {new_tables, tb}},
                                 {"new_refs", {new_refs, rb}}})))
            return st;
        kda::PoolSet set;
        if ((st = make_pools(pools, num_pools, shape->pages, &set)) != KDA_OK) return st;
        if ((st = check_pool_overlap(set, shape->pages,
                                     {{"tables", {tables, tb}}, {"refs", {refs, rb}}, {"new_tables", {new_tables, tb}},
                                      {"new_refs", {new_refs, rb}}, {"page_map", {page_map, rb}}, {"num_live", {num_live, 4}}})) != KDA_OK)
            return st;
        kda::PagePlan p = plan_of(shape, tables, refs, new_tables, new_refs);
        p.page_map = page_map;
        p.num_live = num_live;
        return run_plan(p, kda::kPagesFork, true, set, stream);
    });
}

kda_status kda_pages_copy(int32_t pages, int32_t count, const int32_t* src, const int32_t* dst,
                          const kda_pool* pools, int32_t num_pools, void* stream) {
    return guarded([&] {
        if (pages < 0 || pages > (1 << 30) || count < 0 || count > (1 << 30))
            return fail(KDA_ERR_INVALID_ARGUMENT, "pages and count must be in [0, 2^30] (got %d, %d)", pages, count);
        kda_status st;
        if ((st = check_pointer("src", src, (size_t)count * 4, 4)) || (st = check_pointer("dst", dst, (size_t)count * 4, 4))) return st;
        kda::PoolSet set;
        if ((st = make_pools(pools, num_pools, pages, &set)) != KDA_OK) return st;
        if ((st = check_pool_overlap(set, pages, {{"src", {src, (size_t)count * 4}}, {"dst", {dst, (size_t)count * 4}}})) != KDA_OK)
            return st;
        int dev = 0;
        DeviceInfo* di = nullptr;
        if ((st = current_device(&dev, &di)) != KDA_OK) return st;
        const cudaError_t e = kda::launch_page_copy(set, pages, src, dst, nullptr, count, di->status, di->sm_count, (cudaStream_t)stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "page copy launch");
    });
}

kda_status kda_kvcache_append(const kda_kvcache* cache, const void* k, const void* v,
                              int32_t act_dtype, int64_t k_stride, int64_t v_stride,
                              int64_t num_tokens, const int32_t* lens, const int32_t* cu_tokens,
                              void* stream) {
    return guarded([&] {
        kda_status st = check_cache(cache, num_tokens, lens, cu_tokens);
        if (st != KDA_OK) return st;
        if (act_dtype != KDA_ACT_BF16 && act_dtype != KDA_ACT_F16)
            return fail(KDA_ERR_INVALID_ARGUMENT, "unknown act_dtype %d", act_dtype);
        const int64_t inner = (int64_t)cache->num_kv_heads * cache->head_dim;
        if ((st = check_act("k", k, num_tokens, k_stride, inner)) || (st = check_act("v", v, num_tokens, v_stride, inner))) return st;
        const size_t blocks = (size_t)cache->pages * cache->num_kv_heads, codes = blocks * cache->page_tokens * cache->head_dim;
        if ((st = check_overlap({{"k_codes", {cache->k_codes, codes}}, {"v_codes", {cache->v_codes, codes}},
                                 {"k_scale", {cache->k_scale, blocks * 4}}, {"v_scale", {cache->v_scale, blocks * 4}}},
                                {{"k", {k, span(num_tokens, k_stride, inner)}}, {"v", {v, span(num_tokens, v_stride, inner)}},
                                 {"tables", {cache->tables, (size_t)cache->rows * cache->width * 4}},
                                 {"lens", {lens, (size_t)cache->rows * 4}},
                                 {"cu_tokens", {cu_tokens, ((size_t)cache->rows + 1) * 4}}})) != KDA_OK)
            return st;
        const int64_t units = cu_tokens ? num_tokens / cache->page_tokens + 2ll * cache->rows : 0;
        if (units > 0x7fffffff || 2 * num_tokens * cache->num_kv_heads > 0x7fffffffll * 4)
            return fail(KDA_ERR_INVALID_ARGUMENT, "too many tokens for one launch");
        int dev = 0;
        DeviceInfo* di = nullptr;
        if ((st = current_device(&dev, &di)) != KDA_OK) return st;
        kda::AppendParams p{};
        p.c = cache_params(cache, num_tokens, lens, cu_tokens, di->status);
        p.x[0] = k;
        p.x[1] = v;
        p.stride[0] = k_stride;
        p.stride[1] = v_stride;
        const cudaError_t e = kda::launch_append(p, act_dtype == KDA_ACT_F16, (cudaStream_t)stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "cache append launch");
    });
}

kda_status kda_kvcache_append_rotary(const kda_kvcache* cache, const void* q, const void* k, const void* v,
                                     int32_t num_q_heads, int32_t act_dtype, int64_t q_stride,
                                     int64_t k_stride, int64_t v_stride, int64_t num_tokens,
                                     const int32_t* lens, const int32_t* cu_tokens, const float* rotary,
                                     int64_t num_positions, int32_t rotary_dim, int32_t interleaved,
                                     const int32_t* positions, void* q_out, int64_t out_stride,
                                     void* stream) {
    return guarded([&] {
        kda_status st = check_cache(cache, num_tokens, lens, cu_tokens);
        if (st != KDA_OK) return st;
        if (act_dtype != KDA_ACT_BF16 && act_dtype != KDA_ACT_F16)
            return fail(KDA_ERR_INVALID_ARGUMENT, "unknown act_dtype %d", act_dtype);
        if (num_q_heads < 1 || num_q_heads > (1 << 16))
            return fail(KDA_ERR_INVALID_ARGUMENT, "num_q_heads must be in [1, 2^16] (got %d)", num_q_heads);
        if (rotary_dim < 16 || rotary_dim % 16 != 0 || rotary_dim > cache->head_dim)
            return fail(KDA_ERR_INVALID_ARGUMENT, "rotary_dim must be a multiple of 16 in [16, head_dim] (got %d)", rotary_dim);
        if (num_positions < 0 || num_positions > (int64_t)1 << 31)
            return fail(KDA_ERR_INVALID_ARGUMENT, "num_positions must be in [0, 2^31] (got %lld)", (long long)num_positions);
        const int64_t inner = (int64_t)cache->num_kv_heads * cache->head_dim, q_inner = (int64_t)num_q_heads * cache->head_dim;
        if ((st = check_act("q", q, num_tokens, q_stride, q_inner)) || (st = check_act("k", k, num_tokens, k_stride, inner)) ||
            (st = check_act("v", v, num_tokens, v_stride, inner)) || (st = check_act("q_out", q_out, num_tokens, out_stride, q_inner)))
            return st;
        const size_t table = (size_t)num_positions * rotary_dim * 4;
        if ((st = check_pointer("rotary", rotary, table, 16))) return st;
        if (positions && !aligned(positions, 4)) return fail(KDA_ERR_INVALID_ARGUMENT, "positions is not 4-byte aligned");
        const size_t blocks = (size_t)cache->pages * cache->num_kv_heads, codes = blocks * cache->page_tokens * cache->head_dim;
        const Range out_r{q_out, span(num_tokens, out_stride, q_inner)};
        const Buffer tables{"tables", {cache->tables, (size_t)cache->rows * cache->width * 4}}, lens_b{"lens", {lens, (size_t)cache->rows * 4}},
            cu_b{"cu_tokens", {cu_tokens, ((size_t)cache->rows + 1) * 4}}, rotary_b{"rotary", {rotary, table}},
            positions_b{"positions", {positions, (size_t)num_tokens * 4}};
        if ((st = check_overlap({{"k_codes", {cache->k_codes, codes}}, {"v_codes", {cache->v_codes, codes}},
                                 {"k_scale", {cache->k_scale, blocks * 4}}, {"v_scale", {cache->v_scale, blocks * 4}}},
                                {{"q", {q, span(num_tokens, q_stride, q_inner)}}, {"k", {k, span(num_tokens, k_stride, inner)}},
                                 {"v", {v, span(num_tokens, v_stride, inner)}}, {"q_out", out_r}, tables, lens_b, cu_b, rotary_b, positions_b})) ||
            (st = check_overlap({{"q_out", out_r}}, {tables, lens_b, cu_b, rotary_b, positions_b})))
            return st;
        if (strided_overlap(q_out, out_stride, q_inner, k, k_stride, inner, num_tokens)) return fail(KDA_ERR_ALIASING, "q_out overlaps k");
        if (strided_overlap(q_out, out_stride, q_inner, v, v_stride, inner, num_tokens)) return fail(KDA_ERR_ALIASING, "q_out overlaps v");
        if ((q_out != q || out_stride != q_stride) && strided_overlap(q_out, out_stride, q_inner, q, q_stride, q_inner, num_tokens))
            return fail(KDA_ERR_ALIASING, "q_out overlaps q");
        const int64_t units = cu_tokens ? num_tokens / cache->page_tokens + 2ll * cache->rows : 0;
        if (units > 0x7fffffff || 2 * num_tokens * cache->num_kv_heads > 0x7fffffffll * 2 || num_tokens * num_q_heads > 0x7fffffffll * 4)
            return fail(KDA_ERR_INVALID_ARGUMENT, "too many tokens for one launch");
        int dev = 0;
        DeviceInfo* di = nullptr;
        if ((st = current_device(&dev, &di)) != KDA_OK) return st;
        kda::RotaryParams p{};
        p.c = cache_params(cache, num_tokens, lens, cu_tokens, di->status);
        p.x[0] = k;
        p.x[1] = v;
        p.stride[0] = k_stride;
        p.stride[1] = v_stride;
        p.q = q;
        p.q_out = q_out;
        p.q_stride = q_stride;
        p.out_stride = out_stride;
        p.q_heads = num_q_heads;
        p.table = rotary;
        p.positions = positions;
        p.num_positions = num_positions;
        p.rot = rotary_dim;
        p.interleaved = interleaved != 0;
        const cudaError_t e = kda::launch_rotary_append(p, act_dtype == KDA_ACT_F16, (cudaStream_t)stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "rotary append launch");
    });
}

kda_status kda_kvcache_attention(const kda_kvcache* cache, const void* q, int32_t num_q_heads,
                                 int32_t act_dtype, int64_t q_stride, int64_t num_tokens,
                                 const int32_t* lens, const int32_t* cu_tokens, float scale,
                                 void* out, int64_t out_stride, void* stream) {
    return guarded([&] {
        return attend(cache, q, num_q_heads, act_dtype, q_stride, num_tokens, lens, cu_tokens, nullptr, 0, scale, out, out_stride, stream);
    });
}

kda_status kda_kvcache_attention_shared(const kda_kvcache* cache, const void* q, int32_t num_q_heads,
                                        int32_t act_dtype, int64_t q_stride, int64_t num_tokens,
                                        const int32_t* lens, const int32_t* cu_tokens,
                                        const int32_t* cu_rows, int32_t num_groups, float scale,
                                        void* out, int64_t out_stride, void* stream) {
    return guarded([&] {
        const int32_t rows = cache ? cache->rows : 0;
        if (num_groups < 0 || num_groups > (1 << 24) || (num_groups == 0 && rows > 0))
            return fail(KDA_ERR_INVALID_ARGUMENT, "num_groups must be in [1, 2^24] (got %d)", num_groups);
        const kda_status st = check_pointer("cu_rows", cu_rows, ((size_t)num_groups + 1) * 4, 4);
        if (st != KDA_OK) return st;
        return attend(cache, q, num_q_heads, act_dtype, q_stride, num_tokens, lens, cu_tokens, cu_rows, num_groups, scale, out, out_stride, stream);
    });
}

kda_status kda_logits_penalize(const kda_logits_rules* rules, int64_t rows, int32_t vocab,
                               const void* logits, int32_t logits_dtype, int64_t logits_stride,
                               void* out, int64_t out_stride, void* stream) {
    return guarded([&] {
        if (!rules) return fail(KDA_ERR_INVALID_ARGUMENT, "rules is NULL");
        const kda_logits_rules& r = *rules;
        if (rows < 0 || rows > (1 << 30) || vocab < 1 || vocab > (1 << 30))
            return fail(KDA_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^30], vocab in [1, 2^30] (got %lld, %d)", (long long)rows, vocab);
        if (logits_dtype != KDA_LOGITS_F32 && logits_dtype != KDA_LOGITS_BF16 && logits_dtype != KDA_LOGITS_F16)
            return fail(KDA_ERR_INVALID_ARGUMENT, "unknown logits_dtype %d", logits_dtype);
        for (const int64_t s : {logits_stride, out_stride})
            if (s < vocab || s > (int64_t)1 << 32)
                return fail(KDA_ERR_INVALID_ARGUMENT, "logits_stride and out_stride must be at least vocab (got %lld)", (long long)s);
        // (A token's count has 30 bits.)
        if (r.history_width < 0 || r.history_width >= (1 << 30) || r.num_bias < 0 || r.num_bias > (1 << 30))
            return fail(KDA_ERR_INVALID_ARGUMENT, "history_width must be in [0, 2^30), num_bias in [0, 2^30] (got %d, %d)", r.history_width, r.num_bias);
        const int64_t words = ((int64_t)vocab + 31) / 32;
        if (r.mask && (r.mask_stride < words || r.mask_stride > (int64_t)1 << 32))
            return fail(KDA_ERR_INVALID_ARGUMENT, "mask_stride must be at least %lld (got %lld)", (long long)words, (long long)r.mask_stride);
        const size_t elem = logits_dtype == KDA_LOGITS_F32 ? 4 : 2, n = (size_t)rows;
        auto bytes = [&](int64_t stride) { return rows > 0 ? (size_t)((rows - 1) * stride + vocab) * elem : 0; };
        const size_t lb = bytes(logits_stride), ob = bytes(out_stride);
        const size_t hb = n * r.history_width * 4, bb = n * r.num_bias * 4;
        const size_t mb = r.mask && rows > 0 ? (size_t)((rows - 1) * r.mask_stride + words) * 4 : 0;
        kda_status st;
        if ((st = check_pointer("logits", logits, lb, elem)) || (st = check_pointer("out", out, ob, elem)) ||
            (st = check_pointer("history", r.history, hb, 4)) || (st = check_pointer("bias_tokens", r.bias_tokens, bb, 4)) ||
            (st = check_pointer("bias", r.bias, bb, 4)) || (st = check_pointer("mask", r.mask, mb, 4)))
            return st;
        const Buffer per_row[] = {{"lens", {r.lens, n * 4}}, {"prompt_lens", {r.prompt_lens, n * 4}}, {"repetition", {r.repetition, n * 4}},
                                  {"presence", {r.presence, n * 4}}, {"frequency", {r.frequency, n * 4}}};
        for (const Buffer& b : per_row)
            if (b.r.p && !aligned(b.r.p, 4)) return fail(KDA_ERR_INVALID_ARGUMENT, "%s is not 4-byte aligned", b.name);
        const Buffer out_b{"out", {out, ob}};
        if ((st = check_overlap({out_b}, {{"history", {r.history, hb}}, {"bias_tokens", {r.bias_tokens, bb}}, {"bias", {r.bias, bb}}, {"mask", {r.mask, mb}},
                                          per_row[0], per_row[1], per_row[2], per_row[3], per_row[4]})) != KDA_OK)
            return st;
        if ((out != logits || out_stride != logits_stride) && (st = check_overlap({out_b}, {{"logits", {logits, lb}}})) != KDA_OK) return st;
        int dev = 0;
        DeviceInfo* di = nullptr;
        if ((st = current_device(&dev, &di)) != KDA_OK) return st;
        if (rows == 0) return KDA_OK;
        kda::LogitsParams p{};
        p.logits = logits;
        p.out = out;
        p.stride = logits_stride;
        p.out_stride = out_stride;
        p.rows = rows;
        p.vocab = vocab;
        // (Without penalties a history changes nothing.)
        const bool counted = r.repetition || r.presence || r.frequency;
        p.history = r.history;
        p.width = counted ? r.history_width : 0;
        p.lens = r.lens;
        p.prompt_lens = r.prompt_lens;
        p.repetition = r.repetition;
        p.presence = r.presence;
        p.frequency = r.frequency;
        p.bias_tokens = r.bias_tokens;
        p.bias = r.bias;
        p.num_bias = r.num_bias;
        p.mask = reinterpret_cast<const uint32_t*>(r.mask);
        p.mask_stride = r.mask_stride;
        p.status = di->status;
        p.sm_count = di->sm_count;
        if (rows * ((int64_t)vocab / 1024 + 2) > 0x7fffffff) return fail(KDA_ERR_INVALID_ARGUMENT, "rows * vocab is too large for one launch");
        const cudaError_t e = kda::launch_penalize(p, logits_dtype, (cudaStream_t)stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "logits penalties launch");
    });
}

kda_status kda_beam_select(int32_t batch, int32_t beams, int32_t vocab, int32_t num_out,
                           const void* logits, int32_t logits_dtype, int64_t logits_stride,
                           const float* scores, const uint8_t* done, int32_t eos,
                           float* new_scores, int32_t* tokens, int32_t* parents,
                           uint8_t* new_done, void* stream) {
    return guarded([&] {
        if (batch < 0 || beams < 1 || beams > 64 || num_out < 1 || num_out > 64)
            return fail(KDA_ERR_INVALID_ARGUMENT, "batch must be >= 0, beams and num_out in [1, 64] (got %d, %d, %d)", batch, beams, num_out);
        if (vocab < 1 || (int64_t)beams * vocab > (1 << 30) || (int64_t)batch * beams > (1 << 30))
            return fail(KDA_ERR_INVALID_ARGUMENT, "vocab must be >= 1, beams * vocab at most 2^30, batch * beams at most 2^30 (got %d)", vocab);
        if (logits_dtype != KDA_LOGITS_F32 && logits_dtype != KDA_LOGITS_BF16 && logits_dtype != KDA_LOGITS_F16)
            return fail(KDA_ERR_INVALID_ARGUMENT, "unknown logits_dtype %d", logits_dtype);
        if (logits_stride < vocab || logits_stride > (int64_t)1 << 32)
            return fail(KDA_ERR_INVALID_ARGUMENT, "logits_stride must be at least vocab (got %lld)", (long long)logits_stride);
        if (eos < -1 || eos >= vocab) return fail(KDA_ERR_INVALID_ARGUMENT, "eos must be in [0, vocab) or -1 (got %d)", eos);
        if (done && eos < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "done needs an eos token");
        const int64_t rows = (int64_t)batch * beams, outs = (int64_t)batch * num_out;
        const size_t elem = logits_dtype == KDA_LOGITS_F32 ? 4 : 2;
        const size_t lb = rows > 0 ? (size_t)((rows - 1) * logits_stride + vocab) * elem : 0;
        const size_t sb = (size_t)rows * 4, ob = (size_t)outs * 4;
        kda_status st;
        if ((st = check_pointer("logits", logits, lb, elem)) || (st = check_pointer("scores", scores, sb, 4)) ||
            (st = check_pointer("new_scores", new_scores, ob, 4)) || (st = check_pointer("tokens", tokens, ob, 4)) ||
            (st = check_pointer("parents", parents, ob, 4)))
            return st;
        if ((st = check_overlap({{"new_scores", {new_scores, ob}}, {"tokens", {tokens, ob}}, {"parents", {parents, ob}},
                                 {"new_done", {new_done, (size_t)outs}}},
                                {{"logits", {logits, lb}}, {"scores", {scores, sb}}, {"done", {done, (size_t)rows}}})) != KDA_OK)
            return st;
        int dev = 0;
        DeviceInfo* di = nullptr;
        if ((st = current_device(&dev, &di)) != KDA_OK) return st;
        if (batch == 0) return KDA_OK;
        kda::BeamParams p{};
        p.logits = logits;
        p.stride = logits_stride;
        p.dtype = logits_dtype;
        p.scores = scores;
        p.done = done;
        p.eos = eos;
        p.batch = batch;
        p.beams = beams;
        p.vocab = vocab;
        p.k = num_out;
        p.new_scores = new_scores;
        p.tokens = tokens;
        p.parents = parents;
        p.new_done = new_done;
        p.seg_len = kda::beam_seg_len(rows, vocab, (int)elem, di->sm_count);
        // Rows that do not all start on 16 bytes are cut at 16-byte boundaries: up to one
        // load's elements more.
        const bool even = aligned(logits, 16) && (size_t)logits_stride * elem % 16 == 0;
        p.segs = (int32_t)(((int64_t)vocab + (even ? 0 : 16 / elem - 1) + p.seg_len - 1) / p.seg_len);
        if (rows * p.segs > 0x7fffffffll) return fail(KDA_ERR_INVALID_ARGUMENT, "batch * beams * vocab is too large");
        const size_t pb = (size_t)rows * p.segs * 16, cb = (size_t)rows * p.segs * (num_out + 1) * 8;
        Scratch ws;
        if ((st = ws.take(dev, stream, cb + pb)) != KDA_OK) return st;
        p.part = reinterpret_cast<float4*>(ws.base);
        p.cand = reinterpret_cast<uint64_t*>(ws.base + pb);
        const cudaError_t e = kda::launch_beam(p, (cudaStream_t)stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "beam selection launch");
    });
}

}  // extern "C"
