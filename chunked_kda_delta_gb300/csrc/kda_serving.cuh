// kda_serving.cuh -- declarations shared by the serving operators (page operations, 8-bit
// key/value cache, beam selection) and their host entries.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.cuh"

namespace kda {

constexpr int32_t kStatusBadIndex = kStatusBadSeqlens;  // KDA_ERR_INVALID_ARGUMENT
constexpr int32_t kStatusNoFreePage = 8;
constexpr int32_t kStatusNonfinite = 9;

// Records the first condition since the last read.
__device__ __forceinline__ void report(int32_t* status, int32_t code) { atomicCAS(status, kStatusOk, code); }

// The serving operators' launches are a few microseconds each, so each may be set up while the
// one before it in the stream runs: launched with launch_early, a kernel calls follow_stream before
// it reads or writes anything that another launch writes, on every path.  There it waits until the
// launches before it are complete; the one after it may be set up from then on, which is why all
// that a kernel's own predecessor did not write may be read before the call.
__device__ __forceinline__ void follow_stream() {
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
}
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- recurrent step on pages ------------------------------------------------------------
// s0 == sfin is a pool: sequence n's states are at element state_pages[n] * page_stride;
// negative pages are idle sequences.
struct PagedDecodeParams : DecodeParams {
    const int32_t* state_pages;
    int32_t num_pages;
    int64_t page_stride;
    int32_t* status;
};
cudaError_t launch_decode_paged(const PagedDecodeParams& p, cudaStream_t stream);

// ---- pages ----------------------------------------------------------------------------
constexpr int kMaxPools = 64;

struct PoolSet {
    struct One {
        char* base;
        int64_t page_bytes, page_stride, layer_stride;
        int32_t layers;
        int32_t chunks;  // copy chunks of one page of one layer
        int32_t unit;    // bytes of a load: 16, 4 or 1, dividing every address and size
    } pool[kMaxPools];
    int32_t n;
    int64_t chunks;  // copy chunks of one page over all pools and layers
};
constexpr int kCopyChunk = 32768;  // bytes of one copy chunk

enum PageMode { kPagesFork = 0, kPagesAlloc = 1, kPagesFree = 2 };

struct PagePlan {
    const int32_t* tables;
    const int32_t* refs;
    const int32_t* parents;   // fork
    const int32_t* lens;      // fork with page_tokens > 0
    const int32_t* want;      // alloc
    const uint8_t* drop;      // free
    int32_t page_tokens;
    int32_t rows, width, pages;
    int32_t* new_tables;
    int32_t* new_refs;
    int32_t* page_map;        // compact
    int32_t* num_live;        // compact
    // scratch
    int32_t* held;            // [pages]
    int32_t* first;           // [pages]
    int32_t* list;            // [pages]: free pages in order
    int32_t* copies;          // [1]: pairs in src / dst
    int32_t* src;             // [rows * width] (compact: [pages])
    int32_t* dst;
    int32_t* status;
};
cudaError_t launch_page_plan(const PagePlan& p, int mode, cudaStream_t stream);
cudaError_t launch_page_compact(const PagePlan& p, cudaStream_t stream);
// Copies pages src[i] -> dst[i], i < *count (device) or < limit where count is null.
cudaError_t launch_page_copy(const PoolSet& pools, int32_t pages, const int32_t* src, const int32_t* dst,
                             const int32_t* count, int32_t limit, int32_t* status, int sm_count,
                             cudaStream_t stream);

// ---- 8-bit key/value cache ------------------------------------------------------------
struct CacheParams {
    uint8_t* k_codes;
    uint8_t* v_codes;
    float* k_scale;
    float* v_scale;
    const int32_t* tables;
    const int32_t* lens;
    const int32_t* cu;        // [rows + 1] or nullptr: one token a row
    int32_t pages, page_tokens, heads, dim, rows, width;
    int64_t tokens;
    int32_t* status;
};

struct AppendParams {
    CacheParams c;
    const void* x[2];         // k, v
    int64_t stride[2];
};
cudaError_t launch_append(const AppendParams& p, bool f16, cudaStream_t stream);
// With the positions' rotation (kda_kvcache_rotary.cu).
struct RotaryParams : AppendParams {
    const void* q;
    void* q_out;              // may be q, at q's stride
    int64_t q_stride, out_stride;
    int32_t q_heads;
    const float* table;       // [num_positions][rot]: cosines, then sines
    const int32_t* positions; // [tokens] or nullptr: places in the cache
    int64_t num_positions;
    int32_t rot;              // multiple of 16
    bool interleaved;
};
cudaError_t launch_rotary_append(const RotaryParams& p, bool f16, cudaStream_t stream);

// Rows that share a prefix.
struct SharedGroup {
    int64_t begin;            // first token of its rows
    int32_t tokens;           // of all its rows; 0: nothing is shared
    int32_t shared;           // tokens of the prefix, a multiple of kSharedUnit
    int32_t row;              // whose table is read
    int32_t unused;
};
constexpr int kSharedUnit = 128;

struct AttentionParams {
    CacheParams c;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    int32_t q_heads;
    float scale;              // times log2(e)
    // scratch
    void* split_items;    // scratch of 32 bytes a CTA (items of 128 query rows)
    int64_t* first_work;      // [rows + 1]
    float* part_o;            // [slots][cols * dim], in the layout of the product's fragments
    float* part_ml;           // [slots][cols][2]: maximum and sum
    int32_t ctas, sm_count;
    // shared prefixes
    const SharedGroup* group; // [groups]
    int32_t groups, least;    // least: SharedPlan's
    const int32_t* from;      // [rows]: tokens of the prefix
    float* state_o;           // [tokens * q_heads][dim], what the prefix left: outputs,
    float4* state_ml;         // [tokens * q_heads]: maximum, sum, what a log2 of v's scale counts as at least
    int64_t* first_item;      // [groups + 1] (kda_kvcache_prefix.cu)
};
size_t attention_slots(int ctas);
int attention_cols(const CacheParams& c, int32_t group, int sm_count);
int attention_ctas(int32_t dim, int cols, bool f16, int sm_count);
cudaError_t launch_attention(const AttentionParams& p, int cols, bool f16, cudaStream_t stream);
// Items of 128 query rows on tcgen05 (kda_kvcache_block.cu): two CTAs an SM, two parts each.
constexpr int kBlockRows = 128;
cudaError_t launch_block_attention(const AttentionParams& p, bool f16, cudaStream_t stream);
// The parts of attention with shared prefixes (kda_kvcache_shared.cu): the groups' prefixes are found, then
// worked out into the state, then the rows go on from there.
struct SharedPlan {
    CacheParams c;
    const int32_t* cu_rows;   // [groups + 1]
    int32_t groups;
    int32_t least;            // rows with tokens that a group must have to share
    SharedGroup* group;
    int32_t* from;
};
bool sharing_pays(const AttentionParams& p, int cols, int32_t least);  // cols: attention_cols
cudaError_t launch_shared_plan(const SharedPlan& p, cudaStream_t stream);
constexpr int kPrefixLanes = 256;  // query rows of an item, and of a part
int64_t prefix_items(const AttentionParams& p, int32_t least);  // at most
constexpr size_t kMostSharedScratch = (size_t)1 << 31;  // bytes; calls that would take more share nothing
cudaError_t launch_prefix(const AttentionParams& p, bool f16, cudaStream_t stream);
cudaError_t launch_block_suffix(const AttentionParams& p, bool f16, cudaStream_t stream);
cudaError_t launch_suffix(const AttentionParams& p, int cols, bool f16, cudaStream_t stream);

// ---- beam selection -------------------------------------------------------------------
struct BeamParams {
    const void* logits;
    int64_t stride;
    int32_t dtype;            // KDA_LOGITS_*
    const float* scores;
    const uint8_t* done;
    int32_t eos;
    int32_t batch, beams, vocab, k;
    float* new_scores;
    int32_t* tokens;
    int32_t* parents;
    uint8_t* new_done;
    // scratch
    uint64_t* cand;           // [batch * beams][segs][k + 1]
    float4* part;             // [batch * beams][segs]: sums of exponentials (kda_beam.cu)
    int32_t segs, seg_len;
};
int beam_seg_len(int64_t rows, int32_t vocab, int elem, int sm_count);
cudaError_t launch_beam(const BeamParams& p, cudaStream_t stream);

// ---- penalties, biases and masks on logits ----------------------------------------------
struct LogitsParams {
    const void* logits;
    void* out;
    int64_t stride, out_stride;
    int64_t rows;
    int32_t vocab;
    const int32_t* history;   // [rows][width]
    int32_t width;
    const int32_t* lens;      // [rows] or nullptr
    const int32_t* prompt_lens;
    const float* repetition;  // [rows] or nullptr, as the next two
    const float* presence;
    const float* frequency;
    const int32_t* bias_tokens;  // [rows][num_bias]
    const float* bias;
    int32_t num_bias;
    const uint32_t* mask;     // [rows][mask_stride] or nullptr
    int64_t mask_stride;
    int32_t* status;
    int32_t sm_count;
    // set by the launch
    int32_t segs, seg_len;    // segments of a row, their tokens
    int32_t entries, shift;   // of the table of a segment's touched tokens: 2^(32 - shift), or
    bool direct;              // one for each token
};
cudaError_t launch_penalize(LogitsParams p, int dtype, cudaStream_t stream);

}  // namespace kda
