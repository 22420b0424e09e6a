// Launch arguments of the kernels that run between the products of a decode
// step: q/k norms with rotation and cache append, attention over the paged
// cache, and sampling. The contract of every operator is in include/qmm.h;
// the host checks are in qmm_step.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmm {

// q/k norm, rotation and cache append (qmm_rope.hip).
struct RopeArgs {
    const void *q, *k, *v;                    // [M, heads * D], row strides below
    int64_t q_stride, k_stride, v_stride;     // elements between rows
    const float *q_weight, *k_weight;         // [D]
    const int32_t *positions, *slots;         // [M]
    const float *inv_freq;                    // [R / 2]
    void *q_out;                              // [M, Hq, D]
    void *k_cache, *v_cache;                  // [num_pages, Hkv, page_size, D]
    int M, Hq, Hkv, D, R, page_size;
    uint64_t page_magic;                      // division by page_size (magic_div)
    int page_shift;
    int slot_count;                           // num_pages * page_size
    float eps, weight_offset;
};
hipError_t launch_qk_norm_rope(const RopeArgs &a, int in_type, bool bf16_out, bool interleaved, hipStream_t stream);

// Attention over the paged cache (qmm_attn.hip).
struct AttnArgs {
    const void *q;                            // [T, Hq, D], q_stride elements between rows
    const void *k_cache, *v_cache;            // [num_pages, Hkv, page_size, D]
    const int32_t *block_table;               // [B, max_pages]
    const int32_t *context_lens;              // [B]
    const int32_t *row_starts;                // [B + 1]
    void *out;                                // [T, Hq, D]
    float *lse;                               // [T, Hq] or null
    int2 *joins;                              // [B, chunks, Hkv]: first and last run of an item
    float *part_acc, *part_ml;                // partials, two slots a run: [2 groups, columns, D] and [.., 2]
    int64_t q_stride;
    int T, B, Hq, Hkv, page_size, num_pages, max_pages;
    int window, sinks;
    float scale_log2;                         // scale * log2(e)
    uint64_t page_magic;                      // division by page_size (magic_div)
    int page_shift;
    uint64_t group_magic;                     // division by G = Hq / Hkv
    int group_shift, G;
    int chunks;                               // column chunks of one (sequence, kv head)
    int groups;                               // runs
    int whole, pieces;                        // how items are dealt out (qmm_attn.hip)
    int one_page;                             // page_size is a multiple of 16
};
// How a call is laid out on the GPU; a function of host arguments only.
struct AttnPlan {
    int col_tiles;    // 16-column tiles of a workgroup
    int chunks, groups, join_columns, join_threads;
    bool whole, pieces;
    int64_t blocks, items;
    size_t join_bytes, workspace_bytes;
};
constexpr int kAttnMostTile = 128;  // tokens of the largest tile
bool attn_head_dim_supported(int D);
AttnPlan attn_plan(int B, int Hq, int Hkv, int D, int max_rows, int max_context, int window, int sinks,
                   int page_size, int max_pages);
hipError_t launch_paged_attention(AttnArgs a, const AttnPlan &p, int D, bool bf16, void *workspace, hipStream_t stream);

// Sampling (qmm_sample.hip).
struct SampleArgs {
    const void *logits;                       // [M, V], row_stride elements between rows
    int64_t row_stride;
    const float *u, *temperature, *top_p, *min_p;  // [M]; all but u may be null
    const int32_t *top_k;                     // [M] or null
    int32_t *tokens;                          // [M]
    float *logprobs;                          // [M] or null
    void *workspace;
    int M, V;
};
bool sample_size_supported(int V);
size_t sample_workspace_bytes(int M, int V);
hipError_t launch_sample(const SampleArgs &a, int type, hipStream_t stream);

// n / d = (n * magic) >> (32 + shift) for 0 <= n < 2^31, with
// magic = ceil(2^(32 + shift) / d) and d <= 2^(shift + 1): the magic's excess
// over the exact quotient is below 2^-(shift + 32) * d <= 2^-31 of a unit per
// n, so it never reaches the next multiple. magic has up to 33 bits (d = 1).
struct MagicDiv {
    uint64_t magic;
    int shift;
};
inline MagicDiv magic_div(uint32_t d)
{
    int s = 0;
    while (((uint64_t)2 << s) < d)
        ++s;
    return MagicDiv{(((uint64_t)1 << (32 + s)) + d - 1) / d, s};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, uint64_t magic, int shift)
{
    return (uint32_t)(((uint64_t)n * magic) >> (32 + shift));
}

}  // namespace qmm
