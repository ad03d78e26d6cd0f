// launch.h -- host-side entry points of the kernels (internal to libpagedkv.so).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "decode_common.cuh"

namespace pkv {

// A launch that may overlap the end of the kernel before it (see depend_wait in step_utils.cuh), as a cluster of
// `cluster` CTAs where that is more than one.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster,
                              cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// kMathFp8: tensor-core (f16 mma.sync) math over e4m3 pools with per-head
// scales; chosen by the fp8 entry points, not by the math option.
// kMathTensorCoreGroups: kMathTensorCore plus the prefix units of prefix
// groups; chosen for a launch that has groups (a kernel of its own, so that
// launches without groups keep the leaner register allocation).
enum DecodeMath { kMathCudaCore = 1, kMathTensorCore = 2, kMathFp8 = 3, kMathTensorCoreGroups = 4 };

// True when the (head_dim, block_size, padded group, math) combination is compiled in.
bool decode_variant_exists(int head_dim, int block_size, int group_pad, int math);

// Shared-memory bytes per CTA of a decode variant (num_stages = stages per consumer warp).
size_t decode_smem_bytes(int head_dim, int block_size, int group_pad, int group, int math, int num_stages,
                         int num_seqs, int pack);

// Sets the variant's dynamic shared-memory limit (once per device) and returns
// how many CTAs of it fit on one SM.
cudaError_t decode_prepare(int head_dim, int block_size, int group_pad, int math, size_t smem_bytes,
                           int *ctas_per_sm);

cudaError_t decode_launch(int head_dim, int block_size, int group_pad, int math, const CUtensorMap &tm_k,
                          const CUtensorMap &tm_v, const DecodeArgs &args, int grid, size_t smem_bytes,
                          cudaStream_t stream);


cudaError_t append_launch(const void *k, const void *v, void *k_cache, void *v_cache, const int64_t *slot_mapping,
                          int num_tokens, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                          int32_t *status, cudaStream_t stream);

// Multi-query paged attention (prefill.cu).
struct PrefillArgs {
    void *out;                    // bf16 [T][Hq][D]
    const void *q;                // bf16 [T][Hq][D]
    const int32_t *block_tables;  // [S][MB]
    const int32_t *context_lens;  // [S]
    const int32_t *query_start;   // [S + 1]
    int32_t *status;
    int num_seqs, num_tokens, num_q_heads, num_kv_heads, group, max_blocks_per_seq, num_blocks, max_query_len;
    float scale_log2;
};

size_t prefill_smem_bytes(int head_dim, int block_size, int max_blocks_per_seq);
cudaError_t prefill_launch(int head_dim, int block_size, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                           const PrefillArgs &args, int tiles, size_t smem_bytes, cudaStream_t stream);
int prefill_rows_per_cta();

size_t prefill_tc_smem_bytes(int head_dim, int max_blocks_per_seq);
cudaError_t prefill_tc_launch(int head_dim, int block_size, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                              const CUtensorMap &tm_v, const PrefillArgs &args, int tiles, size_t smem_bytes,
                              cudaStream_t stream);
int prefill_tc_rows_per_cta();

// Attention of drafted trees (tree.cu).
struct TreeArgs {
    void *out;                    // bf16 [T][Hq][D]
    const void *q;                // bf16 [T][Hq][D]
    const void *k_cache;          // [NB][BS][Hkv][D], bf16 or e4m3 codes
    const void *v_cache;
    const float *k_scale;         // e4m3 pools: fp32 [Hkv]
    const float *v_scale;
    const int32_t *block_tables;  // [S][MB]
    const int32_t *context_lens;  // [S], the drafts included
    const int32_t *query_start;   // [S + 1]
    const int32_t *tree_mask;     // [T][mask_words]
    int32_t *status;
    int num_seqs, num_tokens, max_query_len, mask_words, num_q_heads, num_kv_heads, group, block_size,
        max_blocks_per_seq, num_blocks;
    float scale_log2;             // not zero
    int tile_drafts;              // drafts of a 128-row tile: 128 / group
    int lists;                    // 2: some sequence may take a second row tile
    int piece_cost;               // a segment's fixed weight, in iterations
    int min_weight;               // iterations that make another CTA worth it
    int whole;                    // 1: no segment is cut
    float *o_part;                // fp32 [2 * CTAs][D / 4][128][4]: a CTA's partials of a continued and of a begun segment
    float2 *ml_part;              // their rows' maximum (log2 domain) and sum
    int4 *cuts;                   // [CTAs]: the segment of over two pieces that a CTA begins (see tree_merge_kernel)
    unsigned *arrivals;           // [CTAs], by a two-piece segment's first CTA: pieces that have ended + 16 x warps that
                                  // have stored the first one's partial; 0 between launches
};

// Sequences of one launch: their weights share the memory of two CTAs per SM with the operands, and with the rings
// of codes over e4m3 pools.
constexpr int kTreeMaxSeqs = 1024, kTreeMaxSeqsFp8 = 512;
constexpr int kTreeMaxCtas = 320;

cudaError_t tree_launch(bool fp8, int head_dim, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                        const CUtensorMap &tm_v, const TreeArgs &args, int ctas, cudaStream_t stream);

// A step's bookkeeping on the GPU (tables.cu).
cudaError_t tables_grow_launch(int32_t *block_tables, const int32_t *context_lens, const int32_t *new_tokens,
                               const int32_t *free_blocks, const int32_t *num_free, int32_t *new_lens,
                               int32_t *query_start, int64_t *slot_mapping, int32_t *num_free_out, int num_seqs,
                               int num_slots, int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                               cudaStream_t stream);
cudaError_t tables_trim_launch(const int32_t *block_tables, const int32_t *context_lens, const int32_t *keep_lens,
                               int32_t *free_blocks, const int32_t *num_free, int32_t *num_free_out, int num_seqs,
                               int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                               cudaStream_t stream);
cudaError_t tree_mask_launch(int32_t *tree_mask, int32_t *depths, const int32_t *parents, const int32_t *query_start,
                             int num_seqs, int num_tokens, int max_query_len, int mask_words, int32_t *status,
                             cudaStream_t stream);
cudaError_t cache_keep_launch(void *k_cache, void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *query_start, const int32_t *accepted, const int32_t *num_accepted,
                              int32_t *new_lens, int num_seqs, int max_accepted, int row_bytes, int block_size,
                              int max_blocks_per_seq, int num_blocks, int32_t *status, cudaStream_t stream);

cudaError_t append_fp8_launch(const void *k, const void *v, void *k_cache, void *v_cache, const int64_t *slot_mapping,
                              const float *k_scale, const float *v_scale, int num_tokens, int num_kv_heads,
                              int head_dim, int block_size, int num_blocks, int32_t *status, cudaStream_t stream);

cudaError_t block_copy_launch(void *k_cache, void *v_cache, const int32_t *src, const int32_t *dst,
                              int num_copies, int block_size, int num_kv_heads, int row_bytes, int num_blocks,
                              int32_t *status, cudaStream_t stream);

cudaError_t validate_launch(const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                            int max_blocks_per_seq, int block_size, int num_blocks, int32_t *status,
                            cudaStream_t stream);

// Launches a kernel whose bounded wait must give up (see selftest.cu).
cudaError_t selftest_bounded_wait_launch(int32_t *status, cudaStream_t stream);

}  // namespace pkv
