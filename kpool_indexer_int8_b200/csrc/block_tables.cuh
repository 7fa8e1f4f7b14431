// block_tables.cuh -- launchers of the block-table build and of the commit of accepted drafts.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace glm {

constexpr int kBtMaxBatch = 8192;   // requests whose offsets fit in shared memory

struct BlockTableArgs {
    const int32_t *len, *n_new, *n_blocks, *pad;   // [batch] (pad or null)
    int batch, block_size;
    int32_t *table;                                // [batch][ld_blocks]
    int64_t ld_blocks;
    const int32_t *free_list, *n_free;             // [free_cap], [1]
    int free_cap, pool_blocks;
    int64_t *slots;                                // [n_cap]
    int32_t *q_seq, *q_pos;
    int64_t n_cap;
    int64_t *slot_map;                             // [batch][ld_slot] or null
    int64_t ld_slot;
    int32_t *len_out, *n_blocks_out, *cu_new, *free_out, *n_free_out;
};
cudaError_t launch_block_tables(const BlockTableArgs &a, cudaStream_t stream, int num_sms);

struct TreeCommitArgs {
    const uint8_t *draft;                          // [batch * n_nodes] rows of row_bytes
    int row_bytes;
    const int32_t *path;                           // [batch][ld_path]
    int batch, n_nodes;
    int64_t ld_path;
    const int64_t *slots;                          // [n_cap]
    const int32_t *q_seq, *q_pos, *cu_new;
    int64_t n_cap;
    uint8_t *cache;
    int64_t n_rows;
    const uint16_t *draft_k, *draft_gate;          // bf16 [batch][n_nodes][128] or null
    uint16_t *k, *gate;                            // bf16 [batch][ld_tokens][128] or null
    int64_t ld_tokens;
};
cudaError_t launch_tree_commit(const TreeCommitArgs &a, cudaStream_t stream, int num_sms);

}  // namespace glm
