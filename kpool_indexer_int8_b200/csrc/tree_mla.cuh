// tree_mla.cuh -- launchers of the tree attention.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace glm {

constexpr int kTreeMaxNodes = 64;             // one word of visibility bits per node
constexpr int kTreeMaxWidth = 1 << 20;        // index entries of a sequence
constexpr int kTreePairKeys = 96;             // keys of a tile of the two-CTA kernel

struct TreeArgs {
    const uint16_t *q;              // bf16 [batch][n_nodes][n_heads][512]
    const uint8_t *cache;           // rows of the format
    int64_t n_rows;
    const int32_t *rows;            // [batch][width]
    const int32_t *row_len;         // [batch] or null (= width)
    int width;
    const uint8_t *draft;           // rows of the format [batch * n_nodes]
    const uint64_t *mask;           // [batch][n_nodes]
    const int32_t *n_tree;          // [batch] or null (= n_nodes)
    int batch, n_nodes, n_heads;
    float sm_scale;
    uint16_t *out;                  // bf16 [batch][n_nodes][n_heads][512]
    float *lse;                     // [batch][n_nodes][n_heads] or null
    int *status;
    bool give_up;                   // a test: every wait but the last gives up at once
};

// How a call is cut: query rows (node, head) in tiles of `nq` (128: the two-CTA kernel), the keys of
// a sequence in at most `parts` runs; with one part the attention kernel writes the output itself.
// units: SMs (pairs of SMs) that take runs; levels: waves of runs that the kernel may choose from.
struct TreePlan {
    int nq, q_tiles, parts, units, levels;
};
TreePlan tree_plan(int batch, int n_nodes, int n_heads, int width, int num_sms);
// Partials (rows of 512 fp32 + 2) that a call of this shape and every smaller one may need.
size_t tree_partials(int batch, int n_nodes, int n_heads, int width, int num_sms);
cudaError_t launch_tree_mla(const TreePlan &plan, const TreeArgs &a, int format, float *part_acc, float *part_ml,
                            cudaStream_t stream);

// Merges the `parts` partials of each of n_rows = batch * n_nodes * n_heads query rows.
cudaError_t launch_tree_combine(const float *part_acc, const float *part_ml, int n_rows, int n_heads, int parts, int num_sms,
                                uint16_t *out, float *lse, cudaStream_t stream);
cudaError_t launch_tree_pair(const TreePlan &plan, const TreeArgs &a, int format, float *part_acc, float *part_ml,
                             cudaStream_t stream);

}  // namespace glm
