// pa_tree.h -- launch interface of the attention of drafted trees over the paged cache.
#pragma once

#include "pa_internal.h"

namespace pa {

struct TreeArgs {
    void* out;
    const void* q;
    const void* k_pool;
    const void* v_pool;
    const int32_t* block_tables;
    const int32_t* start_pos;
    const int32_t* cu_q;
    const int32_t* mask;     // [total_q][mask_words]
    int32_t* err;
    void* workspace;
    int num_seqs, total_q, max_chunk, mask_words;
    int num_q_heads, num_kv_heads, head_dim, max_blocks, num_blocks;
    float scale;
    pa_dtype dtype;          // of the pools
};

// Work is handed out in key tiles, evenly over the CTAs (pa_tree.cuh), so that at most two items
// of a CTA are incomplete: their partial results are what the workspace holds.
constexpr int kTreeCtas = 160;               // CTAs at most of the tensor-core kernel, one per SM,
constexpr int kTreeF32Ctas = 3 * kTreeCtas;  // and of the f32 kernel
constexpr int kTreeF32Rows = 32;             // query rows of an f32 item
constexpr int kTreeJointBytes = 16;          // of what a CTA says of an item that it shares
// Query rows of an item of the tensor-core kernel: one or two tiles of 128.
inline int tree_tile_rows(long long rows) { return rows > 128 ? 256 : 128; }
size_t tree_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim, int max_chunk);

cudaError_t launch_tree_f32(const TreeArgs& a, cudaStream_t stream);
// What a call with a bound of no nodes says of its sequences: PA_DEV_ERR_HINT where there are some, PA_DEV_ERR_BAD_CU.
cudaError_t launch_tree_bound(const int32_t* cu_q, int num_seqs, int total_q, int32_t* err, cudaStream_t stream);
cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream);      // every other type

}  // namespace pa
