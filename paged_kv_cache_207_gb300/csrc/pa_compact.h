// pa_compact.h -- launch interface of the moving of rows within the paged cache.
#pragma once

#include "pa_internal.h"

namespace pa {

struct CompactArgs {
    void* k_pool;
    void* v_pool;
    const int32_t* block_tables;
    const int32_t* dst_tables;   // block_tables again in place
    const int32_t* src_pos;
    const int32_t* dst_start;
    const int32_t* cu_rows;
    int32_t* err;
    int max_blocks, max_dst_blocks, num_seqs, total_rows, num_blocks, num_kv_heads, head_dim;
    bool in_place;
    pa_dtype dtype;              // of the pools
};
cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream);

}  // namespace pa
