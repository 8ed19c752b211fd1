// pa_window.h -- launch interfaces of the rotary append and of the sliding-window attention.
#pragma once

#include "pa_internal.h"

namespace pa {

struct RopeArgs {
    void* k_pool;
    void* v_pool;
    void* q_out;             // null (with q): no queries
    const void* q;
    const void* k_new;
    const void* v_new;
    long long q_out_stride, q_stride, k_stride, v_stride;   // elements from row to row
    const double* inv_freq;  // [rotary_dim / 2], radians per position
    const int32_t* positions = nullptr;    // of the form with axes: [num_axes][total_new],
    const int32_t* plane_axis = nullptr;   // [rotary_dim / 2] or null
    int num_axes = 0;
    const int32_t* block_tables;
    const int32_t* start_pos;
    const int32_t* cu_new;
    int32_t* err;
    int rotary_dim;
    bool interleaved;
    int max_blocks, num_seqs, total_new, num_blocks, num_q_heads, num_kv_heads, head_dim;
    pa_dtype dtype;          // of the pools
};
cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_rope_append_axes(const RopeArgs& a, cudaStream_t stream);

// Positions of a sequence that stay visible to a row at position L - 1: the first `sinks`
// and the last `window`.
struct WindowArgs {
    void* out;
    const void* q;
    const void* k_pool;
    const void* v_pool;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* err;
    int num_seqs, num_q_heads, num_kv_heads, head_dim;
    int max_blocks, num_blocks;
    int window, sinks;
    float scale;
    pa_dtype dtype;          // of the pools
};
cudaError_t launch_window_decode(const WindowArgs& a, cudaStream_t stream);

// The prefill of pa_prefill.cu with every row limited to the window and the sinks.
cudaError_t launch_prefill_window(const PrefillArgs& a, int total_q, int window, int sinks, cudaStream_t stream);

// The blocks of a sequence that rows at positions first .. last attend to, as one list: the
// blocks of the sinks, then those from the first row's window on.  `first_visible` is the
// first row's oldest window position, max(0, first - window + 1).
struct VisibleBlocks {
    int sink_blocks;         // leading entries of the list that are blocks 0, 1, ...
    int jump;                // the list's later entries are this many blocks further on
    int count;               // length of the list
    __host__ __device__ int block(int i) const { return i < sink_blocks ? i : i + jump; }
};
__host__ __device__ inline VisibleBlocks visible_blocks(int first_visible, int last, int sinks) {
    VisibleBlocks v;
    // sinks that reach the window hide nothing between them
    const int n = sinks < first_visible ? sinks : first_visible;
    v.sink_blocks = n / kBlockTokens + (n % kBlockTokens != 0 ? 1 : 0);
    const int skip = first_visible / kBlockTokens - v.sink_blocks;
    v.jump = skip > 0 ? skip : 0;
    v.count = last / kBlockTokens + 1 - v.jump;
    return v;
}

// Bit t: slot t of the block whose first position is tok0 holds a position below `len` that
// is one of the sinks or not before `first_visible`.
__host__ __device__ inline uint32_t visible_slots(int tok0, int len, int first_visible, int sinks) {
    const int n = len - tok0, a = first_visible - tok0, b = sinks - tok0;
    const uint32_t live = n >= kBlockTokens ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u;
    const uint32_t near = a <= 0 ? 0xffffu : a >= kBlockTokens ? 0u : 0xffffu << a;
    const uint32_t far = b <= 0 ? 0u : b >= kBlockTokens ? 0xffffu : (1u << b) - 1u;
    return live & (near | far);
}

}  // namespace pa
