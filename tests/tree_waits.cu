// The tree attention on the tensor cores, in a build of its own whose waits give up after a time that is set here.
#define PA_TREE_TEST_WAITS
#include "pa_ptx.cuh"
#include "pa_tc.cuh"
// (a look that does not wait itself; what is in flight when a CTA ends is waited for as ever)
#define mbar_try_wait mbar_test
#include "pa_tree_tc.cu"

extern "C" {

int tree_waits_limit(unsigned long long ns) {
    const uint64_t x = ns;
    return (int)cudaMemcpyToSymbol(pa::kWaitNs, &x, sizeof(x));
}

int tree_waits_call(void* out, const void* q, const void* k_pool, const void* v_pool, const int32_t* tables, int32_t max_blocks,
                    const int32_t* start, const int32_t* cu, const int32_t* mask, int32_t words, int32_t seqs, int32_t total,
                    int32_t max_chunk, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t blocks, float scale, int32_t dtype,
                    void* workspace, int32_t* err, void* stream) {
    pa::TreeArgs a;
    a.out = out;
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.block_tables = tables;
    a.start_pos = start;
    a.cu_q = cu;
    a.mask = mask;
    a.err = err;
    a.workspace = workspace;
    a.num_seqs = seqs;
    a.total_q = total;
    a.max_chunk = max_chunk;
    a.mask_words = words;
    a.num_q_heads = q_heads;
    a.num_kv_heads = kv_heads;
    a.head_dim = head_dim;
    a.max_blocks = max_blocks;
    a.num_blocks = blocks;
    a.scale = scale;
    a.dtype = (pa_dtype)dtype;
    return (int)pa::launch_tree_tc(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
