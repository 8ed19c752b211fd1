// pa_tree.cuh -- how the work of the tree attention is handed out, for its kernels.
//
// An item is (sequence, kv head, row tile): ROWS query rows at most of one kv head, whole tokens,
// against all keys of the sequence, cut into key tiles.  The items' key tiles, in the order of the
// sequences, then heads, then row tiles, form one line, and CTA c of C takes the tiles c T / C ..
// (c + 1) T / C - 1 of its T: contexts may be as uneven as they like, every CTA has the same work,
// and no lengths are needed on the host.  A CTA's run of tiles of one item is a piece.  A piece that
// is a whole item gives its outputs; others leave partial results (sums, maxima, unnormalised
// outputs), of which a CTA has two at most, its first and its last piece, and the merge kernel joins
// those of each item in the order of its keys.  Everything is a function of the lengths, so equal
// calls give equal bits.
#pragma once

#include <cuda_bf16.h>

#include "pa_flags.cuh"
#include "pa_ptx.cuh"
#include "pa_tree.h"

namespace pa {

namespace {

constexpr float kTreeLog2e = 1.4426950408889634f;

// What a CTA says of the item that its first tile cuts: the CTAs that have parts of it, from its first
// (the one before) on, and its rows.  count 0: no item, or an earlier CTA says it.
struct Joint {
    int count;               // parts
    int late;                // the first part is its CTA's last piece, not its first
    int row0, rows;          // the row of out, of all heads' rows, of its first one; and its rows
};

static_assert(sizeof(Joint) == kTreeJointBytes, "the workspace's size");

struct TParams {
    void* out;
    const void* q;
    const char* k_pool;
    const char* v_pool;
    const int32_t* tables;
    const int32_t* start_pos;
    const int32_t* cu;
    const int32_t* mask;
    int32_t* err;
    float* part_o;           // [2 CTAs][slot_rows][D]
    float2* part_ml;         // [2 CTAs][slot_rows]: maximum (log2 units) and sum
    Joint* joints;           // [CTAs]
    int slot_rows;
    int S, total_q, max_chunk, words;
    int Hq, Hkv, G, max_blocks, num_blocks;
    int TQ;                  // tokens of a row tile
    int ctas;                // C, before the least number of tiles
    float scale_log2;
};

struct TreeSeq {
    int q0, n, start;        // first row of q, nodes, tokens before them
    int tiles, rts;          // key tiles, row tiles
    int bad;                 // PA_DEV_ERR_ bits; then n is 0
};

template <int KT>
__device__ __forceinline__ TreeSeq tree_seq(const TParams& p, int s) {
    TreeSeq x;
    const int q0 = __ldg(p.cu + s), q1 = __ldg(p.cu + s + 1), start = __ldg(p.start_pos + s);
    const int cap = p.max_blocks * kBlockTokens;
    x.bad = 0;
    x.q0 = q0;
    x.start = start;
    x.n = 0;
    if (q0 < 0 || q0 > q1 || q1 > p.total_q) x.bad = PA_DEV_ERR_BAD_CU;
    else x.n = q1 - q0;
    if (x.n > p.max_chunk) {
        x.bad = PA_DEV_ERR_HINT;
        x.n = p.max_chunk;
    }
    if (x.n > 0 && (start < 0 || start > cap - x.n)) {
        x.bad |= PA_DEV_ERR_BAD_POS;
        x.n = 0;
    }
    x.tiles = x.n > 0 ? (start + x.n + KT - 1) / KT : 0;
    x.rts = (x.n + p.TQ - 1) / p.TQ;
    return x;
}

// A place in the line of tiles.
struct Cursor {
    int s, h, rt, j;         // sequence, kv head, row tile, key tile
    TreeSeq q;
};

// C and the first tile of CTA c.
struct Line {
    long long total;
    int ctas;
    __device__ __forceinline__ long long begin(int c) const { return total / ctas * c + total % ctas * c / ctas; }
};

// The line, and the place of tile `begin_of(line)` in it where there is one (begin >= 0 and below
// the total), found by all NT threads.  `sm`: NT / 32 + 6 words of 64 bits.
template <int NT, int KT, int MIN_TILES, typename Begin>
__device__ __forceinline__ Line tree_locate(const TParams& p, long long* sm, bool report, Begin begin_of, Cursor& cur) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (p.S + NT - 1) / NT, s0 = min(tid * each, p.S), s1 = min(s0 + each, p.S);
    long long mine = 0;
    TreeSeq one{};
    for (int s = s0; s < s1; ++s) {
        one = tree_seq<KT>(p, s);
        if (report && one.bad) raise_flag(p.err, one.bad);
        mine += (long long)one.tiles * one.rts * p.Hkv;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long u = sm[w];
        before += w < warp ? u : 0;
        total += u;
    }
    Line line;
    line.total = total;
    const long long most = (total + MIN_TILES - 1) / MIN_TILES;
    line.ctas = most < 1 ? 1 : most < p.ctas ? (int)most : p.ctas;
    const long long begin = begin_of(line);
    long long at = before + incl - mine;
    if (begin >= at && begin < at + mine) {
        int s = s0;
        for (; each > 1; ++s) {
            one = tree_seq<KT>(p, s);
            const long long len = (long long)one.tiles * one.rts * p.Hkv;
            if (begin < at + len || s + 1 >= s1) break;
            at += len;
        }
        // (with what is known of the sequence: the others need not read it again)
        int* to = reinterpret_cast<int*>(sm + NT / 32 + 1);
        sm[NT / 32] = begin - at;
        to[0] = s;
        to[1] = one.q0;
        to[2] = one.n;
        to[3] = one.start;
        to[4] = one.tiles;
        to[5] = one.rts;
    }
    __syncthreads();
    if (begin >= 0 && begin < total) {
        const int* from = reinterpret_cast<const int*>(sm + NT / 32 + 1);
        cur.s = from[0];
        cur.q = TreeSeq{from[1], from[2], from[3], from[4], from[5], 0};
        const long long off = sm[NT / 32];
        const int item = (int)(off / cur.q.tiles);
        cur.j = (int)(off - (long long)item * cur.q.tiles);
        cur.h = item / cur.q.rts;
        cur.rt = item - cur.h * cur.q.rts;
    }
    return line;
}

// The item after the cursor's (there is one).
template <int KT>
__device__ __forceinline__ void next_item(const TParams& p, Cursor& c) {
    c.j = 0;
    if (++c.rt < c.q.rts) return;
    c.rt = 0;
    if (++c.h < p.Hkv) return;
    c.h = 0;
    do c.q = tree_seq<KT>(p, ++c.s);
    while (c.q.tiles == 0 && c.s + 1 < p.S);
}

// The rows of an item: its tokens.
__device__ __forceinline__ int item_tokens(const TParams& p, const Cursor& c) { return min(c.q.n - c.rt * p.TQ, p.TQ); }

// True when some CTA has already given up on a wait (nothing is written from then on).
__device__ __forceinline__ bool tree_aborted(const int32_t* err) {
    return err && (*reinterpret_cast<const volatile int32_t*>(err) & PA_DEV_ERR_TIMEOUT) != 0;
}

// Fills in what every tree kernel takes.
inline TParams tree_params(const TreeArgs& a, int rows, int ctas) {
    TParams p;
    p.out = a.out;
    p.q = a.q;
    p.k_pool = static_cast<const char*>(a.k_pool);
    p.v_pool = static_cast<const char*>(a.v_pool);
    p.tables = a.block_tables;
    p.start_pos = a.start_pos;
    p.cu = a.cu_q;
    p.mask = a.mask;
    p.err = a.err;
    p.S = a.num_seqs;
    p.total_q = a.total_q;
    p.max_chunk = a.max_chunk;
    p.words = a.mask_words;
    p.Hq = a.num_q_heads;
    p.Hkv = a.num_kv_heads;
    p.G = a.num_q_heads / a.num_kv_heads;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.TQ = rows / p.G;
    const long long used = (long long)p.G * (a.max_chunk < p.TQ ? a.max_chunk : p.TQ);
    p.slot_rows = (int)used;
    p.ctas = ctas;
    p.scale_log2 = a.scale * kTreeLog2e;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)2 * ctas * p.slot_rows * a.head_dim);
    p.joints = reinterpret_cast<Joint*>(p.part_ml + (size_t)2 * ctas * p.slot_rows);
    return p;
}

// What CTA c says of the item that its begin cuts (one thread of it).
__device__ __forceinline__ void say_joint(const TParams& p, const Line& line, const Cursor& cur, int c, bool any) {
    Joint x{0, 0, 0, 0};
    if (any && cur.j > 0) {
        const long long from = line.begin(c) - cur.j, to = from + cur.q.tiles;
        if (line.begin(c - 1) <= from) {
            int last = c;
            while (last + 1 < line.ctas && line.begin(last + 1) < to) ++last;
            x.count = last - c + 2;
            x.late = line.begin(c - 1) < from ? 1 : 0;
            x.row0 = (cur.q.q0 + cur.rt * p.TQ) * p.Hq + cur.h * p.G;
            x.rows = item_tokens(p, cur) * p.G;
        }
    }
    p.joints[c] = x;
}

// Joins the partial results of the items that CTA boundaries cut.  Block b takes the item that CTA
// b + 1 tells of, blockIdx.y eight of its rows, a warp each: the weights of the parts on the lanes,
// then the parts' outputs, eight loads under way together.
constexpr int kMergeThreads = 256;
template <int D, typename Out>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TParams p) {
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
    const int r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);
    grid_dependency_wait();
    grid_launch_dependents();
    const Joint x = p.joints[c];
    if (r >= x.rows || tree_aborted(p.err)) return;                       // (rows: 0 where nothing is to be joined)
    // part i: piece 2 (c - 1 + i), the first one perhaps the piece after it
    auto at = [&](int i) { return (size_t)(2 * (c - 1 + i) + (i == 0 ? x.late : 0)) * p.slot_rows + r; };
    float m = -INFINITY;
    for (int i = lane; i < x.count; i += 32) {
        const float y = p.part_ml[at(i)].x;
        m = (y > m || y != y) ? y : m;                                    // (NaN stays)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, m, o);
        m = (y > m || y != y) ? y : m;
    }
    const float z = m == -INFINITY ? 0.f : m;
    constexpr int N = D / 32, B = 8;
    float l = 0.f, o[N] = {};
    for (int i0 = 0; i0 < x.count; i0 += 32) {
        const float2 ml = i0 + lane < x.count ? p.part_ml[at(i0 + lane)] : make_float2(-INFINITY, 0.f);
        // a part without a key that the row sees counts for nothing, whatever its outputs are
        const float w = ml.y == 0.f ? 0.f : fast_exp2(ml.x - z);
        const uint32_t with = __ballot_sync(0xffffffffu, ml.y != 0.f);
        l = __fmaf_rn(w, ml.y, l);
        const int n = min(32, x.count - i0);
        for (int i = 0; i < n; i += B) {
            float v[B][N];
#pragma unroll
            for (int b = 0; b < B; ++b)
                if (i + b < n) {
                    const float* from = p.part_o + at(i0 + i + b) * D + lane * N;
                    if constexpr (N == 4) {
                        const float4 y = *reinterpret_cast<const float4*>(from);
                        v[b][0] = y.x; v[b][1] = y.y; v[b][2] = y.z; v[b][3] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2*>(from);
                        v[b][0] = y.x; v[b][1] = y.y;
                    }
                }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float wb = __shfl_sync(0xffffffffu, w, (i + b) & 31);
                if (i + b < n && ((with >> (i + b)) & 1u))
#pragma unroll
                    for (int k = 0; k < N; ++k) o[k] = __fmaf_rn(wb, v[b][k], o[k]);
            }
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    const int tok = r / p.G, g = r - tok * p.G;
    const size_t dst = ((size_t)(uint32_t)x.row0 + (size_t)tok * p.Hq + g) * D + lane * N;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = inv != 0.f ? o[k] * inv : 0.f;
    if constexpr (sizeof(Out) == 4) {
        float* to = static_cast<float*>(p.out) + dst;
#pragma unroll
        for (int k = 0; k < N; k += 2) *reinterpret_cast<float2*>(to + k) = make_float2(o[k], o[k + 1]);
    } else {
        uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + dst);
#pragma unroll
        for (int k = 0; k < N; k += 2) to[k / 2] = pack_bf16x2(o[k], o[k + 1]);
    }
}
inline dim3 tree_merge_grid(const TParams& p) {
    return dim3(p.ctas - 1, (p.slot_rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32));
}

inline int tree_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 1;
    return n;
}

// Launches as a programmatic dependent of the previous kernel of the stream.
template <typename K, typename... A>
cudaError_t tree_launch(K kernel, dim3 grid, int threads, int smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

}  // namespace pa
