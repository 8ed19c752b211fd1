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
// the total), found by all NT threads.  `sm`: NT / 32 + 4 words of 64 bits.
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
        for (; s < s1 - 1; ++s) {
            if (each > 1) one = tree_seq<KT>(p, s);
            const long long len = (long long)one.tiles * one.rts * p.Hkv;
            if (begin < at + len) break;
            at += len;
        }
        sm[NT / 32] = s;
        sm[NT / 32 + 1] = begin - at;
    }
    __syncthreads();
    if (begin >= 0 && begin < total) {
        cur.s = (int)sm[NT / 32];
        cur.q = tree_seq<KT>(p, cur.s);
        const long long off = sm[NT / 32 + 1];
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
    return p;
}

// Joins the partial results of the items that CTA boundaries cut.  Block b takes the item that
// boundary b lies in, if no earlier boundary does; blockIdx.y a share of its rows.
constexpr int kMergeThreads = 256;
template <int D, int KT, int MIN_TILES, typename Out>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TParams p) {
    __shared__ long long sm[kMergeThreads / 32 + 4];
    const int b = blockIdx.x + 1;
    // (the lengths are no output of the kernel before, which waited for what came before it)
    Cursor cur{};
    const Line line = tree_locate<kMergeThreads, KT, MIN_TILES>(
        p, sm, false, [&](const Line& l) { return b < l.ctas ? l.begin(b) : -1ll; }, cur);
    grid_dependency_wait();
    grid_launch_dependents();
    if (b >= line.ctas || cur.j == 0 || tree_aborted(p.err)) return;
    const long long x = line.begin(b), from = x - cur.j, to = from + cur.q.tiles;
    if (line.begin(b - 1) > from) return;
    int last = b;
    while (last + 1 < line.ctas && line.begin(last + 1) < to) ++last;
    const int first = b - 1, rows = item_tokens(p, cur) * p.G;
    const size_t slot0 = (size_t)(2 * first + (line.begin(first) < from ? 1 : 0));
    // a warp a row: lane l has dims of (D / 32) l
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int N = D / 32;
    for (int r = blockIdx.y * (kMergeThreads / 32) + warp; r < rows; r += gridDim.y * (kMergeThreads / 32)) {
        float m = -INFINITY;
        for (int c = first; c <= last; ++c) {
            const float2 ml = p.part_ml[(c == first ? slot0 : (size_t)2 * c) * p.slot_rows + r];
            m = (ml.x > m || ml.x != ml.x) ? ml.x : m;      // (NaN stays)
        }
        const float z = m == -INFINITY ? 0.f : m;
        float l = 0.f, o[N] = {};
        for (int c = first; c <= last; ++c) {
            const size_t at = (c == first ? slot0 : (size_t)2 * c) * p.slot_rows + r;
            const float2 ml = p.part_ml[at];
            const float w = fast_exp2(ml.x - z);
            if (ml.y == 0.f) continue;               // no key that this row sees (its outputs count for nothing)
            l = __fmaf_rn(w, ml.y, l);
            float v[N];
            if constexpr (N == 4) {
                const float4 y = reinterpret_cast<const float4*>(p.part_o + at * D)[lane];
                v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
            } else {
                const float2 y = reinterpret_cast<const float2*>(p.part_o + at * D)[lane];
                v[0] = y.x; v[1] = y.y;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = __fmaf_rn(w, v[i], o[i]);
        }
        const int tok = r / p.G, g = r - tok * p.G;
        const size_t dst = ((size_t)(cur.q.q0 + cur.rt * p.TQ + tok) * p.Hq + (size_t)cur.h * p.G + g) * D + lane * N;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = inv != 0.f ? o[i] * inv : 0.f;
        if constexpr (sizeof(Out) == 4) {
            float* to4 = static_cast<float*>(p.out) + dst;
#pragma unroll
            for (int i = 0; i < N; i += 2) *reinterpret_cast<float2*>(to4 + i) = make_float2(o[i], o[i + 1]);
        } else {
            uint32_t* to2 = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + dst);
#pragma unroll
            for (int i = 0; i < N; i += 2) to2[i / 2] = pack_bf16x2(o[i], o[i + 1]);
        }
    }
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
