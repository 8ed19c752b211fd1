// pa_tree.cuh -- how the work of the tree attention is handed out, for its kernels.
//
// An item is (sequence, kv head, row tile): ROWS query rows at most of one kv head, whole tokens,
// against all keys of the sequence, cut into key tiles.  The items, in the order of the sequences,
// then heads, then row tiles, form one line, each item_cost() places (what its beginning and end cost,
// in tiles: 64 sequences of 400 to 7800 tokens, 32 / 8 heads, 32 nodes, 244 us without, 179 with four) and one
// for every tile, and CTA c of C takes the places c T / C .. (c + 1) T / C - 1 of its T: contexts may be as uneven
// as they like, every CTA has the same work, and no lengths are needed on the host.  A CTA's run of
// tiles of one item is a piece.  A piece that
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

// (in tiles of 128 keys on the tensor cores, of 64 on the FMA units)
constexpr int item_cost(int KT) { return KT == 128 ? 4 : 1; }

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
    float* part_o;           // [2 CTAs][D / 4][slot_rows][4]: a thread's row lies beside its neighbours'
    float2* part_ml;         // [2 CTAs][slot_rows]: maximum (log2 units) and sum
    Joint* joints;           // [CTAs]
    int slot_rows;
    int S, total_q, max_chunk, words;
    int Hq, Hkv, G, max_blocks, num_blocks;
    int TQ;                  // tokens of a row tile
    int ctas;                // C, before the number of places
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

// A place in the line.
template <int KT>
struct Cursor {
    static constexpr int COST = item_cost(KT);
    int s, h, rt, at;        // sequence, kv head, row tile, place of the item
    TreeSeq q;
    __device__ __forceinline__ int cost() const { return q.tiles + COST; }
    // the first key tile from a place on
    static __device__ __forceinline__ int tile(int at) { return max(at - COST, 0); }
};

// The line: its places, C, and the first place of CTA c.
struct Line {
    long long total, base;   // base = total / ctas
    uint32_t rest;           // total % ctas
    int ctas;
    // (short lines: a place to a CTA, as many as there are: a tree of 8 nodes after 600 tokens 8.9 us, with
    // three places to a CTA 10.9)
    __device__ __forceinline__ Line(long long places, int limit) {
        total = places;
        ctas = places < 1 ? 1 : places < limit ? (int)places : limit;
        // (a division of 64 bits takes as long as a trip to L2)
        if (places < 1ll << 32) {
            base = (uint32_t)places / (uint32_t)ctas;
            rest = (uint32_t)places % (uint32_t)ctas;
        } else {
            base = places / ctas;
            rest = (uint32_t)(places % ctas);
        }
    }
    __device__ __forceinline__ long long begin(int c) const { return base * c + rest * (uint32_t)c / (uint32_t)ctas; }
};

// The line, and the cursor of place `begin_of(line)` in it where there is one (begin >= 0 and below
// the total), found by all NT threads.  `sm`: NT / 32 + 6 words of 64 bits.
template <int NT, int KT, typename Begin>
__device__ __forceinline__ Line tree_locate(const TParams& p, long long* sm, bool report, Begin begin_of, Cursor<KT>& cur) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto cost = [&](const TreeSeq& q) { return (long long)(q.tiles + item_cost(KT)) * q.rts * p.Hkv; };
    auto scan = [&](long long x) {                        // inclusive, of the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += u;
        }
        return x;
    };
    auto place = [&](long long off) {                     // of the sequence's items
        // (a sequence's heads, row tiles and keys hardly ever pass 2^32)
        const int item = off < 1ll << 32 ? (int)((uint32_t)off / (uint32_t)cur.cost()) : (int)(off / cur.cost());
        cur.at = (int)(off - (long long)item * cur.cost());
        cur.h = item / cur.q.rts;
        cur.rt = item - cur.h * cur.q.rts;
    };
    if (p.S <= 32) {
        // every warp by itself, a lane a sequence (a call's first microseconds: 8.8 us instead of 9.2 for a tree
        // of 8 nodes after 600 tokens)
        TreeSeq one{};
        if (lane < p.S) {
            one = tree_seq<KT>(p, lane);
            if (report && warp == 0 && one.bad) raise_flag(p.err, one.bad);
        }
        const long long mine = lane < p.S ? cost(one) : 0, incl = scan(mine);
        const Line line(__shfl_sync(0xffffffffu, incl, 31), p.ctas);
        const long long begin = begin_of(line), at = incl - mine;
        const uint32_t hit = __ballot_sync(0xffffffffu, begin >= at && begin < incl);
        if (hit) {
            cur.s = __ffs(hit) - 1;
            auto of = [&](int x) { return __shfl_sync(0xffffffffu, x, cur.s); };
            cur.q = TreeSeq{of(one.q0), of(one.n), of(one.start), of(one.tiles), of(one.rts), 0};
            place(begin - __shfl_sync(0xffffffffu, at, cur.s));
        }
        return line;
    }
    const int each = (p.S + NT - 1) / NT, s0 = min(tid * each, p.S), s1 = min(s0 + each, p.S);
    long long mine = 0;
    TreeSeq one{};
    for (int s = s0; s < s1; ++s) {
        one = tree_seq<KT>(p, s);
        if (report && one.bad) raise_flag(p.err, one.bad);
        mine += cost(one);
    }
    const long long incl = scan(mine);
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    const long long sums = scan(lane < NT / 32 ? sm[lane] : 0);
    const Line line(__shfl_sync(0xffffffffu, sums, 31), p.ctas);
    const long long begin = begin_of(line);
    const long long before = __shfl_sync(0xffffffffu, sums, max(warp - 1, 0));
    long long at = (warp > 0 ? before : 0) + incl - mine;
    if (begin >= at && begin < at + mine) {
        int s = s0;
        for (; each > 1; ++s) {
            one = tree_seq<KT>(p, s);
            const long long len = cost(one);
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
    if (begin >= 0 && begin < line.total) {
        const int* from = reinterpret_cast<const int*>(sm + NT / 32 + 1);
        cur.s = from[0];
        cur.q = TreeSeq{from[1], from[2], from[3], from[4], from[5], 0};
        place(sm[NT / 32]);
    }
    return line;
}

// The item after the cursor's (there is one).
template <int KT>
__device__ __forceinline__ void next_item(const TParams& p, Cursor<KT>& c) {
    c.at = 0;
    if (++c.rt < c.q.rts) return;
    c.rt = 0;
    if (++c.h < p.Hkv) return;
    c.h = 0;
    do c.q = tree_seq<KT>(p, ++c.s);
    while (c.q.tiles == 0 && c.s + 1 < p.S);
}

// The rows of an item: its tokens.
template <int KT>
__device__ __forceinline__ int item_tokens(const TParams& p, const Cursor<KT>& c) { return min(c.q.n - c.rt * p.TQ, p.TQ); }

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
template <int KT>
__device__ __forceinline__ void say_joint(const TParams& p, const Line& line, const Cursor<KT>& cur, int c, bool any) {
    Joint x{0, 0, 0, 0};
    const int j = cur.tile(cur.at);
    if (any && j > 0) {
        const long long from = line.begin(c) - cur.at, to = from + cur.cost();
        // (the CTA before has tiles of the item, and is the first that has)
        if (line.begin(c - 1) <= from + item_cost(KT)) {
            // the CTA of the item's last tile: where it would be with even shares, or beside that
            const uint32_t each = line.base > 0 && line.base < 1ll << 31 ? (uint32_t)line.base : line.base > 0 ? 1u << 31 : 1u;
            int last = (int)min((long long)line.ctas - 1, c + (long long)((uint32_t)(cur.cost() - cur.at) / each));
            while (line.begin(last) >= to) --last;
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
// b + 1 tells of, blockIdx.y eight of its rows: a thread four dims of a row, over the parts in their
// order with a running maximum, B parts' loads under way together (which is what registers go to).
constexpr int kMergeRows = 8;
template <int D, typename Out, int B>
__global__ void __launch_bounds__(2 * D, (B == 8 ? 768 : 1536) / (2 * D)) tree_merge_kernel(const TParams p) {
    const int c = blockIdx.x + 1, unit = threadIdx.x / kMergeRows;
    const int r = blockIdx.y * kMergeRows + threadIdx.x % kMergeRows;
    grid_dependency_wait();
    grid_launch_dependents();
    const Joint x = p.joints[c];
    if (r >= x.rows || tree_aborted(p.err)) return;                       // (rows: 0 where nothing is to be joined)
    // part i: piece 2 (c - 1 + i), the first one perhaps the piece after it
    auto slot = [&](int i) { return (size_t)(2 * (c - 1 + i) + (i == 0 ? x.late : 0)); };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < x.count; i0 += B) {
        float2 ml[B];
        float4 v[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            ml[b] = make_float2(-INFINITY, 0.f);
            v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + b < x.count) {
                const size_t at = slot(i0 + b);
                ml[b] = p.part_ml[at * p.slot_rows + r];
                v[b] = reinterpret_cast<const float4*>(p.part_o)[(at * (D / 4) + unit) * p.slot_rows + r];
            }
        }
        float top = m;
#pragma unroll
        for (int b = 0; b < B; ++b) top = (ml[b].x > top || ml[b].x != ml[b].x) ? ml[b].x : top;      // (NaN stays)
        const float z = top == -INFINITY ? 0.f : top, was = fast_exp2(m - z);
        m = top;
        l *= was;
        o = make_float4(o.x * was, o.y * was, o.z * was, o.w * was);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            // (a part without a key that the row sees counts for nothing, whatever its outputs are)
            if (ml[b].y == 0.f) continue;
            const float w = fast_exp2(ml[b].x - z);
            l = __fmaf_rn(w, ml[b].y, l);
            o = make_float4(__fmaf_rn(w, v[b].x, o.x), __fmaf_rn(w, v[b].y, o.y), __fmaf_rn(w, v[b].z, o.z), __fmaf_rn(w, v[b].w, o.w));
        }
    }
    const int tok = r / p.G, g = r - tok * p.G;
    const size_t dst = ((size_t)(uint32_t)x.row0 + (size_t)tok * p.Hq + g) * D + 4 * unit;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    o = inv != 0.f ? make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (sizeof(Out) == 4)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + dst) = o;
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + dst) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
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

template <int D, typename Out>
cudaError_t launch_merge(const TParams& p, cudaStream_t stream) {
    if (p.ctas == 1) return cudaSuccess;
    const dim3 grid(p.ctas - 1, (p.slot_rows + kMergeRows - 1) / kMergeRows);
    // Two parts at a time and six blocks an SM where an item has few parts (at least a third as many items
    // as CTAs), else eight and three: 16 sequences of 2500 tokens, 64 nodes, 53.3 us, with eight 60.0; one of
    // 32768, two kv heads, 8 nodes, 18.9 us, with two 28.3.
    const long long items = (long long)p.S * p.Hkv * ((p.max_chunk + p.TQ - 1) / p.TQ);
    return 3 * items >= p.ctas ? tree_launch(tree_merge_kernel<D, Out, 2>, grid, 2 * D, 0, stream, p)
                               : tree_launch(tree_merge_kernel<D, Out, 8>, grid, 2 * D, 0, stream, p);
}

}  // namespace

}  // namespace pa
