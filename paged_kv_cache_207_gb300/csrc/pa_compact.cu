// pa_compact.cu -- moving rows of a sequence to consecutive positions of the paged cache: the
// accepted path of a drafted tree behind its root, the tokens that an eviction keeps, in place; or
// kept rows into other blocks.
//
// Row i of sequence s goes from position src_pos[cu[s] + i] to dst_start[s] + i, in every kv head of
// both pools, as stored (codes and scales alike).  In place a row's source is not before its
// destination, so no row is written where a later one still has to be read if rows are read in
// order, each before what it is read over by is written: a CTA takes all rows of its share of a (sequence, kv
// head, pool) -- the 16-byte pieces, dims or words that a pool's tile consists of do not mix --
// chunk by chunk, loads chunks ahead into registers, waits for all its threads, and stores the first of
// them.  Into other blocks nothing is in the way, and the rows too are shared out.
//
// Chunks are whole blocks of the destination, so that a block's bytes that hold several slots (the
// 8- and 4-bit values, transposed in their tiles) have one writer.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "pa_compact.h"
#include "pa_flags.cuh"
#include "pa_ptx.cuh"

namespace pa {

namespace {

constexpr int kCompactThreads = 256;
constexpr int kBatchBlocks = 64, kBatchRows = kBatchBlocks * kBlockTokens;   // whose places are looked up together
// 16-byte pieces of a thread's chunk, and chunks under way (three and one CTA less: 64 paths of up to 7 rows
// 5.5 us instead of 4.9, 16 windows of 4100 tokens 94.0 instead of 95.9)
constexpr int kUnits = 2, kDepth = 2;
// CTAs of an SM, which bound the registers: 48, or 64 where units of several slots are put together
// (16 windows of 4100 FP8 tokens, 8 heads: 93 us, with five CTAs 110; 64 gathers of bf16 rows, 2 heads: 10.7 with
// five, 11.9 with four).
constexpr int sm_ctas(bool mix) { return mix ? 4 : 5; }

struct KParams {
    char* k_pool;
    char* v_pool;
    const int32_t* src_tables;
    const int32_t* dst_tables;
    const int32_t* src_pos;
    const int32_t* dst_start;
    const int32_t* cu;
    int32_t* err;
    int src_blocks, dst_blocks;            // widths of the tables
    int total, num_blocks, Hkv;
    int slice_bits, segs;                  // of a (sequence, kv head, pool): 2^slice_bits shares of its tiles, shares of its rows
};

// Where a row comes from: its tile's byte offset in the pool (a multiple of 16) and its slot; -1: it does not move.
using From = int64_t;
__device__ __forceinline__ int slot_of(From f) { return (int)f & (kBlockTokens - 1); }

// The geometry of a (block, kv head) tile.
template <pa_dtype T, int D>
struct Tile {
    static constexpr size_t BYTES = T == PA_F32 ? 64 * D : T == PA_BF16 ? 32 * D : T == PA_FP8_E4M3 ? 16 * D + 64 : 8 * D + D / 2;
    static constexpr int CODES = T == PA_FP8_E4M3 ? 16 * D : T == PA_FP4_E2M1 ? 8 * D : (int)BYTES;
    static constexpr int PIECES = CODES / (16 * kBlockTokens);         // 16-byte pieces of a row of keys
    static constexpr int SCALE = T == PA_FP8_E4M3 ? 4 : T == PA_FP4_E2M1 ? D / 32 : 0;   // scale bytes of a row
    static constexpr bool VALUES_MIX = T == PA_FP8_E4M3 || T == PA_FP4_E2M1;
    // units of a tile of values whose slots share bytes: FP8 a dim (16 bytes), FP4 four words
    static constexpr int MIXED = T == PA_FP8_E4M3 ? D : D / 2;
    // byte offset of a row's piece
    static __device__ __forceinline__ uint32_t piece(int c, int slot) {
        return T == PA_FP4_E2M1 ? slot * (D / 2) + c * 16 : (c * kBlockTokens + slot) * 16;
    }
};

// One dim's 16 slots of FP8 values (16 bytes), or the four words of 16 dims mi and r of FP4 values.
struct Mixed { uint32_t w[4]; };

template <pa_dtype T, int D>
__device__ __forceinline__ uint32_t mixed_at(int u, int i) {       // byte offset of word i
    return T == PA_FP8_E4M3 ? u * 16 + i * 4 : ((4 * (u / (D / 16)) + i) * (D / 16) + u % (D / 16)) * 4;
}
template <pa_dtype T, int D>
__device__ __forceinline__ Mixed load_mixed(const char* tile, int u) {
    Mixed x;
    if constexpr (T == PA_FP8_E4M3) {
        const uint4 v = *reinterpret_cast<const uint4*>(tile + u * 16);
        x = Mixed{{v.x, v.y, v.z, v.w}};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.w[i] = *reinterpret_cast<const uint32_t*>(tile + mixed_at<T, D>(u, i));
    }
    return x;
}
template <pa_dtype T, int D>
__device__ __forceinline__ void store_mixed(char* tile, int u, const Mixed& x) {
    if constexpr (T == PA_FP8_E4M3)
        *reinterpret_cast<uint4*>(tile + u * 16) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    else
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(tile + mixed_at<T, D>(u, i)) = x.w[i];
}
// Slot t (compile-time) of x becomes slot `slot` (the same in the warp, as a rule) of y.
template <pa_dtype T>
__device__ __forceinline__ void move_slot(Mixed& x, int t, const Mixed& y, int slot) {
    const int i = T == PA_FP8_E4M3 ? slot >> 2 : (slot >> 1) & 3;
    const uint32_t w = i & 2 ? (i & 1 ? y.w[3] : y.w[2]) : (i & 1 ? y.w[1] : y.w[0]);
    if constexpr (T == PA_FP8_E4M3) {
        const int sh = 4 * (t & 3);
        x.w[t >> 2] = __byte_perm(x.w[t >> 2], w, (0x3210u & ~(0xfu << sh)) | (4u + (slot & 3)) << sh);
    } else {
        // bytes (dh, half) of word c hold slots 2 c + 8 half, + 1: the two dims' nibbles of a slot
        const int sh = 8 * (t >> 3) + 4 * (t & 1);
        const uint32_t v = (w >> (8 * (slot >> 3) + 4 * (slot & 1))) & 0x000f000fu;
        x.w[(t >> 1) & 3] = (x.w[(t >> 1) & 3] & ~(0x000f000fu << sh)) | v << sh;
    }
}
// Units u of a destination's tile from the rows f, and which of its slots move.  A source's tile
// is read as whole units, once for the rows in turn that come from it: rows mostly lie in few blocks.
template <pa_dtype T, int D, int NU>
__device__ __forceinline__ uint32_t gather_mixed(const char* pool, const From* f, const char* dst, const int (&u)[NU], Mixed (&got)[NU]) {
    Mixed have[NU];
    From at = -1;
    uint32_t moved = 0u;
#pragma unroll
    for (int t = 0; t < kBlockTokens; ++t) {
        const From x = f[t];
        if (x < 0) continue;
        if ((x & ~(From)(kBlockTokens - 1)) != at) {
            at = x & ~(From)(kBlockTokens - 1);
#pragma unroll
            for (int k = 0; k < NU; ++k) have[k] = load_mixed<T, D>(pool + at, u[k]);
        }
        moved |= 1u << t;
#pragma unroll
        for (int k = 0; k < NU; ++k) move_slot<T>(got[k], t, have[k], slot_of(x));
    }
    if (moved != 0u && moved != 0xffffu) {
#pragma unroll
        for (int k = 0; k < NU; ++k) have[k] = load_mixed<T, D>(dst, u[k]);
#pragma unroll
        for (int t = 0; t < kBlockTokens; ++t)
            if (!((moved >> t) & 1u)) {
#pragma unroll
                for (int k = 0; k < NU; ++k) move_slot<T>(got[k], t, have[k], t);
            }
    }
    return moved;
}

// FP8: what one source tile gives the units of a destination's, as byte permutations: word w takes
// (x, y, z) of words 0 and 1, of words 2 and 3, and of those two results, under the mask w.
constexpr int kRuns = 2;                  // tiles that a block's rows come from in turn, at most; more go slot by slot
struct Runs {
    uint4 word[kRuns][4];
    From tile[kRuns];
    uint16_t count, moves;                 // how many there are, and the slots that move
};
template <int D, int NU>
__device__ __forceinline__ void gather_runs(const char* pool, const Runs& x, const char* dst, const int (&u)[NU], Mixed (&got)[NU]) {
    constexpr pa_dtype T = PA_FP8_E4M3;
    Mixed have[kRuns][NU];
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
        if (r < x.count) {
            const char* tile = pool + x.tile[r];
#pragma unroll
            for (int k = 0; k < NU; ++k) have[r][k] = load_mixed<T, D>(tile, u[k]);
        }
    if (x.moves != 0xffffu) {
#pragma unroll
        for (int k = 0; k < NU; ++k) got[k] = load_mixed<T, D>(dst, u[k]);
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
        if (r < x.count) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint4 q = x.word[r][w];
#pragma unroll
                for (int k = 0; k < NU; ++k) {
                    const uint32_t* h = have[r][k].w;
                    const uint32_t z = __byte_perm(__byte_perm(h[0], h[1], q.x), __byte_perm(h[2], h[3], q.y), q.z);
                    got[k].w[w] = (got[k].w[w] & ~q.w) | (z & q.w);
                }
            }
        }
}

template <pa_dtype T, int D, bool IN_PLACE>
__global__ void __launch_bounds__(kCompactThreads, sm_ctas(Tile<T, D>::VALUES_MIX)) compact_kernel(const KParams p) {
    using G = Tile<T, D>;
    __shared__ From from[kBatchRows];
    __shared__ int64_t to[kBatchBlocks];      // byte offsets of the destination's tiles, -1: none
    constexpr bool RUNS = IN_PLACE && T == PA_FP8_E4M3;               // (values of FP4 share bytes: slot by slot)
    __shared__ Runs runs[RUNS ? kBatchBlocks : 1];
    __shared__ uint8_t run_of[RUNS ? kBatchRows : 1];                 // of a row
    const int tid = threadIdx.x, s = blockIdx.z, h = blockIdx.y;
    int x = blockIdx.x;
    const int seg = x % p.segs;
    x /= p.segs;
    const int slice = x & ((1 << p.slice_bits) - 1), which = x >> p.slice_bits;
    grid_dependency_wait();
    grid_launch_dependents();
    const bool report = blockIdx.x == 0 && h == 0 && tid == 0;
    const int q0 = __ldg(p.cu + s), q1 = __ldg(p.cu + s + 1), start = __ldg(p.dst_start + s);
    if (q0 < 0 || q1 < q0 || q1 > p.total) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_CU);
        return;
    }
    const int n = q1 - q0;
    const long long cap = (long long)p.dst_blocks * kBlockTokens, src_cap = (long long)p.src_blocks * kBlockTokens;
    if (n == 0) return;
    if (start < 0 || start > cap - n) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
        return;
    }
    // this CTA's blocks of the destination
    const int first = start / kBlockTokens, nblk = (start + n - 1) / kBlockTokens - first + 1;
    const int each = (nblk + p.segs - 1) / p.segs;
    const int b0 = min(seg * each, nblk), b1 = min(b0 + each, nblk);
    char* const pool = which ? p.v_pool : p.k_pool;
    const int32_t* strow = p.src_tables + (size_t)s * p.src_blocks;
    const int32_t* dtrow = p.dst_tables + (size_t)s * p.dst_blocks;
    auto tile = [&](int32_t blk) { return ((int64_t)blk * p.Hkv + h) * (int64_t)G::BYTES; };
    auto source = [&](From f) -> const char* { return pool + (f & ~(int64_t)(kBlockTokens - 1)); };
    const bool flags = h == 0 && which == 0 && slice == 0;
    for (int base = b0; base < b1; base += kBatchBlocks) {
        const int blocks = min(kBatchBlocks, b1 - base);
        // Values of FP8 by whole tiles' permutations where there are blocks to make up for preparing them, in
        // place (16 windows of 4100 tokens, 8 heads: 93 us, slot by slot 141; 64 paths of up to 7 rows
        // 8.5 us, slot by slot 7.9; 24 scattered halves into other blocks 44, slot by slot 36).
        const bool by_runs = RUNS && which == 1 && blocks > 4;
        __syncthreads();                       // (the last batch's reads of the places are done)
        if (tid < blocks) {
            const int32_t blk = __ldg(dtrow + first + base + tid);
            const bool ok = blk >= 0 && blk < p.num_blocks;
            if (!ok && flags) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
            to[tid] = ok ? tile(blk) : -1;
        }
        for (int i = tid; i - tid % 32 < blocks * kBlockTokens; i += kCompactThreads) {      // (whole warps)
            const int pos = (first + base) * kBlockTokens + i, row = pos - start;
            From f = -1;
            if (i < blocks * kBlockTokens && row >= 0 && row < n) {
                const int src = __ldg(p.src_pos + q0 + row);
                if (src < 0 || src >= src_cap || (IN_PLACE && src < pos)) {
                    if (flags) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
                } else if (!(IN_PLACE && src == pos)) {
                    const int32_t blk = __ldg(strow + src / kBlockTokens);
                    if (blk < 0 || blk >= p.num_blocks) {
                        if (flags) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
                    } else {
                        f = tile(blk) | (src % kBlockTokens);
                    }
                }
            }
            if (i < blocks * kBlockTokens) from[i] = f;
            if constexpr (RUNS) {
                if (by_runs) {
                    const int lane = tid % 32, t = i % kBlockTokens, b = i / kBlockTokens;
                    const From tile = f < 0 ? f : f & ~(From)(kBlockTokens - 1), before = __shfl_up_sync(0xffffffffu, tile, 1);
                    const bool starts = f >= 0 && (t == 0 || before != tile);
                    const uint32_t all = __ballot_sync(0xffffffffu, starts) >> (lane & 16) & 0xffffu;
                    const uint32_t moves = __ballot_sync(0xffffffffu, f >= 0) >> (lane & 16) & 0xffffu;
                    const int mine = __popc(all & ((2u << t) - 1u)) - 1;
                    if (b < blocks) {
                        run_of[i] = f < 0 ? 255 : mine;
                        if (starts && mine < kRuns) runs[b].tile[mine] = tile;
                        if (t == 0) {
                            runs[b].count = __popc(all);
                            runs[b].moves = moves;
                        }
                    }
                }
            }
        }
        __syncthreads();
        if constexpr (RUNS) {
            if (by_runs) {
                for (int i = tid; i < blocks * kRuns * 4; i += kCompactThreads) {
                    const int b = i / (kRuns * 4), r = i / 4 % kRuns, w = i % 4;
                    uint4 q = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = b * kBlockTokens + 4 * w + j, slot = slot_of(from[row]);
                        if (run_of[row] != r) continue;
                        (slot < 8 ? q.x : q.y) |= (uint32_t)(slot % 8) << (4 * j);
                        q.z |= (uint32_t)(slot < 8 ? j : 4 + j) << (4 * j);
                        q.w |= 0xffu << (8 * j);
                    }
                    runs[b].word[r][w] = q;
                }
                __syncthreads();
            }
        }
        // (a row moves if it has both places)
        auto moves = [&](int row) { return from[row] >= 0 && to[row / kBlockTokens] >= 0; };
        if (!G::VALUES_MIX || which == 0) {
            // pieces: lanes on a block's slots, then the slice's pieces, then blocks
            constexpr int PIECE_BITS = G::PIECES == 2 ? 1 : G::PIECES == 4 ? 2 : G::PIECES == 8 ? 3 : G::PIECES == 16 ? 4 : 5;
            const int bits = PIECE_BITS - p.slice_bits, c0 = slice << bits;
            const int units = blocks << (bits + 4), chunk = kUnits * kCompactThreads;
            auto row_at = [&](int i) { return (i >> (bits + 4)) * kBlockTokens + i % kBlockTokens; };
            auto piece_at = [&](int i) { return c0 + ((i >> 4) & ((1 << bits) - 1)); };
            auto load = [&](int at, uint4 (&v)[kUnits]) {
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    const int i = at + k * kCompactThreads + tid;
                    v[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (i < units) {
                        const From f = from[row_at(i)];
                        if (f >= 0) v[k] = *reinterpret_cast<const uint4*>(source(f) + G::piece(piece_at(i), slot_of(f)));
                    }
                }
            };
            auto store = [&](int at, const uint4 (&v)[kUnits]) {
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    const int i = at + k * kCompactThreads + tid, row = row_at(i);
                    if (i < units && moves(row))
                        *reinterpret_cast<uint4*>(pool + to[row / kBlockTokens] + G::piece(piece_at(i), row % kBlockTokens)) = v[k];
                }
            };
            uint4 v[kDepth][kUnits];
#pragma unroll
            for (int d = 0; d + 1 < kDepth; ++d) load(d * chunk, v[d]);
            for (int at = 0; at < units; at += kDepth * chunk) {
#pragma unroll
                for (int d = 0; d < kDepth; ++d) {
                    // (chunks past the last: nothing is loaded or stored, the barrier is passed by all)
                    load(at + (d + kDepth - 1) * chunk, v[(d + kDepth - 1) % kDepth]);
                    if (IN_PLACE) __syncthreads();
                    store(at + d * chunk, v[d]);
                }
            }
        } else {
            // units that hold all slots of a block, of a slice's: two to a thread where they are many, four of
            // FP8 into other blocks (the slots' places are found once for all: 24 scattered FP8 halves 36.4 us
            // with four, 42.9 with two, 49.6 with one)
            const int per = G::MIXED >> p.slice_bits;
            auto run = [&](auto number) {
                constexpr int NU = decltype(number)::value;
                const int groups = per / NU, units = blocks * groups;
                for (int at = 0; at < units; at += kCompactThreads) {
                    const int i = at + tid, b = i < units ? i / groups : 0, j = i % groups;
                    int u[NU];
#pragma unroll
                    for (int k = 0; k < NU; ++k) u[k] = slice * per + (NU == 1 ? j : (j / 32 * NU + k) * 32 + j % 32);
                    Mixed got[NU] = {};
                    uint32_t moved = 0u;
                    if (i < units && to[b] >= 0) {
                        bool in_runs = false;
                        if constexpr (RUNS) {
                            if (by_runs && runs[b].count <= kRuns) {
                                in_runs = true;
                                moved = runs[b].moves;
                                if (moved != 0u) gather_runs<D>(pool, runs[b], pool + to[b], u, got);
                            }
                        }
                        if (!in_runs) moved = gather_mixed<T, D>(pool, from + b * kBlockTokens, pool + to[b], u, got);
                    }
                    if (IN_PLACE) __syncthreads();
                    if (moved != 0u) {
#pragma unroll
                        for (int k = 0; k < NU; ++k) store_mixed<T, D>(pool + to[b], u[k], got[k]);
                    }
                }
            };
            constexpr int MOST = !IN_PLACE && T == PA_FP8_E4M3 && D == 128 ? 4 : 2;
            if (per % (32 * MOST) == 0) run(std::integral_constant<int, MOST>{});
            else run(std::integral_constant<int, 1>{});
        }
        if constexpr (G::SCALE > 0) {
            if (slice == 0) {
                uint32_t v[kBatchRows / kCompactThreads];
#pragma unroll
                for (int k = 0; k < kBatchRows / kCompactThreads; ++k) {
                    const int i = k * kCompactThreads + tid;
                    if (i >= blocks * kBlockTokens || from[i] < 0) continue;
                    const char* at = source(from[i]) + G::CODES + slot_of(from[i]) * G::SCALE;
                    v[k] = G::SCALE == 4 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kBatchRows / kCompactThreads; ++k) {
                    const int i = k * kCompactThreads + tid;
                    if (i >= blocks * kBlockTokens || !moves(i)) continue;
                    char* at = pool + to[i / kBlockTokens] + G::CODES + i % kBlockTokens * G::SCALE;
                    if constexpr (G::SCALE == 4) *reinterpret_cast<uint32_t*>(at) = v[k];
                    else *reinterpret_cast<uint16_t*>(at) = (uint16_t)v[k];
                }
            }
        }
    }
}

template <pa_dtype T, int D, bool IN_PLACE>
cudaError_t launch(KParams p, int num_seqs, cudaStream_t stream) {
    using G = Tile<T, D>;
    int dev = 0, sms = 1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // CTAs for the whole GPU: in place by shares of the tiles (one window of 4096 bf16 tokens, 8 heads: 24 us,
    // without shares 86; four paths 3.1 and 5.0), else by shares of the rows, four times what runs at once (24
    // scattered bf16 sequences of up to 4000: 44.1 us, with two or eight times 46.3)
    const long long pairs = 2ll * p.Hkv * num_seqs, room = (long long)sm_ctas(G::VALUES_MIX) * sms;
    p.slice_bits = 0;
    p.segs = 1;
    if (IN_PLACE) {
        while ((2 << p.slice_bits) <= std::min(G::PIECES, 8) && (pairs << p.slice_bits) * 2 <= room) ++p.slice_bits;
    } else {
        const long long blocks = (p.total / num_seqs + kBlockTokens - 1) / kBlockTokens;
        p.segs = (int)std::max(1ll, std::min((blocks + 3) / 4, 4 * room / pairs));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((2 << p.slice_bits) * p.segs, p.Hkv, num_seqs);
    cfg.blockDim = dim3(kCompactThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, compact_kernel<T, D, IN_PLACE>, p);
}

template <int D, bool IN_PLACE>
cudaError_t launch_type(const KParams& p, pa_dtype dtype, int num_seqs, cudaStream_t stream) {
    switch (dtype) {
        case PA_F32: return launch<PA_F32, D, IN_PLACE>(p, num_seqs, stream);
        case PA_BF16: return launch<PA_BF16, D, IN_PLACE>(p, num_seqs, stream);
        case PA_FP8_E4M3: return launch<PA_FP8_E4M3, D, IN_PLACE>(p, num_seqs, stream);
        case PA_FP4_E2M1: return launch<PA_FP4_E2M1, D, IN_PLACE>(p, num_seqs, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
    KParams p;
    p.k_pool = static_cast<char*>(a.k_pool);
    p.v_pool = static_cast<char*>(a.v_pool);
    p.src_tables = a.block_tables;
    p.dst_tables = a.dst_tables;
    p.src_pos = a.src_pos;
    p.dst_start = a.dst_start;
    p.cu = a.cu_rows;
    p.err = a.err;
    p.src_blocks = a.max_blocks;
    p.dst_blocks = a.max_dst_blocks;
    p.total = a.total_rows;
    p.num_blocks = a.num_blocks;
    p.Hkv = a.num_kv_heads;
    if (a.head_dim == 64)
        return a.in_place ? launch_type<64, true>(p, a.dtype, a.num_seqs, stream) : launch_type<64, false>(p, a.dtype, a.num_seqs, stream);
    return a.in_place ? launch_type<128, true>(p, a.dtype, a.num_seqs, stream) : launch_type<128, false>(p, a.dtype, a.num_seqs, stream);
}

}  // namespace pa
