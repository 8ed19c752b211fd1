// pa_compact.cu -- moving rows of a sequence to consecutive positions of the paged cache: the
// accepted path of a drafted tree behind its root, the tokens that an eviction keeps, in place; or
// kept rows into other blocks.
//
// Row i of sequence s goes from position src_pos[cu[s] + i] to dst_start[s] + i, in every kv head of
// both pools, as stored (codes and scales alike).  In place a row's source is not before its
// destination, so no row is written where a later one still has to be read if rows are read in
// order, each before what it is read over by is written: a CTA takes all rows of its share of a (sequence, kv
// head, pool) -- the 16-byte pieces, dims or words that a pool's tile consists of do not mix --
// chunk by chunk, loads the next chunk into registers, waits for all its threads, and stores the one
// before.  Into other blocks nothing is in the way, and the rows too are shared out.
//
// Chunks are whole blocks of the destination, so that a block's bytes that hold several slots (the
// 8- and 4-bit values, transposed in their tiles) have one writer.
#include <algorithm>
#include <cstdint>

#include "pa_compact.h"
#include "pa_flags.cuh"
#include "pa_ptx.cuh"

namespace pa {

namespace {

constexpr int kCompactThreads = 256;
constexpr int kBatchBlocks = 64, kBatchRows = kBatchBlocks * kBlockTokens;   // whose places are looked up together
constexpr int kUnits = 4;                  // 16-byte pieces of a thread under way

struct KParams {
    char* pool[2];
    const int32_t* src_tables;
    const int32_t* dst_tables;
    const int32_t* src_pos;
    const int32_t* dst_start;
    const int32_t* cu;
    int32_t* err;
    int src_blocks, dst_blocks;            // widths of the tables
    int total, num_blocks, Hkv;
    int slices, segs;                      // of a (sequence, kv head, pool): shares of its tiles, of its rows
    bool in_place;
};

struct From { int32_t blk, slot; };        // where a row comes from; blk -1: it does not move

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

// One dim's 16 slots of FP8 values, or the four words of 16 dims mi and r of FP4 values.
struct Mixed { uint32_t w[4]; };

template <pa_dtype T, int D>
__device__ __forceinline__ Mixed load_mixed(const char* rec, int u) {
    Mixed x;
    if constexpr (T == PA_FP8_E4M3) {
        const uint4 v = *reinterpret_cast<const uint4*>(rec + u * 16);
        x.w[0] = v.x; x.w[1] = v.y; x.w[2] = v.z; x.w[3] = v.w;
    } else {
        const int r = u / (D / 16), mi = u % (D / 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) x.w[c] = *reinterpret_cast<const uint32_t*>(rec + ((4 * r + c) * (D / 16) + mi) * 4);
    }
    return x;
}
template <pa_dtype T, int D>
__device__ __forceinline__ void store_mixed(char* rec, int u, const Mixed& x) {
    if constexpr (T == PA_FP8_E4M3) {
        *reinterpret_cast<uint4*>(rec + u * 16) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    } else {
        const int r = u / (D / 16), mi = u % (D / 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint32_t*>(rec + ((4 * r + c) * (D / 16) + mi) * 4) = x.w[c];
    }
}
__device__ __forceinline__ uint32_t pick(const Mixed& x, int i) {
    return i & 2 ? (i & 1 ? x.w[3] : x.w[2]) : (i & 1 ? x.w[1] : x.w[0]);
}
// Slot t of a unit (compile-time t) becomes slot `from` of another.
template <pa_dtype T>
__device__ __forceinline__ void put_slot(Mixed& x, int t, const Mixed& y, int from) {
    if constexpr (T == PA_FP8_E4M3) {
        const uint32_t v = (pick(y, from >> 2) >> (8 * (from & 3))) & 0xffu;
        const int sh = 8 * (t & 3);
        x.w[t >> 2] = (x.w[t >> 2] & ~(0xffu << sh)) | v << sh;
    } else {
        // bytes (dh, half) of word c hold slots 2 c + 8 half, + 1
        const uint32_t v = (pick(y, (from >> 1) & 3) >> (8 * (from >> 3) + 4 * (from & 1))) & 0x000f000fu;
        const int sh = 8 * (t >> 3) + 4 * (t & 1);
        x.w[(t >> 1) & 3] = (x.w[(t >> 1) & 3] & ~(0x000f000fu << sh)) | v << sh;
    }
}

template <pa_dtype T, int D>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const KParams p) {
    using G = Tile<T, D>;
    __shared__ From from[kBatchRows];
    __shared__ int32_t to[kBatchBlocks];
    const int tid = threadIdx.x, s = blockIdx.z, h = blockIdx.y;
    int x = blockIdx.x;
    const int seg = x % p.segs;
    x /= p.segs;
    const int slice = x % p.slices, which = x / p.slices;
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
    char* const pool = p.pool[which];
    const int32_t* strow = p.src_tables + (size_t)s * p.src_blocks;
    const int32_t* dtrow = p.dst_tables + (size_t)s * p.dst_blocks;
    auto tile = [&](int32_t blk) { return pool + ((size_t)blk * p.Hkv + h) * G::BYTES; };
    const bool flags = h == 0 && which == 0 && slice == 0;
    for (int base = b0; base < b1; base += kBatchBlocks) {
        const int blocks = min(kBatchBlocks, b1 - base);
        __syncthreads();                       // (the last batch's reads of the places are done)
        for (int i = tid; i < blocks; i += kCompactThreads) {
            int32_t blk = __ldg(dtrow + first + base + i);
            if (blk < 0 || blk >= p.num_blocks) {
                if (flags) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
                blk = -1;
            }
            to[i] = blk;
        }
        for (int i = tid; i < blocks * kBlockTokens; i += kCompactThreads) {
            const int pos = (first + base) * kBlockTokens + i, row = pos - start;
            From f{-1, 0};
            if (row >= 0 && row < n) {
                const int src = __ldg(p.src_pos + q0 + row);
                if (src < 0 || src >= src_cap || (p.in_place && src < pos)) {
                    if (flags) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
                } else if (!(p.in_place && src == pos)) {
                    f.blk = __ldg(strow + src / kBlockTokens);
                    f.slot = src % kBlockTokens;
                    if (f.blk < 0 || f.blk >= p.num_blocks) {
                        if (flags) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
                        f.blk = -1;
                    }
                }
            }
            from[i] = f;
        }
        __syncthreads();
        // (rows without a destination)
        for (int i = tid; i < blocks * kBlockTokens; i += kCompactThreads)
            if (to[i / kBlockTokens] < 0) from[i].blk = -1;
        __syncthreads();
        if (!G::VALUES_MIX || which == 0) {
            // pieces: lanes on a block's slots, then the slice's pieces, then blocks
            const int per = G::PIECES / p.slices, c0 = slice * per;
            const int units = blocks * per * kBlockTokens, chunk = kUnits * kCompactThreads;
            auto place = [&](int i, int& row, int& c) {
                const int y = i / kBlockTokens;
                c = c0 + y % per;
                row = y / per * kBlockTokens + i % kBlockTokens;
            };
            auto load = [&](int at, uint4 (&v)[kUnits]) {
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    const int i = at + k * kCompactThreads + tid;
                    if (i >= units) continue;
                    int row, c;
                    place(i, row, c);
                    const From f = from[row];
                    if (f.blk >= 0) v[k] = *reinterpret_cast<const uint4*>(tile(f.blk) + G::piece(c, f.slot));
                }
            };
            auto store = [&](int at, const uint4 (&v)[kUnits]) {
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    const int i = at + k * kCompactThreads + tid;
                    if (i >= units) continue;
                    int row, c;
                    place(i, row, c);
                    if (from[row].blk >= 0)
                        *reinterpret_cast<uint4*>(tile(to[row / kBlockTokens]) + G::piece(c, row % kBlockTokens)) = v[k];
                }
            };
            uint4 a[kUnits], b[kUnits];
            load(0, a);
            for (int at = 0; at < units; at += 2 * chunk) {
                load(at + chunk, b);
                __syncthreads();
                store(at, a);
                load(at + 2 * chunk, a);
                __syncthreads();
                store(at + chunk, b);
            }
        } else {
            // units that hold all slots of a block: gathered slot by slot, from few blocks as a rule
            const int per = G::MIXED / p.slices, u0 = slice * per, units = blocks * per;
            for (int at = 0; at < units; at += kCompactThreads) {
                const int i = at + tid, b = i / per, u = u0 + i % per;
                Mixed got{};
                uint32_t moved = 0u;
                if (i < units && to[b] >= 0) {
                    const From* f = from + b * kBlockTokens;
#pragma unroll
                    for (int t = 0; t < kBlockTokens; ++t) moved |= f[t].blk >= 0 ? 1u << t : 0u;
                    if (moved != 0u && moved != 0xffffu) got = load_mixed<T, D>(tile(to[b]), u);
                    Mixed was{};
                    int32_t last = -1;
#pragma unroll
                    for (int t = 0; t < kBlockTokens; ++t) {
                        const From y = f[t];
                        if (y.blk < 0) continue;
                        if (y.blk != last) {
                            was = load_mixed<T, D>(tile(y.blk), u);
                            last = y.blk;
                        }
                        put_slot<T>(got, t, was, y.slot);
                    }
                }
                __syncthreads();
                if (moved != 0u) store_mixed<T, D>(tile(to[b]), u, got);
            }
        }
        if constexpr (G::SCALE > 0) {
            if (slice == 0) {
                uint32_t v[kBatchRows / kCompactThreads];
#pragma unroll
                for (int k = 0; k < kBatchRows / kCompactThreads; ++k) {
                    const int i = k * kCompactThreads + tid;
                    if (i >= blocks * kBlockTokens || from[i].blk < 0) continue;
                    const char* at = tile(from[i].blk) + G::CODES + from[i].slot * G::SCALE;
                    v[k] = G::SCALE == 4 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kBatchRows / kCompactThreads; ++k) {
                    const int i = k * kCompactThreads + tid;
                    if (i >= blocks * kBlockTokens || from[i].blk < 0) continue;
                    char* at = tile(to[i / kBlockTokens]) + G::CODES + i % kBlockTokens * G::SCALE;
                    if constexpr (G::SCALE == 4) *reinterpret_cast<uint32_t*>(at) = v[k];
                    else *reinterpret_cast<uint16_t*>(at) = (uint16_t)v[k];
                }
            }
        }
    }
}

template <pa_dtype T, int D>
cudaError_t launch(KParams p, int num_seqs, cudaStream_t stream) {
    using G = Tile<T, D>;
    int dev = 0, sms = 1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // CTAs for the whole GPU: in place by shares of the tiles, else by shares of the rows
    const long long pairs = 2ll * p.Hkv * num_seqs;
    p.slices = p.segs = 1;
    if (p.in_place) {
        while (2 * p.slices <= std::min(G::PIECES, 8) && pairs * p.slices < 2ll * sms) p.slices *= 2;
    } else {
        const long long blocks = (p.total / num_seqs + kBlockTokens - 1) / kBlockTokens;
        p.segs = (int)std::max(1ll, std::min((blocks + 3) / 4, 8ll * sms / pairs));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.slices * p.segs, p.Hkv, num_seqs);
    cfg.blockDim = dim3(kCompactThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, compact_kernel<T, D>, p);
}

template <int D>
cudaError_t launch_type(const KParams& p, pa_dtype dtype, int num_seqs, cudaStream_t stream) {
    switch (dtype) {
        case PA_F32: return launch<PA_F32, D>(p, num_seqs, stream);
        case PA_BF16: return launch<PA_BF16, D>(p, num_seqs, stream);
        case PA_FP8_E4M3: return launch<PA_FP8_E4M3, D>(p, num_seqs, stream);
        case PA_FP4_E2M1: return launch<PA_FP4_E2M1, D>(p, num_seqs, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
    KParams p;
    p.pool[0] = static_cast<char*>(a.k_pool);
    p.pool[1] = static_cast<char*>(a.v_pool);
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
    p.in_place = a.in_place;
    return a.head_dim == 64 ? launch_type<64>(p, a.dtype, a.num_seqs, stream) : launch_type<128>(p, a.dtype, a.num_seqs, stream);
}

}  // namespace pa
