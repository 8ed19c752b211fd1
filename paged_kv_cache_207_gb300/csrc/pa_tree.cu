// pa_tree.cu -- attention of a tree of drafted tokens over an f32 cache (other types: pa_tree_tc.cu).
//
// Row (i, h) of sequence s, the query of node i and query head h, sees the positions before
// start_pos[s] and those nodes j, at positions start_pos[s] + j, whose bit its mask row sets:
//   out = sum_t softmax_t(scale <q, K[t][g]>) V[t][g] over the visible t,  g = h / G.
//
// One pass over the keys with running maxima and sums (f32).  A CTA keeps up to 32 query rows of one kv
// head (tokens x G) in shared memory; a warp takes every fourth block of 16 keys with maxima, sums and
// outputs of its own, which the CTA joins at a piece's end: no barrier between blocks, and each
// warp copies its own, the next block's keys under the products with the values, a block's values under its
// scores.  Scores are register tiles of up to 4 rows by 4 keys, outputs of up to 4 rows by D / 4 dims,
// rows in steps of eight (a piece of 8 rows costs a quarter of one of 32).
//
// Where it is bound: by the FMA units once 32 rows share the keys (32 sequences of 2048 tokens, 32 / 8
// heads of 128, 8 nodes: 238 us, 36 of 74 TFLOP/s; packed pairs of fp32 FMAs, whose six operands come
// from the registers at half the pace, 320 us; four warps on one tile of 64 keys with barriers between, 366),
// else by latency: 8 sequences of 20 to 1000 tokens, 12 heads of 64, up to 21 nodes, 20 us.
#include <algorithm>
#include <cfloat>

#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {

namespace {

constexpr int kRows = kTreeF32Rows, kThreads = 128, kWarps = kThreads / 32, kKeys = kWarps * kBlockTokens;
constexpr int f32_ctas(int D) { return D == 64 ? 3 : 2; }      // of an SM: what registers (168) and shared memory (94 KB) allow

__device__ __forceinline__ float4 quad_at(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void fma4(float4& acc, float a, const float4& b) {
    acc = make_float4(fmaf(a, b.x, acc.x), fmaf(a, b.y, acc.y), fmaf(a, b.z, acc.z), fmaf(a, b.w, acc.w));
}

template <int D>
struct F32Layout {
    static constexpr int KS = kBlockTokens + 1;           // 16-byte pieces from one d4 to the next
    static constexpr int HALF = D / 4 * KS * 16;          // a block's keys or values: [D / 4][KS][4]
    static constexpr int OS = D / 4 + 1;                  // pieces from row to row of a warp's outputs (over its keys and values)
    static_assert(kRows * OS * 16 <= 2 * HALF, "a warp's outputs, where its keys and values were");
    static constexpr int KV = 0;                          // [warp][keys, values]
    static constexpr int Q = KV + kWarps * 2 * HALF;      // [D / 4][kRows][4]
    static constexpr int P = Q + D / 4 * kRows * 16;      // [warp][16 keys][8][4]: rows ty + 8 r
    static constexpr int ML = P + kWarps * kBlockTokens * kRows * 4;   // [warp][kRows]
    static constexpr int SM = ML + kWarps * kRows * 8;
    static constexpr int BYTES = SM + (kWarps + 6) * 8;
};

// One piece: tiles j0 .. j1 - 1 of the cursor's item, by rows ty + 8 r, r < NR.
template <int D, int NR>
__device__ __forceinline__ void tree_f32_piece(const TParams& p, const Cursor<kKeys>& cur, uint8_t* smem, int j0, int j1, bool first_piece) {
    using L = F32Layout<D>;
    constexpr int NX = D / 16;                            // float4 of outputs per row and thread
    constexpr size_t TILE = kBlockTokens * D * 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tx = lane & 3, ty = lane >> 2;
    float* const sK = reinterpret_cast<float*>(smem + L::KV + warp * 2 * L::HALF);
    float* const sV = reinterpret_cast<float*>(smem + L::KV + warp * 2 * L::HALF + L::HALF);
    float* const sQ = reinterpret_cast<float*>(smem + L::Q);
    float* const sP = reinterpret_cast<float*>(smem + L::P) + warp * (kBlockTokens * kRows);
    float2* const sML = reinterpret_cast<float2*>(smem + L::ML);
    const int tokens = item_tokens(p, cur), rows = tokens * p.G;
    const int qrow = cur.q.q0 + cur.rt * p.TQ, end = cur.q.start + cur.q.n;
    const int32_t* trow = p.tables + (size_t)cur.s * p.max_blocks;
    // the warp's block of tile j; -1: past the last key, or no block of the pool (flagged)
    auto block_of = [&](int j) -> int32_t {
        const int tok = j * kKeys + warp * kBlockTokens;
        if (j >= j1 || tok >= end) return -1;
        const int32_t blk = __ldg(trow + tok / kBlockTokens);
        if (blk >= 0 && blk < p.num_blocks) return blk;
        if (lane == 0) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
        return -1;
    };
    // keys past the last and those of a bad block count as zeros, and no row sees the former
    auto copy = [&](int j, int32_t blk, const char* pool, float* to) {
        const int slot = lane & 15, tok = j * kKeys + warp * kBlockTokens;
        const bool live = blk >= 0 && tok + slot < end;
        const char* rec = pool + ((size_t)(live ? blk : 0) * p.Hkv + cur.h) * TILE;
        if (j < j1 && tok < end) {
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
                const int d4 = 2 * u + (lane >> 4);
                float* at = to + (d4 * L::KS + slot) * 4;
                if (live) cp_async_16(smem_u32(at), rec + (d4 * kBlockTokens + slot) * 16);
                else *reinterpret_cast<float4*>(at) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        cp_async_commit();
    };
    __syncthreads();                                      // (the piece before has read its outputs)
    int32_t blk = block_of(j0);
    copy(j0, blk, p.k_pool, sK);
    // the query rows, zeros past the last
    for (int i = tid; i < D / 4 * 8 * NR; i += kThreads) {
        const int d4 = i % (D / 4), r = i / (D / 4), tok = r / p.G, g = r - tok * p.G;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const size_t at = ((size_t)(qrow + tok) * p.Hq + (size_t)cur.h * p.G + g) * D + 4 * d4;
            v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
        }
        *reinterpret_cast<float4*>(sQ + (d4 * kRows + r) * 4) = v;
    }
    __syncthreads();
    const int32_t* mrow[NR];                              // the rows' mask words; null: no row
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = ty + 8 * r;
        mrow[r] = row < rows ? p.mask + (size_t)(qrow + row / p.G) * p.words : nullptr;
    }
    float m[NR], l[NR];
    float4 o[NR][NX];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int x = 0; x < NX; ++x) o[r][x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int j = j0; j < j1; ++j) {
        const int tok0 = j * kKeys + warp * kBlockTokens, node0 = tok0 - cur.q.start, left = end - tok0;
        if (left <= 0) break;                             // (the warp's blocks end)
        copy(j, blk, p.v_pool, sV);
        blk = block_of(j + 1);
        // the keys that a row sees: 16 bits
        uint32_t see[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            see[r] = 0xffffu;
            if (node0 > -kBlockTokens) {
                uint32_t v = 0u;
                if (mrow[r]) {
                    if (node0 < 0) {
                        v = ~(0xffffffffu << -node0) | (uint32_t)__ldg(mrow[r]) << -node0;
                    } else {
                        const uint32_t lo = (uint32_t)__ldg(mrow[r] + node0 / 32);
                        const uint32_t hi = (node0 & 31) > 16 && node0 / 32 + 1 < p.words ? (uint32_t)__ldg(mrow[r] + node0 / 32 + 1) : 0u;
                        v = __funnelshift_r(lo, hi, node0 & 31);
                    }
                }
                see[r] = left < kBlockTokens ? v & ~(0xffffffffu << left) : v;
            }
        }
        cp_async_wait<1>();
        __syncwarp();                                     // (the keys)
        // scores of rows ty + 8 r and keys tx + 4 i
        float s[4][4] = {};
#pragma unroll 4
        for (int d4 = 0; d4 < D / 4; ++d4) {
            float4 q[NR], k[4];
#pragma unroll
            for (int r = 0; r < NR; ++r) q[r] = quad_at(sQ + (d4 * kRows + ty + 8 * r) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = quad_at(sK + (d4 * L::KS + tx + 4 * i) * 4);
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[r][i] = fmaf(q[r].w, k[i].w, fmaf(q[r].z, k[i].z, fmaf(q[r].y, k[i].y, fmaf(q[r].x, k[i].x, s[r][i]))));
        }
        __syncwarp();                                     // (the keys are read)
        copy(j + 1, blk, p.k_pool, sK);
        // hidden keys score -inf (a select: they may hold anything)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[r][i] = (see[r] >> (tx + 4 * i)) & 1u ? s[r][i] * p.scale_log2 : -INFINITY;
                top = fmaxf(top, s[r][i]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float n = fmaxf(m[r], top), z = n == -INFINITY ? 0.f : n;
            const float al = fast_exp2(m[r] - z);
            m[r] = n;
            l[r] *= al;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[r][i] = fast_exp2(s[r][i] - z);
                l[r] += s[r][i];
            }
            if (al != 1.f) {
#pragma unroll
                for (int x = 0; x < NX; ++x) o[r][x] = make_float4(o[r][x].x * al, o[r][x].y * al, o[r][x].z * al, o[r][x].w * al);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(sP + ((tx + 4 * i) * 8 + ty) * 4) = make_float4(s[0][i], s[1][i], s[2][i], s[3][i]);
        cp_async_wait<1>();
        __syncwarp();                                     // (the values, and the probabilities)
        // values of the tree's tokens that are no finite numbers must not reach the rows that do
        // not see them (0 times an infinity): such a block takes a select for each product
        bool odd = false;
        if (node0 > -kBlockTokens) {
            const int slot = lane & 15;
            for (int u = 0; u < D / 8; ++u) {
                const float4 v = *reinterpret_cast<const float4*>(sV + ((2 * u + (lane >> 4)) * L::KS + slot) * 4);
                odd |= !(fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX);
            }
            odd = __any_sync(0xffffffffu, odd && node0 + slot >= 0);
        }
#pragma unroll 4
        for (int k = 0; k < kBlockTokens; ++k) {
            const float4 pr = *reinterpret_cast<const float4*>(sP + (k * 8 + ty) * 4);
            const float pv[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const float4 v = quad_at(sV + ((tx + 4 * x) * L::KS + k) * 4);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    if (odd && pv[r] == 0.f) continue;
                    fma4(o[r][x], pv[r], v);
                }
            }
        }
        __syncwarp();                                     // (the values and the probabilities are read)
    }
    // the warps' rows as one
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = ty + 8 * r;
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (tx == 0) sML[warp * kRows + row] = make_float2(m[r], l[r]);
#pragma unroll
        for (int x = 0; x < NX; ++x)
            *reinterpret_cast<float4*>(sK + (row * L::OS + tx + 4 * x) * 4) = o[r][x];
    }
    __syncthreads();
    const bool whole = j0 == 0 && j1 == cur.q.tiles;
    const size_t part = (size_t)(2 * blockIdx.x + (first_piece ? 0 : 1));
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
        const int d4 = i % (D / 4), row = i / (D / 4), tok = row / p.G, g = row - tok * p.G;
        float top = -INFINITY, sum = 0.f;
        float2 ml[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            ml[w] = sML[w * kRows + row];
            top = fmaxf(top, ml[w].x);
        }
        const float z = top == -INFINITY ? 0.f : top;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(ml[w].x - z);
            if (ml[w].x == -INFINITY && ml[w].y == ml[w].y) continue;      // (sees none of the warp's keys)
            const float4 y = *reinterpret_cast<const float4*>(smem + L::KV + w * 2 * L::HALF + (row * L::OS + d4) * 16);
            sum += ml[w].y * f;
            v = make_float4(v.x + y.x * f, v.y + y.y * f, v.z + y.z * f, v.w + y.w * f);
        }
        if (!whole) {
            reinterpret_cast<float4*>(p.part_o)[(part * (D / 4) + d4) * p.slot_rows + row] = v;
            if (d4 == 0) p.part_ml[part * p.slot_rows + row] = make_float2(top, sum);
            continue;
        }
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        v = inv != 0.f ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
        const size_t dst = ((size_t)(qrow + tok) * p.Hq + (size_t)cur.h * p.G + g) * D + 4 * d4;
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + dst) = v;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, f32_ctas(D)) tree_f32_kernel(const TParams given) {
    using L = F32Layout<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dependency_wait();
    grid_launch_dependents();
    Cursor<kKeys> cur{};
    TParams p = given;
    auto locate = [&](bool report) {
        return tree_locate<kThreads, kKeys>(
            p, reinterpret_cast<long long*>(smem + L::SM), report,
            [&](const Line& l) { return (int)blockIdx.x < l.ctas ? l.begin(blockIdx.x) : l.total; }, cur);
    };
    Line line = locate(blockIdx.x == 0);
    // a line that leaves half of the CTAs without a tile shares out rows too, 16 or 8 to an item: four warps
    // take 4 us for 32 rows of head dim 128 against 64 keys (9 sequences of 600 tokens, 32 rows 20.2 -> 16.3 us, 33 of 40
    // with 64 rows 18.6 -> 14.6; three of 500 with 36, head dim 64, 11.6 -> 12.0)
    if (2 * line.total <= p.ctas && p.TQ * p.G > 8) {
        p.TQ = max(1, (4 * line.total <= p.ctas ? 8 : 16) / p.G);
        __syncthreads();
        line = locate(false);
    }
    const bool any = (int)blockIdx.x < line.ctas && line.total > 0;
    if (threadIdx.x == 0) say_joint(p, line, cur, blockIdx.x, any);
    if (__syncthreads_or(!any || (threadIdx.x == 0 && tree_aborted(p.err)))) return;
    long long left = line.begin(blockIdx.x + 1) - line.begin(blockIdx.x);
    if (left <= item_cost(kKeys) - cur.at) return;
    for (bool first_piece = true; left > 0; first_piece = false) {
        const int j0 = cur.tile(cur.at), j1 = cur.tile((int)min((long long)cur.cost(), cur.at + left));
        switch ((item_tokens(p, cur) * p.G + 7) / 8) {
            case 1: tree_f32_piece<D, 1>(p, cur, smem, j0, j1, first_piece); break;
            case 2: tree_f32_piece<D, 2>(p, cur, smem, j0, j1, first_piece); break;
            case 3: tree_f32_piece<D, 3>(p, cur, smem, j0, j1, first_piece); break;
            default: tree_f32_piece<D, 4>(p, cur, smem, j0, j1, first_piece); break;
        }
        left -= cur.cost() - cur.at;
        if (left <= item_cost(kKeys)) break;             // (ends before an item's first tile)
        next_item<kKeys>(p, cur);
    }
}

__global__ void tree_bound_kernel(const int32_t* cu, int num_seqs, int total_q, int32_t* err) {
    grid_dependency_wait();
    grid_launch_dependents();
    for (int s = threadIdx.x; s < num_seqs; s += blockDim.x) {
        const int q0 = __ldg(cu + s), q1 = __ldg(cu + s + 1);
        if (q0 < 0 || q0 > q1 || q1 > total_q) raise_flag(err, PA_DEV_ERR_BAD_CU);
        else if (q1 > q0) raise_flag(err, PA_DEV_ERR_HINT);
    }
}

template <int D>
cudaError_t launch_f32(const TreeArgs& a, cudaStream_t stream) {
    constexpr int smem = F32Layout<D>::BYTES;
    cudaError_t e = cudaFuncSetAttribute(tree_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(f32_ctas(D) * tree_sms(), kTreeF32Ctas);
    const TParams p = tree_params(a, kRows, ctas);
    e = tree_launch(tree_f32_kernel<D>, dim3(ctas), kThreads, smem, stream, p);
    return e != cudaSuccess ? e : launch_merge<D, float>(p, stream);
}

}  // namespace

size_t tree_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim, int max_chunk) {
    const long long G = num_q_heads / num_kv_heads, rows = G * max_chunk;
    const long long tile = tree_tile_rows(rows) / G * G, tile32 = kTreeF32Rows / G * G;
    const long long tc = 2ll * kTreeCtas * std::min(rows, tile), f32 = 2ll * kTreeF32Ctas * std::min(rows, tile32);
    return (size_t)std::max(tc, f32) * (head_dim + 2) * sizeof(float) + kTreeF32Ctas * kTreeJointBytes;
}

cudaError_t launch_tree_bound(const int32_t* cu_q, int num_seqs, int total_q, int32_t* err, cudaStream_t stream) {
    return tree_launch(tree_bound_kernel, dim3(1), 256, 0, stream, cu_q, num_seqs, total_q, err);
}

cudaError_t launch_tree_f32(const TreeArgs& a, cudaStream_t stream) {
    return a.head_dim == 64 ? launch_f32<64>(a, stream) : launch_f32<128>(a, stream);
}

}  // namespace pa
