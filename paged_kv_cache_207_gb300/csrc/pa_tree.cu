// pa_tree.cu -- attention of a tree of drafted tokens over an f32 cache (other types: pa_tree_tc.cu).
//
// Row (i, h) of sequence s, the query of node i and query head h, sees the positions before
// start_pos[s] and those nodes j, at positions start_pos[s] + j, whose bit its mask row sets:
//   out = sum_t softmax_t(scale <q, K[t][g]>) V[t][g] over the visible t,  g = h / G.
//
// One pass over the keys with a running maximum and sum (f32).  A CTA keeps 32 query rows of one kv
// head (tokens x G) in shared memory and goes through key tiles of 64 tokens: scores by register
// tiles of 4 rows x 4 keys, the probabilities through shared memory, outputs by register tiles of
// 4 rows x D / 16 dims, all in packed pairs of fp32 FMAs.
#include <algorithm>
#include <cfloat>

#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {

namespace {

constexpr int kRows = kTreeF32Rows, kKeys = 64, kThreads = 128, kMinTiles = 2;
constexpr int f32_ctas(int D) { return D == 64 ? 3 : 2; }      // of an SM: what shared memory (91 KB at 128) and registers allow

// Packed pairs of fp32: the first in the low 32 bits.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float pair_lo(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float pair_hi(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
struct Quad { uint64_t a, b; };
__device__ __forceinline__ Quad quad_at(const float* p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    return Quad{v.x, v.y};
}

template <int D>
struct F32Layout {
    static constexpr int KS = kKeys + 1;                  // 16-byte pieces from one d4 to the next
    static constexpr int K = 0;                           // [D / 4][KS][4]
    static constexpr int V = K + D / 4 * KS * 16;
    static constexpr int Q = V + D / 4 * KS * 16;         // [D / 4][kRows + 1][4]
    static constexpr int P = Q + D / 4 * (kRows + 1) * 16;   // [kKeys][kRows]
    static constexpr int SM = P + kKeys * kRows * 4;
    static constexpr int BYTES = SM + (kThreads / 32 + 6) * 8;
};

template <int D>
__global__ void __launch_bounds__(kThreads, f32_ctas(D)) tree_f32_kernel(const TParams p) {
    using L = F32Layout<D>;
    constexpr int ND = D / 64;                            // float4 of outputs per row and thread
    constexpr size_t TILE = kBlockTokens * D * 4;
    extern __shared__ __align__(16) uint8_t smem[];
    float* const sK = reinterpret_cast<float*>(smem + L::K);
    float* const sV = reinterpret_cast<float*>(smem + L::V);
    float* const sQ = reinterpret_cast<float*>(smem + L::Q);
    float* const sP = reinterpret_cast<float*>(smem + L::P);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    grid_dependency_wait();
    grid_launch_dependents();
    Cursor<kKeys> cur{};
    const Line line = tree_locate<kThreads, kKeys, kMinTiles>(
        p, reinterpret_cast<long long*>(smem + L::SM), blockIdx.x == 0,
        [&](const Line& l) { return (int)blockIdx.x < l.ctas ? l.begin(blockIdx.x) : l.total; }, cur);
    const bool any = (int)blockIdx.x < line.ctas && line.total > 0;
    if (tid == 0) say_joint(p, line, cur, blockIdx.x, any);
    if (!any || tree_aborted(p.err)) return;
    long long left = line.begin(blockIdx.x + 1) - line.begin(blockIdx.x);
    if (left <= item_cost(kKeys) - cur.at) return;
    for (bool first_piece = true; left > 0; first_piece = false) {
        const int j0 = cur.tile(cur.at), j1 = cur.tile((int)min((long long)cur.cost(), cur.at + left));
        const int tokens = item_tokens(p, cur), rows = tokens * p.G;
        const int qrow = cur.q.q0 + cur.rt * p.TQ, end = cur.q.start + cur.q.n;
        const int32_t* trow = p.tables + (size_t)cur.s * p.max_blocks;
        // the query rows, zeros past the last
        __syncthreads();
        for (int i = tid; i < D / 4 * kRows; i += kThreads) {
            const int d4 = i % (D / 4), r = i / (D / 4), tok = r / p.G, g = r - tok * p.G;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const size_t at = ((size_t)(qrow + tok) * p.Hq + (size_t)cur.h * p.G + g) * D + 4 * d4;
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
            }
            *reinterpret_cast<float4*>(sQ + (d4 * (kRows + 1) + r) * 4) = v;
        }
        float m[4], l[4];
        uint64_t o[4][2 * ND];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int x = 0; x < 2 * ND; ++x) o[r][x] = 0ull;
        }
        // Thread t copies slot t % 16 of blocks t / 16 % 4, pieces from t / 64 on; keys past the last and
        // those of a bad block count as zeros, and no row sees them.  A tile's keys come under the products
        // with the values of the tile before, its values under its scores.
        const int slot = tid & 15, b = (tid >> 4) & 3;
        auto block_of = [&](int j) -> int32_t {
            const int tok = j * kKeys + b * kBlockTokens;
            if (j >= j1 || tok >= end) return -1;
            const int32_t blk = __ldg(trow + tok / kBlockTokens);
            if (blk >= 0 && blk < p.num_blocks) return blk;
            if (slot == 0) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
            return -1;
        };
        auto copy = [&](int j, int32_t blk, const char* pool, float* to) {
            const bool live = blk >= 0 && j * kKeys + b * kBlockTokens + slot < end;
            const char* rec = pool + ((size_t)(live ? blk : 0) * p.Hkv + cur.h) * TILE;
#pragma unroll 8
            for (int d4 = tid >> 6; d4 < D / 4 && j < j1; d4 += 2) {
                float* at = to + (d4 * L::KS + b * 16 + slot) * 4;
                if (live) cp_async_16(smem_u32(at), rec + (d4 * kBlockTokens + slot) * 16);
                else *reinterpret_cast<float4*>(at) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            cp_async_commit();
        };
        int32_t blk = block_of(j0);
        copy(j0, blk, p.k_pool, sK);
        for (int j = j0; j < j1; ++j) {
            const int tok0 = j * kKeys;
            copy(j, blk, p.v_pool, sV);
            blk = block_of(j + 1);
            cp_async_wait<1>();
            __syncthreads();                              // (the keys, and before the first tile the queries)
            // scores of rows 4 ty .. + 3 and keys tx + 16 i, in pairs of dims
            uint64_t s2[4][4] = {};
#pragma unroll 4
            for (int d4 = 0; d4 < D / 4; ++d4) {
                Quad q[4], k[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) q[r] = quad_at(sQ + (d4 * (kRows + 1) + 4 * ty + r) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = quad_at(sK + (d4 * L::KS + tx + 16 * i) * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        fma2(s2[r][i], q[r].a, k[i].a);
                        fma2(s2[r][i], q[r].b, k[i].b);
                    }
            }
            __syncthreads();                              // (the keys are read)
            copy(j + 1, blk, p.k_pool, sK);
            // hidden keys score -inf (a select: they may hold anything)
            float s[4][4], top[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                top[r] = -INFINITY;
                const int row = 4 * ty + r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = tok0 + tx + 16 * i;
                    bool see = key < end;
                    if (key >= cur.q.start && see)
                        see = row < rows && ((uint32_t)__ldg(p.mask + (size_t)(qrow + row / p.G) * p.words + (key - cur.q.start) / 32) >>
                                             ((key - cur.q.start) & 31)) & 1u;
                    s[r][i] = see ? (pair_lo(s2[r][i]) + pair_hi(s2[r][i])) * p.scale_log2 : -INFINITY;
                    top[r] = fmaxf(top[r], s[r][i]);
                }
            }
            float al[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
                const float n = fmaxf(m[r], top[r]), z = n == -INFINITY ? 0.f : n;
                al[r] = fast_exp2(m[r] - z);
                m[r] = n;
                l[r] *= al[r];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[r][i] = fast_exp2(s[r][i] - z);
                    l[r] += s[r][i];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(sP + (tx + 16 * i) * kRows + 4 * ty) = make_float4(s[0][i], s[1][i], s[2][i], s[3][i]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint64_t a2 = pair_of(al[r], al[r]);
#pragma unroll
                for (int x = 0; x < 2 * ND; ++x) o[r][x] = mul2(o[r][x], a2);
            }
            cp_async_wait<1>();
            __syncthreads();                              // (the values)
            // values of the tree's tokens that are no finite numbers must not reach the rows that do
            // not see them (0 times an infinity): such a tile takes a select for each product
            bool odd = false;
            if (tok0 + kKeys > cur.q.start)
                for (int i = tid; i < D / 4 * kKeys; i += kThreads) {
                    const int key = tok0 + i % kKeys;
                    const float4 v = *reinterpret_cast<const float4*>(sV + (i / kKeys * L::KS + i % kKeys) * 4);
                    odd |= key >= cur.q.start && !(fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX && fabsf(v.w) <= FLT_MAX);
                }
            odd = __syncthreads_or(odd);                  // (the probabilities are in place)
#pragma unroll 2
            for (int k = 0; k < kKeys; ++k) {
                const float4 pr = *reinterpret_cast<const float4*>(sP + k * kRows + 4 * ty);
                const float pv[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
                for (int x = 0; x < ND; ++x) {
                    const Quad v = quad_at(sV + ((tx + 16 * x) * L::KS + k) * 4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (odd && pv[r] == 0.f) continue;
                        const uint64_t w = pair_of(pv[r], pv[r]);
                        fma2(o[r][2 * x], w, v.a);
                        fma2(o[r][2 * x + 1], w, v.b);
                    }
                }
            }
            __syncthreads();                              // (the values and the probabilities are read)
        }
        cp_async_wait<0>();
        // the lanes' shares of the sums as one
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
        const bool whole = j0 == 0 && j1 == cur.q.tiles;
        const size_t part = (size_t)(2 * blockIdx.x + (first_piece ? 0 : 1));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 4 * ty + r;
            if (row >= rows) continue;
            const int tok = row / p.G, g = row - tok * p.G;
            const size_t dst = ((size_t)(qrow + tok) * p.Hq + (size_t)cur.h * p.G + g) * D;
            const float inv = l[r] > 0.f || l[r] != l[r] ? 1.f / l[r] : 0.f;
#pragma unroll
            for (int x = 0; x < ND; ++x) {
                const int d = 4 * (tx + 16 * x);
                float4 v = make_float4(pair_lo(o[r][2 * x]), pair_hi(o[r][2 * x]), pair_lo(o[r][2 * x + 1]), pair_hi(o[r][2 * x + 1]));
                if (!whole) {
                    reinterpret_cast<float4*>(p.part_o)[(part * (D / 4) + d / 4) * p.slot_rows + row] = v;
                    continue;
                }
                v = inv != 0.f ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(static_cast<float*>(p.out) + dst + d) = v;
            }
            if (!whole && tx == 0) p.part_ml[part * p.slot_rows + row] = make_float2(m[r], l[r]);
        }
        left -= cur.cost() - cur.at;
        if (left <= item_cost(kKeys)) break;             // (ends before an item's first tile)
        next_item<kKeys>(p, cur);
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

cudaError_t launch_tree_f32(const TreeArgs& a, cudaStream_t stream) {
    return a.head_dim == 64 ? launch_f32<64>(a, stream) : launch_f32<128>(a, stream);
}

}  // namespace pa
