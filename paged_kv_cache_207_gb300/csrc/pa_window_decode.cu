// pa_window_decode.cu -- single-token attention over a sliding window of the paged cache
// and a few first tokens that stay visible.
//
// The query of sequence s, at position L - 1 (L = context_lens[s]), attends to positions
// j < L with j >= L - window or j < sinks:
//   out[s][h] = sum_j softmax_j(scale <q[s][h], K[s][j][g]>) V[s][j][g],  g = h / G.
// Only the blocks that hold such positions are read (VisibleBlocks lists them: the sinks'
// blocks, then the window's), so the work does not grow with the context, and a cache may
// free the blocks between; hidden slots of a listed block are masked, whatever they hold.
//
// One warp-level pass over the keys with a running maximum and sum (fp32): each warp takes
// every NW-th listed block through a private ring of shared-memory stages, two bulk copies
// (K and V tile of the (block, kv head)) per stage on its mbarrier.  Scores of 16 tokens x 8
// heads (the kv head's G <= 8 query heads) come from the tensor cores (mma.sync, tokens on M),
// probabilities are transposed in registers and multiplied with V on the tensor cores again;
// the f32 cache uses FMAs, for fp32 accuracy.  The bound is HBM: about G operations per byte.
#include <cuda_bf16.h>

#include <cmath>

#include "pa_ptx.cuh"
#include "pa_rows.cuh"
#include "pa_window.h"

namespace pa {

namespace {

constexpr uint64_t kWaitLimitNs = 200000000ull;   // 200 ms: a real tile copy takes microseconds
constexpr float kLog2e = 1.4426950408889634f;

struct WParams {
    void* out;
    const void* q;
    const char* k_pool;
    const char* v_pool;
    const int32_t* tables;
    const int32_t* lens;
    int32_t* err;
    int Hq, Hkv, G, max_blocks, num_blocks;
    int window, sinks;
    float scale_log2;
};

// Running maxima (log2 units) and this lane's share of the sums of heads 2c, 2c + 1.
struct Running {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
};

// The cache types.  A lane is r = lane / 4, c = lane % 4; it holds the scores of two tokens,
// lo() and hi() of the block, for heads 2c and 2c + 1.  o[mi] accumulates dims 16 mi + r, + 8
// of the same heads.

template <int D>
struct Bf16Cache {
    static constexpr int TILE = kBlockTokens * D * 2;         // bytes of a (block, kv head) tile
    static constexpr int KS = D / 16;
    uint32_t qb[KS][2];                                       // query fragments (B operand)
    int lane, r, c;
    __device__ __forceinline__ Bf16Cache(int lane_) : lane(lane_), r(lane_ >> 2), c(lane_ & 3) {}
    __device__ __forceinline__ int lo() const { return r; }
    __device__ __forceinline__ int hi() const { return r + 8; }
    __device__ __forceinline__ void load_q(const void* q, size_t row0, int G) {
        const uint16_t* qrow = static_cast<const uint16_t*>(q) + (row0 + (r < G ? r : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            qb[kk][0] = r < G ? *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * c) : 0u;
            qb[kk][1] = r < G ? *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 8 + 2 * c) : 0u;
        }
    }
    __device__ __forceinline__ void scores(const uint8_t* kt, float scale, float (&s)[4]) const {
        const uint32_t addr = smem_u32(kt) + lane * 16;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            uint32_t a0, a1, a2, a3;
            ldmatrix_x4(addr + kk * 512, a0, a1, a2, a3);
            mma_bf16_16816(acc, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = acc[i] * scale;
    }
    // Probabilities are rounded to bf16 for the tensor cores, and the sums take the rounded
    // ones, so that a weighted mean of equal values stays exact.
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[4], uint32_t vis, bool, bool,
                                       Running& run, float al0, float al1, bool rescale, float (&o)[KS][4]) {
        const uint32_t x0 = pack_bf16x2(pr[0], pr[1]), x1 = pack_bf16x2(pr[2], pr[3]);
        run.l0 = run.l0 * al0 + (bf16_lo_to_f32(x0) + bf16_lo_to_f32(x1));
        run.l1 = run.l1 * al1 + (bf16_hi_to_f32(x0) + bf16_hi_to_f32(x1));
        const uint32_t pb0 = movmatrix_trans(x0), pb1 = movmatrix_trans(x1);
        // V^T fragments hold tokens 2c, 2c+1 (regs 0, 1) and 2c+8, 2c+9 (regs 2, 3); hidden
        // slots may hold anything (even NaN), so zero them
        uint32_t ma = 0xffffffffu, mb = 0xffffffffu;
        if (vis != 0xffffu) {
            const uint32_t w = vis >> (2 * c);
            ma = ((w & 1u) ? 0x0000ffffu : 0u) | ((w & 2u) ? 0xffff0000u : 0u);
            mb = ((w & 0x100u) ? 0x0000ffffu : 0u) | ((w & 0x200u) ? 0xffff0000u : 0u);
        }
        const int vm = lane >> 3;
        const uint32_t addr = smem_u32(vt) + (uint32_t)(((vm & 1) * 16 + (vm >> 1) * 8 + (lane & 7)) * 16);
#pragma unroll
        for (int mi = 0; mi < KS; ++mi) {
            uint32_t v0, v1, v2, v3;
            ldmatrix_x4_trans(addr + mi * 512, v0, v1, v2, v3);
            v0 &= ma; v1 &= ma; v2 &= mb; v3 &= mb;
            if (rescale) { o[mi][0] *= al0; o[mi][1] *= al1; o[mi][2] *= al0; o[mi][3] *= al1; }
            mma_bf16_16816(o[mi], v0, v1, v2, v3, pb0, pb1);
        }
    }
    __device__ __forceinline__ void finish(Running&, float (&)[KS][4]) {}
};

// E4M3 records: codes become f16 in registers (exact), the products run in f16.
//   K: ldmatrix gives a lane 4 consecutive dims of one token, so the dot product's index is
//   permuted alike in the query; the tokens come in the order lo() = 4 (r / 2) + r % 2,
//   hi() = lo() + 2, which lines the transposed probabilities up with V's 16-token rows.
//   The key's scale multiplies its scores; the value's multiplies its probability, with 2^8
//   to keep the product in f16's normal range (taken out of the sums at the end).
template <int D>
struct Fp8Cache {
    static constexpr int TILE = 16 * D + 64;
    static constexpr int KS = D / 16;
    static constexpr float kPScale = 256.f;
    uint32_t qb[KS][2];
    int lane, r, c;
    __device__ __forceinline__ Fp8Cache(int lane_) : lane(lane_), r(lane_ >> 2), c(lane_ & 3) {}
    __device__ __forceinline__ int lo() const { return 4 * (r >> 1) + (r & 1); }
    __device__ __forceinline__ int hi() const { return lo() + 2; }
    __device__ __forceinline__ void load_q(const void* q, size_t row0, int G) {
        const uint16_t* qrow = static_cast<const uint16_t*>(q) + (row0 + (r < G ? r : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            const uint2 u = r < G ? *reinterpret_cast<const uint2*>(qrow + 16 * kk + 4 * c) : make_uint2(0u, 0u);
            qb[kk][0] = pack_f16x2(bf16_lo_to_f32(u.x), bf16_hi_to_f32(u.x));
            qb[kk][1] = pack_f16x2(bf16_lo_to_f32(u.y), bf16_hi_to_f32(u.y));
        }
    }
    static __device__ __forceinline__ uint32_t half(uint32_t x, int i) {
        return e4m3x2_to_f16x2((uint16_t)(i ? x >> 16 : x & 0xffffu));
    }
    __device__ __forceinline__ void scores(const uint8_t* kt, float scale, float (&s)[4]) const {
        const int km = lane >> 3, kr = lane & 7;
        const int tok = 4 * (kr >> 1) + (kr & 1) + ((km & 1) ? 2 : 0);
        const uint32_t addr = smem_u32(kt) + (uint32_t)(((km >> 1) * kBlockTokens + tok) * 16);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KS; kk += 2) {
            uint32_t x0, x1, x2, x3;
            ldmatrix_x4(addr + kk * 256, x0, x1, x2, x3);
            mma_f16_16816(acc, half(x0, 0), half(x1, 0), half(x0, 1), half(x1, 1), qb[kk][0], qb[kk][1]);
            mma_f16_16816(acc, half(x2, 0), half(x3, 0), half(x2, 1), half(x3, 1), qb[kk + 1][0], qb[kk + 1][1]);
        }
        const float* ks = reinterpret_cast<const float*>(kt + 16 * D);
        const float s0 = ks[lo()] * scale, s1 = ks[hi()] * scale;
        s[0] = acc[0] * s0;
        s[1] = acc[1] * s0;
        s[2] = acc[2] * s1;
        s[3] = acc[3] * s1;
    }
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[4], uint32_t vis, bool ok0, bool ok1,
                                       Running& run, float al0, float al1, bool rescale, float (&o)[KS][4]) {
        run.l0 = run.l0 * al0 + (pr[0] + pr[2]);
        run.l1 = run.l1 * al1 + (pr[1] + pr[3]);
        // hidden slots carry arbitrary scales (even inf): select rather than multiply
        const float* vs = reinterpret_cast<const float*>(vt + 16 * D);
        const float v0 = vs[lo()] * kPScale, v1 = vs[hi()] * kPScale;
        const uint32_t pb0 = movmatrix_trans(pack_f16x2(ok0 ? pr[0] * v0 : 0.f, ok0 ? pr[1] * v0 : 0.f));
        const uint32_t pb1 = movmatrix_trans(pack_f16x2(ok1 ? pr[2] * v1 : 0.f, ok1 ? pr[3] * v1 : 0.f));
        // a V register holds tokens 4c .. 4c+3 of one dim: hidden ones' codes may be NaN
        uint32_t vm = 0xffffffffu;
        if (vis != 0xffffu) {
            const uint32_t w = vis >> (4 * c);
            vm = ((w & 1u) ? 0xffu : 0u) | ((w & 2u) ? 0xff00u : 0u) | ((w & 4u) ? 0xff0000u : 0u) |
                 ((w & 8u) ? 0xff000000u : 0u);
        }
        const uint32_t addr = smem_u32(vt) + lane * 16;
#pragma unroll
        for (int mi = 0; mi < KS; mi += 2) {
            uint32_t y[4];                       // dims 16 mi .. + 7, + 8 .., 16 (mi + 1) .., + 8 ..
            ldmatrix_x4(addr + mi * 256, y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float(&om)[4] = o[mi + x];
                const uint32_t ya = y[2 * x] & vm, yb = y[2 * x + 1] & vm;
                if (rescale) { om[0] *= al0; om[1] *= al1; om[2] *= al0; om[3] *= al1; }
                mma_f16_16816(om, half(ya, 0), half(yb, 0), half(ya, 1), half(yb, 1), pb0, pb1);
            }
        }
    }
    __device__ __forceinline__ void finish(Running& run, float (&)[KS][4]) {
        run.l0 *= kPScale;                       // the products carry the same factor
        run.l1 *= kPScale;
    }
};

// MXFP4 records: codes become f16 in registers (exact).
//   K: the scale varies along the dot product, so each 32-dim block of it is a product of
//   its own, times the token's scale, summed in fp32.
//   V: the scale varies along the tokens, so it multiplies the probabilities: block b's dims
//   take P_b = p 2^(e_b(t) - 127) c_b with c_b = 2^(135 - R_b), R_b the largest scale code of
//   block b so far (raised, and the block's accumulators rescaled, when a tile brings a
//   larger one), so that P_b stays at most 2^8, in f16's range.
template <int D>
struct Fp4Cache {
    static constexpr int TILE = 8 * D + D / 2;
    static constexpr int KS = D / 16;
    static constexpr int NB = D / 32;                         // scale blocks of a row
    uint32_t qb[KS][2];
    int ref[NB];
    float cb[NB];
    uint32_t ref_packed = 0;
    int lane, r, c;
    __device__ __forceinline__ Fp4Cache(int lane_) : lane(lane_), r(lane_ >> 2), c(lane_ & 3) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            ref[b] = 0;
            cb[b] = exp2i(127);
        }
    }
    __device__ __forceinline__ int lo() const { return r; }
    __device__ __forceinline__ int hi() const { return r + 8; }
    __device__ __forceinline__ void load_q(const void* q, size_t row0, int G) {
        const uint16_t* qrow = static_cast<const uint16_t*>(q) + (row0 + (r < G ? r : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            const uint32_t u0 = r < G ? *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * c) : 0u;
            const uint32_t u1 = r < G ? *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 8 + 2 * c) : 0u;
            qb[kk][0] = pack_f16x2(bf16_lo_to_f32(u0), bf16_hi_to_f32(u0));
            qb[kk][1] = pack_f16x2(bf16_lo_to_f32(u1), bf16_hi_to_f32(u1));
        }
    }
    static __device__ __forceinline__ uint32_t scale_bytes(const uint8_t* at) {
        if constexpr (NB == 4) return *reinterpret_cast<const uint32_t*>(at);
        else return *reinterpret_cast<const uint16_t*>(at);
    }
    // scale byte b of w: 2^(code - 127) (the code is the exponent field; code 0 gives 0)
    static __device__ __forceinline__ float scale_value(uint32_t w, int b) {
        return __uint_as_float(((w >> (8 * b)) & 0xffu) << 23);
    }
    __device__ __forceinline__ void scores(const uint8_t* kt, float scale, float (&s)[4]) const {
        uint32_t k0[NB], k1[NB];
#pragma unroll
        for (int w = 0; w < NB; ++w) {
            k0[w] = *reinterpret_cast<const uint32_t*>(kt + r * (D / 2) + c * (D / 8) + 4 * w);
            k1[w] = *reinterpret_cast<const uint32_t*>(kt + (r + 8) * (D / 2) + c * (D / 8) + 4 * w);
        }
        const uint32_t e0 = scale_bytes(kt + 8 * D + r * NB), e1 = scale_bytes(kt + 8 * D + (r + 8) * NB);
        s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t a[4], a8[4];
            e2m1x8_to_f16x2x4(k0[b], a);
            e2m1x8_to_f16x2x4(k1[b], a8);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(acc, a[0], a8[0], a[1], a8[1], qb[2 * b][0], qb[2 * b][1]);
            mma_f16_16816(acc, a[2], a8[2], a[3], a8[3], qb[2 * b + 1][0], qb[2 * b + 1][1]);
            const float f0 = scale_value(e0, b) * scale, f1 = scale_value(e1, b) * scale;
            s[0] = fmaf(acc[0], f0, s[0]);
            s[1] = fmaf(acc[1], f0, s[1]);
            s[2] = fmaf(acc[2], f1, s[2]);
            s[3] = fmaf(acc[3], f1, s[3]);
        }
    }
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[4], uint32_t, bool ok0, bool ok1,
                                       Running& run, float al0, float al1, bool rescale, float (&o)[KS][4]) {
        run.l0 = run.l0 * al0 + (pr[0] + pr[2]);
        run.l1 = run.l1 * al1 + (pr[1] + pr[3]);
        // hidden slots count with scale code 0 (their codes are finite whatever they are)
        const uint32_t e0 = ok0 ? scale_bytes(vt + 8 * D + r * NB) : 0u;
        const uint32_t e1 = ok1 ? scale_bytes(vt + 8 * D + (r + 8) * NB) : 0u;
        uint32_t top = __vmaxu4(e0, e1);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) top = __vmaxu4(top, __shfl_xor_sync(0xffffffffu, top, x));
        if (__vmaxu4(top, ref_packed) != ref_packed) {        // warp-uniform, rare after the first tile
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int eb = (int)((top >> (8 * b)) & 0xffu);
                if (eb > ref[b]) {
                    const float cn = exp2i(min(135 - eb, 127)), f = cn / cb[b];    // a power of two: exact
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        o[2 * b][x] *= f;
                        o[2 * b + 1][x] *= f;
                    }
                    ref[b] = eb;
                    cb[b] = cn;
                }
            }
            ref_packed = __vmaxu4(top, ref_packed);
        }
        if (rescale) {
#pragma unroll
            for (int mi = 0; mi < KS; ++mi) { o[mi][0] *= al0; o[mi][1] *= al1; o[mi][2] *= al0; o[mi][3] *= al1; }
        }
        uint32_t vw[KS];
#pragma unroll
        for (int w = 0; w < KS; ++w) vw[w] = *reinterpret_cast<const uint32_t*>(vt + (r * 4 + c) * (KS * 4) + 4 * w);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float g0 = scale_value(e0, b) * cb[b], g1 = scale_value(e1, b) * cb[b];
            const uint32_t pb0 = movmatrix_trans(pack_f16x2(pr[0] * g0, pr[1] * g0));
            const uint32_t pb1 = movmatrix_trans(pack_f16x2(pr[2] * g1, pr[3] * g1));
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
                uint32_t a[4];
                e2m1x8_to_f16x2x4(vw[2 * b + h2], a);
                mma_f16_16816(o[2 * b + h2], a[0], a[2], a[1], a[3], pb0, pb1);
            }
        }
    }
    __device__ __forceinline__ void finish(Running&, float (&o)[KS][4]) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float f = 1.f / cb[b];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                o[2 * b][x] *= f;
                o[2 * b + 1][x] *= f;
            }
        }
    }
};

// Shared memory: the stage rings (reused at the end by the warps' results: 8 rows of D + 4
// floats each, their maxima and sums), then the barriers.
template <int D, int TILE, int NW, int NST>
struct Layout {
    static constexpr int OS = D + 4;
    static constexpr int RING = NW * NST * 2 * TILE;
    static constexpr int MERGE = NW * 8 * (OS + 2) * 4;
    static constexpr int BAR = ((RING > MERGE ? RING : MERGE) + 15) / 16 * 16;
    static constexpr int BYTES = BAR + NW * NST * 8;
};

// The listed blocks of one sequence as one warp walks them: entry i of this warp is listed
// block first + i * NW, and the table entries are read 32 at a time.
struct BlockWalk {
    const int32_t* trow;
    VisibleBlocks v;
    int first, step, n, lane, page;
    int32_t ent;
    __device__ __forceinline__ void fetch() {
        const int i = page * 32 + lane;
        ent = i < n ? __ldg(trow + v.block(first + i * step)) : -1;
    }
    __device__ __forceinline__ int32_t entry(int i) {          // i in order, the whole warp
        if ((i >> 5) != page) {
            page = i >> 5;
            fetch();
        }
        return __shfl_sync(0xffffffffu, ent, i & 31);
    }
};

struct Row {
    int len, first;          // context length (clamped to the table), oldest window position
    VisibleBlocks v;
};
__device__ __forceinline__ Row row_of(const WParams& p, int s, bool report) {
    Row x;
    x.len = __ldg(p.lens + s);
    const int cap = p.max_blocks * kBlockTokens;
    if (x.len < 0 || x.len > cap) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
        x.len = x.len < 0 ? 0 : cap;
    }
    x.first = x.len > p.window ? x.len - p.window : 0;
    if (x.len > 0) x.v = visible_blocks(x.first, x.len - 1, p.sinks);
    else x.v = VisibleBlocks{0, 0, 0};
    return x;
}

// True when some CTA has already given up on a copy (nothing is written from then on).
__device__ __forceinline__ bool aborted(const int32_t* err) {
    return err && (*reinterpret_cast<const volatile int32_t*>(err) & PA_DEV_ERR_TIMEOUT) != 0;
}

// The warps' partial results (sm_o rows, sm_m, sm_l per warp and head) as one, written to
// `out`.  A CTA in which a copy wait gave up writes NaN: its result is incomplete.
template <int D, int NW, typename Out>
__device__ __forceinline__ void store_merged(const WParams& p, const float* sm_o, const float* sm_m, const float* sm_l,
                                             size_t row0, bool failed) {
    constexpr int OS = D + 4;
    for (int i = threadIdx.x; i < p.G * D; i += NW * 32) {
        const int g = i / D, d = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, sm_m[w * 8 + g]);
        float acc = 0.f, l = 0.f;
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float wt = fast_exp2(sm_m[w * 8 + g] - M);
                acc += wt * sm_o[(w * 8 + g) * OS + d];
                l += wt * sm_l[w * 8 + g];
            }
        }
        const float x = failed ? __int_as_float(0x7fc00000) : l > 0.f ? acc / l : 0.f;
        if constexpr (sizeof(Out) == 2) static_cast<__nv_bfloat16*>(p.out)[(row0 + g) * D + d] = __float2bfloat16_rn(x);
        else static_cast<float*>(p.out)[(row0 + g) * D + d] = x;
    }
}

template <template <int> class Cache, int D, int NW, int NST>
__global__ void __launch_bounds__(NW * 32) window_decode_kernel(const WParams p) {
    using C = Cache<D>;
    using L = Layout<D, C::TILE, NW, NST>;
    constexpr int KS = C::KS, TILE = C::TILE;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.x, s = blockIdx.y;
    uint8_t* stage0 = smem + warp * NST * 2 * TILE;
    const uint32_t bar0 = smem_u32(smem) + L::BAR + warp * NST * 8;
    if (lane == 0) {
#pragma unroll
        for (int st = 0; st < NST; ++st) mbar_init(bar0 + st * 8, 1);
        fence_proxy_async_smem();
    }
    __syncwarp();
    // lengths, tables, queries and pools may all be the previous kernels' output
    grid_dependency_wait();
    grid_launch_dependents();
    if (aborted(p.err)) return;
    const size_t row0 = (size_t)s * p.Hq + (size_t)kvh * p.G;
    C cache(lane);
    cache.load_q(p.q, row0, p.G);
    const Row row = row_of(p, s, kvh == 0 && threadIdx.x == 0);
    BlockWalk walk{p.tables + (size_t)s * p.max_blocks, row.v, warp, NW, 0, lane, 0, -1};
    walk.n = row.v.count > warp ? (row.v.count - warp + NW - 1) / NW : 0;
    walk.fetch();

    const uint64_t pol = l2_policy_evict_first();
    uint32_t issued = 0, phase = 0;
    auto issue = [&](int i) {
        const int st = i % NST;
        const int32_t blk = walk.entry(i);
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
            return;
        }
        if (lane == 0) {
            const size_t off = ((size_t)blk * p.Hkv + kvh) * (size_t)TILE;
            const uint32_t k = smem_u32(stage0) + st * 2 * TILE, bar = bar0 + st * 8;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, 2 * TILE);
            bulk_g2s(k, p.k_pool + off, TILE, bar, pol);
            bulk_g2s(k + TILE, p.v_pool + off, TILE, bar, pol);
        }
        issued |= 1u << st;
    };
    for (int i = 0; i < NST && i < walk.n; ++i) issue(i);

    Running run;
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    bool failed = false;
    for (int i = 0; i < walk.n; ++i) {
        const int st = i % NST;
        if ((issued >> st) & 1u) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + st * 8, (phase >> st) & 1u, kWaitLimitNs))) {
                failed = true;
                break;
            }
            phase ^= 1u << st;
            issued &= ~(1u << st);
            const uint8_t* kt = stage0 + st * 2 * TILE;
            const int tok0 = row.v.block(warp + i * NW) * kBlockTokens;
            const uint32_t vis = visible_slots(tok0, row.len, row.first, p.sinks);
            float sc[4];
            cache.scores(kt, p.scale_log2, sc);
            const bool ok0 = (vis >> cache.lo()) & 1u, ok1 = (vis >> cache.hi()) & 1u;
            // hidden slots may hold anything: select, never multiply
            const float s0 = ok0 ? sc[0] : -INFINITY, s1 = ok0 ? sc[1] : -INFINITY;
            const float s2 = ok1 ? sc[2] : -INFINITY, s3 = ok1 ? sc[3] : -INFINITY;
            float t0 = fmaxf(s0, s2), t1 = fmaxf(s1, s3);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
            }
            const float n0 = fmaxf(run.m0, t0), n1 = fmaxf(run.m1, t1);
            // (a maximum still at -inf, from keys that score -inf, must not give inf - inf)
            const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
            const float al0 = fast_exp2(run.m0 - z0), al1 = fast_exp2(run.m1 - z1);
            run.m0 = n0;
            run.m1 = n1;
            const float pr[4] = {fast_exp2(s0 - z0), fast_exp2(s1 - z1), fast_exp2(s2 - z0), fast_exp2(s3 - z1)};
            const bool rescale = __any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f);
            cache.pv(kt + TILE, pr, vis, ok0, ok1, run, al0, al1, rescale, o);
        }
        __syncwarp();
        if (i + NST < walk.n) issue(i + NST);
    }
    if (failed) {
        // drain every copy still in flight before the shared memory is reused
        if (lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        for (int st = 0; st < NST; ++st)
            if ((issued >> st) & 1u) mbar_wait_bounded(bar0 + st * 8, (phase >> st) & 1u, kWaitLimitNs);
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        run.l0 += __shfl_xor_sync(0xffffffffu, run.l0, x);
        run.l1 += __shfl_xor_sync(0xffffffffu, run.l1, x);
    }
    cache.finish(run, o);
    const bool cta_failed = __syncthreads_or(failed);          // every warp is done with its stages
    float* sm_o = reinterpret_cast<float*>(smem);
    float* sm_m = sm_o + NW * 8 * L::OS;
    float* sm_l = sm_m + NW * 8;
    {
        const int r = lane >> 2, c = lane & 3;
        float* ow = sm_o + warp * 8 * L::OS;
#pragma unroll
        for (int mi = 0; mi < KS; ++mi) {
            const int d = 16 * mi + r;
            ow[(2 * c) * L::OS + d] = o[mi][0];
            ow[(2 * c + 1) * L::OS + d] = o[mi][1];
            ow[(2 * c) * L::OS + d + 8] = o[mi][2];
            ow[(2 * c + 1) * L::OS + d + 8] = o[mi][3];
        }
        if (r == 0) {
            sm_m[warp * 8 + 2 * c] = run.m0;
            sm_m[warp * 8 + 2 * c + 1] = run.m1;
            sm_l[warp * 8 + 2 * c] = run.l0;
            sm_l[warp * 8 + 2 * c + 1] = run.l1;
        }
    }
    __syncthreads();
    store_merged<D, NW, __nv_bfloat16>(p, sm_o, sm_m, sm_l, row0, cta_failed);
}

// The f32 cache: the same walk with fp32 FMAs (no tensor-core product has fp32 accuracy).
// Lane (t, half) takes token t's dot products over half of the dims; the G probabilities of a
// block pass through shared memory, and a lane then owns D / 32 dims of the output.
template <int D, int NW, int NST>
__global__ void __launch_bounds__(NW * 32) window_decode_f32_kernel(const WParams p) {
    constexpr int TILE = kBlockTokens * D * 4;
    using L = Layout<D, TILE, NW, NST>;
    constexpr int NCH = D / 4;          // 16-byte pieces of a row
    constexpr int DPL = D / 32;         // output dims of a lane
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.x, s = blockIdx.y;
    uint8_t* stage0 = smem + warp * NST * 2 * TILE;
    const uint32_t bar0 = smem_u32(smem) + L::BAR + warp * NST * 8;
    float* sq = reinterpret_cast<float*>(smem + L::BYTES);              // [8][D] query rows
    float* sp = sq + 8 * D + warp * 8 * kBlockTokens;                   // [8][16] this warp's probabilities
    if (lane == 0) {
#pragma unroll
        for (int st = 0; st < NST; ++st) mbar_init(bar0 + st * 8, 1);
        fence_proxy_async_smem();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (aborted(p.err)) return;
    const size_t row0 = (size_t)s * p.Hq + (size_t)kvh * p.G;
    const float* qrow = static_cast<const float*>(p.q) + row0 * D;
    for (int i = threadIdx.x; i < 8 * D; i += NW * 32) sq[i] = i < p.G * D ? qrow[i] : 0.f;
    __syncthreads();
    const Row row = row_of(p, s, kvh == 0 && threadIdx.x == 0);
    BlockWalk walk{p.tables + (size_t)s * p.max_blocks, row.v, warp, NW, 0, lane, 0, -1};
    walk.n = row.v.count > warp ? (row.v.count - warp + NW - 1) / NW : 0;
    walk.fetch();
    const uint64_t pol = l2_policy_evict_first();
    uint32_t issued = 0, phase = 0;
    auto issue = [&](int i) {
        const int st = i % NST;
        const int32_t blk = walk.entry(i);
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
            return;
        }
        if (lane == 0) {
            const size_t off = ((size_t)blk * p.Hkv + kvh) * (size_t)TILE;
            const uint32_t k = smem_u32(stage0) + st * 2 * TILE, bar = bar0 + st * 8;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, 2 * TILE);
            bulk_g2s(k, p.k_pool + off, TILE, bar, pol);
            bulk_g2s(k + TILE, p.v_pool + off, TILE, bar, pol);
        }
        issued |= 1u << st;
    };
    for (int i = 0; i < NST && i < walk.n; ++i) issue(i);
    float m[8], l[8], o[8][DPL];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int k = 0; k < DPL; ++k) o[g][k] = 0.f;
    }
    bool failed = false;
    const int t = lane & 15, half = lane >> 4;
    for (int i = 0; i < walk.n; ++i) {
        const int st = i % NST;
        if ((issued >> st) & 1u) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + st * 8, (phase >> st) & 1u, kWaitLimitNs))) {
                failed = true;
                break;
            }
            phase ^= 1u << st;
            issued &= ~(1u << st);
            const float* kt = reinterpret_cast<const float*>(stage0 + st * 2 * TILE);
            const float* vt = kt + TILE / 4;
            const int tok0 = row.v.block(warp + i * NW) * kBlockTokens;
            const uint32_t vis = visible_slots(tok0, row.len, row.first, p.sinks);
            float acc[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) acc[g] = 0.f;
#pragma unroll 4
            for (int ch = half * (NCH / 2); ch < (half + 1) * (NCH / 2); ++ch) {
                const float4 kv = *reinterpret_cast<const float4*>(kt + (ch * kBlockTokens + t) * 4);
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if (g < p.G) {
                        const float4 qv = *reinterpret_cast<const float4*>(sq + g * D + ch * 4);
                        acc[g] = fmaf(qv.x, kv.x, acc[g]);
                        acc[g] = fmaf(qv.y, kv.y, acc[g]);
                        acc[g] = fmaf(qv.z, kv.z, acc[g]);
                        acc[g] = fmaf(qv.w, kv.w, acc[g]);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                if (g < p.G) {
                    float sc = acc[g] + __shfl_xor_sync(0xffffffffu, acc[g], 16);
                    sc = (vis >> t) & 1u ? sc * p.scale_log2 : -INFINITY;
                    float top = sc;
#pragma unroll
                    for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float mn = fmaxf(m[g], top);
                    const float z = mn == -INFINITY ? 0.f : mn;
                    const float al = exp2f(m[g] - z), pr = exp2f(sc - z);
                    float sum = pr;
#pragma unroll
                    for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                    m[g] = mn;
                    l[g] = l[g] * al + sum;
#pragma unroll
                    for (int k = 0; k < DPL; ++k) o[g][k] *= al;
                    if (half == 0) sp[g * kBlockTokens + t] = pr;
                }
            }
            __syncwarp();
            for (int tt = 0; tt < kBlockTokens; ++tt) {
                if (!((vis >> tt) & 1u)) continue;             // (a hidden slot's V may be NaN)
#pragma unroll
                for (int k = 0; k < DPL; ++k) {
                    const int d = lane + 32 * k;
                    const float v = vt[((d >> 2) * kBlockTokens + tt) * 4 + (d & 3)];
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        if (g < p.G) o[g][k] = fmaf(sp[g * kBlockTokens + tt], v, o[g][k]);
                }
            }
        }
        __syncwarp();
        if (i + NST < walk.n) issue(i + NST);
    }
    if (failed) {
        if (lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        for (int st = 0; st < NST; ++st)
            if ((issued >> st) & 1u) mbar_wait_bounded(bar0 + st * 8, (phase >> st) & 1u, kWaitLimitNs);
    }
    const bool cta_failed = __syncthreads_or(failed);
    float* sm_o = reinterpret_cast<float*>(smem);
    float* sm_m = sm_o + NW * 8 * L::OS;
    float* sm_l = sm_m + NW * 8;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
#pragma unroll
        for (int k = 0; k < DPL; ++k) sm_o[(warp * 8 + g) * L::OS + lane + 32 * k] = o[g][k];
        if (lane == g) {
            sm_m[warp * 8 + g] = m[g];
            sm_l[warp * 8 + g] = l[g];
        }
    }
    __syncthreads();
    store_merged<D, NW, float>(p, sm_o, sm_m, sm_l, row0, cta_failed);
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int threads, int smem, cudaStream_t stream, const WParams& p) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <template <int> class Cache, int D, int NST>
cudaError_t launch_mma(const WParams& p, dim3 grid, cudaStream_t stream) {
    constexpr int NW = 4;
    return launch(window_decode_kernel<Cache, D, NW, NST>, grid, NW * 32, Layout<D, Cache<D>::TILE, NW, NST>::BYTES,
                  stream, p);
}

template <int D>
cudaError_t launch_type(const WParams& p, pa_dtype dtype, dim3 grid, cudaStream_t stream) {
    switch (dtype) {
        case PA_BF16: return launch_mma<Bf16Cache, D, 2>(p, grid, stream);
        case PA_FP8_E4M3: return launch_mma<Fp8Cache, D, 2>(p, grid, stream);
        case PA_FP4_E2M1: return launch_mma<Fp4Cache, D, 4>(p, grid, stream);
        case PA_F32: {
            constexpr int NW = 4, NST = 2;
            constexpr int smem = Layout<D, kBlockTokens * D * 4, NW, NST>::BYTES + (8 * D + NW * 8 * kBlockTokens) * 4;
            return launch(window_decode_f32_kernel<D, NW, NST>, grid, NW * 32, smem, stream, p);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_window_decode(const WindowArgs& a, cudaStream_t stream) {
    WParams p;
    p.out = a.out;
    p.q = a.q;
    p.k_pool = static_cast<const char*>(a.k_pool);
    p.v_pool = static_cast<const char*>(a.v_pool);
    p.tables = a.block_tables;
    p.lens = a.context_lens;
    p.err = a.err;
    p.Hq = a.num_q_heads;
    p.Hkv = a.num_kv_heads;
    p.G = a.num_q_heads / a.num_kv_heads;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.window = a.window;
    p.sinks = a.sinks;
    p.scale_log2 = a.scale * kLog2e;
    const dim3 grid(a.num_kv_heads, a.num_seqs);
    return a.head_dim == 64 ? launch_type<64>(p, a.dtype, grid, stream) : launch_type<128>(p, a.dtype, grid, stream);
}

}  // namespace pa
