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
// One warp-level pass over the keys with a running maximum and sum (fp32): the listed blocks
// go to the warps in pairs, through a stage of shared memory of the warp's own that bulk copies
// fill.  Its K half and V half have an mbarrier each: K is refilled as soon as the scores are
// taken, V after the products (more stages gained nothing: the CTAs of an SM hide the copies).  Scores of 32 tokens x 8 heads (the kv head's G <= 8 query
// heads) come from the tensor cores (mma.sync, tokens on M), the probabilities are transposed
// in registers and multiplied with V on the tensor cores again.  Two blocks at a time because
// the chain scores -> maximum -> probabilities -> products is what a warp waits for when few
// CTAs run, and its shuffles and rescaling are shared by the pair.  The bound is HBM: about G
// operations per byte.
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>

#include "pa_flags.cuh"
#include "pa_ptx.cuh"
#include "pa_window.h"

namespace pa {

namespace {

constexpr uint64_t kWaitLimitNs = 200000000ull;   // 200 ms: a real tile copy takes microseconds
constexpr float kLog2e = 1.4426950408889634f;
// Times below are of one call on GB300, inputs in L2 or not as they come in turn.  "A": 32 / 8
// heads of 128, "B": 14 / 2 heads of 64.
//
// Warps of a CTA.  At head_dim 64 a block is half the work and eight warps keep a CTA as short
// as four at 128 (B, window 2048, 128 sequences, eight against four: bf16 23.8 / 25.6 us, FP8
// 20.8 / 26.1, FP4 20.0 / 23.0; one sequence, window 512: bf16 5.3 / 6.7, FP8 6.1 / 7.9).  At 128,
// eight win with many blocks for each and many CTAs (A, window 4096: FP8, 256 sequences, 326 /
// 333; bf16, 16 sequences, 41.6 / 45.6) and lose elsewhere (window 1024: one sequence, bf16 8.8 /
// 7.2, FP8 9.7 / 7.8, bf16, 32 of them 26.1 / 23.3; FP4, window 2047, 128 sequences, 90.5 / 81.0).
constexpr int warps_for(pa_dtype t, int head_dim) { return head_dim == 64 && t != PA_F32 ? 8 : 4; }
// CTAs that an SM is to hold, which bounds the registers: as many as shared memory allows for
// bf16 and f32 (A, f32, window 4096, 12 sequences: 92 us with 255 registers, one CTA, against
// 137 with 168), four of FP8 and FP4, whose conversions want the warps more than the registers
// (four against three: FP8, 64 sequences of window 1024, 25.6 / 35.7 us, a mixed batch of 64 25.0 /
// 29.7, but of 96 43.6 / 38.8; FP4 with 128 sequences 81.7 / 91.6).
constexpr int ctas_for(pa_dtype t, int head_dim) {
    return t == PA_F32 ? (head_dim == 64 ? 3 : 1) : head_dim == 64 ? 2 : t == PA_BF16 ? 3 : 4;
}
// Blocks of a part, at least.  A part's end costs a warp about as much as a block or two (FP4:
// two to four, with its scale references to set again), so longer parts are cheaper where one
// CTA goes through all of them and shorter ones faster where CTAs share them (16 / 32 blocks, A,
// window 1024, one sequence: bf16 7.2 / 10.7 us, FP8 7.8 / 10.7, f32 12.2 / 17.4; 64 sequences,
// FP8: 25.6 / 24.8; B, window 2048, FP8, 24 sequences 14.2 / 11.9.  FP4, 32 / 64 blocks: window 2048, one sequence, 11.4 / 17.6, 128 of them
// 81.0 / 77.1).
constexpr int min_part(pa_dtype t) { return t == PA_FP4_E2M1 ? 32 : 16; }
// Pairs of blocks for each warp below which a sequence is one part, since joining parts costs
// about 1 us (4 against 5 and 6: A, bf16, window 512, one sequence 7.3 / 7.6, 16 sequences 10.3 /
// 8.2; window 700, one sequence 7.5 / 7.5 / 8.8; f32, window 512, one sequence 12.5 / 15.7).
constexpr int min_pairs(pa_dtype t) { return t == PA_F32 ? 4 : 5; }
// Whether clusters are to leave an SM to each CTA: one of eight warps fills it (B, window 2048, 24
// sequences, an SM each against as many as fit: bf16 13.0 / 14.7 us, FP8 14.2 / 15.5; 32 / 8 heads
// of 64, window 4096, bf16, 16 sequences, 25.1 / 29.2; but FP4, window 8192, 48 sequences of B, 46.7
// / 38.4).
constexpr bool one_each(pa_dtype t, int head_dim) { return head_dim == 64 && (t == PA_BF16 || t == PA_FP8_E4M3); }
// Parts, at most.  Clusters of up to 8 find room in every part of the GPU; 16 pay only where an
// SM holds three CTAs that are long (16 against 8: f32, 12 heads of 64, window 4096, one
// sequence 13.6 / 14.3 us; A, window 4096, 8 sequences: bf16 27.8 / 25.5, f32 56.0 / 52.4;
// FP8, 16 sequences, 37.4 / 29.7).
constexpr int most_parts(pa_dtype t, int head_dim) { return t == PA_F32 && head_dim == 64 ? 16 : 8; }

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
    int parts, part_len;     // at most so many, of so many listed blocks (the last takes what is left too)
    int per;                 // parts of a cluster's CTA, each kept by itself; 0: a CTA alone folds all parts
    float scale_log2;
};

struct Row {
    int len, first;          // context length (clamped to the table), oldest window position
    VisibleBlocks v;
};

// Running maxima (log2 units) and this lane's share of the sums of heads 2c, 2c + 1, and the
// factors that the last pair's maxima put on what was summed before.
struct Running {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float al0 = 1.f, al1 = 1.f;
    bool rescale = false;        // any lane's factor is not 1
};

template <int KS>
__device__ __forceinline__ void rescale_rows(const Running& run, float (&o)[KS][4]) {
#pragma unroll
    for (int mi = 0; mi < KS; ++mi) {
        o[mi][0] *= run.al0; o[mi][1] *= run.al1; o[mi][2] *= run.al0; o[mi][3] *= run.al1;
    }
}

// The cache types.  A lane is r = lane / 4, c = lane % 4; of each block it holds the scores of
// two tokens, lo() and hi(), for heads 2c and 2c + 1: s[0..1] and s[2..3].  o[mi] accumulates
// dims 16 mi + r, + 8 of the same heads.  finish() gives the factor that is left on o.

template <int D>
struct Bf16Cache {
    static constexpr pa_dtype TYPE = PA_BF16;
    using Out = __nv_bfloat16;
    static constexpr int TILE = kBlockTokens * D * 2;         // bytes of a (block, kv head) tile
    static constexpr int KS = D / 16;
    static constexpr int SCRATCH = 0;
    uint32_t qb[KS][2];                                       // query fragments (B operand)
    int lane, r, c;
    __device__ __forceinline__ Bf16Cache(int lane_, float*) : lane(lane_), r(lane_ >> 2), c(lane_ & 3) {}
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
    __device__ __forceinline__ void set_q(float) {}
    __device__ __forceinline__ void scores(const uint8_t* kt, const WParams& p, float (&s)[2][4]) const {
        const uint32_t addr = smem_u32(kt) + lane * 16;
        float acc[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t a0, a1, a2, a3;
                ldmatrix_x4(addr + b * TILE + kk * 512, a0, a1, a2, a3);
                mma_bf16_16816(acc[b], a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
            }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][i] = acc[b][i] * p.scale_log2;
    }
    // Hidden slots of a V tile may hold anything (even NaN): zero them, 16-byte pieces of 16 slots.
    __device__ __forceinline__ void hide(uint8_t* vt, uint32_t vis) const {
        for (int i = lane; i < TILE / 16; i += 32)
            if (!((vis >> (i % kBlockTokens)) & 1u)) *reinterpret_cast<uint4*>(vt + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    // Probabilities are rounded to bf16 for the tensor cores, whose factors have one type (f16
    // would need every value converted and scaled), and the sums take the rounded ones, so that
    // a weighted mean of equal values stays exact.
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[2][4], Running& run,
                                       float (&o)[KS][4]) {
        uint32_t pb[2][2];
        run.l0 *= run.al0;
        run.l1 *= run.al1;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t x0 = pack_bf16x2(pr[b][0], pr[b][1]), x1 = pack_bf16x2(pr[b][2], pr[b][3]);
            run.l0 += bf16_lo_to_f32(x0) + bf16_lo_to_f32(x1);
            run.l1 += bf16_hi_to_f32(x0) + bf16_hi_to_f32(x1);
            pb[b][0] = movmatrix_trans(x0);
            pb[b][1] = movmatrix_trans(x1);
        }
        if (run.rescale) rescale_rows(run, o);
        const int vm = lane >> 3;
        const uint32_t addr = smem_u32(vt) + (uint32_t)(((vm & 1) * 16 + (vm >> 1) * 8 + (lane & 7)) * 16);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int mi = 0; mi < KS; ++mi) {
                uint32_t v0, v1, v2, v3;
                ldmatrix_x4_trans(addr + b * TILE + mi * 512, v0, v1, v2, v3);
                mma_bf16_16816(o[mi], v0, v1, v2, v3, pb[b][0], pb[b][1]);
            }
        }
    }
    __device__ __forceinline__ void reset() {}
    __device__ __forceinline__ float finish(float (&)[KS][4]) const { return 1.f; }
};

// Query rows of the 8- and 4-bit caches, bf16 in q and f16 for the tensor cores: each row times
// the power of two that takes its largest magnitude to 2^4 .. 2^5, which the row's scores give
// back.  So no element overflows f16, and one loses bits only where it is 2^18 below its row's
// largest: at most 2^-29 of that, less than the sum's fp32.  (Not higher: FP4's sums over a scale
// block are multiplied with scales of up to 2^114 before the row's power of two.)  `qb`: the
// fragments, bf16 on entry; s0, s1: what the scores of heads 2c and 2c + 1 are multiplied with.
template <int KS>
__device__ __forceinline__ void rows_to_f16(uint32_t (&qb)[KS][2], float scale, int c, float& s0, float& s1) {
    uint32_t top = 0u;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) top = __vmaxu2(top, __vmaxu2(qb[kk][0] & 0x7fff7fffu, qb[kk][1] & 0x7fff7fffu));
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int shift = min(131 - (int)(top >> 7), 110);        // (2^110 makes bf16's smallest an f16)
    const float f = exp2i(shift), back = scale * exp2i(-shift);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i) qb[kk][i] = pack_f16x2(bf16_lo_to_f32(qb[kk][i]) * f, bf16_hi_to_f32(qb[kk][i]) * f);
    s0 = __shfl_sync(0xffffffffu, back, 8 * c);
    s1 = __shfl_sync(0xffffffffu, back, 8 * c + 4);
}

// E4M3 records: codes become f16 in registers (exact), the products run in f16.
//   K: ldmatrix gives a lane 4 consecutive dims of one token, so the dot product's index is
//   permuted alike in the query; the tokens come in the order lo() = 4 (r / 2) + r % 2,
//   hi() = lo() + 2, which lines the transposed probabilities up with V's 16-token rows.
//   The key's scale multiplies its scores; the value's multiplies its probability, with a power
//   of two c that keeps the product in f16's range whatever the values' size: below 2^12 at one
//   scale of the part's first pair, so that three octaves more need no other c (a pair with a
//   larger scale lowers c and rescales the accumulators).  f16 because its 11 bits keep
//   a product eight times as exact as bf16 would; one below its normal range is off by at most
//   2^-25 / c, 2^-36 of the largest scale so far.
template <int D>
struct Fp8Cache {
    static constexpr pa_dtype TYPE = PA_FP8_E4M3;
    using Out = __nv_bfloat16;
    static constexpr int TILE = 16 * D + 64;
    static constexpr int KS = D / 16;
    static constexpr int SCRATCH = 0;
    uint32_t qb[KS][2];
    float q0, q1;                                             // factors of the scores
    float unit;                                               // c; 0: the part has no pair yet
    int lane, r, c;
    __device__ __forceinline__ Fp8Cache(int lane_, float*) : lane(lane_), r(lane_ >> 2), c(lane_ & 3) { reset(); }
    __device__ __forceinline__ int lo() const { return 4 * (r >> 1) + (r & 1); }
    __device__ __forceinline__ int hi() const { return lo() + 2; }
    __device__ __forceinline__ void load_q(const void* q, size_t row0, int G) {
        const uint16_t* qrow = static_cast<const uint16_t*>(q) + (row0 + (r < G ? r : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            const uint2 u = r < G ? *reinterpret_cast<const uint2*>(qrow + 16 * kk + 4 * c) : make_uint2(0u, 0u);
            qb[kk][0] = u.x;
            qb[kk][1] = u.y;
        }
    }
    __device__ __forceinline__ void set_q(float scale) { rows_to_f16<KS>(qb, scale, c, q0, q1); }
    static __device__ __forceinline__ uint32_t half(uint32_t x, int i) {
        return e4m3x2_to_f16x2((uint16_t)(i ? x >> 16 : x & 0xffffu));
    }
    __device__ __forceinline__ void scores(const uint8_t* kt, const WParams&, float (&s)[2][4]) const {
        const int km = lane >> 3, kr = lane & 7;
        const int tok = 4 * (kr >> 1) + (kr & 1) + ((km & 1) ? 2 : 0);
        const uint32_t addr = smem_u32(kt) + (uint32_t)(((km >> 1) * kBlockTokens + tok) * 16);
        float acc[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < KS; kk += 2)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t x0, x1, x2, x3;
                ldmatrix_x4(addr + b * TILE + kk * 256, x0, x1, x2, x3);
                mma_f16_16816(acc[b], half(x0, 0), half(x1, 0), half(x0, 1), half(x1, 1), qb[kk][0], qb[kk][1]);
                mma_f16_16816(acc[b], half(x2, 0), half(x3, 0), half(x2, 1), half(x3, 1), qb[kk + 1][0], qb[kk + 1][1]);
            }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float* ks = reinterpret_cast<const float*>(kt + b * TILE + 16 * D);
            const float k0 = ks[lo()], k1 = ks[hi()];
            s[b][0] = acc[b][0] * (k0 * q0);
            s[b][1] = acc[b][1] * (k0 * q1);
            s[b][2] = acc[b][2] * (k1 * q0);
            s[b][3] = acc[b][3] * (k1 * q1);
        }
    }
    // Hidden slots may hold anything (NaN codes, scales of inf): a dim's 16 slots are 16 bytes.
    __device__ __forceinline__ void hide(uint8_t* vt, uint32_t vis) const {
        uint32_t m[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t v = vis >> (4 * w);
            m[w] = ((v & 1u) ? 0xffu : 0u) | ((v & 2u) ? 0xff00u : 0u) | ((v & 4u) ? 0xff0000u : 0u) | ((v & 8u) ? 0xff000000u : 0u);
        }
        for (int d = lane; d < D; d += 32) {
            uint4* row = reinterpret_cast<uint4*>(vt + d * 16);
            const uint4 x = *row;
            *row = make_uint4(x.x & m[0], x.y & m[1], x.z & m[2], x.w & m[3]);
        }
        if (lane < kBlockTokens && !((vis >> lane) & 1u)) *reinterpret_cast<float*>(vt + 16 * D + 4 * lane) = 0.f;
    }
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[2][4], Running& run,
                                       float (&o)[KS][4]) {
        uint32_t pb[2][2];
        run.l0 = run.l0 * run.al0 + ((pr[0][0] + pr[0][2]) + (pr[1][0] + pr[1][2]));
        run.l1 = run.l1 * run.al1 + ((pr[0][1] + pr[0][3]) + (pr[1][1] + pr[1][3]));
        float v[2][2];                                        // the scales of the lane's tokens
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float* vs = reinterpret_cast<const float*>(vt + b * TILE + 16 * D);
            v[b][0] = vs[lo()];
            v[b][1] = vs[hi()];
        }
        float top = fmaxf(fmaxf(fabsf(v[0][0]), fabsf(v[0][1])), fmaxf(fabsf(v[1][0]), fabsf(v[1][1])));
        // (a part's first pair: by its first scale, which every lane reads, as good as any)
        if (unit == 0.f) unit = unit_for(*reinterpret_cast<const float*>(vt + 16 * D));
        if (__any_sync(0xffffffffu, top * unit >= 32768.f)) {                      // rare
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float was = unit;
            unit = unit_for(top);
            const float f = exp2i(exponent(unit) - exponent(was));                 // exact
#pragma unroll
            for (int mi = 0; mi < KS; ++mi)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[mi][x] *= f;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float v0 = v[b][0] * unit, v1 = v[b][1] * unit;
            pb[b][0] = movmatrix_trans(pack_f16x2(pr[b][0] * v0, pr[b][1] * v0));
            pb[b][1] = movmatrix_trans(pack_f16x2(pr[b][2] * v1, pr[b][3] * v1));
        }
        if (run.rescale) rescale_rows(run, o);
        const uint32_t addr = smem_u32(vt) + lane * 16;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int mi = 0; mi < KS; mi += 2) {
                uint32_t y[4];                       // dims 16 mi .. + 7, + 8 .., 16 (mi + 1) .., + 8 ..
                ldmatrix_x4(addr + b * TILE + mi * 256, y[0], y[1], y[2], y[3]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t ya = y[2 * x], yb = y[2 * x + 1];
                    mma_f16_16816(o[mi + x], half(ya, 0), half(yb, 0), half(ya, 1), half(yb, 1), pb[b][0], pb[b][1]);
                }
            }
        }
    }
    // c for a largest scale in 2^(e - 127) .. 2^(e - 126): their product from 2^11 on, below 2^12
    static __device__ __forceinline__ float unit_for(float top) { return exp2i(min(138 - (int)(__float_as_uint(fabsf(top)) >> 23), 127)); }
    // log2 of a power of two
    static __device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
    __device__ __forceinline__ void reset() { unit = 0.f; }
    __device__ __forceinline__ float finish(float (&)[KS][4]) const { return unit > 0.f ? exp2i(-exponent(unit)) : 1.f; }
};

// The first product of a sum: D = A B.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// MXFP4 records: codes become f16 in registers (exact).
//   K: the scale varies along the dot product, so each 32-dim block of it is a product of
//   its own, times the token's scale, summed in fp32.
//   V: the scale varies along the tokens, so it multiplies the probabilities: block b's dims
//   take P_b = p 2^(e_b(t) - 127) c_b with c_b = 2^(142 - R_b), R_b at least the largest scale
//   code of block b so far (raised, and the block's accumulators rescaled, when a pair brings
//   a larger one), so that P_b stays at most 2^15, in f16's range.  As with FP8, f16 for its 11
//   bits; R_b lies up to three octaves above the largest code, so a P_b below f16's normal range
//   is off by at most 2^-25 / c_b, 2^-37 of the largest scale.
// The bound is latency: an SM's 16 warps fill 60 % of the issue slots (64 sequences of window
// 2040, 32 / 8 heads of 128), waiting for the chain conversion, product, product, sum of each 32
// dims.  Conversions, selections and packing run at half the rate of FMAs (that pipe is 45 %
// busy), so scale codes are read as bytes (their fp32 is one multiply away, on the other pipe),
// and lane c watches the codes of block c alone for a raise.
template <int D>
struct Fp4Cache {
    static constexpr pa_dtype TYPE = PA_FP4_E2M1;
    using Out = __nv_bfloat16;
    static constexpr int TILE = 8 * D + D / 2;
    static constexpr int KS = D / 16;
    static constexpr int SCRATCH = 0;
    static constexpr int NB = D / 32;                         // scale blocks of a row
    uint32_t qb[KS][2];
    float q0, q1;                                             // factors of the scores
    float cb[NB];
    int ref;                                                  // R_b of b = c % NB
    int lane, r, c;
    __device__ __forceinline__ Fp4Cache(int lane_, float*) : lane(lane_), r(lane_ >> 2), c(lane_ & 3) {
        reset();
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int b = 0; b < NB; ++b) cb[b] = exp2i(127);
        ref = 0;
    }
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
    __device__ __forceinline__ void set_q(float scale) { rows_to_f16<KS>(qb, scale, c, q0, q1); }
    // N adjacent 32-bit words
    template <int N>
    static __device__ __forceinline__ void words(const uint8_t* at, uint32_t (&w)[N]) {
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(at + 4 * i);
                w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
            }
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            w[0] = v.x; w[1] = v.y;
        }
    }
    // 2^(code - 127): the code is the exponent field (code 0 gives 0)
    static __device__ __forceinline__ float scale_value(uint8_t code) { return __uint_as_float((uint32_t)code * 0x800000u); }
    // log2 of a block's c_b, from its R_b: at most 127
    static __device__ __forceinline__ int c_exp(int R) { return min(142 - R, 127); }
    __device__ __forceinline__ void scores(const uint8_t* kt, const WParams&, float (&s)[2][4]) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* k = kt + t * TILE;
            uint32_t k0[NB], k1[NB];
            words<NB>(k + r * (D / 2) + c * (D / 8), k0);
            words<NB>(k + (r + 8) * (D / 2) + c * (D / 8), k1);
            const uint8_t* e0 = k + 8 * D + r * NB;
            const uint8_t* e1 = e0 + 8 * NB;
            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t a[4], a8[4];
                e2m1x8_to_f16x2x4(k0[b], a);
                e2m1x8_to_f16x2x4(k1[b], a8);
                float acc[4];
                mma_f16_zero(acc, a[0], a8[0], a[1], a8[1], qb[2 * b][0], qb[2 * b][1]);
                mma_f16_16816(acc, a[2], a8[2], a[3], a8[3], qb[2 * b + 1][0], qb[2 * b + 1][1]);
                const float f0 = scale_value(e0[b]), f1 = scale_value(e1[b]);
                s[t][0] = fmaf(acc[0], f0, s[t][0]);
                s[t][1] = fmaf(acc[1], f0, s[t][1]);
                s[t][2] = fmaf(acc[2], f1, s[t][2]);
                s[t][3] = fmaf(acc[3], f1, s[t][3]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][i] *= (i & 1) ? q1 : q0;
        }
    }
    // Hidden slots count with scale code 0 (their codes are finite whatever they are).
    __device__ __forceinline__ void hide(uint8_t* vt, uint32_t vis) const {
        if (lane < kBlockTokens && !((vis >> lane) & 1u))
#pragma unroll
            for (int b = 0; b < NB; ++b) vt[8 * D + lane * NB + b] = 0;
    }
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[2][4], Running& run,
                                       float (&o)[KS][4]) {
        run.l0 = run.l0 * run.al0 + ((pr[0][0] + pr[0][2]) + (pr[1][0] + pr[1][2]));
        run.l1 = run.l1 * run.al1 + ((pr[0][1] + pr[0][3]) + (pr[1][1] + pr[1][3]));
        const uint8_t* sc = vt + 8 * D + r * NB;              // scale codes of token r, then r + 8
        int top = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            top = max(top, max((int)sc[t * TILE + c % NB], (int)sc[t * TILE + 8 * NB + c % NB]));
        if (__any_sync(0xffffffffu, top > ref)) {             // rare after a part's first pair
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
            // (three octaves above the largest seen, so that the next ones hardly raise it again)
            const int raised = top > ref ? min(top + 3, 255) : ref;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int en = c_exp(__shfl_sync(0xffffffffu, raised, b)), eo = c_exp(__shfl_sync(0xffffffffu, ref, b));
                const float f = exp2i(en - eo);               // exact
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[2 * b][x] *= f;
                    o[2 * b + 1][x] *= f;
                }
                cb[b] = exp2i(en);
            }
            ref = raised;
        }
        if (run.rescale) rescale_rows(run, o);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t vw[KS];
            words<KS>(vt + t * TILE + (r * 4 + c) * (KS * 4), vw);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float g0 = scale_value(sc[t * TILE + b]) * cb[b], g1 = scale_value(sc[t * TILE + 8 * NB + b]) * cb[b];
                const uint32_t pb0 = movmatrix_trans(pack_f16x2(pr[t][0] * g0, pr[t][1] * g0));
                const uint32_t pb1 = movmatrix_trans(pack_f16x2(pr[t][2] * g1, pr[t][3] * g1));
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    uint32_t a[4];
                    e2m1x8_to_f16x2x4(vw[2 * b + h2], a);
                    mma_f16_16816(o[2 * b + h2], a[0], a[2], a[1], a[3], pb0, pb1);
                }
            }
        }
    }
    __device__ __forceinline__ float finish(float (&o)[KS][4]) const {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float f = exp2i(-c_exp(__shfl_sync(0xffffffffu, ref, b)));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                o[2 * b][x] *= f;
                o[2 * b + 1][x] *= f;
            }
        }
        return 1.f;
    }
};

// f32 tiles: each operand x is split into two tf32 numbers, h (x rounded) and l (x - h
// rounded), and a product is h h' + (h l' + l h') on the tensor cores: the dropped l l' and the
// roundings of l are 2^-21 of the product at most, near fp32's own rounding, and the work does
// not grow with G as with FMAs.  The tensor cores' own sums are cut, not rounded, at each step,
// so they are kept short: h h' and the small products apart, a few steps each, added in fp32
// (the outputs' relative error: 2.5e-7 to 3.5e-7; with one long sum 8e-7).
// K and V fragments are plain 32-bit reads of the tiles (K's are free of bank conflicts, V's
// two-way); the probabilities pass through shared memory to reach the B operand's order.
// An infinity has no such two numbers (its l is NaN), and the rounding of h takes finite numbers
// within 2^-12 of the largest to infinity.  Either leaves its mark on the part: a score that is
// NaN on the part's sum, a value on its outputs, which come out NaN or infinite.  Such a part of a
// warp is done again with fp32 FMAs, token by token (a check of each pair's results instead: 10 to
// 37 % of the time).
struct Split { uint32_t h, l; };
__device__ __forceinline__ Split split_tf32(float x) {
    // (integer operations: the conversion instruction runs at a fraction of their rate)
    Split s;
    s.h = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    s.l = __float_as_uint(x - __uint_as_float(s.h)) & 0xffffe000u;
    return s;
}
__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// large += h h', small += h l' + l h' over 8 of the contraction's elements, a in fp32, b split
__device__ __forceinline__ void mma_split(float (&large)[4], float (&small)[4], const float (&a)[4], Split b0, Split b1) {
    Split x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = split_tf32(a[i]);
    mma_tf32_1688(large, x[0].h, x[1].h, x[2].h, x[3].h, b0.h, b1.h);
    mma_tf32_1688(small, x[0].l, x[1].l, x[2].l, x[3].l, b0.h, b1.h);
    mma_tf32_1688(small, x[0].h, x[1].h, x[2].h, x[3].h, b0.l, b1.l);
}

template <int D>
struct F32Cache {
    static constexpr pa_dtype TYPE = PA_F32;
    using Out = float;
    static constexpr int TILE = kBlockTokens * D * 4;
    static constexpr int KS = D / 16;
    static constexpr int SCRATCH = 32 * 8 * 4;                // a warp's probabilities, [32 tokens][8 heads]
    float q[D / 8][2];
    float* sp;
    int lane, r, c;
    __device__ __forceinline__ F32Cache(int lane_, float* scratch) : sp(scratch), lane(lane_), r(lane_ >> 2), c(lane_ & 3) {}
    __device__ __forceinline__ int lo() const { return r; }
    __device__ __forceinline__ int hi() const { return r + 8; }
    __device__ __forceinline__ void load_q(const void* q_, size_t row0, int G) {
        const float* qrow = static_cast<const float*>(q_) + (row0 + (r < G ? r : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < D / 8; ++kk) {
            q[kk][0] = r < G ? qrow[8 * kk + c] : 0.f;
            q[kk][1] = r < G ? qrow[8 * kk + 4 + c] : 0.f;
        }
    }
    __device__ __forceinline__ void set_q(float) {}
    __device__ __forceinline__ void scores(const uint8_t* kt, const WParams& p, float (&s)[2][4]) const {
        const float* k = reinterpret_cast<const float*>(kt);
        float large[2][2][4] = {}, small[2][4] = {};          // two sums of h h' per block, of every other step
#pragma unroll
        for (int kk = 0; kk < D / 8; ++kk) {
            const Split b0 = split_tf32(q[kk][0]), b1 = split_tf32(q[kk][1]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float* at = k + b * (TILE / 4) + (2 * kk * kBlockTokens + r) * 4 + c;
                const float a[4] = {at[0], at[32], at[64], at[96]};
                mma_split(large[b][kk & 1], small[b], a, b0, b1);
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][i] = (large[b][0][i] + large[b][1][i] + small[b][i]) * p.scale_log2;
    }
    // (as for bf16)
    __device__ __forceinline__ void hide(uint8_t* vt, uint32_t vis) const {
        for (int i = lane; i < TILE / 16; i += 32)
            if (!((vis >> (i % kBlockTokens)) & 1u)) *reinterpret_cast<uint4*>(vt + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void pv(const uint8_t* vt, const float (&pr)[2][4], Running& run,
                                       float (&o)[KS][4]) {
        run.l0 = run.l0 * run.al0 + ((pr[0][0] + pr[0][2]) + (pr[1][0] + pr[1][2]));
        run.l1 = run.l1 * run.al1 + ((pr[0][1] + pr[0][3]) + (pr[1][1] + pr[1][3]));
        __syncwarp();                                         // (the last pair's reads are done)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            *reinterpret_cast<float2*>(sp + (16 * b + r) * 8 + 2 * c) = make_float2(pr[b][0], pr[b][1]);
            *reinterpret_cast<float2*>(sp + (16 * b + r + 8) * 8 + 2 * c) = make_float2(pr[b][2], pr[b][3]);
        }
        __syncwarp();
        if (run.rescale) rescale_rows(run, o);
        Split p0[4], p1[4];                                   // of tokens c and c + 4 of 8, four times
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            p0[kk] = split_tf32(sp[(8 * kk + c) * 8 + r]);
            p1[kk] = split_tf32(sp[(8 * kk + c + 4) * 8 + r]);
        }
        const float* v = reinterpret_cast<const float*>(vt) + ((r >> 2) * kBlockTokens + c) * 4 + (r & 3);
#pragma unroll
        for (int mi = 0; mi < KS; ++mi) {
            float large[4] = {}, small[4] = {};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const float* at = v + (kk >> 1) * (TILE / 4) + mi * (4 * kBlockTokens * 4) + (kk & 1) * 32;
                const float a[4] = {at[0], at[2 * kBlockTokens * 4], at[16], at[2 * kBlockTokens * 4 + 16]};
                mma_split(large, small, a, p0[kk], p1[kk]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) o[mi][x] += large[x] + small[x];
        }
    }
    __device__ __forceinline__ void reset() {}
    __device__ __forceinline__ float finish(float (&)[KS][4]) const { return 1.f; }
    // The part of entries first .. last - 1 of a walk again, from the pools: its maxima and outputs,
    // and its whole sums in every lane.
    template <typename Walk>
    __device__ __forceinline__ void again(const WParams& p, const Walk& walk, const Row& row, int first, int last, Running& run,
                                          float (&o)[KS][4]) const {
        const size_t row0 = (size_t)blockIdx.z * p.Hq + (size_t)blockIdx.y * p.G;
        // (lanes of heads past G: the first head's, which nothing stores)
        const float* q0 = static_cast<const float*>(p.q) + (row0 + (2 * c < p.G ? 2 * c : 0)) * D;
        const float* q1 = static_cast<const float*>(p.q) + (row0 + (2 * c + 1 < p.G ? 2 * c + 1 : 0)) * D;
        run.m0 = run.m1 = -INFINITY;
        run.l0 = run.l1 = 0.f;
#pragma unroll
        for (int mi = 0; mi < KS; ++mi) o[mi][0] = o[mi][1] = o[mi][2] = o[mi][3] = 0.f;
#pragma unroll 1
        for (int e = first; e < last; ++e) {
            const int at = walk.block(e);
            const int32_t blk = __ldg(walk.trow + at);
            if (blk < 0 || blk >= p.num_blocks) continue;
            const uint32_t vis = visible_slots(at * kBlockTokens, row.len, row.first, p.sinks);
            const size_t tile = ((size_t)blk * p.Hkv + blockIdx.y) * TILE;
#pragma unroll 1
            for (int t = 0; t < kBlockTokens; ++t) {
                if (!((vis >> t) & 1u)) continue;
                const float* k = reinterpret_cast<const float*>(p.k_pool + tile) + t * 4;
                const float* v = reinterpret_cast<const float*>(p.v_pool + tile) + t * 4;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll 1
                for (int d = 0; d < D; ++d) {
                    const float x = k[(d >> 2) * (kBlockTokens * 4) + (d & 3)];
                    s0 = __fmaf_rn(q0[d], x, s0);
                    s1 = __fmaf_rn(q1[d], x, s1);
                }
                s0 *= p.scale_log2;
                s1 *= p.scale_log2;
                const float n0 = fmaxf(run.m0, s0), n1 = fmaxf(run.m1, s1);
                const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
                const float a0 = fast_exp2(run.m0 - z0), a1 = fast_exp2(run.m1 - z1);
                const float w0 = fast_exp2(s0 - z0), w1 = fast_exp2(s1 - z1);
                run.m0 = n0;
                run.m1 = n1;
                run.l0 = __fmaf_rn(run.l0, a0, w0);
                run.l1 = __fmaf_rn(run.l1, a1, w1);
#pragma unroll
                for (int mi = 0; mi < KS; ++mi)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int d = 16 * mi + r + (x >> 1) * 8;
                        o[mi][x] = __fmaf_rn((x & 1) ? w1 : w0, v[(d >> 2) * (kBlockTokens * 4) + (d & 3)], o[mi][x] * ((x & 1) ? a1 : a0));
                    }
            }
        }
    }
};

// Shared memory: the warps' stages, each the K tiles then the V tiles of a pair of blocks;
// the warps' scratch; the barriers, two of each warp; and the warps' folded results.  A result is
// the outputs as the lanes hold them (per pair of heads, 16 dims and r: a float4, dims r and
// r + 8 of one head, then of the other; CS floats for a pair of heads, no two lanes in the same banks), then the
// heads' maxima and sums.
template <class C, int D, int NW>
struct Layout {
    static constexpr int STAGE = 4 * C::TILE;
    static constexpr int WARP = NW * STAGE;
    static constexpr int BAR = WARP + NW * C::SCRATCH;
    static constexpr int OUT = BAR + NW * 16;
    static constexpr int CS = 2 * D + 8;
    static __host__ __device__ constexpr int outs(int G) { return CS * ((G + 1) / 2); }         // floats of a warp
    static __host__ __device__ constexpr int result(int G) { return NW * (outs(G) + 2 * G); }   // and of all
    static constexpr int bytes(int G, int results) { return OUT + results * result(G) * 4; }
};

// The listed blocks of one sequence as one warp walks them: entry e is block e % 2 of its pair
// e / 2, pairs lie 2 NW blocks apart, and the table entries are read 32 at a time.
template <int NW>
struct BlockWalk {
    const int32_t* trow;
    VisibleBlocks v;
    int first, n, lane, page, num_blocks;      // n: entries
    int32_t* err;
    int32_t ent;                                // -1: names no block of the pool (flagged)
    __device__ __forceinline__ int block(int e) const { return v.block(first + (e >> 1) * 2 * NW + (e & 1)); }
    __device__ __forceinline__ void fetch() {
        const int e = page * 32 + lane;
        ent = -1;
        if (e < n) {
            const int32_t b = __ldg(trow + block(e));
            if (b >= 0 && b < num_blocks) ent = b;
            else raise_flag(err, PA_DEV_ERR_BAD_BLOCK);
        }
    }
    __device__ __forceinline__ int32_t entry(int e) {          // in order, the whole warp
        if ((e >> 5) != page) {
            page = e >> 5;
            fetch();
        }
        return __shfl_sync(0xffffffffu, ent, e & 31);
    }
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// another CTA's address of what this CTA has at shared address `addr`, and a float there
__device__ __forceinline__ uint32_t peer_at(uint32_t addr, int rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    return at;
}
__device__ __forceinline__ float peer_f32(uint32_t at) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}

// Parts.  The listed blocks are cut into parts of p.part_len (the last takes what is left), and
// in every part warp w takes the same blocks whatever CTA it belongs to.  A (warp, part) has
// its own maximum, sum and outputs; a warp's parts are folded into one in their order, and the
// warps merged in theirs.  So the result is the same, bit for bit, whether one CTA goes through
// all parts (many sequences: no joining at all) or a cluster of CTAs has p.per parts each (few:
// every SM gets work), and a sequence's result does not depend on the batch.
struct Partial { float m, l, o; };         // of one head and dim; a part without keys: -inf, 0, 0
__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.f : m; }
// The joint maximum of two parts and what their sums are scaled by.
struct Fold { float m, a, s; };
__device__ __forceinline__ Fold fold_factors(float a, float s) {
    // (NaN, from a part that was given up, must stay)
    const float m = (s > a || s != s) ? s : a, z = safe_max(m);
    return Fold{m, fast_exp2(a - z), fast_exp2(s - z)};
}
__device__ __forceinline__ float fold_add(const Fold& f, float a, float s) { return __fmaf_rn(s, f.s, __fmul_rn(a, f.a)); }
__device__ __forceinline__ void fold(Partial& a, const Partial& s) {
    const Fold f = fold_factors(a.m, s.m);
    a = Partial{f.m, fold_add(f, a.l, s.l), fold_add(f, a.o, s.o)};
}

// The warps' results of one head as one: their maxima and sums first, then each output.
template <int NW>
struct Merge {
    float m[NW], l[NW], sum;          // m: after weigh(), the warps' weights
    __device__ __forceinline__ void set(int w, float m_, float l_) {
        m[w] = m_;
        l[w] = l_;
    }
    __device__ __forceinline__ void weigh() {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = (m[w] > M || m[w] != m[w]) ? m[w] : M;
        const float z = safe_max(M);
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            m[w] = fast_exp2(m[w] - z);
            sum = __fmaf_rn(l[w], m[w], sum);
        }
    }
    __device__ __forceinline__ float add(float acc, int w, float o) const { return __fmaf_rn(o, m[w], acc); }
    __device__ __forceinline__ float result(float acc) const { return sum > 0.f || sum != sum ? acc / sum : 0.f; }
};

template <typename Out>
__device__ __forceinline__ void store_out(void* out, size_t at, float x) {
    if constexpr (sizeof(Out) == 2) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
    else static_cast<float*>(out)[at] = x;
}

template <template <int> class Cache, int D, int NW>
__global__ void __launch_bounds__(NW * 32, ctas_for(Cache<D>::TYPE, D)) window_decode_kernel(const WParams p) {
    using C = Cache<D>;
    using L = Layout<C, D, NW>;
    constexpr int KS = C::KS, TILE = C::TILE;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.y, s = blockIdx.z;
    uint8_t* const stage = smem + warp * L::STAGE;
    const uint32_t bars = smem_u32(smem) + L::BAR + warp * 16;         // K's, V's
    if (lane == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        fence_proxy_async_smem();
    }
    __syncwarp();
    // lengths, tables, queries and pools may all be the previous kernels' output
    grid_dependency_wait();
    grid_launch_dependents();
    // (each warp for itself; a warp that skips reads no tiles and the CTA writes nothing)
    const bool skip = __any_sync(0xffffffffu, aborted(p.err));
    const size_t row0 = (size_t)s * p.Hq + (size_t)kvh * p.G;
    C cache(lane, reinterpret_cast<float*>(smem + L::WARP + warp * C::SCRATCH));
    cache.load_q(p.q, row0, p.G);
    const Row row = row_of(p, s, blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0);
    const int parts = max(1, min(p.parts, (row.v.count + p.part_len - 1) / p.part_len));
    const int begin = blockIdx.x * p.per * p.part_len;
    if (p.per && (int)blockIdx.x * p.per >= parts) return;     // (a CTA that leaves is not waited for)
    // this CTA's parts and listed blocks
    const int mine = p.per ? min(p.per, parts - (int)blockIdx.x * p.per) : parts;
    const int count = (p.per && (int)(blockIdx.x + 1) * p.per < parts ? begin + p.per * p.part_len : row.v.count) - begin;
    BlockWalk<NW> walk{p.tables + (size_t)s * p.max_blocks, row.v, begin + 2 * warp, 0, lane, 0, p.num_blocks, p.err, -1};
    {
        // whole pairs before the last, then what is left of it
        const int from = count - 2 * warp;
        const int pairs = from > 0 && !skip ? (from + 2 * NW - 1) / (2 * NW) : 0;
        walk.n = pairs > 0 ? 2 * (pairs - 1) + min(2, from - 2 * NW * (pairs - 1)) : 0;
    }
    const int npairs = (walk.n + 1) >> 1;
    walk.fetch();

    const uint64_t pol = l2_policy_evict_first();
    // Pair i's tiles into the stage, HALF 0 K, 1 V (a table entry that names no block is flagged
    // and left out).
    uint32_t have = 0;                         // of the pair whose K was issued last, a bit a block: it is copied
    uint32_t phase = 0, in_flight = 0;         // a bit a half: the phase that its next copy ends; it has a copy under way
    int32_t blk[2];                            // that pair's blocks, kept from K's issue to V's
    auto issue = [&](int i, int half) {
        if (half == 0) {
            blk[0] = walk.entry(2 * i);
            blk[1] = walk.entry(2 * i + 1);                    // (-1 past the last)
            have = (blk[0] >= 0 ? 1u : 0u) | (blk[1] >= 0 ? 2u : 0u);
        }
        if (have == 0u) return;
        in_flight |= 1u << half;
        if (lane == 0) {
            const uint32_t bar = bars + half * 8, dst = smem_u32(stage) + half * 2 * TILE;
            const char* pool = half == 0 ? p.k_pool : p.v_pool;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, have == 3u ? 2 * TILE : TILE);
            if (have & 1u) bulk_g2s(dst, pool + ((size_t)blk[0] * p.Hkv + kvh) * (size_t)TILE, TILE, bar, pol);
            if (have & 2u) bulk_g2s(dst + TILE, pool + ((size_t)blk[1] * p.Hkv + kvh) * (size_t)TILE, TILE, bar, pol);
        }
    };
    auto landed = [&](int half) -> bool {
        const bool ok = mbar_wait_bounded(bars + half * 8, (phase >> half) & 1u, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, ok)) return false;
        phase ^= 1u << half;
        in_flight &= ~(1u << half);
        return true;
    };
    if (npairs > 0) {
        issue(0, 0);
        issue(0, 1);
    }
    cache.set_q(p.scale_log2);                 // (the queries are waited for with the copies under way)

    Running run;
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // A part's end: the lanes' sums as one, the cache's own factors out, and into the warp's
    // folded result (its outputs in shared memory, every lane its own elements); in a cluster,
    // where parts before this CTA's are still to be folded, into a result of the part's own.
    const int slot = L::result(p.G), outs = L::outs(p.G), G2 = (p.G + 1) / 2;
    float* sm_o = reinterpret_cast<float*>(smem + L::OUT);     // [NW][G2][KS][8][4]
    float* sm_m = sm_o + NW * outs;                            // [NW][G]
    float* sm_l = sm_m + NW * p.G;                             // [NW][G]
    int at_slot = 0;                                           // floats from the first result
    float all_m0 = -INFINITY, all_m1 = -INFINITY, all_l0 = 0.f, all_l1 = 0.f;
    bool folded = false;
    auto put_sums = [&](float m0, float m1, float l0, float l1) {
        const int r = lane >> 2, g = 2 * (lane & 3), at = at_slot + warp * p.G + g;
        if (r == 0 && g < p.G) {
            sm_m[at] = m0;
            sm_l[at] = l0;
        }
        if (r == 0 && g + 1 < p.G) {
            sm_m[at + 1] = m1;
            sm_l[at + 1] = l1;
        }
    };
    auto end_part = [&](int from, int to) {                    // (of the pairs from .. to - 1)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            run.l0 += __shfl_xor_sync(0xffffffffu, run.l0, x);
            run.l1 += __shfl_xor_sync(0xffffffffu, run.l1, x);
        }
        if constexpr (C::TYPE == PA_F32) {
            bool fine = run.l0 == run.l0 && run.l1 == run.l1;
#pragma unroll
            for (int mi = 0; mi < KS; ++mi)
#pragma unroll
                for (int x = 0; x < 4; ++x) fine = fine && fabsf(o[mi][x]) <= FLT_MAX;
            if (!__all_sync(0xffffffffu, fine)) cache.again(p, walk, row, 2 * from, min(2 * to, walk.n), run, o);
        }
        const float factor = cache.finish(o);
        const int r = lane >> 2, c = lane & 3;
        const Fold f0 = fold_factors(all_m0, run.m0), f1 = fold_factors(all_m1, run.m1);
        const Fold o0{f0.m, f0.a, f0.s * factor}, o1{f1.m, f1.a, f1.s * factor};
        if (c < G2) {
            float4* at = reinterpret_cast<float4*>(sm_o + at_slot + warp * outs + c * L::CS) + r;
#pragma unroll
            for (int mi = 0; mi < KS; ++mi, at += 8) {
                const float4 was = folded ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                *at = make_float4(fold_add(o0, was.x, o[mi][0]), fold_add(o0, was.y, o[mi][2]),
                                  fold_add(o1, was.z, o[mi][1]), fold_add(o1, was.w, o[mi][3]));
            }
        }
        all_l0 = fold_add(f0, all_l0, run.l0);
        all_l1 = fold_add(f1, all_l1, run.l1);
        all_m0 = f0.m;
        all_m1 = f1.m;
        folded = true;
        if (p.per) {
            put_sums(all_m0, all_m1, all_l0, all_l1);
            at_slot += slot;
            all_m0 = all_m1 = -INFINITY;
            all_l0 = all_l1 = 0.f;
            folded = false;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        run.m0 = run.m1 = -INFINITY;
        run.l0 = run.l1 = 0.f;
        cache.reset();
    };
    const int part_pairs = p.part_len / (2 * NW);      // of a warp
    const int last_end = (mine - 1) * part_pairs;
    int end_at = mine > 1 ? part_pairs : INT_MAX;      // pair before which a part ends (the last one: never)
    bool failed = false;
    for (int i = 0; i < npairs; ++i) {
        const bool more = i + 1 < npairs;
        if (i == end_at) {
            end_part(i - part_pairs, i);
            end_at = end_at < last_end ? end_at + part_pairs : INT_MAX;
        }
        const uint32_t h = have;
        if (h == 0u) {                         // no block of the pair is in the pool
            if (more) {
                issue(i + 1, 0);
                issue(i + 1, 1);
            }
            continue;
        }
        uint32_t vis[2];                       // 16 bits, a slot each
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int tok0 = walk.block(2 * i + b) * kBlockTokens;
            const bool inner = tok0 >= row.first && tok0 + kBlockTokens <= row.len;
            vis[b] = !((h >> b) & 1u) ? 0u : inner ? 0xffffu : visible_slots(tok0, row.len, row.first, p.sinks);
        }
        const bool full = (vis[0] & vis[1]) == 0xffffu;
        if (!landed(0)) {
            failed = true;
            break;
        }
        float sc[2][4];
        cache.scores(stage, p, sc);
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (!full) {
                // hidden slots may hold anything: select, never multiply
                const bool ok0 = (vis[b] >> cache.lo()) & 1u, ok1 = (vis[b] >> cache.hi()) & 1u;
                sc[b][0] = ok0 ? sc[b][0] : -INFINITY;
                sc[b][1] = ok0 ? sc[b][1] : -INFINITY;
                sc[b][2] = ok1 ? sc[b][2] : -INFINITY;
                sc[b][3] = ok1 ? sc[b][3] : -INFINITY;
            }
            t0 = fmaxf(t0, fmaxf(sc[b][0], sc[b][2]));
            t1 = fmaxf(t1, fmaxf(sc[b][1], sc[b][3]));
        }
        // K is read: the stage's next K tiles may land under the rest of the pair
        __syncwarp();
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        const float n0 = fmaxf(run.m0, t0), n1 = fmaxf(run.m1, t1);
        // (a maximum still at -inf, from keys that score -inf, must not give inf - inf)
        const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
        run.al0 = fast_exp2(run.m0 - z0);
        run.al1 = fast_exp2(run.m1 - z1);
        run.m0 = n0;
        run.m1 = n1;
        float pr[2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            pr[b][0] = fast_exp2(sc[b][0] - z0);
            pr[b][1] = fast_exp2(sc[b][1] - z1);
            pr[b][2] = fast_exp2(sc[b][2] - z0);
            pr[b][3] = fast_exp2(sc[b][3] - z1);
        }
        run.rescale = __any_sync(0xffffffffu, run.al0 != 1.f || run.al1 != 1.f);
        if (more) issue(i + 1, 0);
        if (!landed(1)) {
            failed = true;
            break;
        }
        if (!full) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (vis[b] != 0xffffu) cache.hide(stage + (2 + b) * TILE, vis[b]);
            fence_proxy_async_smem();      // (before the stage's next copy)
            __syncwarp();
        }
        cache.pv(stage + 2 * TILE, pr, run, o);
        __syncwarp();
        if (more) issue(i + 1, 1);
    }
    if (failed) {
        // drain every copy still in flight before the shared memory is reused
        if (lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        for (int half = 0; half < 2; ++half)
            if ((in_flight >> half) & 1u) mbar_wait_bounded(bars + half * 8, (phase >> half) & 1u, kWaitLimitNs);
    }
    const int results = p.per ? min(p.per, parts - (int)blockIdx.x * p.per) : 1;
    int from = end_at == INT_MAX ? last_end : end_at - part_pairs;
    do {                                       // (a warp without blocks in the last parts: empty ones)
        end_part(from, npairs);
        from = npairs;
    } while (p.per && at_slot < results * slot);
    const bool bad = __syncthreads_or(failed || skip), cta_skip = __syncthreads_or(skip);
    if (!p.per) put_sums(all_m0, all_m1, all_l0, all_l1);
    if (bad) {
        // what was given up or skipped passes on NaN: its result is incomplete
        const float nan = __int_as_float(0x7fc00000);
        for (at_slot = 0; at_slot < results * slot; at_slot += slot) put_sums(nan, nan, nan, nan);
    }
    if (!p.per || parts == 1) {
        __syncthreads();
        if (cta_skip) return;
        // two outputs of HT heads a thread
        constexpr int HT = NW == 8 ? 1 : 2;
        for (int i = threadIdx.x; i < G2 * KS * 16 / HT; i += NW * 32) {
            const int x = i * HT / 2, c = x / (KS * 8), d = x / 8 % KS * 16 + x % 8;
            const float* at = sm_o + c * L::CS + x % (KS * 8) * 4;
#pragma unroll
            for (int e = 0; e < HT; ++e) {
                const int h = HT == 2 ? e : i & 1, g = 2 * c + h;
                if (g >= p.G) continue;
                Merge<NW> m;
#pragma unroll
                for (int w = 0; w < NW; ++w) m.set(w, sm_m[w * p.G + g], sm_l[w * p.G + g]);
                m.weigh();
                float lo = 0.f, hi = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float2 o2 = *reinterpret_cast<const float2*>(at + w * outs + 2 * h);
                    lo = m.add(lo, w, o2.x);
                    hi = m.add(hi, w, o2.y);
                }
                store_out<typename C::Out>(p.out, (row0 + g) * D + d, m.result(lo));
                store_out<typename C::Out>(p.out, (row0 + g) * D + d + 8, m.result(hi));
            }
        }
        return;
    }
    // In a cluster each CTA adds up its share of the output elements over all parts, reading the
    // others' shared memory (so nothing goes through a workspace, and one launch does it).
    cluster_arrive();
    cluster_wait();
    const int ctas = (parts + p.per - 1) / p.per;
    // (the loads of JB parts of all warps are under way together: 14 / 2 heads of 64, window 1500, one
    // sequence 8.5 -> 7.2 us)
    constexpr int JB = (C::TYPE == PA_FP4_E2M1 ? 8 : 16) / NW;       // (FP4: registers)
    const uint32_t m_from = NW * outs * 4, l_from = m_from + NW * p.G * 4;
    for (int i = blockIdx.x * (NW * 32) + threadIdx.x; i < G2 * KS * 32; i += ctas * (NW * 32)) {
        const int c = i / (KS * 32), g = 2 * c + (i >> 1 & 1), d = i / 32 % KS * 16 + i / 4 % 8 + (i & 1) * 8;
        if (g >= p.G) continue;
        Partial a[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) a[w] = Partial{-INFINITY, 0.f, 0.f};
        int rank = 0, k = 0;
        for (int j = 0; j < parts; j += JB) {
            Partial x[JB][NW];
#pragma unroll
            for (int jj = 0; jj < JB; ++jj) {
                const uint32_t at = peer_at(smem_u32(sm_o), rank) + k * slot * 4;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    x[jj][w] = Partial{-INFINITY, 0.f, 0.f};
                    if (j + jj < parts)
                        x[jj][w] = Partial{peer_f32(at + m_from + (w * p.G + g) * 4), peer_f32(at + l_from + (w * p.G + g) * 4),
                                           peer_f32(at + (w * outs + c * L::CS + i % (KS * 32)) * 4)};
                }
                if (++k == p.per) {
                    k = 0;
                    rank = min(rank + 1, ctas - 1);
                }
            }
#pragma unroll
            for (int jj = 0; jj < JB; ++jj)
#pragma unroll
                for (int w = 0; w < NW; ++w) fold(a[w], x[jj][w]);
        }
        Merge<NW> m;
#pragma unroll
        for (int w = 0; w < NW; ++w) m.set(w, a[w].m, a[w].l);
        m.weigh();
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) y = m.add(y, w, a[w].o);
        if (!cta_skip) store_out<typename C::Out>(p.out, (row0 + g) * D + d, m.result(y));
    }
    // no CTA leaves while another may still read its shared memory
    cluster_arrive();
    cluster_wait();
}

constexpr int kSmemMax = 232448;       // shared memory of an SM that one CTA can have

// Attributes of a kernel, set once per device; and the device's SMs.
template <void (*Kernel)(const WParams)>
cudaError_t prepare_kernel(int& dev, int& sms) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    // clusters of up to 16 CTAs
    if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Clusters of `ctas` CTAs that the (empty) GPU runs at once.  What the runtime answers is kept,
// one answer for each number of CTAs, with what it was asked for.
template <void (*Kernel)(const WParams)>
long long clusters_at_once(int dev, int ctas, int threads, int smem) {
    static std::atomic<uint64_t> kept[17];         // device + 1, bytes, answer
    const uint64_t key = (uint64_t)(dev + 1) << 48 | (uint64_t)smem << 16;
    const uint64_t was = kept[ctas].load(std::memory_order_relaxed);
    if ((was & ~0xffffull) == key) return (long long)(was & 0xffff);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    n = n < 0xffff ? n : 0xffff;
    kept[ctas].store(key | (uint64_t)n, std::memory_order_relaxed);
    return n;
}

template <void (*Kernel)(const WParams)>
cudaError_t launch(WParams p, int num_seqs, int threads, bool one_each, int smem, int smem_result, cudaStream_t stream) {
    const int parts = p.parts;
    int dev = 0, sms = 1;
    const cudaError_t e = prepare_kernel<Kernel>(dev, sms);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const long long pairs = (long long)p.Hkv * num_seqs;
    // As many CTAs for a sequence's parts as the GPU has room for at once (clusters' CTAs start
    // together, and what does not fit waits for a whole cluster to end).  bf16, window 4096, 1, 4,
    // 8 and 16 sequences of 32 / 8 heads of 128: 10.2, 17.3, 25.5 and 45.6 us, against 37.6,
    // 38.3, 39.4 and 46.5 with a CTA for each (sequence, kv head); FP8, 16 sequences: 29.1 / 43.1.
    // Clusters of more CTAs than fit: f32, 2 sequences, window 2048, 24.6 / 18.3.
    p.per = 0;
    for (int per = 1; per < parts; per *= 2) {
        const int bytes = smem + (per - 1) * smem_result;
        if (bytes > kSmemMax) break;
        const int ctas = (parts + per - 1) / per;
        if ((!one_each || pairs * ctas <= sms) && pairs <= clusters_at_once<Kernel>(dev, ctas, threads, bytes)) {
            p.per = per;
            break;
        }
    }
    const int ctas = p.per ? (parts + p.per - 1) / p.per : 1;
    cfg.gridDim = dim3(ctas, p.Hkv, num_seqs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = p.per ? smem + (p.per - 1) * smem_result : smem;
    // No more CTAs on an SM than the grid has for each: a grid of less than the GPU holds would
    // fill some SMs and leave others empty, so its CTAs ask for the memory that keeps them apart
    // (32 sequences of 32 / 8 heads of 128, bf16, window 1024: 27.2 -> 23.8 us).  Not so for
    // clusters, which may not find as many SMs together.
    const long long per_sm = (pairs + sms - 1) / sms, apart = kSmemMax / (per_sm + 1) + 1;
    if (ctas == 1 && apart > smem && apart <= kSmemMax / per_sm - 1024) cfg.dynamicSmemBytes = (size_t)(apart + 15) / 16 * 16;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, Kernel, p);
    if (launched == cudaSuccess || ctas == 1) return launched;
    // a GPU (or a part of one) without room for the cluster: one CTA for all parts, the same result
    cudaGetLastError();
    p.per = 0;
    cfg.gridDim.x = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, Kernel, p);
}

template <template <int> class Cache, int D>
cudaError_t launch_cache(const WParams& p, int num_seqs, cudaStream_t stream) {
    constexpr int NW = warps_for(Cache<D>::TYPE, D);
    using L = Layout<Cache<D>, D, NW>;
    return launch<window_decode_kernel<Cache, D, NW>>(p, num_seqs, NW * 32, one_each(Cache<D>::TYPE, D), L::bytes(p.G, 1),
                                                           L::bytes(p.G, 2) - L::bytes(p.G, 1), stream);
}

template <int D>
cudaError_t launch_type(const WParams& p, pa_dtype dtype, int num_seqs, cudaStream_t stream) {
    switch (dtype) {
        case PA_BF16: return launch_cache<Bf16Cache, D>(p, num_seqs, stream);
        case PA_FP8_E4M3: return launch_cache<Fp8Cache, D>(p, num_seqs, stream);
        case PA_FP4_E2M1: return launch_cache<Fp4Cache, D>(p, num_seqs, stream);
        case PA_F32: return launch_cache<F32Cache, D>(p, num_seqs, stream);
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
    // the blocks that a sequence can have listed: the window's (one more when it starts inside
    // one) and the sinks'
    long long n = ((long long)a.window + 2 * kBlockTokens - 2) / kBlockTokens +
                  ((long long)a.sinks + kBlockTokens - 1) / kBlockTokens;
    if (n > a.max_blocks) n = a.max_blocks;
    const int unit = 2 * warps_for(a.dtype, a.head_dim);       // blocks: a pair for every warp
    const int blocks = (int)n, least = min_part(a.dtype), limit = most_parts(a.dtype, a.head_dim);
    p.parts = 1;
    while (blocks >= min_pairs(a.dtype) * unit && 2 * p.parts <= limit && 2 * p.parts * least <= blocks) p.parts *= 2;
    p.part_len = blocks / p.parts / unit * unit;
    if (p.part_len == 0 || blocks - p.parts * p.part_len > unit) {
        p.part_len += unit;
        p.parts = (blocks + p.part_len - 1) / p.part_len;
    }
    p.per = 0;
    p.scale_log2 = a.scale * kLog2e;
    return a.head_dim == 64 ? launch_type<64>(p, a.dtype, a.num_seqs, stream)
                            : launch_type<128>(p, a.dtype, a.num_seqs, stream);
}

}  // namespace pa
