// pa_rope.cuh -- appending new tokens with the position rotation applied on the way: the kernels
// and their launch, compiled for rows turned by their place in the sequence (pa_rope.cu) and for
// rows turned by positions of their own on several axes (pa_rope_axes.cu).
//
// Row i of sequence s is the token at position p = start_pos[s] + i.  Its queries and keys
// are rotated by the angles p * inv_freq[f], f < R / 2 (R = rotary_dim) -- with AXES by
// positions[axis of f][row] * inv_freq[f], while p still is where the row goes --: dims (f, f + R / 2),
// or (2 f, 2 f + 1) when interleaved, are turned as a plane,
//   y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin,
// and dims R and up pass through.  The keys and values then go to the row's slot of the pool
// in the pool's type, the queries to q_out: one read and one write of each, in one launch.
//
// Angles.  In 32 bits p * inv_freq loses the angle of a far position (at p = 131072 an ulp of
// the product is 1/128 radian), and 64-bit arithmetic per angle is slow on this GPU.  So each
// frequency becomes a 64-bit fixed-point number of turns, F = inv_freq / (2 pi) * 2^64 mod
// 2^64 (once per CTA and frequency), and the angle of position p is the low 64 bits of p * F:
// the wrap of the integer product is the reduction modulo a turn, exact for every int32
// position.  The nearest quarter turn comes off in integers and the rest, at most an eighth of
// a turn, goes to sincospif, so that sine and cosine carry about one fp32 rounding each.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "pa_flags.cuh"
#include "pa_ptx.cuh"
#include "pa_window.h"

namespace pa {

namespace {

struct RParams {
    char* k_pool;
    char* v_pool;
    char* q_out;
    const char* q;
    const char* k_new;
    const char* v_new;
    long long q_out_stride, q_stride, k_stride, v_stride;      // bytes from row to row
    const double* inv_freq;
    const int32_t* positions;                                  // AXES: [axes][total], and the axis of each plane
    const int32_t* plane_axis;                                 // (null: the only one)
    int axes;
    const int32_t* tables;
    const int32_t* start_pos;
    const int32_t* cu;
    int32_t* err;
    int max_blocks, S, total, num_blocks, Hq, Hkv, half;       // half = rotary_dim / 2
};

// Threads of a tile's CTA: its 16 rows times a head's items, or more.  128 against 256, 32 / 8
// heads of 128: 37 chunks of 1 to 131, bf16 14.0 / 17.5 us and FP8 17.2 / 22.0; 16 of 512, 34.8 /
// 36.2 and 38.4 / 40.6 (the SMs' loads come out more even).
constexpr int tile_threads(pa_dtype t, int head_dim) { return t == PA_F32 && head_dim == 128 ? 256 : 128; }
constexpr int kRowThreads = 128;      // of a row's
// Items of a row's thread that are loaded together (32 / 8 heads of 128 have three for each; two
// leave the quantised types' registers), and CTAs of an SM that the registers are bounded for (7
// against what comes of it, 6 or 9: 1024 rows of 32 / 8 heads, bf16 5.5 / 7.0 us, f32 9.5 / 10.6).
constexpr int row_items(pa_dtype t, int head_dim) { return head_dim == 64 || (t != PA_F32 && t != PA_BF16) ? 2 : 3; }
constexpr int kRowCtas = 7;
// A call goes row by row (a CTA each, no row waits for another) or tile by tile (a pool's tile
// is written in whole runs).  Rows are faster for few of them, and for short chunks, whose
// tiles are mostly empty; runs matter more where a value is a byte.  Rows against tiles, 32 / 8
// heads of 128, us: one chunk of 256 bf16 3.0 / 3.5, FP8 6.3 / 6.3; of 500 bf16 4.1 / 4.3, FP8
// 13.2 / 6.5; 256 chunks of 8, 11.6 / 17.6 and 27.4 / 28.2; 64 of 16, 5.5 / 7.7 and 16.2 / 13.4;
// 100 of 1 to 40, 11.0 / 14.2 and 27.2 / 19.1; 256 of 16, 24.0 / 24.2 and 51.6 / 34.8; 16 of 512,
// 40.3 / 34.8 and 99.4 / 38.4.
constexpr bool quantised(pa_dtype t) { return t == PA_FP8_E4M3 || t == PA_FP4_E2M1; }
constexpr int rows_alone(pa_dtype t) { return quantised(t) ? 256 : 512; }     // up to so many rows in all
constexpr int tile_min_rows(pa_dtype t) { return quantised(t) ? 16 : 32; }    // and below so many per sequence
// Heads of a tile's thread, at least and at most (four against two and six, 14 / 2 heads of 64,
// FP8, 37 chunks of 1 to 131: 6.5, 7.3 and 6.8 us; 16 chunks of 512, 32 / 8 of 128, bf16, 24
// and 48 heads: 34.8 and 39.2).
constexpr int kLeastHeads = 4, kMostHeads = 36;
// Threads of tiles' CTAs for each SM while their shares are picked.  An SM holds 512; a handful of
// CTAs more cost less than a whole share fewer for every tile (4 chunks of 600, 153 tiles, 32 / 8
// heads of 128, 520 against 512, four shares against three: bf16 11.9 / 13.9 us, FP8 14.4 / 15.8;
// f32, two against one, 21.7 / 26.9).
constexpr int kTileRoom = 520;
constexpr int kTileHeads = 3;          // heads of a thread that are loaded together (four spill)

// A frequency in radians per position as turns * 2^64, modulo 2^64.  Below 1024 in integers
// (FP64 instructions take 64 times as long here): x = m 2^e with a 53-bit m, and 2^64 x / (2 pi)
// is m (2^66 / (2 pi)) 2^(e - 2), good to less than 2^10 / 2^64 turns.
__device__ __forceinline__ uint64_t fixed_turns(double inv_freq) {
    const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
    const int e = (int)(bits >> 52 & 0x7ff);                   // x = m 2^(e - 1075)
    uint64_t t;
    if (e < 1023 + 10) {
        const uint64_t m = e > 0 ? (bits & ((1ull << 52) - 1)) | 1ull << 52 : 0;    // (denormal: none)
        const uint64_t hi = __umul64hi(m, 0xa2f9836e4e44152aull), lo = m * 0xa2f9836e4e44152aull;
        const int sh = 1077 - e;                               // from 45 on
        t = sh < 64 ? lo >> sh | hi << (64 - sh) : sh == 64 ? hi : sh < 128 ? hi >> (sh - 64) : 0;
    } else {
        double r = fabs(inv_freq) * 0.15915494309189533577;    // 1 / (2 pi)
        r -= rint(r);
        t = (uint64_t)__double2ll_rn(r * 18446744073709551616.0);
    }
    return bits >> 63 ? 0 - t : t;
}

// cos and sin of `phase` / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));     // within +-2^61
    const float x = (float)(int32_t)(rest >> 30) * 1.16415321826934814453125e-10f;   // 2^-33: half turns
    float s, c;
    sincospif(x, &s, &c);
    const float a = (quarter & 1) ? s : c, b = (quarter & 1) ? c : s;
    return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b);
}

// The axis of plane f where rows have positions of their own, -1 (flagged by `report`): it has none.
__device__ __forceinline__ int plane_axis(const RParams& p, int f, bool report) {
    const int axis = p.plane_axis ? __ldg(p.plane_axis + f) : 0;
    const bool ok = axis >= 0 && axis < p.axes;
    if (!ok && report) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
    return ok ? axis : -1;
}
// The position of row `row` on an axis; a plane without one does not turn.
__device__ __forceinline__ int32_t own_position(const RParams& p, int row, int axis) {
    return axis >= 0 ? __ldg(p.positions + (size_t)axis * p.total + row) : 0;
}

// Elements of one 16-byte piece of a row.
template <int E>
struct Piece { float x[E]; };

template <int E>
__device__ __forceinline__ Piece<E> unpack(uint4 v) {
    Piece<E> r;
    if constexpr (E == 4) {
        r.x[0] = __uint_as_float(v.x); r.x[1] = __uint_as_float(v.y);
        r.x[2] = __uint_as_float(v.z); r.x[3] = __uint_as_float(v.w);
    } else {
        r.x[0] = bf16_lo_to_f32(v.x); r.x[1] = bf16_hi_to_f32(v.x);
        r.x[2] = bf16_lo_to_f32(v.y); r.x[3] = bf16_hi_to_f32(v.y);
        r.x[4] = bf16_lo_to_f32(v.z); r.x[5] = bf16_hi_to_f32(v.z);
        r.x[6] = bf16_lo_to_f32(v.w); r.x[7] = bf16_hi_to_f32(v.w);
    }
    return r;
}

template <int E>
__device__ __forceinline__ uint4 pack(const Piece<E>& r) {
    if constexpr (E == 4)
        return make_uint4(__float_as_uint(r.x[0]), __float_as_uint(r.x[1]), __float_as_uint(r.x[2]),
                          __float_as_uint(r.x[3]));
    else
        return make_uint4(pack_bf16x2(r.x[0], r.x[1]), pack_bf16x2(r.x[2], r.x[3]),
                          pack_bf16x2(r.x[4], r.x[5]), pack_bf16x2(r.x[6], r.x[7]));
}

template <int E>
__device__ __forceinline__ float max_abs(const Piece<E>& r) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(r.x[e]));
    return m;
}

// x / scale, correctly rounded, for one scale and many x: with the correctly rounded reciprocal
// y, q = x y and two steps q + (x - q scale) y, the remainders exact by fused multiply-add, give
// the quotient's rounding (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) while nothing underflows.  At scales from 2^-80 the remainders
// of quotients that round to a code above 0 do not; other scales (infinity too) divide.  The
// steps make +0 of a quotient of -0 (and may of one that underflows): x gives the sign.
struct Divisor {
    float scale, y;
    bool plain;
    __device__ __forceinline__ explicit Divisor(float s) {
        scale = s;
        y = __frcp_rn(s);
        plain = !(s >= 0x1p-80f && s <= 0x1p80f);
    }
    __device__ __forceinline__ float quotient(float x) const {
        float q = __fmul_rn(x, y);
        q = __fmaf_rn(__fmaf_rn(-q, scale, x), y, q);
        return copysignf(__fmaf_rn(__fmaf_rn(-q, scale, x), y, q), x);
    }
};

// Eight E4M3 codes of x / scale, in the order of the dims (scale 0: an all-zero row).
__device__ __forceinline__ uint2 e4m3_codes(const Piece<8>& r, const Divisor& by) {
    if (!(by.scale > 0.f)) return make_uint2(0u, 0u);
    float q[8];
    if (by.plain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(r.x[i], by.scale);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = by.quotient(r.x[i]);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)pack_e4m3x2(q[4 * i], q[4 * i + 1]) | (uint32_t)pack_e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16;
    return make_uint2(w[0], w[1]);
}

// The two pieces of a head's row that work item u (of D / (2 E)) takes: the two sides of its
// planes, or two neighbours.
struct Pair { int a, b; };
template <int E>
__device__ __forceinline__ Pair pieces_of(int u, int half, bool split) {
    const int h = half / E;
    if (split && u < h) return Pair{u, u + h};
    return Pair{2 * u, 2 * u + 1};         // (past the planes of a split row: 2 h + 2 (u - h))
}
// The item that takes piece y, and whether as its first or second one.
template <int E>
__device__ __forceinline__ int item_of_piece(int y, int half, bool split, bool& second) {
    const int h = half / E;
    if (split && y < 2 * h) {
        second = y >= h;
        return second ? y - h : y;
    }
    second = y & 1;
    return y >> 1;
}

// Turns the planes of item u: `cs` the cosines and sines of its row's frequencies.
template <int E, bool INTERLEAVED>
__device__ __forceinline__ void turn_item(Piece<E>& a, Piece<E>& b, const float2 (&c)[E]) {
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 ca = c[e / 2], cb = c[E / 2 + e / 2];
            const float a0 = a.x[e], a1 = a.x[e + 1], b0 = b.x[e], b1 = b.x[e + 1];
            a.x[e] = a0 * ca.x - a1 * ca.y;
            a.x[e + 1] = a1 * ca.x + a0 * ca.y;
            b.x[e] = b0 * cb.x - b1 * cb.y;
            b.x[e + 1] = b1 * cb.x + b0 * cb.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x1 = a.x[e], x2 = b.x[e];
            a.x[e] = x1 * c[e].x - x2 * c[e].y;
            b.x[e] = x2 * c[e].x + x1 * c[e].y;
        }
    }
}
// Item u's E cosines and sines: its planes are u E .. u E + E - 1 of the row's.
template <int E>
__device__ __forceinline__ void item_turns(const float2* cs, int u, float2 (&c)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float4 v = *reinterpret_cast<const float4*>(cs + u * E + e);
        c[e] = make_float2(v.x, v.y);
        c[e + 1] = make_float2(v.z, v.w);
    }
}

// One item of a key or value row into a quantised pool (u-adjacent lanes hold a head's items;
// every lane of the warp calls it).
template <int D, pa_dtype T>
__device__ __forceinline__ void put_quantised(const RParams& p, char* pool, int32_t blk, int h, int slot, bool is_k,
                                              bool live, int u, Pair at, bool split, const Piece<8>& a,
                                              const Piece<8>& b) {
    constexpr int E = 8, PH = D / 16;
    if constexpr (T == PA_FP8_E4M3) {
        float m = fmaxf(max_abs<E>(a), max_abs<E>(b));
#pragma unroll
        for (int x = 1; x < PH; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (live) {
            const float scale = __fdiv_rn(m, 448.f);
            char* rec = pool + ((size_t)blk * p.Hkv + h) * fp8_record_bytes(D);
            const Divisor by(scale);
            const uint2 ca = e4m3_codes(a, by), cb = e4m3_codes(b, by);
            if (is_k) {
                *reinterpret_cast<uint2*>(rec + ((at.a >> 1) * kBlockTokens + slot) * 16 + (at.a & 1) * 8) = ca;
                *reinterpret_cast<uint2*>(rec + ((at.b >> 1) * kBlockTokens + slot) * 16 + (at.b & 1) * 8) = cb;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    rec[(at.a * 8 + e) * kBlockTokens + slot] = (char)((e < 4 ? ca.x : ca.y) >> (8 * (e & 3)));
                    rec[(at.b * 8 + e) * kBlockTokens + slot] = (char)((e < 4 ? cb.x : cb.y) >> (8 * (e & 3)));
                }
            }
            if (u == 0) *reinterpret_cast<float*>(rec + (size_t)16 * D + 4 * slot) = scale;
        }
    } else {
        // the largest magnitude of each piece's 32-value block: its four pieces' maxima,
        // wherever in the head's lanes they are
        const float ma = max_abs<E>(a), mb = max_abs<E>(b);
        const int lane = threadIdx.x & 31, base = lane - u;
        char* rec = pool + ((size_t)blk * p.Hkv + h) * fp4_record_bytes(D);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int pc = k ? at.b : at.a;
            float m = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                bool second;
                const int from = base + item_of_piece<E>((pc & ~3) + y, p.half, split, second);
                const float va = __shfl_sync(0xffffffffu, ma, from), vb = __shfl_sync(0xffffffffu, mb, from);
                m = fmaxf(m, second ? vb : va);
            }
            if (!live) continue;
            const int code = m > 0.f ? max((int)(__float_as_uint(m) >> 23) - 2, 0) : 0;
            const float inv = exp2i(127 - code);                  // 1 / scale, exact
            const Piece<E>& x = k ? b : a;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t two = m > 0.f ? pack_e2m1x2(x.x[2 * c] * inv, x.x[2 * c + 1] * inv) : 0u;
                if (is_k) {
                    rec[(size_t)slot * (D / 2) + c * (D / 8) + pc] = (char)two;
                } else {
                    // a byte holds two slots of one dim, and rows of one call may share it
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at_byte = (((2 * c + e) * 4 + (slot % 8) / 2) * (D / 16) + pc / 2) * 4 +
                                            (pc & 1) * 2 + slot / 8;
                        unsigned int* word = reinterpret_cast<unsigned int*>(rec + (at_byte & ~3));
                        const int shift = (at_byte & 3) * 8 + (slot & 1) * 4;
                        atomicAnd(word, ~(0xfu << shift));
                        atomicOr(word, ((two >> (4 * e)) & 0xfu) << shift);
                    }
                }
            }
            if ((pc & 3) == 0) rec[8 * D + slot * (D / 32) + (pc >> 2)] = (char)code;
        }
    }
}

// Flags cu_new_tokens where it is not a prefix sum that ends at the rows (one CTA's N threads).
template <int N>
__device__ __forceinline__ void check_cu(const RParams& p) {
    bool bad = threadIdx.x == 0 && (__ldg(p.cu) != 0 || __ldg(p.cu + p.S) != p.total);
    for (int s = threadIdx.x; s < p.S; s += N) bad |= __ldg(p.cu + s) > __ldg(p.cu + s + 1);
    if (bad) raise_flag(p.err, PA_DEV_ERR_BAD_CU);
}

// The last of n sequences from lo on whose first unit (from(s), not falling) is at most x, found
// by all N threads of the CTA: a probe each narrows the range N times.
template <int N, typename From>
__device__ __forceinline__ int last_from(int lo, int n, int x, From from) {
    while (n > 1) {
        const int step = (n + N - 1) / N, at = threadIdx.x * step;
        const int hits = __syncthreads_count(at < n && from(lo + at) <= x);
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// The place of new row `row`, the same in every thread; false: it has none (flagged).
__device__ __forceinline__ bool find_row(const RParams& p, int row, int& pos_out, int32_t& blk_out) {
    // its sequence if all append as many rows (a decode step), with its place in the same round trip
    int s = min((int)((long long)row * p.S / p.total), p.S - 1);
    int first = __ldg(p.cu + s), next = __ldg(p.cu + s + 1);
    long long start = __ldg(p.start_pos + s);
    const bool report = threadIdx.x == 0;
    if (row < first || row >= next) {
        s = last_from<kRowThreads>(0, p.S, row, [&](int x) { return __ldg(p.cu + x); });
        first = __ldg(p.cu + s);
        next = __ldg(p.cu + s + 1);
        start = __ldg(p.start_pos + s);
        if (row < first || row >= next) {
            if (report) raise_flag(p.err, PA_DEV_ERR_BAD_CU);
            return false;
        }
    }
    const long long pos = start + (row - first);
    if (pos < 0 || pos >= (long long)p.max_blocks * kBlockTokens) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
        return false;
    }
    const int32_t blk = __ldg(p.tables + (size_t)s * p.max_blocks + (int)(pos / kBlockTokens));
    pos_out = (int)pos;
    blk_out = blk;
    return true;
}

// One CTA per row: its frequencies' cosines and sines once, then every (head, item) of the
// keys, values and queries, a thread an item at a time: two 16-byte loads, two stores.  The
// row's data do not depend on its place, so the first N items of a thread are under way while
// the place is looked up.  T: the pool's type.
template <int D, pa_dtype T, bool INTERLEAVED, bool AXES>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) rope_append_kernel(const RParams p) {
    constexpr int E = T == PA_F32 ? 4 : 8;       // elements of a piece (the rows are f32 or bf16)
    constexpr int PH = D / (2 * E);              // items of a head
    constexpr int N = row_items(T, D);
    __shared__ __align__(16) float2 cs[D / 2];
    // the rows may come from the kernel before (a projection), and the pools be in use by it
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x, tid = threadIdx.x;
    const int items = (2 * p.Hkv + p.Hq) * PH;
    struct Item { int h, u; bool live, is_k, is_v; Pair at; };
    auto item = [&](int i) {
        Item x;
        const int head = i / PH;
        x.live = i < items;
        x.u = i % PH;
        x.is_k = head < p.Hkv;
        x.is_v = !x.is_k && head < 2 * p.Hkv;
        x.h = x.is_k ? head : x.is_v ? head - p.Hkv : head - 2 * p.Hkv;
        x.at = pieces_of<E>(x.u, p.half, !INTERLEAVED && !x.is_v);
        return x;
    };
    uint4 ra[N], rb[N];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const Item x = item(i0 + j * kRowThreads + tid);
            ra[j] = rb[j] = make_uint4(0u, 0u, 0u, 0u);
            if (!x.live) continue;
            const char* src = (x.is_k ? p.k_new + row * p.k_stride : x.is_v ? p.v_new + row * p.v_stride
                                                                            : p.q + row * p.q_stride) + (size_t)x.h * (PH * 32);
            ra[j] = *reinterpret_cast<const uint4*>(src + x.at.a * 16);
            rb[j] = *reinterpret_cast<const uint4*>(src + x.at.b * 16);
        }
    };
    load(0);
    // (at most one plane a thread, whose position does not depend on the row's place either)
    static_assert(D / 2 <= kRowThreads, "a thread has one plane");
    int32_t own = 0;
    if (AXES && tid < p.half) own = own_position(p, row, plane_axis(p, tid, true));
    if (row == 0) check_cu<kRowThreads>(p);
    int pos = 0;
    int32_t blk = 0;
    if (!find_row(p, row, pos, blk)) return;
    for (int f = tid; f < p.half; f += kRowThreads) {
        if constexpr (AXES) cs[f] = cos_sin(fixed_turns(p.inv_freq[f]) * (uint64_t)(int64_t)own);
        else cs[f] = cos_sin(fixed_turns(p.inv_freq[f]) * (uint64_t)pos);
    }
    if (blk < 0 || blk >= p.num_blocks) {        // no place: the row is skipped
        if (tid == 0) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
        return;
    }
    __syncthreads();
    const int slot = pos % kBlockTokens;
    // every lane runs every iteration: the quantised types share maxima by shuffles
    for (int i0 = 0; i0 < items; i0 += N * kRowThreads) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (i0 + j * kRowThreads >= items) break;
            const Item x = item(i0 + j * kRowThreads + tid);
            const Pair at = x.at;
            Piece<E> a = unpack<E>(ra[j]), b = unpack<E>(rb[j]);
            if (!x.is_v && x.u < p.half / E) {
                float2 c[E];
                item_turns<E>(cs, x.u, c);
                turn_item<E, INTERLEAVED>(a, b, c);
            }
            const bool to_pool = x.live && (x.is_k || x.is_v);
            if (x.live && !to_pool) {
                char* dst = p.q_out + row * p.q_out_stride + (size_t)x.h * (PH * 32);
                *reinterpret_cast<uint4*>(dst + at.a * 16) = pack<E>(a);
                *reinterpret_cast<uint4*>(dst + at.b * 16) = pack<E>(b);
            }
            char* pool = x.is_v ? p.v_pool : p.k_pool;
            if constexpr (T == PA_F32 || T == PA_BF16) {
                if (to_pool) {
                    char* dst = pool + ((((size_t)blk * p.Hkv + x.h) * (2 * PH)) * kBlockTokens + slot) * 16;
                    *reinterpret_cast<uint4*>(dst + at.a * 256) = pack<E>(a);
                    *reinterpret_cast<uint4*>(dst + at.b * 256) = pack<E>(b);
                }
            } else if (__any_sync(0xffffffffu, to_pool)) {
                put_quantised<D, T>(p, pool, blk, to_pool ? x.h : 0, slot, x.is_k, to_pool, x.u, at, !INTERLEAVED && !x.is_v, a, b);
            }
        }
    }
}

// Chunks.  A CTA takes a tile: the rows of one sequence that fall into one block, at most 16,
// so that a pool's tile is written in whole runs and the place is looked up once.  Tile t
// belongs to the last sequence s with cu[s] / 16 + 2 s <= t (a sequence of n rows touches at
// most n / 16 + 2 blocks, so its tiles stay below the next one's): no counts are summed, and a
// search by all threads finds s.  blockIdx.y picks a share of the heads.
//
// A thread keeps one item index u of one row, with its cosines and sines in registers, and
// goes through the heads of its share: keys with the rows on adjacent lanes (16 slots of a
// piece are 256 bytes of a pool tile), queries with the items on adjacent lanes.  FP8 values
// are transposed through shared memory: a warp takes a head's 16 rows, and every lane stores
// whole 16-slot runs of four dims.
constexpr int kTileRows = kBlockTokens;

struct Tile {
    int32_t row0;            // first row of the new rows, of slot `lo`
    int pos0;                // position of the block's slot 0
    int lo, hi;              // slots lo .. hi - 1
    int32_t blk;             // as read from the table
};

__device__ __forceinline__ int tile_base(const RParams& p, int s) {
    return (__ldg(p.cu + s) >> 4) + 2 * s;        // (arithmetic shift: also of a bad negative entry)
}

// The CTA's tile, the same in every thread; false: none, or at no position of the table
// (flagged).  The block is checked by the caller, when its load has had time to land.
template <int NT>
__device__ __forceinline__ bool find_tile(const RParams& p, int t, Tile& out) {
    const int tid = threadIdx.x;
    // the sequence if all have as many rows, and its place with it: often right, one round trip
    int lo = min(t / (p.total / (kTileRows * p.S) + 2), p.S - 1);
    int first = __ldg(p.cu + lo), next = __ldg(p.cu + lo + 1);
    long long start = __ldg(p.start_pos + lo);
    const bool guessed = t >= (first >> 4) + 2 * lo && (lo + 1 == p.S || t < (next >> 4) + 2 * (lo + 1));
    if (!guessed) {
        lo = last_from<NT>(0, p.S, t, [&](int s) { return tile_base(p, s); });
        first = __ldg(p.cu + lo);
        next = __ldg(p.cu + lo + 1);
        start = __ldg(p.start_pos + lo);
    }
    const bool report = tid == 0 && blockIdx.y == 0;
    if (first < 0 || next > p.total || next < first) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_CU);
        return false;
    }
    const long long from = start >> 4;                              // block of the first row
    const long long b = from + (t - ((first >> 4) + 2 * lo));
    const long long begin = max(start, b * kTileRows), end = min(start + (next - first), (b + 1) * kTileRows);
    if (b < from || begin >= end) return false;                     // (a gap between sequences)
    if (b < 0 || b >= p.max_blocks) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
        return false;
    }
    out.blk = __ldg(p.tables + (size_t)lo * p.max_blocks + (int)b);
    out.pos0 = (int)(b * kTileRows);
    out.lo = (int)(begin - b * kTileRows);
    out.hi = (int)(end - b * kTileRows);
    out.row0 = first + (int)(begin - start);
    return true;
}

// FP8 values of one head: lane = (slot, half of the dims), D / 16 pieces of its row.
template <int D>
__device__ __forceinline__ void load_values(const RParams& p, const Tile& tile, int h, uint4 (&v)[D / 16]) {
    const int lane = threadIdx.x & 31, slot = lane & 15, half = lane >> 4;
    const bool live = h < p.Hkv && slot >= tile.lo && slot < tile.hi;
    const char* src = p.v_new + (long long)(tile.row0 + slot - tile.lo) * p.v_stride + (size_t)h * (2 * D) + half * D;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
        v[i] = live ? *reinterpret_cast<const uint4*>(src + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
}
// ... and into the pool.  `sm`: D / 4 x 16 words of the warp.
template <int D>
__device__ __forceinline__ void put_fp8_values(const RParams& p, const Tile& tile, int h, const uint4 (&v)[D / 16],
                                               uint32_t* sm) {
    constexpr int NP = D / 16;
    const int lane = threadIdx.x & 31, slot = lane & 15, half = lane >> 4;
    const bool live = slot >= tile.lo && slot < tile.hi;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) m = fmaxf(m, max_abs<8>(unpack<8>(v[i])));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    const float scale = __fdiv_rn(m, 448.f);
    const Divisor by(scale);
    __syncwarp();                               // (the last head's reads are done)
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint2 c = e4m3_codes(unpack<8>(v[i]), by);
        const int d4 = half * (D / 8) + 2 * i;
        sm[d4 * 16 + slot] = c.x;
        sm[(d4 + 1) * 16 + slot] = c.y;
    }
    __syncwarp();
    char* rec = p.v_pool + ((size_t)tile.blk * p.Hkv + h) * fp8_record_bytes(D);
    for (int d4 = lane; d4 < D / 4; d4 += 32) {
        uint32_t y[4][4];                       // [dim][four slots]
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint4 x = *reinterpret_cast<const uint4*>(sm + d4 * 16 + 4 * w);
            const uint32_t a = __byte_perm(x.x, x.y, 0x5140), b = __byte_perm(x.z, x.w, 0x5140);
            const uint32_t c = __byte_perm(x.x, x.y, 0x7362), d = __byte_perm(x.z, x.w, 0x7362);
            y[0][w] = __byte_perm(a, b, 0x5410);
            y[1][w] = __byte_perm(a, b, 0x7632);
            y[2][w] = __byte_perm(c, d, 0x5410);
            y[3][w] = __byte_perm(c, d, 0x7632);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            char* dst = rec + (4 * d4 + j) * 16;
            if (tile.lo == 0 && tile.hi == kTileRows) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(y[j][0], y[j][1], y[j][2], y[j][3]);
                continue;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (4 * w >= tile.lo && 4 * w + 4 <= tile.hi) {
                    *reinterpret_cast<uint32_t*>(dst + 4 * w) = y[j][w];
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (4 * w + k >= tile.lo && 4 * w + k < tile.hi) dst[4 * w + k] = (char)(y[j][w] >> (8 * k));
                }
            }
        }
    }
    if (live && half == 0) *reinterpret_cast<float*>(rec + (size_t)16 * D + 4 * slot) = scale;
}

template <int D, pa_dtype T, bool INTERLEAVED, bool AXES>
__global__ void __launch_bounds__(tile_threads(T, D), 512 / tile_threads(T, D)) rope_append_tile_kernel(const RParams p) {
    constexpr int E = T == PA_F32 ? 4 : 8;
    constexpr int PH = D / (2 * E);
    constexpr int NT = tile_threads(T, D), NW = NT / 32;
    constexpr int GROUPS = NT / (kTileRows * PH);      // threads of a (row, item), a share of the heads each
    constexpr int PAD = D / 2 + 2;                           // (rows on different banks)
    __shared__ __align__(16) float2 cs[kTileRows * PAD];
    __shared__ uint64_t turns[D / 2];
    __shared__ int axis[AXES ? D / 2 : 1];
    __shared__ __align__(16) uint32_t sm_v[T == PA_FP8_E4M3 ? NW * (D / 4) * 16 : 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_cu<NT>(p);
    if (tid < p.half) turns[tid] = fixed_turns(p.inv_freq[tid]);
    if constexpr (AXES)
        if (tid < p.half) axis[tid] = plane_axis(p, tid, blockIdx.y == 0);
    Tile tile;
    if (!find_tile<NT>(p, blockIdx.x, tile)) return;
    const int share = blockIdx.y * GROUPS, stride = gridDim.y * GROUPS;
    auto row_at = [&](int slot) { return (long long)(tile.row0 + slot - tile.lo); };
    // Queries: items on adjacent lanes.  N heads are loaded while the N before them are turned
    // and stored (q_out may be q, so the compiler would not move loads past stores); the first
    // ones are under way while the cosines are made.
    constexpr int N = kTileHeads;
    const int qu = tid % PH, qslot = (tid / PH) % kTileRows, qg = share + tid / (PH * kTileRows);
    const bool q_here = p.Hq > 0 && qslot >= tile.lo && qslot < tile.hi;
    const Pair qat = pieces_of<E>(qu, p.half, !INTERLEAVED);
    // (a row's heads span less than 2^26 bytes: 32-bit offsets)
    const char* q_src = p.q + row_at(qslot) * p.q_stride + qat.a * 16 + (uint32_t)(qg * (PH * 32));
    const int q_ab = (qat.b - qat.a) * 16, q_step = stride * (PH * 32);
    const int q_heads = q_here && qg < p.Hq ? (p.Hq - qg + stride - 1) / stride : 0;     // of this thread
    // its heads first .. first + N - 1
    auto load_q = [&](int first, uint4 (&ra)[N], uint4 (&rb)[N]) {
        const char* s = q_src + (uint32_t)(first * q_step);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (first + i < q_heads) {
                ra[i] = *reinterpret_cast<const uint4*>(s + i * q_step);
                rb[i] = *reinterpret_cast<const uint4*>(s + i * q_step + q_ab);
            }
    };
    uint4 a0[N], b0[N];
    load_q(0, a0, b0);
    __syncthreads();
    const int rows = tile.hi - tile.lo;
    for (int i = tid; i < rows * p.half; i += NT) {
        const int r = i / p.half, f = i - r * p.half;
        if constexpr (AXES) {
            cs[(tile.lo + r) * PAD + f] = cos_sin(turns[f] * (uint64_t)(int64_t)own_position(p, tile.row0 + r, axis[f]));
        } else {
            cs[(tile.lo + r) * PAD + f] = cos_sin(turns[f] * (uint64_t)(tile.pos0 + tile.lo + r));
        }
    }
    if (tile.blk < 0 || tile.blk >= p.num_blocks) {        // no place: the tile is skipped
        if (tid == 0 && blockIdx.y == 0) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
        return;
    }
    __syncthreads();
    if (q_heads > 0) {
        const bool turn = qu < p.half / E;
        float2 c[E];
        if (turn) item_turns<E>(cs + qslot * PAD, qu, c);
        char* q_dst = p.q_out + row_at(qslot) * p.q_out_stride + qat.a * 16 + (uint32_t)(qg * (PH * 32));
        auto store_q = [&](int first, const uint4 (&ra)[N], const uint4 (&rb)[N]) {
            char* d = q_dst + (uint32_t)(first * q_step);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (first + i < q_heads) {
                    Piece<E> a = unpack<E>(ra[i]), b = unpack<E>(rb[i]);
                    if (turn) turn_item<E, INTERLEAVED>(a, b, c);
                    *reinterpret_cast<uint4*>(d + i * q_step) = pack<E>(a);
                    *reinterpret_cast<uint4*>(d + i * q_step + q_ab) = pack<E>(b);
                }
        };
        uint4 a1[N], b1[N];
        for (int i = 0; i < q_heads; i += 2 * N) {
            load_q(i + N, a1, b1);
            store_q(i, a0, b0);
            load_q(i + 2 * N, a0, b0);
            store_q(i + N, a1, b1);
        }
    }
    if constexpr (T == PA_F32 || T == PA_BF16) {
        // keys and values: rows on adjacent lanes
        const int slot = tid % kTileRows, u = (tid / kTileRows) % PH, g = share + tid / (PH * kTileRows);
        if (slot < tile.lo || slot >= tile.hi) return;
        const Pair at = pieces_of<E>(u, p.half, !INTERLEAVED);
        const bool turn = u < p.half / E;
        float2 c[E];
        if (turn) item_turns<E>(cs + slot * PAD, u, c);
        const char* ks = p.k_new + row_at(slot) * p.k_stride;
        const char* vs = p.v_new + row_at(slot) * p.v_stride;
        constexpr int NK = 2;
        for (int h0 = g; h0 < p.Hkv; h0 += NK * stride) {
            uint4 ra[NK], rb[NK], va[NK], vb[NK];
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const size_t off = (size_t)(h0 + i * stride) * (PH * 32);
                if (h0 + i * stride < p.Hkv) {
                    ra[i] = *reinterpret_cast<const uint4*>(ks + off + at.a * 16);
                    rb[i] = *reinterpret_cast<const uint4*>(ks + off + at.b * 16);
                    va[i] = *reinterpret_cast<const uint4*>(vs + off + u * 32);
                    vb[i] = *reinterpret_cast<const uint4*>(vs + off + u * 32 + 16);
                }
            }
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int h = h0 + i * stride;
                if (h < p.Hkv) {
                    Piece<E> a = unpack<E>(ra[i]), b = unpack<E>(rb[i]);
                    if (turn) turn_item<E, INTERLEAVED>(a, b, c);
                    const size_t to = ((((size_t)tile.blk * p.Hkv + h) * (2 * PH)) * kBlockTokens + slot) * 16;
                    *reinterpret_cast<uint4*>(p.k_pool + to + at.a * 256) = pack<E>(a);
                    *reinterpret_cast<uint4*>(p.k_pool + to + at.b * 256) = pack<E>(b);
                    *reinterpret_cast<uint4*>(p.v_pool + to + u * 512) = va[i];
                    *reinterpret_cast<uint4*>(p.v_pool + to + u * 512 + 256) = vb[i];
                }
            }
        }
    } else {
        // keys (and FP4 values): a head's items on adjacent lanes, which share its maxima; the next
        // head is loaded while one is stored (two or three ahead: 41.9 us for 40.6)
        const int u = tid % PH, slot = (tid / PH) % kTileRows, g = share + tid / (PH * kTileRows);
        const bool here = slot >= tile.lo && slot < tile.hi;
        const bool turn = u < p.half / E;
        float2 c[E];
        if (turn && here) item_turns<E>(cs + slot * PAD, u, c);
        constexpr bool FP8 = T == PA_FP8_E4M3;
        // FP8 values: by warps, from the last share on, loaded while the keys are turned
        const int warp = tid >> 5;
        int vh = (gridDim.y - 1 - blockIdx.y) * NW + warp;
        uint4 v[D / 16];
        if constexpr (FP8) load_values<D>(p, tile, vh, v);
#pragma unroll
        for (int kind = 0; kind < (FP8 ? 1 : 2); ++kind) {
            const bool split = !INTERLEAVED && kind == 0;
            const Pair at = pieces_of<E>(u, p.half, split);
            const char* src = kind == 0 ? p.k_new + row_at(slot) * p.k_stride : p.v_new + row_at(slot) * p.v_stride;
            uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
            auto load = [&](int h) {
                if (!here || h >= p.Hkv) return;
                ra = *reinterpret_cast<const uint4*>(src + (size_t)h * (PH * 32) + at.a * 16);
                rb = *reinterpret_cast<const uint4*>(src + (size_t)h * (PH * 32) + at.b * 16);
            };
            load(g);
            for (int h0 = share; h0 < p.Hkv; h0 += stride) {             // (the same trips in every lane)
                const int h = h0 + (g - share);
                const bool live = here && h < p.Hkv;
                Piece<E> a = unpack<E>(ra), b = unpack<E>(rb);
                load(h + stride);
                if (kind == 0 && turn && live) turn_item<E, INTERLEAVED>(a, b, c);
                put_quantised<D, T>(p, kind == 0 ? p.k_pool : p.v_pool, tile.blk, live ? h : 0, slot, kind == 0, live, u, at,
                                    split, a, b);
            }
        }
        if constexpr (FP8) {
            for (; vh < p.Hkv; vh += gridDim.y * NW) {
                put_fp8_values<D>(p, tile, vh, v, sm_v + warp * (D / 4) * 16);
                load_values<D>(p, tile, vh + gridDim.y * NW, v);
            }
        }
    }
}

template <int D, pa_dtype T, bool INTERLEAVED, bool AXES>
cudaError_t launch_rope(const RParams& p, cudaStream_t stream) {
    const bool tiles = p.total > rows_alone(T) && p.total >= tile_min_rows(T) * (long long)p.S;
    cudaLaunchConfig_t cfg = {};
    // A tile's heads are shared by several CTAs while all of them find room on the GPU (kTileRoom)
    // and a thread keeps kLeastHeads; by two where a thread of 128 had more than kMostHeads.
    constexpr int NT = tile_threads(T, D), GROUPS = NT / (kTileRows * (D / (T == PA_F32 ? 8 : 16)));
    const long long touched = (p.total + (kTileRows - 1ll) * p.S) / kTileRows;      // of chunks that begin anywhere
    const int heads = (p.Hq + 2 * p.Hkv) / GROUPS;                                  // of a thread that has a share alone
    const long long most = std::max(1, std::min(8, heads / kLeastHeads));
    int sms = 1;
    if (tiles) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
    }
    const long long at_once = (long long)sms * kTileRoom / NT / touched, least = NT == 128 && heads > kMostHeads ? 2 : 1;
    const int shares = (int)std::max(least, std::min(most, at_once));
    cfg.gridDim = tiles ? dim3((unsigned)(p.total / kTileRows + 2ll * p.S), shares) : dim3((unsigned)p.total);
    cfg.blockDim = dim3(tiles ? tile_threads(T, D) : kRowThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return tiles ? cudaLaunchKernelEx(&cfg, rope_append_tile_kernel<D, T, INTERLEAVED, AXES>, p)
                 : cudaLaunchKernelEx(&cfg, rope_append_kernel<D, T, INTERLEAVED, AXES>, p);
}

template <int D, bool INTERLEAVED, bool AXES>
cudaError_t launch_rope_type(const RParams& p, pa_dtype dtype, cudaStream_t stream) {
    switch (dtype) {
        case PA_F32: return launch_rope<D, PA_F32, INTERLEAVED, AXES>(p, stream);
        case PA_BF16: return launch_rope<D, PA_BF16, INTERLEAVED, AXES>(p, stream);
        case PA_FP8_E4M3: return launch_rope<D, PA_FP8_E4M3, INTERLEAVED, AXES>(p, stream);
        case PA_FP4_E2M1: return launch_rope<D, PA_FP4_E2M1, INTERLEAVED, AXES>(p, stream);
    }
    return cudaErrorInvalidValue;
}

template <bool AXES>
cudaError_t launch_rows(const RopeArgs& a, cudaStream_t stream) {
    if (a.total_new == 0) return cudaSuccess;
    const long long e = a.dtype == PA_F32 ? 4 : 2;      // bytes of a row's element
    RParams p;
    p.k_pool = static_cast<char*>(a.k_pool);
    p.v_pool = static_cast<char*>(a.v_pool);
    p.q_out = static_cast<char*>(a.q_out);
    p.q = static_cast<const char*>(a.q);
    p.k_new = static_cast<const char*>(a.k_new);
    p.v_new = static_cast<const char*>(a.v_new);
    p.q_out_stride = a.q_out_stride * e;
    p.q_stride = a.q_stride * e;
    p.k_stride = a.k_stride * e;
    p.v_stride = a.v_stride * e;
    p.inv_freq = a.inv_freq;
    p.positions = a.positions;
    p.plane_axis = a.plane_axis;
    p.axes = a.num_axes;
    p.tables = a.block_tables;
    p.start_pos = a.start_pos;
    p.cu = a.cu_new;
    p.err = a.err;
    p.max_blocks = a.max_blocks;
    p.S = a.num_seqs;
    p.total = a.total_new;
    p.num_blocks = a.num_blocks;
    p.Hq = a.q ? a.num_q_heads : 0;
    p.Hkv = a.num_kv_heads;
    p.half = a.rotary_dim / 2;
    if (a.head_dim == 64)
        return a.interleaved ? launch_rope_type<64, true, AXES>(p, a.dtype, stream)
                             : launch_rope_type<64, false, AXES>(p, a.dtype, stream);
    return a.interleaved ? launch_rope_type<128, true, AXES>(p, a.dtype, stream)
                         : launch_rope_type<128, false, AXES>(p, a.dtype, stream);
}

}  // namespace

}  // namespace pa
