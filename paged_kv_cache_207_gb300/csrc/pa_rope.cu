// pa_rope.cu -- appending new tokens with the position rotation applied on the way.
//
// Row i of sequence s is the token at position p = start_pos[s] + i.  Its queries and keys
// are rotated by the angles p * inv_freq[f], f < R / 2 (R = rotary_dim): dims (f, f + R / 2),
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
#include <cuda_bf16.h>

#include <cstdint>

#include "pa_ptx.cuh"
#include "pa_rows.cuh"
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
    const int32_t* tables;
    const int32_t* start_pos;
    const int32_t* cu;
    int32_t* err;
    int max_blocks, S, total, num_blocks, Hq, Hkv, half;       // half = rotary_dim / 2
};

constexpr int kThreads = 256;

// A frequency in radians per position as turns * 2^64, modulo 2^64.
__device__ __forceinline__ uint64_t fixed_turns(double inv_freq) {
    double t = inv_freq * 0.15915494309189533577;              // 1 / (2 pi)
    t -= rint(t);
    return (uint64_t)__double2ll_rn(t * 18446744073709551616.0);
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

// Eight E4M3 codes of x / scale, in the order of the dims (scale 0: an all-zero row).
__device__ __forceinline__ uint2 e4m3_codes(const Piece<8>& r, float scale) {
    if (!(scale > 0.f)) return make_uint2(0u, 0u);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)pack_e4m3x2(__fdiv_rn(r.x[4 * i], scale), __fdiv_rn(r.x[4 * i + 1], scale)) |
               (uint32_t)pack_e4m3x2(__fdiv_rn(r.x[4 * i + 2], scale), __fdiv_rn(r.x[4 * i + 3], scale)) << 16;
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

// One CTA per row: its frequencies' cosines and sines once, then every (head, item) of the
// keys, values and queries, a thread an item at a time: two 16-byte loads, two stores.
// T: the pool's type.
template <int D, pa_dtype T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RParams p) {
    constexpr int E = T == PA_F32 ? 4 : 8;       // elements of a piece (the rows are f32 or bf16)
    constexpr int PH = D / (2 * E);              // items of a head
    __shared__ float2 cs[D / 2];
    // the rows may come from the kernel before (a projection), and the pools be in use by it
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x, tid = threadIdx.x;
    if (row == 0 && tid == 0 && (__ldg(p.cu) != 0 || __ldg(p.cu + p.S) != p.total))
        raise_flag(p.err, PA_DEV_ERR_BAD_CU);
    int s, pos = 0;
    int32_t blk = 0;
    if (!locate_row(p, row, tid == 0, s, pos, blk)) return;      // the same in every thread
    for (int f = tid; f < p.half; f += kThreads) cs[f] = cos_sin(fixed_turns(p.inv_freq[f]) * (uint64_t)pos);
    __syncthreads();
    const int slot = pos % kBlockTokens;
    const int heads = 2 * p.Hkv + p.Hq;
    const int items = heads * PH;
    // every lane runs every iteration: the quantised types share maxima by shuffles
    for (int i0 = 0; i0 < items; i0 += kThreads) {
        const int i = i0 + tid;
        const bool live = i < items;
        const int head = live ? i / PH : 0, u = i % PH;
        const bool is_k = head < p.Hkv, is_v = !is_k && head < 2 * p.Hkv;
        const int h = is_k ? head : is_v ? head - p.Hkv : head - 2 * p.Hkv;
        const bool split = !INTERLEAVED && !is_v;
        const bool turn = !is_v && u < p.half / E;
        const Pair at = pieces_of<E>(u, p.half, split);
        const char* src = (is_k ? p.k_new + row * p.k_stride : is_v ? p.v_new + row * p.v_stride : p.q + row * p.q_stride) +
                          (size_t)h * (PH * 32);
        uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
        if (live) {
            ra = *reinterpret_cast<const uint4*>(src + at.a * 16);
            rb = *reinterpret_cast<const uint4*>(src + at.b * 16);
        }
        Piece<E> a = unpack<E>(ra), b = unpack<E>(rb);
        if (turn) {
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 ca = cs[u * E + e / 2], cb = cs[u * E + E / 2 + e / 2];
                    const float a0 = a.x[e], a1 = a.x[e + 1], b0 = b.x[e], b1 = b.x[e + 1];
                    a.x[e] = a0 * ca.x - a1 * ca.y;
                    a.x[e + 1] = a1 * ca.x + a0 * ca.y;
                    b.x[e] = b0 * cb.x - b1 * cb.y;
                    b.x[e + 1] = b1 * cb.x + b0 * cb.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float2 c = cs[u * E + e];
                    const float x1 = a.x[e], x2 = b.x[e];
                    a.x[e] = x1 * c.x - x2 * c.y;
                    b.x[e] = x2 * c.x + x1 * c.y;
                }
            }
        }
        if (live && !is_k && !is_v) {
            char* dst = p.q_out + row * p.q_out_stride + (size_t)h * (PH * 32);
            *reinterpret_cast<uint4*>(dst + at.a * 16) = pack<E>(a);
            *reinterpret_cast<uint4*>(dst + at.b * 16) = pack<E>(b);
        }
        char* pool = is_v ? p.v_pool : p.k_pool;
        if constexpr (T == PA_F32 || T == PA_BF16) {
            if (live && (is_k || is_v)) {
                char* dst = pool + ((((size_t)blk * p.Hkv + h) * (2 * PH)) * kBlockTokens + slot) * 16;
                *reinterpret_cast<uint4*>(dst + at.a * 256) = pack<E>(a);
                *reinterpret_cast<uint4*>(dst + at.b * 256) = pack<E>(b);
            }
        } else if constexpr (T == PA_FP8_E4M3) {
            float m = fmaxf(max_abs<E>(a), max_abs<E>(b));
#pragma unroll
            for (int x = 1; x < PH; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            if (live && (is_k || is_v)) {
                const float scale = __fdiv_rn(m, 448.f);
                char* rec = pool + ((size_t)blk * p.Hkv + h) * fp8_record_bytes(D);
                const uint2 ca = e4m3_codes(a, scale), cb = e4m3_codes(b, scale);
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
            const int lane = tid & 31, base = lane - u;
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
                if (!live || (!is_k && !is_v)) continue;
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
}

template <int D, pa_dtype T, bool INTERLEAVED>
cudaError_t launch_rope(const RParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.total);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, T, INTERLEAVED>, p);
}

template <int D, bool INTERLEAVED>
cudaError_t launch_rope_type(const RParams& p, pa_dtype dtype, cudaStream_t stream) {
    switch (dtype) {
        case PA_F32: return launch_rope<D, PA_F32, INTERLEAVED>(p, stream);
        case PA_BF16: return launch_rope<D, PA_BF16, INTERLEAVED>(p, stream);
        case PA_FP8_E4M3: return launch_rope<D, PA_FP8_E4M3, INTERLEAVED>(p, stream);
        case PA_FP4_E2M1: return launch_rope<D, PA_FP4_E2M1, INTERLEAVED>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
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
        return a.interleaved ? launch_rope_type<64, true>(p, a.dtype, stream)
                             : launch_rope_type<64, false>(p, a.dtype, stream);
    return a.interleaved ? launch_rope_type<128, true>(p, a.dtype, stream)
                         : launch_rope_type<128, false>(p, a.dtype, stream);
}

}  // namespace pa
